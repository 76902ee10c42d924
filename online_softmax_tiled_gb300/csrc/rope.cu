// Rotary positions: y = m · R(p·w) x on pairs of each head's first rot_dim
// elements, the rest of the head copied, for queries and keys in one launch.
//
// Mathematics. Pair i of a head at position p is turned by the angle p·w_i:
//   y_a = m (x_a cos - x_b sin),  y_b = m (x_b cos + x_a sin),
// (a, b) = (i, i + rot_dim/2) or (2i, 2i + 1). R is orthogonal, so the
// gradient of y = m R x is dx = m Rᵀ dy: the same kernel with sin negated.
//
// Angles: 64-bit fractions of a turn (rope_math.cuh).
//
// Work. Memory bound: 8 bytes per rotated bf16 pair against a few FMAs; the
// sincos of a (token, pair) costs tens of instructions, so a thread computes
// the cos and sin of its pairs once and applies them to a run of heads.
// A thread owns V pairs, 16 bytes of each half (or 32 consecutive bytes when
// interleaved): the 8 threads of a 128-wide bf16 head read its two halves as
// whole 128-byte lines. Shapes, strides or addresses that are not multiples
// of 16 bytes take the same kernel with V = 1.
//
// Measured: 2 x 8192 tokens of 40 bf16 heads of 128 out of a fused projection
// 53.0 us (6.3 TB/s, 0.93 of a plain copy; 88 us where the views start one
// element off and take V = 1). 2 x 4096 tokens of 20 heads, half of each
// turned, interleaved, as a gradient: 16.4 us (5.1 TB/s). One token of 64
// requests: 4.8 us back to back from Python, 2.8 in a CUDA graph.

#include "common.cuh"
#include "launchers.h"
#include "rope_math.cuh"

namespace attn {

namespace {

// Threads per block: a row has at most d / (2V) = 256 chunks with V = 1, 64
// otherwise.
template <int V> constexpr int kThreadsOf = V == 1 ? 256 : 128;

// V adjacent elements as they are in memory (V = 1: one element).
template <typename T, int V> struct Pack;
template <> struct Pack<__nv_bfloat16, 8> {
  using Raw = uint4;
  static ATTN_DEVINL void open(const Raw& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    }
  }
  static ATTN_DEVINL Raw close(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};
template <> struct Pack<float, 4> {
  using Raw = float4;
  static ATTN_DEVINL void open(const Raw& r, float (&x)[4]) {
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
  }
  static ATTN_DEVINL Raw close(const float (&x)[4]) {
    return make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <typename T> struct Pack<T, 1> {
  using Raw = T;
  static ATTN_DEVINL void open(const Raw& r, float (&x)[1]) { x[0] = to_f32(r); }
  static ATTN_DEVINL Raw close(const float (&x)[1]) { return from_f32<T>(x[0]); }
};

// One tensor of the call: heads [0, H) of x, written to y.
template <typename T> struct RopeTensor {
  const T* x;
  T* y;
  attn_strides xs, ys;
};

// Grid: x over groups of tokens (b·N + n), y over groups of `hpt` heads of
// the Hq + Hkv heads. A thread owns one chunk of V pairs (or, past the
// rotated part, 2V elements to copy) of one token, in all heads of the group.
// U heads are in flight at a time, held as they came from memory: 2U
// independent 16-byte loads, the first of them issued before the angles are
// worked out.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreadsOf<V>)
rope_kernel(RopeTensor<T> tq, RopeTensor<T> tk, const int* __restrict__ positions,
            long long pos_stride, const double* __restrict__ inv_freq, int tokens, int N, int Hq,
            int H, int d, int rot, int hpt, float magnitude, int inverse) {
  using P = Pack<T, V>;
  using Raw = typename P::Raw;
  constexpr int U = 4, kThreads = kThreadsOf<V>;
  pdl_launch_dependents();
  const int per_row = d / (2 * V);                     // chunks of a row
  const int chunk = threadIdx.x % per_row;
  const int token = blockIdx.x * (kThreads / per_row) + threadIdx.x / per_row;
  if (threadIdx.x >= kThreads / per_row * per_row || token >= tokens) return;
  const int b = token / N, n = token % N;
  const bool turned = chunk < rot / (2 * V);
  // element offsets of the chunk's two V-element pieces
  const int off0 = kInterleaved || !turned ? chunk * 2 * V : chunk * V;
  const int off1 = kInterleaved || !turned ? off0 + V : off0 + rot / 2;
  const T* xq = tq.x + b * tq.xs.batch + n * tq.xs.token;
  const T* xk = tk.x + b * tk.xs.batch + n * tk.xs.token;
  T* yq = tq.y + b * tq.ys.batch + n * tq.ys.token;
  T* yk = tk.y + b * tk.ys.batch + n * tk.ys.token;
  const int h0 = int(blockIdx.y) * hpt, h1 = min(H, h0 + hpt);

  pdl_wait_primary();
  Raw a[U], c[U];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u < h1) {
        const T* px = h + u < Hq ? xq + (h + u) * tq.xs.head : xk + (h + u - Hq) * tk.xs.head;
        a[u] = *reinterpret_cast<const Raw*>(px + off0);
        c[u] = *reinterpret_cast<const Raw*>(px + off1);
      }
  };
  load(h0);
  float cs[V], sn[V];
  if (turned) {
    const long long p = positions[b * pos_stride + n];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s;
      turn_cos_sin(p, inv_freq[chunk * V + i], magnitude, cs[i], s);
      sn[i] = inverse ? -s : s;
    }
  }
  for (int h = h0; h < h1; h += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u < h1) {
        if (turned) {
          float x[V], z[V], e[2 * V];                  // e: the 2V results in memory order
          P::open(a[u], x);
          P::open(c[u], z);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            // interleaved: pair i is elements 2i, 2i + 1 of the 2V
            const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : V + i;
            const float xa = ia < V ? x[ia % V] : z[ia % V];
            const float xb = ib < V ? x[ib % V] : z[ib % V];
            e[ia] = fmaf(xa, cs[i], -xb * sn[i]);
            e[ib] = fmaf(xb, cs[i], xa * sn[i]);
          }
#pragma unroll
          for (int i = 0; i < V; ++i) {
            x[i] = e[i];
            z[i] = e[V + i];
          }
          a[u] = P::close(x);
          c[u] = P::close(z);
        }
        T* py = h + u < Hq ? yq + (h + u) * tq.ys.head : yk + (h + u - Hq) * tk.ys.head;
        *reinterpret_cast<Raw*>(py + off0) = a[u];
        *reinterpret_cast<Raw*>(py + off1) = c[u];
      }
    }
    if (h + U < h1) load(h + U);
  }
}

template <typename T, int V, bool kInterleaved>
cudaError_t launch_t(const RopeArgs& a) {
  constexpr int kThreads = kThreadsOf<V>;
  const int per_row = a.d / (2 * V);
  const int tpb = kThreads / per_row;                  // tokens per block
  const int tokens = a.B * a.N, H = a.Hq + a.Hkv;
  const long long blocks = (1LL * tokens + tpb - 1) / tpb;
  // Heads per thread, a power of two times the 4 that are in flight: as many as
  // leave eight blocks per SM, of which registers admit six at a time. (2 x 8192
  // tokens of 40 heads: 59.5 us with one to six left, 53.4 with 8, 53 with 12
  // to 32; the gradient of 2 x 4096 tokens of 20: 18.3, 17.3, 20.)
  const long long slots = 8LL * (device_sm_count() > 0 ? device_sm_count() : 1);
  int hpt = 4;
  while (hpt < H && blocks * ((H + 2 * hpt - 1) / (2 * hpt)) >= slots) hpt *= 2;
  const RopeTensor<T> tq{static_cast<const T*>(a.q), static_cast<T*>(a.q_out), a.qs, a.qos};
  const RopeTensor<T> tk{static_cast<const T*>(a.k), static_cast<T*>(a.k_out), a.ks, a.kos};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks), unsigned((H + hpt - 1) / hpt));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<T, V, kInterleaved>, tq, tk, a.positions,
                            a.pos_stride, a.inv_freq, tokens, a.N, a.Hq, H, a.d, a.rot, hpt,
                            a.magnitude, a.inverse);
}

template <typename T, int V>
cudaError_t launch_v(const RopeArgs& a) {
  const bool wide = a.d % (2 * V) == 0 && a.rot % (2 * V) == 0 &&
                    rows16(a.q, a.qs, a.B, a.Hq, a.N, sizeof(T)) &&
                    rows16(a.q_out, a.qos, a.B, a.Hq, a.N, sizeof(T)) &&
                    (a.Hkv == 0 || (rows16(a.k, a.ks, a.B, a.Hkv, a.N, sizeof(T)) &&
                                    rows16(a.k_out, a.kos, a.B, a.Hkv, a.N, sizeof(T))));
  if (wide) return a.interleaved ? launch_t<T, V, true>(a) : launch_t<T, V, false>(a);
  return a.interleaved ? launch_t<T, 1, true>(a) : launch_t<T, 1, false>(a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a) {
  return a.dt == ATTN_BF16 ? launch_v<__nv_bfloat16, 8>(a) : launch_v<float, 4>(a);
}

}  // namespace attn
