// Keys and values into the pages of a cache, with the rotation applied on the
// way (attn_cache_append, attn_cache_append4), and a 4-bit cache's rows back
// as bf16 (attn_cache_read4).
//
// Mathematics. Rotation: y_a = m (x_a cos - x_b sin), y_b = m (x_b cos +
// x_a sin) on pairs of the first rot_dim elements, in the arithmetic of rope.cu:
// a key appended here is bit for bit the key that attn_rope returns. 4 bits:
// per group of 32 elements s = bf16(max |y| / 6) and the e2m1 codes nearest to
// y / s, from the float32 values of the rotation (rounding them to bf16 first
// would add an error and save nothing). max |y| / 6 and y / s are IEEE divisions:
// quotients of bf16 values fall on the borders between codes often enough that a
// reciprocal's last bit would decide. A group with a value that is not finite
// gets the scale NaN.
//
// Work. Memory bound: a token's rows are read once and written once. A thread
// owns 8 adjacent elements of a row (16 bytes of bf16), D/8 lanes a row, through
// a run of heads of its token: query heads, then key heads, then value heads.
// It loads its piece and, where pairs lie rot_dim/2 apart, the piece of the
// partners too: twice the loads of a thread that owns whole pairs (from L1, the
// same bytes from memory), and the four lanes of a 4-bit group are neighbours
// whatever the layout of the pairs. The rows of a warp are whole, so rows turned
// in place are read by all their lanes before any is written (__syncwarp).

#include "common.cuh"
#include "fp4.cuh"
#include "launchers.h"
#include "rope_math.cuh"

namespace attn {

ATTN_DEFINE_ERROR_WORD(take_error_cache_append)

namespace {

constexpr int kThreads = 128;

// 8 adjacent elements as they are in memory.
template <typename T> struct alignas(16) Piece {
  T x[8];
};
template <typename T, bool kWide> ATTN_DEVINL void load_piece(Piece<T>& p, const T* src) {
  if constexpr (kWide) {
#pragma unroll
    for (int i = 0; i < int(sizeof(p) / 16); ++i)
      reinterpret_cast<uint4*>(&p)[i] = reinterpret_cast<const uint4*>(src)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p.x[i] = src[i];
  }
}
template <typename T, bool kWide> ATTN_DEVINL void store_piece(T* dst, const Piece<T>& p) {
  if constexpr (kWide) {
#pragma unroll
    for (int i = 0; i < int(sizeof(p) / 16); ++i)
      reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(&p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i] = p.x[i];
  }
}

template <typename T> struct AppendParams {
  const T *q, *k, *v;
  T* q_out;
  attn_strides qs, qos, ks, vs;
  void *k_pool, *v_pool;                    // T rows, or codes
  __nv_bfloat16 *k_scales, *v_scales;       // 4 bits
  const int *table, *lens, *new_lens, *positions;
  long long pos_stride;
  const double* inv_freq;
  int tokens, N, Hq, Hkv, num_pages, page_size, max_pages, rot, hpt;
  float magnitude;
};

// Codes and scale of the 8 elements y of a lane, whose group's other 24 are
// those of the lanes around it (l ^ 1, l ^ 2, l ^ 3), into a row's D/2 code bytes
// and D/32 scales. All lanes of the warp call it; those of rows that are not
// `live` write nothing.
template <int D>
ATTN_DEVINL void store_row4(const float (&y)[8], uint8_t* codes, __nv_bfloat16* scales, int l,
                            bool live) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // (as integers, infinities and NaN are above every finite value)
  const bool finite = top < 0x7f800000u;
  const __nv_bfloat16 s = __float2bfloat16_rn(
      finite ? __fdiv_rn(__uint_as_float(top), 6.f) : __uint_as_float(0x7fffffffu));
  const float sf = __bfloat162float(s);
  uint32_t x = 0;
  if (finite && sf != 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x |= f32_to_e2m1x2(__fdiv_rn(y[2 * i], sf), __fdiv_rn(y[2 * i + 1], sf)) << (8 * i);
  }
  // The lane's low two bytes are of g = 2t, its high two of 2t + 1, of group c.
  // Lane c of the D/32 that share t writes the c-th word of their D/8 bytes.
  constexpr int kWords = D / 64;                       // words of one g
  const int c = l / 4, t = l % 4, lane = threadIdx.x & 31;
  const int src = (lane & ~(D / 8 - 1)) + 8 * (c % kWords) + t;
  const uint32_t a = __shfl_sync(0xffffffffu, x, src), b = __shfl_sync(0xffffffffu, x, src + 4);
  const uint32_t word = c / kWords ? __byte_perm(a, b, 0x7632) : __byte_perm(a, b, 0x5410);
  if (!live) return;
  *reinterpret_cast<uint32_t*>(codes + t * (D / 8) + 4 * c) = word;
  if (t == 0) scales[c] = s;
}

// Grid: x over groups of tokens (b·N + i), y over runs of `hpt` of the
// Hq + 2 Hkv heads. U heads are in flight at a time.
template <typename T, int D, bool kWide, bool kInterleaved, bool k4>
__global__ void __launch_bounds__(kThreads)
append_kernel(const __grid_constant__ AppendParams<T> p) {
  constexpr int kLanes = D / 8, U = sizeof(T) == 2 ? 4 : 2;
  constexpr int kAngles = kInterleaved ? 4 : 8;        // of the 8 elements
  pdl_launch_dependents();
  const int l = threadIdx.x % kLanes, e0 = 8 * l;
  const int token = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const bool in_grid = token < p.tokens;
  const int b = in_grid ? token / p.N : 0, i = in_grid ? token % p.N : 0;
  const int H = p.Hq + 2 * p.Hkv;
  const int h0 = int(blockIdx.y) * p.hpt, h1 = min(H, h0 + p.hpt);
  // with rows that move in 16-byte pieces a piece is turned as a whole or not
  const bool turned = e0 < p.rot;
  const int half = p.rot / 2;
  const int mate = kInterleaved || !turned ? 0 : e0 < half ? half : -half;
  const T* xq = p.q + b * p.qs.batch + i * p.qs.token + e0;
  const T* xk = p.k + b * p.ks.batch + i * p.ks.token + e0;
  const T* xv = p.v + b * p.vs.batch + i * p.vs.token + e0;
  T* yq = p.q_out + b * p.qos.batch + i * p.qos.token + e0;

  pdl_wait_primary();
  Piece<T> own[U], other[U];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = h + u;
      if (at >= h1 || !in_grid) continue;
      const T* x = at < p.Hq           ? xq + at * p.qs.head
                   : at < p.Hq + p.Hkv ? xk + (at - p.Hq) * p.ks.head
                                       : xv + (at - p.Hq - p.Hkv) * p.vs.head;
      load_piece<T, kWide>(own[u], x);
      if (!kInterleaved && turned && at < p.Hq + p.Hkv) {
        if constexpr (kWide) {
          load_piece<T, true>(other[u], x + mate);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e0 + j < p.rot) other[u].x[j] = x[e0 + j < half ? j + half : j - half];
        }
      }
    }
  };
  load(h0);

  // the token's row of the cache
  int row_of = -1;                                     // its position among the request's keys
  if (in_grid) {
    const int n = p.lens[b], m = p.new_lens != nullptr ? p.new_lens[b] : p.N;
    if (n < 0 || n > p.max_pages * p.page_size || m < 0 || m > min(p.N, n)) {
      if (l == 0 && h0 == 0 && i == 0) attn_flag_error(kErrBadIndex);
    } else if (i < m) {
      row_of = n - m + i;
    }
  }
  const bool live = row_of >= 0;
  long long row = -1;                                  // of the pool, head 0
  if (live && h1 > p.Hq) {
    const int page = p.table[1LL * b * p.max_pages + row_of / p.page_size];
    if (unsigned(page) < unsigned(p.num_pages))
      row = 1LL * page * p.Hkv * p.page_size + row_of % p.page_size;
    else if (l == 0)
      attn_flag_error(kErrBadIndex);
  }
  float cs[kAngles], sn[kAngles];
  if (turned && live && h0 < p.Hq + p.Hkv) {
    const long long at = p.positions != nullptr ? p.positions[b * p.pos_stride + i] : row_of;
#pragma unroll
    for (int j = 0; j < kAngles; ++j) {
      const int e = kInterleaved ? e0 + 2 * j : e0 + j;
      if (kWide || e < p.rot) {
        turn_cos_sin(at, p.inv_freq[kInterleaved ? e / 2 : e < half ? e : e - half],
                     p.magnitude, cs[j], sn[j]);
        if (!kInterleaved && e < half) sn[j] = -sn[j];
      }
    }
  }
  for (int h = h0; h < h1; h += U) {
    // every lane of a row has read what a row turned in place overwrites
    __syncwarp();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = h + u;
      if (at >= h1) break;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = to_f32(own[u].x[j]);
      if (turned && at < p.Hq + p.Hkv) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!kWide && e0 + j >= p.rot) continue;
          const float x = to_f32(own[u].x[j]);
          if constexpr (kInterleaved) {
            const float z = to_f32(own[u].x[j ^ 1]) * sn[j / 2];
            y[j] = fmaf(x, cs[j / 2], j % 2 ? z : -z);
          } else {
            y[j] = fmaf(x, cs[j], to_f32(other[u].x[j]) * sn[j]);
          }
        }
      }
      const bool is_q = at < p.Hq, is_k = at < p.Hq + p.Hkv;
      const int head = is_k ? at - p.Hq : at - p.Hq - p.Hkv;
      const long long to = row + 1LL * head * p.page_size;
      if (k4 && !is_q) {
        uint8_t* codes = static_cast<uint8_t*>(is_k ? p.k_pool : p.v_pool);
        __nv_bfloat16* scales = is_k ? p.k_scales : p.v_scales;
        store_row4<D>(y, codes + to * (D / 2), scales + to * (D / 32), l, row >= 0);
        continue;
      }
      Piece<T> out;
#pragma unroll
      for (int j = 0; j < 8; ++j) out.x[j] = from_f32<T>(y[j]);
      if (is_q) {
        if (live) store_piece<T, kWide>(yq + at * p.qos.head, out);
      } else if (row >= 0) {
        T* pool = static_cast<T*>(is_k ? p.k_pool : p.v_pool);
        store_piece<T, true>(pool + to * D + e0, out);
      }
    }
    if (h + U < h1) load(h + U);
  }
}

// Rows of a 4-bit cache as bf16: four lanes a row, each 8 elements of every
// group, kRows rows a thread. Grid: x over runs of rows, y over (request, KV
// head), z over K and V.
constexpr int kReadRows = 4;
template <int D>
__global__ void __launch_bounds__(kThreads)
read4_kernel(const uint8_t* __restrict__ k_codes, const __nv_bfloat16* __restrict__ k_scales,
             const uint8_t* __restrict__ v_codes, const __nv_bfloat16* __restrict__ v_scales,
             const int* __restrict__ table, const int* __restrict__ lens,
             __nv_bfloat16* __restrict__ k_out, __nv_bfloat16* __restrict__ v_out, int Hkv,
             int num_pages, int page_size, int max_pages, int L) {
  constexpr int kRowsPerStep = kThreads / 4, kGroups = D / 32;
  using Codes = typename std::conditional<D == 128, uint4, uint2>::type;
  using Scales = typename std::conditional<D == 128, uint2, uint32_t>::type;
  pdl_launch_dependents();
  pdl_wait_primary();
  const int b = blockIdx.y / Hkv, h = blockIdx.y % Hkv, t = threadIdx.x % 4;
  int n = lens[b];
  if (n < 0 || n > min(L, max_pages * page_size)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) attn_flag_error(kErrBadIndex);
    n = 0;
  }
  const int j0 = blockIdx.x * (kRowsPerStep * kReadRows) + threadIdx.x / 4;
  if (j0 >= n) return;
  const uint8_t* codes = blockIdx.z ? v_codes : k_codes;
  const __nv_bfloat16* scales = blockIdx.z ? v_scales : k_scales;
  __nv_bfloat16* out = (blockIdx.z ? v_out : k_out) + 1LL * blockIdx.y * L * D;
  long long row[kReadRows];
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const int j = j0 + u * kRowsPerStep;
    row[u] = -1;
    if (j < n) {
      const int page = table[1LL * b * max_pages + j / page_size];
      if (unsigned(page) < unsigned(num_pages))
        row[u] = (1LL * page * Hkv + h) * page_size + j % page_size;
      else
        attn_flag_error(kErrBadIndex);
    }
  }
  Codes w[kReadRows];
  Scales s[kReadRows];
#pragma unroll
  for (int u = 0; u < kReadRows; ++u)
    if (row[u] >= 0) {
      w[u] = *reinterpret_cast<const Codes*>(codes + row[u] * (D / 2) + t * (D / 8));
      s[u] = *reinterpret_cast<const Scales*>(scales + row[u] * (D / 32));
    }
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    if (row[u] < 0) continue;
    const uint32_t* cw = reinterpret_cast<const uint32_t*>(&w[u]);
    const uint32_t* sw = reinterpret_cast<const uint32_t*>(&s[u]);
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      const float scale = c % 2 ? bf16hi(sw[c / 2]) : bf16lo(sw[c / 2]);
      const uint32_t lo = cw[c / 2], hi = cw[D / 64 + c / 2];
      uint32_t f[4], o[4];
      f[0] = c % 2 ? e2m1x2_to_f16x2<2>(lo) : e2m1x2_to_f16x2<0>(lo);
      f[1] = c % 2 ? e2m1x2_to_f16x2<3>(lo) : e2m1x2_to_f16x2<1>(lo);
      f[2] = c % 2 ? e2m1x2_to_f16x2<2>(hi) : e2m1x2_to_f16x2<0>(hi);
      f[3] = c % 2 ? e2m1x2_to_f16x2<3>(hi) : e2m1x2_to_f16x2<1>(hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        o[i] = pack_bf16x2(x.x * scale, x.y * scale);
      }
      *reinterpret_cast<uint4*>(out + 1LL * (j0 + u * kRowsPerStep) * D + 32 * c + 8 * t) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

void dependent_launch(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, dim3 grid,
                      cudaStream_t stream) {
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

template <typename T, int D, bool kWide, bool kInterleaved, bool k4>
cudaError_t launch_t(const AppendArgs& a) {
  AppendParams<T> p{};
  p.q = static_cast<const T*>(a.q);
  p.k = static_cast<const T*>(a.k);
  p.v = static_cast<const T*>(a.v);
  p.q_out = static_cast<T*>(a.q_out);
  p.qs = a.qs;
  p.qos = a.qos;
  p.ks = a.ks;
  p.vs = a.vs;
  p.k_pool = a.k_pool;
  p.v_pool = a.v_pool;
  p.k_scales = static_cast<__nv_bfloat16*>(a.k_scales);
  p.v_scales = static_cast<__nv_bfloat16*>(a.v_scales);
  p.table = a.block_table;
  p.lens = a.seq_lens;
  p.new_lens = a.new_lens;
  p.positions = a.positions;
  p.pos_stride = a.pos_stride;
  p.inv_freq = a.inv_freq;
  p.tokens = a.B * a.N;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.rot = a.rot;
  p.magnitude = a.magnitude;
  const int tpb = kThreads / (D / 8), H = a.Hq + 2 * a.Hkv;
  const long long blocks = (1LL * p.tokens + tpb - 1) / tpb;
  // Heads per thread, a power of two times the 4 that are in flight: as many as
  // leave eight blocks per SM (as in rope.cu).
  const long long slots = 8LL * (device_sm_count() > 0 ? device_sm_count() : 1);
  p.hpt = 4;
  while (p.hpt < H && blocks * ((H + 2 * p.hpt - 1) / (2 * p.hpt)) >= slots) p.hpt *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  dependent_launch(cfg, attr, dim3(unsigned(blocks), unsigned((H + p.hpt - 1) / p.hpt)), a.stream);
  return cudaLaunchKernelEx(&cfg, append_kernel<T, D, kWide, kInterleaved, k4>, p);
}

template <typename T, int D, bool k4>
cudaError_t launch_d(const AppendArgs& a) {
  const bool wide = a.rot % (a.interleaved ? 8 : 16) == 0 &&
                    (a.Hq == 0 || (rows16(a.q, a.qs, a.B, a.Hq, a.N, sizeof(T)) &&
                                   rows16(a.q_out, a.qos, a.B, a.Hq, a.N, sizeof(T)))) &&
                    rows16(a.k, a.ks, a.B, a.Hkv, a.N, sizeof(T)) &&
                    rows16(a.v, a.vs, a.B, a.Hkv, a.N, sizeof(T));
  if (wide)
    return a.interleaved ? launch_t<T, D, true, true, k4>(a) : launch_t<T, D, true, false, k4>(a);
  return a.interleaved ? launch_t<T, D, false, true, k4>(a) : launch_t<T, D, false, false, k4>(a);
}

template <typename T> cudaError_t launch_type(const AppendArgs& a) {
  const bool four = a.k_scales != nullptr;
  if (a.d == 64) return four ? launch_d<T, 64, true>(a) : launch_d<T, 64, false>(a);
  return four ? launch_d<T, 128, true>(a) : launch_d<T, 128, false>(a);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a) {
  return a.dt == ATTN_BF16 ? launch_type<__nv_bfloat16>(a) : launch_type<float>(a);
}

cudaError_t launch_cache_read4(const Read4Args& a) {
  constexpr int kRowsPerBlock = kThreads / 4 * kReadRows;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  dependent_launch(cfg, attr,
                   dim3(unsigned((a.L + kRowsPerBlock - 1) / kRowsPerBlock),
                        unsigned(a.B * a.Hkv), 2),
                   a.stream);
  auto run = [&](auto* kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint8_t*>(a.k_codes),
                              static_cast<const __nv_bfloat16*>(a.k_scales),
                              static_cast<const uint8_t*>(a.v_codes),
                              static_cast<const __nv_bfloat16*>(a.v_scales), a.block_table,
                              a.seq_lens, static_cast<__nv_bfloat16*>(a.k_out),
                              static_cast<__nv_bfloat16*>(a.v_out), a.Hkv, a.num_pages,
                              a.page_size, a.max_pages, a.L);
  };
  return a.d == 64 ? run(read4_kernel<64>) : run(read4_kernel<128>);
}

}  // namespace attn
