// Keys and values into the pages of a cache, with the rotation applied on the
// way (attn_cache_append, attn_cache_append4), and a 4-bit cache's rows back
// as bf16 (attn_cache_read4).
//
// Mathematics. Rotation: y_a = m (x_a cos - x_b sin), y_b = m (x_b cos +
// x_a sin) on pairs of the first rot_dim elements, in the arithmetic of rope.cu:
// a key appended here is bit for bit the key that attn_rope returns. 4 bits:
// per group of 32 elements s = bf16(max |y| / 6) and the e2m1 codes nearest to
// y / s, from the float32 values of the rotation (rounding them to bf16 first
// would add an error and save nothing). max |y| / 6 and y / s are correctly rounded:
// quotients of bf16 values fall on the borders between codes often enough that a
// reciprocal's last bit would decide. A group with a value that is not finite
// gets the scale NaN.
//
// Work. Memory bound: a token's rows are read once and written once. A thread
// owns two pieces of 8 adjacent elements (16 bytes of bf16) that hold whole pairs,
// D/16 lanes a row, through a run of heads of its token: query heads, then key
// heads, then value heads. The block's warps take different heads of the same
// tokens, whose angles they work out together. The pieces of a 4-bit group lie
// with neighbouring lanes; what does not fit that (rows or pairs off multiples of
// 16 bytes, pairs across halves of groups) goes element by element.
//
// Measured (GB300, of a plain copy's 6.7 TB/s): two prompts of 8192 tokens, 32 + 8 heads of
// 128, bf16, 62 us (0.97: memory); one token of 64 requests 3.5 us (3.1 in a CUDA graph: a
// launch and its chain length, table entry, angles, store). 2048 tokens of four requests
// into 4 bits 36 us (0.74): queries are bound by memory; keys and values, 19 us by
// themselves, by neither (issue slots and ALU at 45 %: each thread loads, then
// computes), and the first blocks take them; blocks that mix both took 44. The same
// element by element: rot_dim 32 of 128 88 us, of 64 50 (in pieces 19), bf16 pages 83 to 112
// (33). 8192 keys of four requests back from 4 bits 23.2 us (0.92: memory).

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "fp4.cuh"
#include "launchers.h"
#include "rope_math.cuh"

namespace attn {

ATTN_DEFINE_ERROR_WORD(take_error_cache_append)

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

// V adjacent elements as they are in memory, 16 bytes or 32.
template <typename T, int V> struct alignas(16) Piece {
  T x[V];
};
template <typename T, int V> ATTN_DEVINL void load_piece(Piece<T, V>& p, const T* src) {
#pragma unroll
  for (int i = 0; i < int(sizeof(p) / 16); ++i)
    reinterpret_cast<uint4*>(&p)[i] = reinterpret_cast<const uint4*>(src)[i];
}
template <typename T, int V> ATTN_DEVINL void store_piece(T* dst, const Piece<T, V>& p) {
#pragma unroll
  for (int i = 0; i < int(sizeof(p) / 16); ++i)
    reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(&p)[i];
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
  unsigned blocks, groups;                  // of tokens, of heads
  float magnitude;
};

template <typename T, bool k4> constexpr int kPiece = k4 ? 8 : 16 / int(sizeof(T));

// A token of a block: its request, its number among the request's new ones, and
// its place among the request's keys, -1 where it has none.
struct Token {
  int b, i, key;
};
template <typename T>
ATTN_DEVINL Token token_at(const AppendParams<T>& p, int token, bool report) {
  Token t{0, 0, -1};
  if (token < p.tokens) {
    t.b = token / p.N;
    t.i = token - t.b * p.N;
    const int n = p.lens[t.b], m = p.new_lens != nullptr ? p.new_lens[t.b] : p.N;
    if (n < 0 || n > p.max_pages * p.page_size || m < 0 || m > min(p.N, n)) {
      if (report && t.i == 0) attn_flag_error(kErrBadIndex);
    } else if (t.i < m) {
      t.key = n - m + t.i;
    }
  }
  return t;
}
// Its row of the pool for head 0, -1 where there is none.
template <typename T>
ATTN_DEVINL long long pool_row(const AppendParams<T>& p, const Token& t, bool report) {
  if (t.key < 0) return -1;
  const int page = p.table[1LL * t.b * p.max_pages + t.key / p.page_size];
  if (unsigned(page) < unsigned(p.num_pages))
    return 1LL * page * p.Hkv * p.page_size + t.key % p.page_size;
  if (report) attn_flag_error(kErrBadIndex);
  return -1;
}
template <typename T>
ATTN_DEVINL float2 token_turn(const AppendParams<T>& p, const Token& t, int pair) {
  float2 x = make_float2(1.f, 0.f);
  if (t.key >= 0)
    turn_cos_sin(p.positions != nullptr ? p.positions[t.b * p.pos_stride + t.i] : t.key,
                 p.inv_freq[pair], p.magnitude, x.x, x.y);
  return x;
}

// The largest magnitude, NaN if any is not a number.
ATTN_DEVINL float largest(float a, float b, float c) {
  float x;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(x) : "f"(a), "f"(b), "f"(c));
  return x;
}
template <int V> ATTN_DEVINL float largest(const float (&y)[V]) {
  float top = y[V - 1];
#pragma unroll
  for (int i = 0; i + 1 < V; i += 2) top = largest(top, y[i], y[i + 1]);
  return top;
}
// The largest of four neighbouring lanes (or of two).
template <int kLanes> ATTN_DEVINL float largest_of_lanes(float top) {
#pragma unroll
  for (int off = 1; off < kLanes; off *= 2) {
    const float other = __shfl_xor_sync(0xffffffffu, top, off);
    top = largest(top, other, other);
  }
  return top;
}
// Quotients below are correctly rounded without a division: with r = 1 / s rounded
// once and q = y·r, q + (y - q·s)·r rounds to y / s (Markstein 1990: the residual of a q
// within an ulp is exact in an FMA), as long as reciprocal and residual stay normal
// numbers. r itself comes from an approximation r0 within an ulp in the same way, r0 +
// (1 - r0·s)·r0, which fails for no s but significands of all ones, which no bf16
// value is.
//
// A group's scale from its largest magnitude.
ATTN_DEVINL __nv_bfloat16 scale_of(float top) {
  constexpr float kSixth = 1.f / 6.f;
  float q = top * kSixth;
  q = fmaf(fmaf(-q, 6.f, top), kSixth, q);
  if (top < 0x1p-90f) q = __fdiv_rn(top, 6.f);
  return __float2bfloat16_rn(top < INFINITY ? q : __uint_as_float(0x7fffffffu));
}
// Codes of 8 elements, two a byte; zeros where the scale is 0 or not a number.
template <int V> ATTN_DEVINL uint32_t codes_of(const float (&y)[V], __nv_bfloat16 scale) {
  static_assert(V == 8, "a piece of 4-bit rows is a quarter of a group");
  const float s = __bfloat162float(scale);
  f2 q[V / 2];
  if (s >= 0x1p-90f && s <= 0x1p90f) {
    float r0;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(s));
    const float r = fmaf(fmaf(-r0, s, 1.f), r0, r0);
    const f2 rr{r, r}, ss{-s, -s};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const f2 x{y[2 * i], y[2 * i + 1]}, first = mul2(x, rr);
      q[i] = fma2(fma2(first, ss, x), rr, first);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      q[i] = s > 0.f ? f2{__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s)}
                     : f2{0.f, 0.f};
  }
  return f32_to_e2m1x8(q);
}

// The codes x0, x1 of a lane's two pieces (8 elements a word, of which the low
// half belongs to one g, the high half to the next) into a row's bytes, in which
// the 16-bit halves of one g follow one another by group. Lane c of the row holds
//   interleaved:   elements 16c .. 16c + 15, both of group c / 2;
//   otherwise, of D = 64:  8 (c mod 4) .. of groups 0 and 1;
//              of D = 128: 8 (c mod 4) .. of groups c / 4 and c / 4 + 2, or
//                          (kNear) of groups 2 (c / 4) and 2 (c / 4) + 1.
// Every lane stores 8 bytes. All lanes of the warp call it.
template <int D, bool kInterleaved>
ATTN_DEVINL void store_codes(uint32_t x0, uint32_t x1, uint8_t* row, int c, bool near, bool live) {
  constexpr uint32_t kLow = 0x5410u, kHigh = 0x7632u;  // both words' low or high halves
  uint32_t w0, w1;
  int at;
  if constexpr (D == 64 && !kInterleaved) {
    w0 = __byte_perm(x0, x1, kLow);
    w1 = __byte_perm(x0, x1, kHigh);
    at = 8 * c;
  } else if constexpr (D == 64) {
    // (lanes c and c ^ 2 hold the groups of the same elements)
    const bool second = c / 2;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, second ? x0 : x1, 2);
    const uint32_t a = second ? y : x0, b = second ? x1 : y;
    w0 = __byte_perm(a, b, kLow);
    w1 = __byte_perm(a, b, kHigh);
    at = 16 * (c % 2) + 8 * second;
  } else if constexpr (!kInterleaved) {
    // lanes c and c ^ 4 hold all four groups of the same elements; the first
    // stores the halves of one g, the second those of the next
    const bool second = c / 4;
    const uint32_t y0 = __shfl_xor_sync(0xffffffffu, x0, 4),
                   y1 = __shfl_xor_sync(0xffffffffu, x1, 4);
    const uint32_t l0 = second ? y0 : x0, l1 = second ? y1 : x1, u0 = second ? x0 : y0,
                   u1 = second ? x1 : y1;
    const uint32_t pick = second ? kHigh : kLow;
    w0 = __byte_perm(l0, near ? l1 : u0, pick);
    w1 = __byte_perm(near ? u0 : l1, u1, pick);
    at = 16 * (c % 4) + 8 * second;
  } else {
    // lane c = 2 group + p holds the words 2p and 2p + 1 of its group; it stores
    // those halves (low: group even, high: odd) of all groups' word 2p + group / 2
    const int group = c / 2;
    const bool upper = group / 2, odd = group % 2;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, upper ? x0 : x1, 4);
    const uint32_t lo = upper ? y : x0, hi = upper ? x1 : y;     // groups group % 2, + 2
    const uint32_t own = __byte_perm(lo, hi, odd ? kHigh : kLow);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, __byte_perm(lo, hi, odd ? kLow : kHigh), 2);
    const uint32_t even_ = odd ? other : own, odd_ = odd ? own : other;
    w0 = __byte_perm(even_, odd_, kLow);
    w1 = __byte_perm(even_, odd_, kHigh);
    at = 16 * (2 * (c % 2) + upper) + 8 * odd;
  }
  if (live) *reinterpret_cast<uint2*>(row + at) = make_uint2(w0, w1);
}

// Rows in 16-byte pieces. Grid: groups of tokens (b·N + i), fastest, and runs of the
// Hq + 2 Hkv heads; with 4 bits the last heads, which take longest, first. A thread
// takes `hpt` heads, U in flight at a time, the first while the angles are worked
// out. kSpread: the block's warps take different heads of the same tokens and work out
// their angles together, one or two a thread; otherwise they take different tokens,
// every thread with its own angles.
template <typename T, int D, bool kInterleaved, bool k4, bool kSpread>
__global__ void __launch_bounds__(kThreads, k4 ? 5 : 6)
append_kernel(const __grid_constant__ AppendParams<T> p) {
  // elements of a piece: 16 bytes of them; with 4 bits a quarter of a group
  constexpr int V = kPiece<T, k4>, kLanes = D / (2 * V), U = V * sizeof(T) == 16 ? 4 : 2;
  constexpr int kTokens = (kSpread ? 32 : kThreads) / kLanes, kPairs = D / 2;
  __shared__ alignas(16) float2 turns[kSpread ? kTokens : 1][kPairs];
  pdl_launch_dependents();
  // (uniform, and known to be)
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) / 32, 0);
  const int c = threadIdx.x % kLanes, mine = (kSpread ? threadIdx.x % 32 : threadIdx.x) / kLanes;
  const int H = p.Hq + 2 * p.Hkv;
  const int group = int(blockIdx.x % p.blocks);
  const int run_of = int(blockIdx.x / p.blocks);       // (of heads, from the first: hb)
  const int hb = (k4 ? int(p.groups) - 1 - run_of : run_of) * p.hpt * (kSpread ? kWarps : 1);
  const int h0 = hb + (kSpread ? warp * p.hpt : 0), h1 = min(H, h0 + p.hpt);
  const int token0 = group * kTokens;
  const bool turned = c < p.rot / (2 * V);
  const int half = p.rot / 2;
  // where the lane's two pieces begin
  int off0, off1;
  if (kInterleaved) {
    off0 = 2 * V * c;
    off1 = off0 + V;
  } else if (turned) {
    off0 = V * c;
    off1 = off0 + half;
  } else {
    off0 = p.rot + V * (c - p.rot / (2 * V));
    off1 = off0 + (D - p.rot) / 2;
  }

  pdl_wait_primary();
  const Token own = token_at(p, token0 + mine, c == 0 && hb == 0 && (!kSpread || warp == 0));
  const bool live = own.key >= 0;
  // Padding is not loaded, but for small calls, which do not wait for the lengths.
  const bool fetch = kSpread || p.new_lens == nullptr ? token0 + mine < p.tokens : live;
  // the thread's heads of each kind: [first, end)
  const int q0 = min(h0, p.Hq), q1 = min(h1, p.Hq);
  const int k0 = max(h0 - p.Hq, 0), k1 = min(max(h1 - p.Hq, 0), p.Hkv);
  const int v0 = max(h0 - p.Hq - p.Hkv, 0), v1 = max(h1 - p.Hq - p.Hkv, 0);
  auto rows = [&](const T* x, const attn_strides& s, int head) {
    return x + own.b * s.batch + own.i * s.token + head * s.head;
  };
  Piece<T, V> x0[U], x1[U];
  auto load = [&](const T* x, long long step, int n) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < n && fetch) {
        load_piece(x0[u], x + u * step + off0);
        load_piece(x1[u], x + u * step + off1);
      }
  };
  if (q0 < q1)
    load(rows(p.q, p.qs, q0), p.qs.head, q1 - q0);
  else if (k0 < k1)
    load(rows(p.k, p.ks, k0), p.ks.head, k1 - k0);
  else
    load(rows(p.v, p.vs, v0), p.vs.head, v1 - v0);
  const long long row = h1 > max(h0, p.Hq) ? pool_row(p, own, c == 0) : -1;
  float cs[V], sn[V];
  if (p.rot > 0 && hb < p.Hq + p.Hkv) {                // (the same for the whole block)
    if constexpr (kSpread) {
      for (int a = threadIdx.x; a < kTokens * kPairs; a += kThreads)
        if (a % kPairs < half)
          turns[a / kPairs][a % kPairs] =
              token_turn(p, token_at(p, token0 + a / kPairs, false), a % kPairs);
      __syncthreads();
    }
    if (turned) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 y = kSpread ? turns[kSpread ? mine : 0][V * c + i] : token_turn(p, own, V * c + i);
        cs[i] = y.x;
        sn[i] = y.y;
      }
    }
  }
  // `n` heads of one kind from x on, `step` elements apart; `out`: where the first
  // of them goes, in rows of T `out_step` apart, or (4 bits) its codes and scales. The
  // first U are there already if `loaded`.
  enum { kCopied, kTurned, kCoded };                   // (values stay T; queries, keys; 4 bits)
  auto run = [&](auto kind, const T* x, long long step, T* out, long long out_step, int n,
                 bool loaded, bool stored, bool turn, uint8_t* codes, __nv_bfloat16* scales) {
    constexpr int kKind = decltype(kind)::value;
    if (!loaded) load(x, step, n);
    for (int h = 0; h < n; h += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= n) break;
        if (kKind != kCopied) {
          float y0[V], y1[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            y0[j] = to_f32(x0[u].x[j]);
            y1[j] = to_f32(x1[u].x[j]);
          }
          if (turn) {
            // pair i: elements 2i, 2i + 1 of both pieces, or i of either; two at a time
            auto first = [&](int i) -> float& {
              return !kInterleaved ? y0[i] : i < V / 2 ? y0[2 * i % V] : y1[2 * i % V];
            };
            auto second = [&](int i) -> float& {
              return !kInterleaved ? y1[i] : i < V / 2 ? y0[2 * i % V + 1] : y1[2 * i % V + 1];
            };
#pragma unroll
            for (int i = 0; i < V; i += 2) {
              const f2 a{first(i), first(i + 1)}, b{second(i), second(i + 1)}, c2{cs[i], cs[i + 1]},
                  s2{sn[i], sn[i + 1]};
              const f2 ya = fma2(a, c2, mul2(b, {-s2.x, -s2.y})), yb = fma2(b, c2, mul2(a, s2));
              first(i) = ya.x;
              first(i + 1) = ya.y;
              second(i) = yb.x;
              second(i + 1) = yb.y;
            }
          }
          if constexpr (kKind == kCoded) {
            const float top0 = largest(y0), top1 = largest(y1);
            __nv_bfloat16 s0, s1;
            if constexpr (kInterleaved) {
              s0 = s1 = scale_of(largest_of_lanes<2>(largest(top0, top1, top1)));
            } else {
              s0 = scale_of(largest_of_lanes<4>(top0));
              s1 = scale_of(largest_of_lanes<4>(top1));
            }
            store_codes<D, kInterleaved>(codes_of(y0, s0), codes_of(y1, s1), codes, c,
                                         p.rot == D / 2, stored);
            if (stored && c % (kInterleaved ? 2 : 4) == 0) {
              scales[off0 / 32] = s0;
              if (!kInterleaved) scales[off1 / 32] = s1;
            }
            codes += p.page_size * (D / 2);
            scales += p.page_size * (D / 32);
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              x0[u].x[j] = from_f32<T>(y0[j]);
              x1[u].x[j] = from_f32<T>(y1[j]);
            }
          }
        }
        if (kKind != kCoded && stored) {
          store_piece(out + u * out_step + off0, x0[u]);
          store_piece(out + u * out_step + off1, x1[u]);
        }
      }
      x += U * step;
      out += U * out_step;
      if (h + U < n) load(x, step, n - h - U);
    }
  };
  if (q0 < q1)
    run(std::integral_constant<int, kTurned>{}, rows(p.q, p.qs, q0), p.qs.head,
        p.q_out + own.b * p.qos.batch + own.i * p.qos.token + q0 * p.qos.head, p.qos.head,
        q1 - q0, true, live, turned, nullptr, nullptr);
  const long long head_rows = 1LL * p.page_size * D;
  if constexpr (k4) {
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {             // (one copy of the code for both)
      const int first = kind ? v0 : k0, end = kind ? v1 : k1;
      const long long to = row + 1LL * first * p.page_size;
      if (first < end)
        run(std::integral_constant<int, kCoded>{},
            kind ? rows(p.v, p.vs, first) : rows(p.k, p.ks, first),
            kind ? p.vs.head : p.ks.head, static_cast<T*>(nullptr), 0, end - first,
            q0 >= q1 && (kind == 0 || k0 >= k1), row >= 0, turned && kind == 0,
            static_cast<uint8_t*>(kind ? p.v_pool : p.k_pool) + to * (D / 2),
            (kind ? p.v_scales : p.k_scales) + to * (D / 32));
    }
  } else {
    if (k0 < k1)
      run(std::integral_constant<int, kTurned>{}, rows(p.k, p.ks, k0), p.ks.head,
          static_cast<T*>(p.k_pool) + row * D + k0 * head_rows, head_rows, k1 - k0, q0 >= q1,
          row >= 0, turned, nullptr, nullptr);
    if (v0 < v1)
      run(std::integral_constant<int, kCopied>{}, rows(p.v, p.vs, v0), p.vs.head,
          static_cast<T*>(p.v_pool) + row * D + v0 * head_rows, head_rows, v1 - v0,
          q0 >= q1 && k0 >= k1, row >= 0, false, nullptr, nullptr);
  }
}

// The same element by element: any alignment, any rot_dim. A thread owns 8
// adjacent elements, D/8 lanes a row, and reads the partners of its pairs too; the
// rows of a warp are whole, so that rows turned in place are read by all their
// lanes before any is written.
template <typename T, int D, bool k4>
__global__ void __launch_bounds__(kThreads)
append_any_kernel(const __grid_constant__ AppendParams<T> p, int interleaved) {
  constexpr int kLanes = D / 8, kTokens = 32 / kLanes, kPairs = D / 2;
  __shared__ float2 turns[kTokens][kPairs];
  pdl_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % kLanes, e0 = 8 * l;
  const int mine = lane / kLanes, token0 = int(blockIdx.x % p.blocks) * kTokens, half = p.rot / 2;
  const int H = p.Hq + 2 * p.Hkv, hb = int(blockIdx.x / p.blocks) * p.hpt * kWarps;
  const int h0 = hb + warp * p.hpt, h1 = min(H, h0 + p.hpt);
  pdl_wait_primary();
  const Token own = token_at(p, token0 + mine, l == 0 && hb == 0 && warp == 0);
  const bool live = own.key >= 0;
  const long long row = h1 > max(h0, p.Hq) ? pool_row(p, own, l == 0) : -1;
  for (int a = threadIdx.x; a < kTokens * kPairs; a += kThreads)
    if (a % kPairs < half)
      turns[a / kPairs][a % kPairs] =
          token_turn(p, token_at(p, token0 + a / kPairs, false), a % kPairs);
  __syncthreads();
  for (int at = h0; at < h1; ++at) {
    const bool is_q = at < p.Hq, is_k = at < p.Hq + p.Hkv;
    const int head = is_q ? at : is_k ? at - p.Hq : at - p.Hq - p.Hkv;
    const attn_strides& s = is_q ? p.qs : is_k ? p.ks : p.vs;
    const T* x = (is_q ? p.q : is_k ? p.k : p.v) + own.b * s.batch + own.i * s.token +
                 head * s.head;
    float y[8] = {};
    if (live)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j;
        y[j] = to_f32(x[e]);
        if (is_k && e < p.rot) {
          const bool second = interleaved ? e % 2 : e >= half;
          const int mate = interleaved ? e ^ 1 : second ? e - half : e + half;
          const float2 t = turns[mine][interleaved ? e / 2 : second ? e - half : e];
          const float z = to_f32(x[mate]) * t.y;
          y[j] = fmaf(y[j], t.x, second ? z : -z);
        }
      }
    __syncwarp();
    const long long to = row + 1LL * head * p.page_size;
    if (k4 && !is_q) {
      const __nv_bfloat16 scale = scale_of(largest_of_lanes<4>(largest(y)));
      const uint32_t w = codes_of(y, scale);
      if (row >= 0) {
        const int c = l / 4, t = l % 4;                // group, and which 8 of it
        uint16_t* codes = reinterpret_cast<uint16_t*>(
            static_cast<uint8_t*>(is_k ? p.k_pool : p.v_pool) + to * (D / 2));
        codes[2 * t * (D / 32) + c] = uint16_t(w);
        codes[(2 * t + 1) * (D / 32) + c] = uint16_t(w >> 16);
        if (t == 0) (is_k ? p.k_scales : p.v_scales)[to * (D / 32) + c] = scale;
      }
    } else if (is_q ? live : row >= 0) {
      T* out = is_q ? p.q_out + own.b * p.qos.batch + own.i * p.qos.token + head * p.qos.head
                    : static_cast<T*>(is_k ? p.k_pool : p.v_pool) + to * D;
#pragma unroll
      for (int j = 0; j < 8; ++j) out[e0 + j] = from_f32<T>(y[j]);
    }
  }
}

// Rows of a 4-bit cache as bf16: four lanes a row, each 8 elements of every
// group, kRows rows a thread. Grid: x over runs of rows, y over (request, KV
// head), z over K and V.
constexpr int kReadRows = 4;
template <int D>
__global__ void __launch_bounds__(kThreads)
read4_kernel(const uint8_t* k_codes, const __nv_bfloat16* k_scales, const uint8_t* v_codes,
             const __nv_bfloat16* v_scales, const int* table, const int* lens,
             __nv_bfloat16* k_out, __nv_bfloat16* v_out, int Hkv,
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

void dependent_launch(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, dim3 grid, int threads,
                      cudaStream_t stream) {
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

template <typename T, int D, bool k4>
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
  // Rows in 16-byte pieces where they and their pairs lie so; with 4 bits a pair's
  // pieces have to be whole quarters of groups, too.
  constexpr int V = kPiece<T, k4>;
  const bool wide = a.rot % (k4 && !a.interleaved ? 64 : 2 * V) == 0 &&
                    (a.Hq == 0 || (rows16(a.q, a.qs, a.B, a.Hq, a.N, sizeof(T)) &&
                                   rows16(a.q_out, a.qos, a.B, a.Hq, a.N, sizeof(T)))) &&
                    rows16(a.k, a.ks, a.B, a.Hkv, a.N, sizeof(T)) &&
                    rows16(a.v, a.vs, a.B, a.Hkv, a.N, sizeof(T));
  // Many tokens: 8 heads a thread (4 bits: 16, so that angles are worked out less
  // often), where that gives eight blocks an SM. (16384 tokens in bf16: 75 us at 4, 62 at 8
  // and 16, 63 at 24; 8192 in 4 bits: 42 at 6, 36.9 at 8, 36.0 at 16, 38.7 at 48.) Fewer: the
  // warps spread over the heads, with as many heads each as leave four blocks an SM. (48
  // heads of 64, 1024, 2048, 4096 tokens: spread 3.1, 5.8, 9.0, 18.4 us, otherwise 4.5, 8.3,
  // 9.0, 15.5; in 4 bits 3.2, 6.7, 10.6, 19.6 and 6.8, 8.3, 10.7, 18.3. 512 tokens at two,
  // four, eight blocks: 5.2, 4.7, 6.6.)
  const int H = a.Hq + 2 * a.Hkv, sms = std::max(1, device_sm_count());
  const int rows = 64 * V / D;                         // of a warp
  const long long plain = (1LL * p.tokens + kWarps * rows - 1) / (kWarps * rows);
  const bool spread = !wide || plain * ((H + 7) / 8) < 8LL * sms;
  const int tokens = !wide ? 256 / D : spread ? rows : kWarps * rows;   // of a block
  const long long blocks = (1LL * p.tokens + tokens - 1) / tokens;
  p.hpt = spread ? 4 : k4 && plain * ((H + 15) / 16) >= 8LL * sms ? 16 : 8;
  if (spread)
    while (p.hpt > 1 && blocks * ((H + kWarps * p.hpt - 1) / (kWarps * p.hpt)) < 4LL * sms)
      p.hpt /= 2;
  const int heads = p.hpt * (spread ? kWarps : 1);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  p.blocks = unsigned(blocks);
  p.groups = unsigned((H + heads - 1) / heads);
  if (blocks * p.groups > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  dependent_launch(cfg, attr, dim3(unsigned(blocks * p.groups)), kThreads, a.stream);
  if (!wide) return cudaLaunchKernelEx(&cfg, append_any_kernel<T, D, k4>, p, a.interleaved);
  if (spread)
    return a.interleaved ? cudaLaunchKernelEx(&cfg, append_kernel<T, D, true, k4, true>, p)
                         : cudaLaunchKernelEx(&cfg, append_kernel<T, D, false, k4, true>, p);
  return a.interleaved ? cudaLaunchKernelEx(&cfg, append_kernel<T, D, true, k4, false>, p)
                       : cudaLaunchKernelEx(&cfg, append_kernel<T, D, false, k4, false>, p);
}

template <typename T> cudaError_t launch_type(const AppendArgs& a) {
  const bool four = a.k_scales != nullptr;
  if (a.d == 64) return four ? launch_t<T, 64, true>(a) : launch_t<T, 64, false>(a);
  return four ? launch_t<T, 128, true>(a) : launch_t<T, 128, false>(a);
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
                   kThreads, a.stream);
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
