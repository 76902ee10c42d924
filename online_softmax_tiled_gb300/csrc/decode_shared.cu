// Decode of a batch whose requests share long prefixes: the prefix part and
// the merge (the requests' own keys run the paged split kernel of decode.cu).
//
// Mathematics. Softmax over [prefix keys ; own keys] splits exactly: any set
// of keys leaves (o, m, l) = (Σ e^(s - m) v, max s, Σ e^(s - m)) and sets are
// merged on a common maximum (ML notes, haolingpu.github.io, split-K notes).
// The prefix's keys are the same for all its requests, so their part is a
// small attention problem of its own: the query rows of a KV head are those
// of all requests of the prefix times the G heads of the group, against one
// K and V. Read once for all instead of once per request, it stops being
// bound by memory: R rows do 4·d·R flops per 4·d bytes of K and V, R per
// byte, and belong on the tensor cores.
//
// Prefix kernel. One CTA owns (prefix, KV head, run of query rows, chunk of
// keys) and runs the tensor-core forward's scheme: S = Q Kᵀ and Õ += P̃ V as
// tcgen05.mma with accumulators in tensor memory, one softmax warpgroup per
// 128 accumulator rows, K and V tiles of 128 keys through a ring filled by
// TMA, the reference maximum moved only when a row's maximum grows by more
// than 2^8. P̃ is rounded to bf16 for the P̃ V product, as in the forward
// (relative 2^-8 per weight at most, averaging out over the keys); sums, maxima
// and the partial outputs stay float32.
//   kPair (more than 128 rows a prefix on average): the two warpgroups hold
//     rows 0..127 and 128..255, and every K and V tile feeds both.
//   otherwise: both hold the same 128 rows and take alternate key tiles, so
//     one's softmax overlaps the other's products and a third stage of K and
//     V is loading; they are merged at the end through shared memory.
// Key tiles come from pages by one TMA copy per page piece (128 rows, or the
// largest power of two that divides the page size) that takes whole rows: a
// copy costs about 100 cycles to issue, and 16-key pages need eight a tile as
// it is. Value rows past the
// prefix's end are zeroed in shared memory before the product (a page's
// unused rows may hold anything, and 0 · NaN is NaN).
//
// Measured (32 heads on 8, d = 128): 64 requests behind 8192 keys, 0 to 1024
// of their own each, 16-key pages: 53 us, 168 MB of K and V, of which the own
// keys' 134 MB alone take 40 (short pieces of keys: a CTA's start-up, not the
// bandwidth, bounds them) and the prefix's tiles 43 on 32 SMs beside them.
// 96 requests behind three documents of 16384 to 32768 keys, 64-key pages:
// 113 us, 438 MB. Four requests behind 500 keys: 12.7 us, three launches.
// (With P̃ as one bf16 part: 49, 92 and 11.8.) A key tile takes 1.15 us, 2.2
// where it feeds 256 rows.
// Pairs against single runs at 8192 keys: 256 rows 53 and 55 us, 512 rows 91
// and 93, 128 rows 41 and 34; over three prefixes of 128 rows on average 127
// and 117. The same calls with a prefix_table 16 times as wide take 58, 119 and
// 13 (cut by what the table holds: 162, 317 and 15).
//
// Order. The three kernels of a call are launched as programmatic
// dependents. The prefix kernel lets the split kernel start once what
// precedes the call is complete; the split kernel does not wait for the
// prefix kernel but for its last CTA, so that its CTAs fill the SMs the
// prefix leaves idle; the merge waits for both.

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "launchers.h"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace attn {

ATTN_DEFINE_ERROR_WORD(take_error_decode_shared)

namespace {

constexpr int kBM = 128;             // query rows per accumulator tile
constexpr int kBN = 128;             // keys per K/V tile
constexpr int kThreads = 384;        // TMA warp, MMA warp, two idle, two softmax warpgroups
constexpr int kPagesCached = 256;    // table entries of a chunk kept in shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;

template <int D, bool kPair>
struct Cfg {
  static constexpr int kAtoms = D / 64;                // 128-byte swizzle atoms per row
  static constexpr int kTileBytes = kBM * D * 2;
  static constexpr int kQTiles = kPair ? 2 : 1;
  static constexpr int kStages = (kPair ? 2 : 3) * (128 / D);
  static constexpr int kKOff = kQTiles * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kSmemBytes = kVOff + kStages * kTileBytes;
  static constexpr int kDynSmem = kSmemBytes + 1024;   // slack for 1024-byte alignment
  static constexpr uint32_t kColS = 0, kColO = 256;    // S0, S1 | O0, O1
  // output rows staged for coalesced stores: D floats and 4 of padding, so
  // that 8 lanes' 16-byte pieces of one column cover all banks
  static constexpr int kStagePitch = D + 4;
  // behind the staged rows: m and l of both warpgroups' rows (not kPair)
  static constexpr int kMlOff = 2 * kBM * kStagePitch * 4;
  static_assert(kMlOff + 4 * kBM * 4 <= kSmemBytes, "staging fits Q and the ring");
};

struct Bars {
  uint64_t q_full;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t mma_drain;
  uint32_t tmem_base;
  int abort;
  int unit[5];               // prefix, first request, requests of this CTA's rows; keys, chunk
};

struct PrefixArgs {
  const int* prefix_table;
  const int* prefix_lens;
  const int* prefix_start;
  float* o_part;
  float* m_part;
  float* l_part;
  int B, Hq, Hkv, G, n_prefix, num_pages, page_size, max_pages, box_rows, most, stride;
  SplitCost cost;
  int joined;                // copies that take both 64-column halves of a row
  float scale;
};

// Requests [first, last) of prefix p; an entry outside [0, B] or one below
// its predecessor leaves the group empty.
ATTN_DEVINL bool group_of(const int* start, int p, int B, int& first, int& last) {
  first = __ldcg(start + p);
  last = __ldcg(start + p + 1);
  const bool good = first >= 0 && last >= first && last <= B;
  if (!good) first = last = 0;
  return good;
}

// (rounded operation by operation: two kernels must choose the same splits)
__host__ __device__ inline float split_cost(const SplitCost& c, int tiles, int s) {
#ifdef __CUDA_ARCH__
  auto mul = [](float x, float y) { return __fmul_rn(x, y); };
  auto add = [](float x, float y) { return __fadd_rn(x, y); };
#else
  auto mul = [](float x, float y) { return x * y; };
  auto add = [](float x, float y) { return x + y; };
#endif
  // (divisions take longer than all the rest; 1e-4 is above the product's
  // rounding and below what a part of a wave counts)
  const float waves = fmaxf(1.f, ceilf(add(mul(c.filled, float(s)), -1e-4f)));
  const float cta = mul(mul(float((unsigned(tiles) + s - 1) / unsigned(s) + 4), waves), c.tile);
  const float all = add(mul(float(tiles + 4 * s), c.work), c.own);
  return add(add(fmaxf(cta, all), mul(0.15f, cta)), mul(float(s), c.merge));
}
constexpr int kMostSplits = 64;      // that are chosen

// Keys per split of a prefix of n keys (a whole warp): the cheapest of at most
// `most` splits for the prefix's own length, not for what its table could hold.
ATTN_DEVINL int chunk_of(const SplitCost& c, int n, int most, int lane) {
  const int tiles = (n + kBN - 1) / kBN;
  int s = most;
  if (!c.fixed) {
    uint32_t best = 0xffffffffu;
    for (int s0 = 1; s0 <= most; s0 += 32) {
      const uint32_t cost =
          s0 + lane <= most ? __float_as_uint(split_cost(c, tiles, s0 + lane)) : 0xffffffffu;
      const uint32_t low = __reduce_min_sync(0xffffffffu, cost);
      const uint32_t who = __ballot_sync(0xffffffffu, cost == low);
      if (low < best) {
        best = low;
        s = s0 + __ffs(who) - 1;
      }
    }
  }
  return max(1, (tiles + s - 1) / s) * kBN;
}

ATTN_DEVINL int checked_len(int n, int cap) { return n < 0 || n > cap ? 0 : n; }

// Grid: x chunk of keys, y KV head, z run of rows (the prefixes' runs one
// after another; runs past the last one return).
template <int D, bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
prefix_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, PrefixArgs a) {
  using C = Cfg<D, kPair>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ int pages[kPagesCached];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y;
  constexpr int kRows = kPair ? 2 * kBM : kBM;
  const int per_unit = kRows / a.G;        // requests per run of rows

  if (tid == 0) {
    bars.abort = 0;
    mbar_init(&bars.q_full, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.p_full[t], kBM);
      mbar_init(&bars.o_done[t], 1);
    }
    mbar_init(&bars.mma_drain, 1);
    fence_barrier_init();
    tc::tma_prefetch_desc(&map_q);
    tc::tma_prefetch_desc(&map_k);
    tc::tma_prefetch_desc(&map_v);
  }
  if (warp == 1) {
    tc::tmem_alloc(&bars.tmem_base, 512);
    tc::tmem_relinquish();
  }
  pdl_wait_primary();
  // This CTA's run of rows: warp 0 counts the runs of the prefixes in order.
  if (warp == 0) {
    int seen = 0, p_of = -1, first_of = 0, n_of = 0, len_of = 0;
    bool bad = false;
    for (int p0 = 0; p0 < a.n_prefix && p_of < 0; p0 += 32) {
      int first = 0, last = 0, len = 0;
      if (p0 + lane < a.n_prefix) {
        len = a.prefix_lens[p0 + lane];
        bad |= !group_of(a.prefix_start, p0 + lane, a.B, first, last);
      }
      const int units = (last - first + per_unit - 1) / per_unit;
      int upto = units;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
      }
      const int u = int(blockIdx.z) - (seen + upto - units);   // run within the lane's prefix
      const uint32_t hit = __ballot_sync(0xffffffffu, u >= 0 && u < units);
      if (hit) {
        const int src = __ffs(hit) - 1;
        p_of = p0 + src;
        first_of = __shfl_sync(0xffffffffu, first + u * per_unit, src);
        n_of = min(per_unit, __shfl_sync(0xffffffffu, last, src) - first_of);
        len_of = __shfl_sync(0xffffffffu, len, src);
      }
      seen += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (bad) attn_flag_error(kErrBadIndex);
    const int cap = a.max_pages * a.page_size;
    if ((len_of < 0 || len_of > cap) && lane == 0) attn_flag_error(kErrBadIndex);
    len_of = checked_len(len_of, cap);
    const int chunk = chunk_of(a.cost, len_of, a.most, lane);
    if (lane == 0) {
      bars.unit[0] = p_of;
      bars.unit[1] = first_of;
      bars.unit[2] = n_of;
      bars.unit[3] = len_of;
      bars.unit[4] = chunk;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // (every thread has waited for what precedes the call)
  if (tid == 0) pdl_launch_dependents();
  const uint32_t tmem = bars.tmem_base;
  volatile int* abort_flag = &bars.abort;
  const int p = bars.unit[0], b0 = bars.unit[1], n_req = bars.unit[2];

  // This CTA's keys, and their pages checked (all before any is read).
  int n_keys = 0, key0 = 0;
  const int* table = nullptr;
  bool bad = false;
  if (p >= 0) {
    const int n = bars.unit[3], chunk = bars.unit[4];
    key0 = int(min((long long)n, 1LL * blockIdx.x * chunk));
    n_keys = min(n - key0, chunk);
    table = a.prefix_table + size_t(p) * a.max_pages;
  }
  const int page0 = key0 / a.page_size;
  if (n_keys > 0) {
    const int page1 = (key0 + n_keys - 1) / a.page_size;
    for (int i = page0 + tid; i <= page1; i += kThreads) {
      const int e = table[i];
      bad |= e < 0 || e >= a.num_pages;
      if (i - page0 < kPagesCached) pages[i - page0] = e;
    }
  }
  bad = __syncthreads_or(bad);
  const int nj = bad ? 0 : (n_keys + kBN - 1) / kBN;      // key tiles
  const int rows = n_req * a.G;                            // valid query rows
  // A key tile in shared memory: bytes from 8 keys to the next, and from one
  // 64-column half to the other.
  const uint32_t group = a.joined ? 1024 * C::kAtoms : 1024;
  const uint32_t half = a.joined ? 1024 : kBN * 128;
  // tiles of warpgroup t: all (kPair; none without rows), or every other one
  const int n_t[2] = {kPair ? (rows > 0 ? nj : 0) : (nj + 1) / 2,
                      kPair ? (rows > kBM ? nj : 0) : nj / 2};
  if (bad) {
    // a page index out of range: the chunk reads nothing and leaves no mass
    if (tid == 0) attn_flag_error(kErrBadIndex);
    for (int r = tid; r < rows; r += kThreads) {
      const size_t row = size_t(b0 + r / a.G) * a.Hq + g * a.G + r % a.G;
      a.m_part[row * a.stride + blockIdx.x] = -INFINITY;
      a.l_part[row * a.stride + blockIdx.x] = 0.f;
    }
  }

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (the whole warp)
    regs_dec<80>();
    if (nj > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars.q_full, C::kQTiles * C::kTileBytes);
        for (int t = 0; t < C::kQTiles; ++t)
          for (int at = 0; at < C::kAtoms; ++at)
            tc::tma_load_3d(smem + t * C::kTileBytes + at * (kBM * 128), &map_q, 64 * at, g * a.G,
                            b0 + t * (kBM / a.G), &bars.q_full);
      }
      // Lane i < here issues the copies of the tile's i-th box, for K and V
      // alike; boxes past the chunk's keys are not read. (A single page comes
      // as one box, in halves.)
      const int shift = 31 - __clz(a.box_rows);            // box_rows is a power of two
      int here = 0, row = 0, outer = 0;
      auto look_up = [&](int j) {
        const int at = j * kBN + lane * a.box_rows;
        here = min(kBN, n_keys - j * kBN + a.box_rows - 1) >> shift;
        if (lane < here) {
          const int pi = (key0 + at) / a.page_size;
          row = key0 + at - pi * a.page_size;
          outer = (pi - page0 < kPagesCached ? pages[pi - page0] : table[pi]) * a.Hkv + g;
        }
      };
      auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar) {
        if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(here) * a.box_rows * 128 * C::kAtoms);
        __syncwarp();
        if (lane < here) {
          if (a.joined)
            tc::tma_load_5d(dst + lane * a.box_rows * 128 * C::kAtoms, map, 0, 0, 0, row / 8, outer,
                            bar);
          else
#pragma unroll
            for (int at = 0; at < C::kAtoms; ++at)
              tc::tma_load_3d(dst + at * (kBN * 128), map, 64 * at, row, outer, bar);
        }
      };
      int issued_k = 0, issued_v = 0;
      bool ok = true;
      for (int j = 0; j < nj; ++j) {
        const int st = j % C::kStages;
        const uint32_t ph = (j / C::kStages) & 1;
        look_up(j);
        if (j >= C::kStages) ok = mbar_wait_warp(&bars.k_empty[st], ph ^ 1, abort_flag);
        if (!ok) break;
        load(smem + C::kKOff + st * C::kTileBytes, &map_k, &bars.k_full[st]);
        ++issued_k;
        if (j >= C::kStages) ok = mbar_wait_warp(&bars.v_empty[st], ph ^ 1, abort_flag);
        if (!ok) break;
        load(smem + C::kVOff + st * C::kTileBytes, &map_v, &bars.v_full[st]);
        ++issued_v;
      }
      if (!ok) {
        if (lane == 0) attn_flag_error(kErrTimeout);
        bars.abort = 1;
        // the loads in flight land before the CTA exits
        mbar_wait_warp(&bars.q_full, 0, nullptr);
        for (int j = max(0, issued_k - C::kStages); j < issued_k; ++j)
          mbar_wait_warp(&bars.k_full[j % C::kStages], (j / C::kStages) & 1, nullptr);
        for (int j = max(0, issued_v - C::kStages); j < issued_v; ++j)
          mbar_wait_warp(&bars.v_full[j % C::kStages], (j / C::kStages) & 1, nullptr);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    regs_dec<80>();
    if (nj > 0) {
      constexpr uint32_t idesc_s = tc::idesc_bf16_f32(kBM, kBN, false, false);
      constexpr uint32_t idesc_o = tc::idesc_bf16_f32(kBM, D, false, true);
      const uint32_t q_base = smem_u32(smem);
      const uint32_t k_base = smem_u32(smem + C::kKOff);
      const uint32_t v_base = smem_u32(smem + C::kVOff);
      auto issue_s = [&](int t, int j) {
        const uint32_t qa = q_base + (kPair ? t : 0) * C::kTileBytes;
        const uint32_t ka = k_base + (j % C::kStages) * C::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          tc::mma_ss_warp(tmem + C::kColS + t * kBN,
                          tc::smem_desc(qa + (kk / 4) * (kBM * 128) + (kk % 4) * 32, 16, 1024,
                                        tc::kLayoutSW128),
                          tc::smem_desc(ka + (kk / 4) * half + (kk % 4) * 32, 16, group,
                                        tc::kLayoutSW128),
                          idesc_s, kk > 0);
        }
        tc::mma_commit_warp(&bars.s_full[t]);
      };
      auto issue_pv = [&](int t, int j, bool first) {
        const uint32_t va = v_base + (j % C::kStages) * C::kTileBytes;
        // (P̃'s rounded values lie in the first 64 columns, the rests behind)
#pragma unroll 1
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            tc::mma_ts_warp(tmem + C::kColO + t * D,
                            tmem + C::kColS + t * kBN + part * (kBN / 2) + kk * 8,
                            tc::smem_desc(va + kk * 2 * group, half, group, tc::kLayoutSW128),
                            idesc_o, (!first || part + kk > 0) ? 1u : 0u);
        tc::mma_commit_warp(&bars.o_done[t]);
      };
      auto k_ready = [&](int j) {
        return mbar_wait_warp(&bars.k_full[j % C::kStages], (j / C::kStages) & 1, abort_flag);
      };
      bool ok = mbar_wait_warp(&bars.q_full, 0, abort_flag);
      if (kPair) {
        // S0, S1, PV0, S0', PV1, S1', ... over tiles that feed both
        if (ok) ok = k_ready(0);
        if (ok) {
          tc::fence_after_sync();
          for (int t = 0; t < 2; ++t)
            if (n_t[t] > 0) issue_s(t, 0);
          tc::mma_commit_warp(&bars.k_empty[0]);
        }
        for (int j = 0; j < nj && ok; ++j) {
          const bool next = j + 1 < nj;
          ok = mbar_wait_warp(&bars.v_full[j % C::kStages], (j / C::kStages) & 1, abort_flag);
          if (ok && next) ok = k_ready(j + 1);
          for (int t = 0; t < 2 && ok; ++t) {
            if (n_t[t] == 0) continue;
            ok = mbar_wait_warp(&bars.p_full[t], j & 1, abort_flag);
            if (!ok) break;
            tc::fence_after_sync();
            issue_pv(t, j, j == 0);
            if (next) issue_s(t, j + 1);
          }
          if (!ok) break;
          tc::mma_commit_warp(&bars.v_empty[j % C::kStages]);
          if (next) tc::mma_commit_warp(&bars.k_empty[(j + 1) % C::kStages]);
        }
      } else {
        // tile j belongs to warpgroup j & 1; S of tile j + 2 follows PV of
        // tile j, whose P̃ lies in the same columns
        for (int j = 0; j < min(nj, 2) && ok; ++j) {
          ok = k_ready(j);
          if (!ok) break;
          tc::fence_after_sync();
          issue_s(j, j);
          tc::mma_commit_warp(&bars.k_empty[j % C::kStages]);
        }
        for (int j = 0; j < nj && ok; ++j) {
          const int t = j & 1;
          ok = mbar_wait_warp(&bars.v_full[j % C::kStages], (j / C::kStages) & 1, abort_flag);
          if (ok) ok = mbar_wait_warp(&bars.p_full[t], (j >> 1) & 1, abort_flag);
          if (!ok) break;
          tc::fence_after_sync();
          issue_pv(t, j, j < 2);
          tc::mma_commit_warp(&bars.v_empty[j % C::kStages]);
          if (j + 2 < nj) {
            ok = k_ready(j + 2);
            if (!ok) break;
            tc::fence_after_sync();
            issue_s(t, j + 2);
            tc::mma_commit_warp(&bars.k_empty[(j + 2) % C::kStages]);
          }
        }
      }
      if (!ok && lane == 0) {
        attn_flag_error(kErrTimeout);
        bars.abort = 1;
      }
      __syncwarp();
      // every MMA has completed before tensor memory is freed
      tc::mma_commit_warp(&bars.mma_drain);
      mbar_wait_warp(&bars.mma_drain, 0, nullptr);
    }
  } else if (warp < 4) {
    regs_dec<80>();
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    // 128 x 80 + 256 x 208 registers <= 384 x 168 at launch
    regs_inc<208>();
    const int t = (warp - 4) / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;                     // accumulator row (TMEM lane)
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + C::kColS + t * kBN;
    const uint32_t o_addr = tmem + lane_base + C::kColO + t * D;
    const float c = a.scale * kLog2e;
    const int nt = n_t[t];
    float m_ref = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int i = 0; i < nt; ++i) {
      const int j = kPair ? i : 2 * i + t;                 // key tile
      if (!mbar_wait_warp(&bars.s_full[t], i & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      uint32_t sr[128];
      tc::tmem_ld32(s_addr + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      tc::tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
      tc::tmem_ld32(s_addr + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
      tc::tmem_ld32(s_addr + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
      tc::tmem_ld_wait();
      float* s = reinterpret_cast<float*>(sr);
      const int valid = n_keys - j * kBN;                  // keys of this tile
      if (valid < kBN) {
#pragma unroll
        for (int cc = 0; cc < kBN; ++cc)
          if (cc >= valid) s[cc] = -INFINITY;
      }
      float m8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) m8[k] = fmaxf(s[k], s[k + 8]);
#pragma unroll
      for (int e = 16; e < kBN; e += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) m8[k] = max3(m8[k], s[e + k], s[e + 8 + k]);
      const float mx = fmaxf(max3(m8[0], m8[1], m8[2]),
                             fmaxf(max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])));
      const float m_cand = fmaxf(m_ref, mx * c);
      const bool need = m_cand - m_ref > kRescaleThreshold;   // also true while m_ref = -inf
      float alpha = 1.f;
      if (need) {
        alpha = fast_exp2(m_ref - m_cand);
        m_ref = m_cand;
      }
      const float neg_m = (m_ref == -INFINITY) ? 0.f : -m_ref;
      const f2 cc2{c, c}, nm2{neg_m, neg_m};
      f2 rs2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        uint32_t pk[16], rest[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          f2 x = fma2(f2{s[part * 32 + 2 * e], s[part * 32 + 2 * e + 1]}, cc2, nm2);
          x.x = fast_exp2(x.x);
          x.y = fast_exp2(x.y);
          rs2[e & 3] = add2(rs2[e & 3], x);
          pk[e] = pack_bf16x2(x.x, x.y);
          x = fma2(f2{bf16lo(pk[e]), bf16hi(pk[e])}, f2{-1.f, -1.f}, x);   // exact
          rest[e] = pack_bf16x2(x.x, x.y);
        }
        tc::tmem_st16(s_addr + part * 16, pk);
        tc::tmem_st16(s_addr + kBN / 2 + part * 16, rest);
      }
      const f2 rsa = add2(add2(rs2[0], rs2[1]), add2(rs2[2], rs2[3]));
      l_run = fmaf(alpha, l_run, rsa.x + rsa.y);
      if (i > 0 && __any_sync(0xffffffffu, need)) {
        ok = mbar_wait_warp(&bars.o_done[t], (i - 1) & 1, abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t orr[32];
          tc::tmem_ld32(o_addr + ch * 32, orr);
          tc::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
          tc::tmem_st32(o_addr + ch * 32, orr);
        }
      }
      if (valid < kBN) {
        // the last tile: zero the value rows past the end (row r, if it is
        // one) once they have landed, before the product reads them
        ok = mbar_wait_warp(&bars.v_full[j % C::kStages], (j / C::kStages) & 1, abort_flag);
        if (!ok) break;
        if (r >= valid) {
          uint8_t* vt = smem + C::kVOff + (j % C::kStages) * C::kTileBytes + (r / 8) * group +
                        r % 8 * 128;
#pragma unroll
          for (int at = 0; at < C::kAtoms; ++at)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(vt + at * half + e * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      mbar_arrive(&bars.p_full[t]);
    }
    if (ok && nt > 0) ok = mbar_wait_warp(&bars.o_done[t], (nt - 1) & 1, abort_flag);
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    }
    if (nj > 0) {
      // Both warpgroups are past their last product: the ring is free.
      tc::fence_after_sync();
      float* mine = reinterpret_cast<float*>(smem) + ((warp - 4) * 32 + lane) * C::kStagePitch;
      named_bar_sync(1, 2 * kBM);
      float wgt = 1.f;
      if (!kPair) {
        // the two warpgroups' (o, m, l) of a row onto their common maximum
        float* ml = reinterpret_cast<float*>(smem + C::kMlOff);   // [warpgroup][m, l][row]
        ml[(2 * t) * kBM + r] = m_ref;
        ml[(2 * t + 1) * kBM + r] = l_run;
        named_bar_sync(1, 2 * kBM);
        const float m0 = ml[r], m1 = ml[2 * kBM + r];
        const float mm = fmaxf(m0, m1);
        const float w0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - mm);
        const float w1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - mm);
        wgt = t == 0 ? w0 : w1;
        m_ref = mm;
        l_run = ml[kBM + r] * w0 + ml[3 * kBM + r] * w1;
      }
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        // (a warpgroup that visited no tile never wrote its columns: zeros)
        uint32_t orr[32];
        tc::tmem_ld32(o_addr + ch * 32, orr);
        tc::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (nt > 0)
            x = make_float4(__uint_as_float(orr[4 * e]) * wgt, __uint_as_float(orr[4 * e + 1]) * wgt,
                            __uint_as_float(orr[4 * e + 2]) * wgt,
                            __uint_as_float(orr[4 * e + 3]) * wgt);
          *reinterpret_cast<float4*>(mine + ch * 32 + 4 * e) = x;
        }
      }
      if (kPair) __syncwarp();
      else named_bar_sync(1, 2 * kBM);
      // Rows out, a warp per row: the rows of this warp's quarter of its tile
      // (kPair), or half of the quarter the two warpgroups share.
      const float* st0 = reinterpret_cast<const float*>(smem);
      const int q0 = quarter * 32 + (kPair ? 0 : t * 16);
      if (!bars.abort) {
        for (int i = 0; i < (kPair ? 32 : 16); ++i) {
          const int tr = q0 + i;                           // row of the tile
          const int rr = (kPair ? t * kBM : 0) + tr;       // row of the run
          if (rr >= rows) break;
          const size_t row = size_t(b0 + rr / a.G) * a.Hq + g * a.G + rr % a.G;
          float* dst = a.o_part + (row * a.stride + blockIdx.x) * D;
          if (lane < D / 4) {
            float4 x = reinterpret_cast<const float4*>(
                st0 + ((kPair ? t * kBM : 0) + tr) * C::kStagePitch)[lane];
            if (!kPair) {
              const float4 y =
                  reinterpret_cast<const float4*>(st0 + (kBM + tr) * C::kStagePitch)[lane];
              x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            reinterpret_cast<float4*>(dst)[lane] = x;
          }
        }
        const int rr = (kPair ? t * kBM : 0) + r;
        if ((kPair || t == 0) && rr < rows) {
          const size_t at = (size_t(b0 + rr / a.G) * a.Hq + g * a.G + rr % a.G) * a.stride +
                            blockIdx.x;
          a.m_part[at] = m_ref == -INFINITY ? -INFINITY : m_ref * kLn2;   // natural units
          a.l_part[at] = l_run;
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// One warp per output row: the prefix's partials [0, np) and the request's
// own [s_own, s_own + no), each weighted by exp(m_t - m), fetched eight at a
// time with independent loads. Latency is what it costs: everything that can
// be known before the partials is, and m, l and o come in one round trip.
struct SharedMergeArgs {
  const float* o_part;
  const float* m_part;
  const float* l_part;
  __nv_bfloat16* o;
  float* lse;
  const int* prefix_lens;
  const int* prefix_start;
  const int* seq_lens;
  int rows, Hq, d, B, n_prefix, prefix_cap, own_cap, own_chunk, s_own, stride;
  SplitCost cost;
};

__global__ void __launch_bounds__(256) merge_shared_kernel(SharedMergeArgs a) {
  constexpr int kBatch = 8;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= a.rows) return;
  // (Lengths and starts may be read at once, from L2: the prefix kernel has
  // waited for all that precedes the call before this grid could start.)
  const int b = row / a.Hq;
  int np = 0;
  for (int p0 = 0; p0 < a.n_prefix; p0 += 32) {
    int first = 0, last = 0;
    if (p0 + lane < a.n_prefix) group_of(a.prefix_start, p0 + lane, a.B, first, last);
    const uint32_t hit = __ballot_sync(0xffffffffu, first <= b && b < last);
    if (hit) {
      const int n = checked_len(__ldcg(a.prefix_lens + p0 + __ffs(hit) - 1), a.prefix_cap);
      const int chunk = chunk_of(a.cost, n, a.s_own, lane);
      np = (n + chunk - 1) / chunk;
      break;
    }
  }
  const int no = (checked_len(__ldcg(a.seq_lens + b), a.own_cap) + a.own_chunk - 1) / a.own_chunk;
  const int nv = np + no, d4 = a.d / 4;                // (d4 is 16 or 32: a column per lane)
  auto slot = [&](int t) { return t < np ? t : t - np + a.s_own; };
  const float* mr = a.m_part + size_t(row) * a.stride;
  const float* lr = a.l_part + size_t(row) * a.stride;
  const float4* prow = reinterpret_cast<const float4*>(a.o_part + size_t(row) * a.stride * a.d);
  // (a partial without mass may hold anything)
  auto fetch = [&](float4 (&x)[kBatch], int t0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      x[u] = t0 + u < nv && lane < d4 ? prow[size_t(slot(t0 + u)) * d4 + lane]
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  pdl_wait_primary();
  pdl_launch_dependents();
  // m and l of partials `lane`, and the first batch of o, in one round trip
  const float m0 = lane < nv ? mr[slot(lane)] : -INFINITY;
  const float l0 = lane < nv ? lr[slot(lane)] : 0.f;
  float4 x[kBatch];
  fetch(x, 0);
  float mx = m0;
  for (int t = lane + 32; t < nv; t += 32) mx = fmaxf(mx, mr[slot(t)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  const bool empty = mx == -INFINITY;
  auto weight = [&](float m) { return m == -INFINITY ? 0.f : expf(m - mx); };
  const float w0 = weight(m0);
  float l = w0 != 0.f ? w0 * l0 : 0.f;
  for (int t = lane + 32; t < nv; t += 32) {
    const float w = weight(mr[slot(t)]);
    if (w != 0.f) l = fmaf(w, lr[slot(t)], l);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = 0; t0 < nv; t0 += kBatch) {
    if (t0 > 0) fetch(x, t0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int t = t0 + u;
      const float ws = __shfl_sync(0xffffffffu, w0, t & 31);
      const float w = t < 32 ? ws : t < nv ? weight(mr[slot(t)]) : 0.f;
      if (w == 0.f) continue;
      acc.x = fmaf(w, x[u].x, acc.x);
      acc.y = fmaf(w, x[u].y, acc.y);
      acc.z = fmaf(w, x[u].z, acc.z);
      acc.w = fmaf(w, x[u].w, acc.w);
    }
  }
  const float inv = empty ? 0.f : 1.f / l;
  if (lane < d4)
    reinterpret_cast<uint2*>(a.o + size_t(row) * a.d)[lane] = make_uint2(
        pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse != nullptr && lane == 0) a.lse[row] = empty ? -INFINITY : mx + logf(l);
}

// q as [B][Hq][d] with boxes of the G heads of a group times kBM / G
// requests: the box lands as kBM rows, request-major.
bool make_map_q(CUtensorMap* m, const void* q, int B, int Hq, int d, int G) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(Hq), cuuint64_t(B)};
  const cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(Hq) * d * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(G), cuuint32_t(kBM / G)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kPair>
cudaError_t launch_prefix_t(const SharedArgs& a, const SharedPlan& pl) {
  using C = Cfg<D, kPair>;
  const int G = a.own.Hq / a.own.Hkv;
  const uint64_t outer = uint64_t(a.num_prefix_pages) * a.own.Hkv;
  CUtensorMap mq, mk, mv;
  // (pages have a multiple of 8 rows where a table row has more than one)
  const bool joined = a.max_prefix_pages > 1;
  auto map = [&](CUtensorMap* m, const void* base) {
    return joined ? make_map_bf16_joined(m, base, D, a.prefix_page_size, outer, pl.box_rows)
                  : make_map_bf16_3d(m, base, D, a.prefix_page_size, outer, pl.box_rows);
  };
  if (!make_map_q(&mq, a.own.q, a.own.B, a.own.Hq, D, G) || !map(&mk, a.k_prefix) ||
      !map(&mv, a.v_prefix))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(prefix_kernel<D, kPair>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kDynSmem);
  if (e != cudaSuccess) return e;
  const PrefixArgs pa{a.prefix_table, a.prefix_lens, a.prefix_start, a.own.o_part, a.own.m_part,
                      a.own.l_part, a.own.B, a.own.Hq, a.own.Hkv, G, a.n_prefix,
                      a.num_prefix_pages, a.prefix_page_size, a.max_prefix_pages, pl.box_rows,
                      pl.prefix_splits, pl.prefix_splits + pl.own_splits, pl.cost, joined,
                      a.own.scale};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.prefix_splits, a.own.Hkv, pl.units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kDynSmem;
  cfg.stream = a.own.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_kernel<D, kPair>, mq, mk, mv, pa);
}

}  // namespace

// How a call is cut, as far as its sizes tell (group sizes and lengths are
// only known on the device).
SharedPlan shared_plan(int B, int Hq, int Hkv, int d, int n_prefix, int prefix_page_size,
                       int max_prefix_pages, int page_size, int max_pages, int prefix_splits,
                       int own_splits) {
  SharedPlan pl;
  const long long sms = device_sm_count() > 0 ? device_sm_count() : 152;
  const long long rows = 1LL * B * (Hq / Hkv);
  pl.pair = rows > 128LL * n_prefix;
  const int per = pl.pair ? 2 * kBM : kBM;
  // runs of rows: every prefix may end with a part of one
  pl.units = int(std::min<long long>((rows + per - 1) / per + n_prefix - 1, B));
  const long long cap = 1LL * prefix_page_size * max_prefix_pages;
  const long long tiles = (cap + kBN - 1) / kBN;
  const long long own_cap = 1LL * page_size * max_pages;
  if (own_splits <= 0) {
    // A split per 512 keys of capacity, as many as make one round of the split
    // kernel's three CTAs per SM, or four where that is more (64 requests of up
    // to 1024 keys: 57, 52, 52, 58 us with 1, 2, 4, 8 splits; 128 of up to
    // 8192: 481, 410, 361, 362; 16 of up to 400, 64 heads: 21.4 and 25.8 with
    // 1 and 4).
    const long long want = (3 * sms + 1LL * B * Hkv - 1) / (1LL * B * Hkv);
    own_splits = int(std::min((own_cap + 511) / 512, std::max(4LL, want)));
  }
  // Both parts run at once, so a call takes as long as a prefix CTA, or as
  // the work of both spread over all SMs, then as the merge of the splits;
  // where the two meet, shorter CTAs pack better (0.15 of a CTA's time).
  // In microseconds, as measured: 1.2 for a key tile, 2.3 where it feeds 256
  // rows (1.8 with d = 64); four tiles for a CTA's start and its partial rows;
  // own keys, half their capacity but 512 at most (the capacity says little of
  // the lengths), at 3 TB/s; 0.5 + 0.6 per MB of partials for every split to
  // merge. (64 requests behind 8192 keys: 87, 65, 53, 57, 61 us with 2, 3, 4,
  // 5, 8 splits, 69 with 19, which fill the device; 128 of them 103, 92, 93
  // with 2, 3, 4; 96 behind three prefixes up to 32768: 147, 117, 117, 124
  // with 3, 4, 5, 6.) Here for what the table can hold, which bounds the splits
  // of all prefixes; each prefix's own are chosen by the same costs from its
  // length, on the device.
  pl.cost.tile = pl.pair ? (d == 64 ? 1.8f : 2.3f) : 1.2f;
  pl.cost.filled =
      float(1.0 * Hkv * std::max<long long>(n_prefix, (rows + per - 1) / per) / double(sms));
  pl.cost.work = pl.cost.tile * pl.cost.filled;
  pl.cost.own = float(1.0 * B * Hkv * std::min(own_cap / 2, 512LL) * d * 4 / 3e6);
  pl.cost.merge = float(0.5 + 0.6e-6 * B * Hq * d * 4);
  pl.cost.fixed = prefix_splits > 0;
  if (prefix_splits <= 0) {
    prefix_splits = 1;
    for (int s = 2; s <= kMostSplits && s <= tiles; ++s)
      if (split_cost(pl.cost, int(tiles), s) < split_cost(pl.cost, int(tiles), prefix_splits))
        prefix_splits = s;
  }
  // (as many as the longest prefix would use)
  const long long per_split = (tiles + prefix_splits - 1) / prefix_splits;
  pl.prefix_splits = int((tiles + per_split - 1) / per_split);
  pl.own_splits = own_splits;
  // copies of a key tile: whole tiles of a single page, else the largest
  // power of two that divides the page size
  pl.box_rows = kBN;
  if (max_prefix_pages > 1)
    while (prefix_page_size % pl.box_rows != 0) pl.box_rows /= 2;
  return pl;
}

cudaError_t launch_decode_shared(const SharedArgs& a, const SharedPlan& pl) {
  const bool d64 = a.own.d == 64;
  cudaError_t e = pl.pair ? (d64 ? launch_prefix_t<64, true>(a, pl)
                                 : launch_prefix_t<128, true>(a, pl))
                          : (d64 ? launch_prefix_t<64, false>(a, pl)
                                 : launch_prefix_t<128, false>(a, pl));
  if (e != cudaSuccess) return e;
  // the own keys' partials follow the prefix's in every row
  DecodeArgs own = a.own;
  own.num_splits = pl.own_splits;
  own.part_stride = pl.prefix_splits + pl.own_splits;
  own.o_part += size_t(pl.prefix_splits) * own.d;
  own.m_part += pl.prefix_splits;
  own.l_part += pl.prefix_splits;
  own.after_partner = true;
  e = launch_decode_split(own);
  if (e != cudaSuccess) return e;
  const SharedMergeArgs m{a.own.o_part, a.own.m_part, a.own.l_part,
                          static_cast<__nv_bfloat16*>(a.own.o), a.own.lse, a.prefix_lens,
                          a.prefix_start, a.own.seq_lens, a.own.B * a.own.Hq, a.own.Hq, a.own.d,
                          a.own.B, a.n_prefix, a.max_prefix_pages * a.prefix_page_size,
                          a.own.max_pages * a.own.page_size, decode_chunk(own), pl.prefix_splits,
                          own.part_stride, pl.cost};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((m.rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = a.own.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_shared_kernel, m);
}

}  // namespace attn
