// Attention weight received by each cached key:
//   out[b, g, j] = decay · prev[b, g, j] + Σ_r exp(scale · q_r·k_j - lse_r)
// over the R = G·T query rows r of KV head g (the T query tokens of its G
// heads) that see key j. With the rows' log-sum-exp known the weights need
// no softmax of their own: a matrix product, an exponential per element and
// a sum over one axis.
//
// GB300 mapping. The product is taken transposed, Sᵀ = K Qᵀ: keys are the
// accumulator's rows (TMEM lanes), so that the thread of a key sums its
// weights over the columns in registers and no sum crosses threads. A
// warpgroup owns 128 keys. Per (key, row) the tensor core spends 2·d flops
// (1/32 cycle of an SM at d = 128) and the special-function unit one
// exponential (1/16 cycle): with many rows the exponentials bound it, with
// few the reading of K.
//
//  * At most 256 rows (decode steps, observation windows): the rows of a
//    (request, KV head) stay in shared memory and the keys stream past them.
//    One persistent CTA per SM takes an equal share of all key tiles of the
//    batch; tiles alternate between two warpgroups, so one's exponentials
//    overlap the other's product.
//  * More rows (every token of a prompt as an observer): 256 keys of a
//    (request, KV head) stay in shared memory, 128 per warpgroup, and the
//    rows stream past them in chunks of 128; chunks that see none of the
//    keys are skipped. Few keys are spread over more CTAs by cutting the
//    rows; the partial sums are then added in a fixed order by a second
//    kernel.
//
// Sums are float32; every wait is bounded, as in the other kernels.

#include <algorithm>
#include <climits>

#include "common.cuh"
#include "launchers.h"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace attn {

ATTN_DEFINE_ERROR_WORD(take_error_key_weights)

namespace {

constexpr int kTileKeys = 128;
constexpr int kThreads = 384;     // TMA, MMA, row data, idle warp; two warpgroups of keys
constexpr float kLog2e = 1.4426950408889634f;

struct KwArgs {
  const float* lse;        // [B, Hkv, R]
  const float* prev;
  float* out;              // [B, Hkv, out_len], or partial sums [S][B, Hkv, out_len]
  const int* seq_lens;
  const int* block_table;
  int B, Hkv, R, T, cap, out_len, num_pages, page_size, max_pages, box_rows;
  int causal;
  float c, decay;          // scale · log2 e
};

ATTN_DEVINL int request_len(const KwArgs& a, int b, bool& bad) {
  if (a.seq_lens == nullptr) return a.cap;
  const int n = a.seq_lens[b];
  const bool wrong = n < 0 || n > a.cap;
  bad |= wrong;
  return wrong ? 0 : n;
}

// The copies of one key tile (all lanes of a converged warp): one per (box,
// atom); boxes past the request's keys or behind a bad page index are left
// out, their lanes' sums are not used.
template <int D>
ATTN_DEVINL void load_key_tile(const KwArgs& a, uint8_t* dst, const CUtensorMap* map, int b, int g,
                               int key0, int n, uint64_t* bar, int lane) {
  constexpr int kAtoms = D / 64;
  const int boxes = min(kTileKeys / a.box_rows, (n - key0 + a.box_rows - 1) / a.box_rows);
  int row = 0, outer = 0;
  bool good = lane < boxes;
  if (good) {
    const int key = key0 + lane * a.box_rows;
    if (a.block_table == nullptr) {
      row = key;
      outer = b * a.Hkv + g;
    } else {
      const int pi = key / a.page_size;
      const int page = a.block_table[size_t(b) * a.max_pages + pi];
      good = page >= 0 && page < a.num_pages;
      if (!good) attn_flag_error(kErrBadIndex);
      row = key - pi * a.page_size;
      outer = page * a.Hkv + g;
    }
  }
  const uint32_t live = __ballot_sync(0xffffffffu, good);
  if (lane == 0)
    mbar_arrive_expect_tx(bar, uint32_t(__popc(live)) * a.box_rows * 128 * kAtoms);
  __syncwarp();
  if (good)
#pragma unroll
    for (int at = 0; at < kAtoms; ++at)
      tc::tma_load_3d(dst + at * (kTileKeys * 128) + lane * a.box_rows * 128, map, 64 * at, row,
                      outer, bar);
}

// Whether the page of this thread's key may be read (its lane is in use).
ATTN_DEVINL bool page_good(const KwArgs& a, int b, int j) {
  if (a.block_table == nullptr) return true;
  const int page = a.block_table[size_t(b) * a.max_pages + j / a.page_size];
  return page >= 0 && page < a.num_pages;
}

// What a chunk of query rows needs besides Q: the log-sum-exp in log2 units
// (+inf where the row counts for nothing: past R, or a row that saw no key)
// and the row's token (INT_MIN past R).
struct RowData {
  float lse2;
  int token;
};
ATTN_DEVINL RowData row_data(const KwArgs& a, int head, int r) {
  if (r >= a.R) return RowData{INFINITY, INT_MIN};
  const float l = a.lse[size_t(head) * a.R + r];
  return RowData{l == -INFINITY ? INFINITY : l * kLog2e, r % a.T};
}

// Σ exp2(s·c - lse2) over NC accumulator columns, the row data read from
// shared memory (the same address for all lanes). Masked form: a column
// counts if its token is at least `first` (the first token that sees the key).
template <int NC, bool kMask>
ATTN_DEVINL void add_columns(const uint32_t (&s)[NC], const float* lse2, const int* token, float c,
                             int first, f2 (&sum)[2]) {
  const f2 c2{c, c};
#pragma unroll
  for (int e = 0; e < NC; e += 4) {
    const float4 l = *reinterpret_cast<const float4*>(lse2 + e);
    f2 x = fma2(f2{__uint_as_float(s[e]), __uint_as_float(s[e + 1])}, c2, f2{-l.x, -l.y});
    f2 y = fma2(f2{__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])}, c2, f2{-l.z, -l.w});
    x.x = fast_exp2(x.x);
    x.y = fast_exp2(x.y);
    y.x = fast_exp2(y.x);
    y.y = fast_exp2(y.y);
    if (kMask) {
      const int4 t = *reinterpret_cast<const int4*>(token + e);
      x.x = t.x >= first ? x.x : 0.f;
      x.y = t.y >= first ? x.y : 0.f;
      y.x = t.z >= first ? y.x : 0.f;
      y.y = t.w >= first ? y.y : 0.f;
    }
    sum[0] = add2(sum[0], x);
    sum[1] = add2(sum[1], y);
  }
}

// Columns [0, N) of an accumulator (N a multiple of 16), 32 at a time, the
// next ones on their way from tensor memory while the last are summed.
// masked: every column is tested; otherwise only those past `full`.
ATTN_DEVINL float sum_columns(uint32_t addr, int N, int full, bool masked, const float* lse2,
                              const int* token, float c, int first) {
  f2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
  uint32_t even[32], odd[32];
  const int n32 = N / 32;
  auto add = [&](const uint32_t(&s)[32], int i) {
    if (masked || 32 * i + 32 > full)
      add_columns<32, true>(s, lse2 + 32 * i, token + 32 * i, c, first, sum);
    else
      add_columns<32, false>(s, lse2 + 32 * i, token + 32 * i, c, first, sum);
  };
  if (n32 > 0) tc::tmem_ld32(addr, even);
  for (int i = 0; i < n32; i += 2) {
    tc::tmem_ld_wait();
    if (i + 1 < n32) tc::tmem_ld32(addr + 32 * (i + 1), odd);
    add(even, i);
    if (i + 1 < n32) {
      tc::tmem_ld_wait();
      if (i + 2 < n32) tc::tmem_ld32(addr + 32 * (i + 2), even);
      add(odd, i + 1);
    }
  }
  if (N % 32 != 0) {
    uint32_t rest[16];
    tc::tmem_ld16(addr + 32 * n32, rest);
    tc::tmem_ld_wait();
    add_columns<16, true>(rest, lse2 + 32 * n32, token + 32 * n32, c, first, sum);
  }
  const f2 t = add2(sum[0], sum[1]);
  return t.x + t.y;
}

// The first token that sees key j (any token without a causal mask, but
// never a column past R).
ATTN_DEVINL int first_token(const KwArgs& a, int n, int j) {
  return a.causal ? max(0, j - (n - a.T)) : 0;
}

// ---------------------------------------------------------------- few rows: keys stream

template <int D, int NMAX>
struct KeysCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kTileKeys * D * 2;
  static constexpr int kQBufs = NMAX <= 64 ? 2 : 1;
  static constexpr int kQBytes = NMAX * D * 2;
  static constexpr int kStages = 4 * (128 / D);
  static constexpr int kKOff = kQBufs * kQBytes;
  static constexpr int kDynSmem = kKOff + kStages * kTileBytes + 1024;
  static constexpr uint32_t kTmemCols = 2 * NMAX;    // one accumulator per warpgroup
};

struct KeysBars {
  uint64_t q_full[2], q_empty[2], k_full[8], k_empty[8], acc_full[2], acc_empty[2];
  uint64_t row_full[2], row_empty[2], mma_drain;
  uint32_t tmem_base;
  int abort;
  int warp_sum[kThreads / 32 + 1];
  int start[3];                      // request, head, tile where this CTA begins
  int count;                         // its tiles
};

// The tiles of a CTA in order: (request, head, tile), skipping empty requests.
struct TileWalk {
  int b, g, tile, n, tiles;
  ATTN_DEVINL void open(const KwArgs& a) {
    bool bad = false;
    n = request_len(a, b, bad);
    tiles = (n + kTileKeys - 1) / kTileKeys;
  }
  // Moves to the next tile; true when it belongs to another (request, head).
  ATTN_DEVINL bool next(const KwArgs& a) {
    if (++tile < tiles) return false;
    tile = 0;
    if (++g < a.Hkv) return true;
    g = 0;
    do {
      if (++b >= a.B) return true;
      open(a);
    } while (tiles == 0);
    return true;
  }
};

template <int D, int NMAX>
__global__ void __launch_bounds__(kThreads, 1)
weights_keys_kernel(const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_k, KwArgs a, int N) {
  using C = KeysCfg<D, NMAX>;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ KeysBars bars;
  __shared__ __align__(16) float row_lse[2][NMAX];
  __shared__ __align__(16) int row_token[2][NMAX];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    bars.abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kTileKeys);
      mbar_init(&bars.row_full[i], 32);
      mbar_init(&bars.row_empty[i], 2 * kTileKeys);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
    }
    mbar_init(&bars.mma_drain, 1);
    fence_barrier_init();
    tc::tma_prefetch_desc(&map_q);
    tc::tma_prefetch_desc(&map_k);
  }
  if (warp == 1) {
    tc::tmem_alloc(&bars.tmem_base, C::kTmemCols);
    tc::tmem_relinquish();
  }
  pdl_wait_primary();
  // This CTA's share of the batch's key tiles: thread t counts a run of
  // requests, a scan over the threads gives where each run begins.
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int r0 = min(a.B, tid * per), r1 = min(a.B, r0 + per);
    int mine = 0;
    bool bad = false;
    for (int b = r0; b < r1; ++b)
      mine += (request_len(a, b, bad) + kTileKeys - 1) / kTileKeys * a.Hkv;
    if (bad && blockIdx.x == 0) attn_flag_error(kErrBadIndex);
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) bars.warp_sum[warp] = upto;
    __syncthreads();
    int before = upto - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += bars.warp_sum[w];
      total += bars.warp_sum[w];
    }
    const int first = int(1LL * total * blockIdx.x / gridDim.x);
    const int last = int(1LL * total * (blockIdx.x + 1) / gridDim.x);
    if (tid == 0) bars.count = last - first;
    if (first < last && before <= first && first < before + mine) {
      int at = before;
      for (int b = r0; b < r1; ++b) {
        const int tiles = (request_len(a, b, bad) + kTileKeys - 1) / kTileKeys;
        if (first < at + tiles * a.Hkv) {
          bars.start[0] = b;
          bars.start[1] = (first - at) / tiles;
          bars.start[2] = (first - at) % tiles;
          break;
        }
        at += tiles * a.Hkv;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars.tmem_base;
  volatile int* abort_flag = &bars.abort;
  const int count = bars.count;
  TileWalk w{bars.start[0], bars.start[1], bars.start[2], 0, 0};
  if (count > 0) w.open(a);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (the whole warp)
    bool ok = true, fresh = true;
    int heads = 0, i = 0;
    for (; i < count && ok; ++i) {
      if (fresh) {
        const int qb = heads % C::kQBufs;
        if (heads >= C::kQBufs)
          ok = mbar_wait_warp(&bars.q_empty[qb], (heads / C::kQBufs - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars.q_full[qb], uint32_t(N) * D * 2);
          for (int at = 0; at < C::kAtoms; ++at)
            tc::tma_load_3d(smem + qb * C::kQBytes + at * (NMAX * 128), &map_q, 64 * at, 0,
                            w.b * a.Hkv + w.g, &bars.q_full[qb]);
        }
        __syncwarp();
        ++heads;
      }
      const int st = i % C::kStages;
      if (i >= C::kStages)
        ok = mbar_wait_warp(&bars.k_empty[st], (i / C::kStages - 1) & 1, abort_flag);
      if (!ok) break;
      load_key_tile<D>(a, smem + C::kKOff + st * C::kTileBytes, &map_k, w.b, w.g,
                       w.tile * kTileKeys, w.n, &bars.k_full[st], lane);
      fresh = w.next(a);
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
      // the loads in flight land before the CTA exits
      for (int j = max(0, heads - C::kQBufs); j < heads; ++j)
        mbar_wait_warp(&bars.q_full[j % C::kQBufs], (j / C::kQBufs) & 1, nullptr);
      for (int j = max(0, i - C::kStages); j < i; ++j)
        mbar_wait_warp(&bars.k_full[j % C::kStages], (j / C::kStages) & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the whole warp)
    const uint32_t idesc = tc::idesc_bf16_f32(kTileKeys, N, false, false);
    const uint32_t q_base = smem_u32(smem), k_base = smem_u32(smem + C::kKOff);
    bool ok = true, fresh = true;
    int heads = 0;
    for (int i = 0; i < count && ok; ++i) {
      if (fresh) {
        ok = mbar_wait_warp(&bars.q_full[heads % C::kQBufs], (heads / C::kQBufs) & 1, abort_flag);
        ++heads;
      }
      const int st = i % C::kStages, t = i & 1;
      if (ok) ok = mbar_wait_warp(&bars.k_full[st], (i / C::kStages) & 1, abort_flag);
      if (ok && i >= 2) ok = mbar_wait_warp(&bars.acc_empty[t], ((i >> 1) - 1) & 1, abort_flag);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t qa = q_base + ((heads - 1) % C::kQBufs) * C::kQBytes;
      const uint32_t ka = k_base + st * C::kTileBytes;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        tc::mma_ss_warp(tmem + t * NMAX,
                        tc::smem_desc(ka + (kk / 4) * (kTileKeys * 128) + (kk % 4) * 32, 16, 1024,
                                      tc::kLayoutSW128),
                        tc::smem_desc(qa + (kk / 4) * (NMAX * 128) + (kk % 4) * 32, 16, 1024,
                                      tc::kLayoutSW128),
                        idesc, kk > 0);
      tc::mma_commit_warp(&bars.acc_full[t]);
      tc::mma_commit_warp(&bars.k_empty[st]);
      fresh = w.next(a);
      if (fresh) tc::mma_commit_warp(&bars.q_empty[(heads - 1) % C::kQBufs]);
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    }
    __syncwarp();
    tc::mma_commit_warp(&bars.mma_drain);
    mbar_wait_warp(&bars.mma_drain, 0, nullptr);
  } else if (warp == 2) {
    // ------------------------------------------------------------ row data, one head ahead
    bool ok = true, fresh = true;
    int heads = 0;
    for (int i = 0; i < count && ok; ++i) {
      if (fresh) {
        const int rb = heads & 1;
        if (heads >= 2) ok = mbar_wait_warp(&bars.row_empty[rb], ((heads >> 1) - 1) & 1, abort_flag);
        if (!ok) break;
        for (int r = lane; r < N; r += 32) {
          const RowData x = row_data(a, w.b * a.Hkv + w.g, r);
          row_lse[rb][r] = x.lse2;
          row_token[rb][r] = x.token;
        }
        mbar_arrive(&bars.row_full[rb]);
        ++heads;
      }
      fresh = w.next(a);
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ warpgroups of keys
    const int t = (warp - 4) / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;                   // key of the tile (TMEM lane)
    const uint32_t addr = tmem + (uint32_t(quarter * 32) << 16) + t * NMAX;
    bool ok = true, fresh = true;
    int heads = 0;
    for (int i = 0; i < count && ok; ++i) {
      if (fresh) {
        if (heads > 0) mbar_arrive(&bars.row_empty[(heads - 1) & 1]);
        ok = mbar_wait_warp(&bars.row_full[heads & 1], (heads >> 1) & 1, abort_flag);
        if (!ok) break;
        ++heads;
      }
      if ((i & 1) == t) {
        const int j = w.tile * kTileKeys + r;
        const size_t at = (size_t(w.b) * a.Hkv + w.g) * a.out_len + j;
        const bool live = j < w.n;
        // on their way while the product runs
        const float prev = live && a.prev != nullptr ? a.prev[at] : 0.f;
        const bool good = live && page_good(a, w.b, j);
        ok = mbar_wait_warp(&bars.acc_full[t], (i >> 1) & 1, abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
        // the tile needs its columns tested if the first token misses its last key
        const bool masked = first_token(a, w.n, w.tile * kTileKeys + kTileKeys - 1) > 0;
        const float sum = sum_columns(addr, N, a.R, masked, row_lse[(heads - 1) & 1],
                                      row_token[(heads - 1) & 1], a.c, first_token(a, w.n, j));
        tc::fence_before_sync();
        mbar_arrive(&bars.acc_empty[t]);
        if (live) {
          const float kept = a.prev != nullptr ? a.decay * prev : 0.f;
          a.out[at] = good ? kept + sum : kept;
        }
      }
      fresh = w.next(a);
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- many rows: rows stream

constexpr int kChunk = 128;        // query rows per step

template <int D>
struct RowsCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kTileKeys * D * 2;
  static constexpr int kStages = 4;
  static constexpr int kQOff = 2 * kTileBytes;       // two key tiles first
  static constexpr int kDynSmem = kQOff + kStages * kTileBytes + 1024;
  static constexpr uint32_t kTmemCols = 512;         // two accumulators per warpgroup
};

struct RowsBars {
  uint64_t k_full, q_full[4], q_empty[4], acc_full[2][2], acc_empty[2][2];
  uint64_t row_full[4], row_empty[4], mma_drain;
  uint32_t tmem_base;
  int abort;
};

// Grid: key blocks of 256, the first ones (which the most rows see) of all
// heads first; y splits the chunks of rows.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
weights_rows_kernel(const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_k, KwArgs a) {
  using C = RowsCfg<D>;
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ RowsBars bars;
  __shared__ __align__(16) float row_lse[C::kStages][kChunk];
  __shared__ __align__(16) int row_token[C::kStages][kChunk];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = a.B * a.Hkv;
  const int head = blockIdx.x % heads, b = head / a.Hkv, g = head % a.Hkv;
  const int key0 = int(blockIdx.x / heads) * 2 * kTileKeys;

  if (tid == 0) {
    bars.abort = 0;
    mbar_init(&bars.k_full, 2);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.row_full[i], 32);
      mbar_init(&bars.row_empty[i], 2 * kTileKeys);
    }
    for (int t = 0; t < 2; ++t)
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.acc_full[t][i], 1);
        mbar_init(&bars.acc_empty[t][i], kTileKeys);
      }
    mbar_init(&bars.mma_drain, 1);
    fence_barrier_init();
    tc::tma_prefetch_desc(&map_q);
    tc::tma_prefetch_desc(&map_k);
  }
  if (warp == 1) {
    tc::tmem_alloc(&bars.tmem_base, C::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  pdl_wait_primary();
  const uint32_t tmem = bars.tmem_base;
  volatile int* abort_flag = &bars.abort;

  bool bad = false;
  const int n = request_len(a, b, bad);
  if (bad && tid == 0 && key0 == 0 && g == 0 && blockIdx.y == 0) attn_flag_error(kErrBadIndex);
  // this CTA's chunks of rows; those whose latest token does not see a
  // tile's first key are skipped by every role alike
  const int chunks = (a.R + kChunk - 1) / kChunk;
  const int c0 = int(1LL * chunks * blockIdx.y / gridDim.y);
  const int c1 = int(1LL * chunks * (blockIdx.y + 1) / gridDim.y);
  auto last_token = [&](int c) {
    const int r0 = c * kChunk, r1 = min(a.R, r0 + kChunk) - 1;
    return r1 / a.T > r0 / a.T ? a.T - 1 : r1 % a.T;
  };
  auto first_of_chunk = [&](int c) {
    const int r0 = c * kChunk, r1 = min(a.R, r0 + kChunk) - 1;
    return r1 / a.T > r0 / a.T ? 0 : r0 % a.T;
  };
  const int tiles = key0 >= n ? 0 : key0 + kTileKeys < n ? 2 : 1;
  const int from[2] = {first_token(a, n, key0), first_token(a, n, key0 + kTileKeys)};
  auto sees = [&](int c, int t) { return t < tiles && last_token(c) >= from[t]; };

  if (tiles == 0) {
    // nothing to do (the partial sums of keys past the end are never read)
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (the whole warp)
    for (int t = 0; t < 2; ++t) {
      if (t < tiles)
        load_key_tile<D>(a, smem + t * C::kTileBytes, &map_k, b, g, key0 + t * kTileKeys, n,
                         &bars.k_full, lane);
      else if (lane == 0)
        mbar_arrive(&bars.k_full);
    }
    bool ok = true;
    int i = 0;
    for (int c = c0; c < c1 && ok; ++c) {
      if (!sees(c, 0)) continue;
      const int st = i % C::kStages;
      if (i >= C::kStages)
        ok = mbar_wait_warp(&bars.q_empty[st], (i / C::kStages - 1) & 1, abort_flag);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars.q_full[st], C::kTileBytes);
        for (int at = 0; at < C::kAtoms; ++at)
          tc::tma_load_3d(smem + C::kQOff + st * C::kTileBytes + at * (kChunk * 128), &map_q,
                          64 * at, c * kChunk, head, &bars.q_full[st]);
      }
      __syncwarp();
      ++i;
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
      mbar_wait_warp(&bars.k_full, 0, nullptr);
      for (int j = max(0, i - C::kStages); j < i; ++j)
        mbar_wait_warp(&bars.q_full[j % C::kStages], (j / C::kStages) & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the whole warp)
    constexpr uint32_t idesc = tc::idesc_bf16_f32(kTileKeys, kChunk, false, false);
    const uint32_t k_base = smem_u32(smem), q_base = smem_u32(smem + C::kQOff);
    bool ok = mbar_wait_warp(&bars.k_full, 0, abort_flag);
    int i = 0, used[2] = {0, 0};
    for (int c = c0; c < c1 && ok; ++c) {
      if (!sees(c, 0)) continue;
      const int st = i % C::kStages;
      ok = mbar_wait_warp(&bars.q_full[st], (i / C::kStages) & 1, abort_flag);
      for (int t = 0; t < 2 && ok; ++t) {
        if (!sees(c, t)) continue;
        const int ab = used[t] & 1;
        if (used[t] >= 2)
          ok = mbar_wait_warp(&bars.acc_empty[t][ab], ((used[t] >> 1) - 1) & 1, abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t ka = k_base + t * C::kTileBytes, qa = q_base + st * C::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * (kTileKeys * 128) + (kk % 4) * 32;
          tc::mma_ss_warp(tmem + (2 * t + ab) * kChunk,
                          tc::smem_desc(ka + off, 16, 1024, tc::kLayoutSW128),
                          tc::smem_desc(qa + off, 16, 1024, tc::kLayoutSW128), idesc, kk > 0);
        }
        tc::mma_commit_warp(&bars.acc_full[t][ab]);
        ++used[t];
      }
      if (!ok) break;
      tc::mma_commit_warp(&bars.q_empty[st]);
      ++i;
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    }
    __syncwarp();
    tc::mma_commit_warp(&bars.mma_drain);
    mbar_wait_warp(&bars.mma_drain, 0, nullptr);
  } else if (warp == 2) {
    // ------------------------------------------------------------ row data, chunks ahead
    bool ok = true;
    int i = 0;
    for (int c = c0; c < c1 && ok; ++c) {
      if (!sees(c, 0)) continue;
      const int st = i % C::kStages;
      if (i >= C::kStages)
        ok = mbar_wait_warp(&bars.row_empty[st], (i / C::kStages - 1) & 1, abort_flag);
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < kChunk / 32; ++u) {
        const RowData x = row_data(a, head, c * kChunk + u * 32 + lane);
        row_lse[st][u * 32 + lane] = x.lse2;
        row_token[st][u * 32 + lane] = x.token;
      }
      mbar_arrive(&bars.row_full[st]);
      ++i;
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ warpgroups of keys
    const int t = (warp - 4) / 4, quarter = warp % 4;
    const int j = key0 + t * kTileKeys + quarter * 32 + lane;
    const uint32_t addr = tmem + (uint32_t(quarter * 32) << 16) + 2 * t * kChunk;
    const bool live = j < n;
    const size_t at = size_t(head) * a.out_len + j;
    const float prev = live && a.prev != nullptr ? a.prev[at] : 0.f;
    const bool good = live && page_good(a, b, j);
    const int first = first_token(a, n, j);
    const int all_from = first_token(a, n, key0 + t * kTileKeys + kTileKeys - 1);
    float sum = 0.f;
    bool ok = true;
    int i = 0, used = 0;
    for (int c = c0; c < c1 && ok; ++c) {
      if (!sees(c, 0)) continue;
      const int st = i % C::kStages;
      // (waited for by a warpgroup that skips the chunk too: its arrival below
      // must count for this round of the stage)
      ok = mbar_wait_warp(&bars.row_full[st], (i / C::kStages) & 1, abort_flag);
      if (!ok) break;
      if (sees(c, t)) {
        ok = mbar_wait_warp(&bars.acc_full[t][used & 1], (used >> 1) & 1, abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
        const bool masked = first_of_chunk(c) < all_from;
        sum += sum_columns(addr + (used & 1) * kChunk, kChunk, a.R - c * kChunk, masked,
                           row_lse[st], row_token[st], a.c, first);
        tc::fence_before_sync();
        mbar_arrive(&bars.acc_empty[t][used & 1]);
        ++used;
      }
      mbar_arrive(&bars.row_empty[st]);
      ++i;
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    } else if (live) {
      if (gridDim.y == 1) {
        const float kept = a.prev != nullptr ? a.decay * prev : 0.f;
        a.out[at] = good ? kept + sum : kept;
      } else {
        a.out[size_t(blockIdx.y) * heads * a.out_len + at] = good ? sum : 0.f;
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// out = decay · prev + the S partial sums, in order.
__global__ void __launch_bounds__(256)
weights_join_kernel(KwArgs a, const float* __restrict__ part, int S) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int head = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  bool bad = false;
  if (j >= request_len(a, head / a.Hkv, bad)) return;
  const size_t at = size_t(head) * a.out_len + j, step = size_t(gridDim.y) * a.out_len;
  float sum = 0.f;
#pragma unroll 4
  for (int s = 0; s < S; ++s) sum += part[s * step + at];
  a.out[at] = a.prev != nullptr ? fmaf(a.decay, a.prev[at], sum) : sum;
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream,
                   Args... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int NMAX>
cudaError_t launch_keys(const CUtensorMap& mk, const KeyWeightsArgs& w, const KwArgs& a) {
  const int N = (a.R + 15) / 16 * 16;
  CUtensorMap mq;
  if (!make_map_bf16_3d(&mq, w.q, D, a.R, uint64_t(a.B) * a.Hkv, N)) return cudaErrorInvalidValue;
  const long long tiles = 1LL * a.B * a.Hkv * ((a.cap + kTileKeys - 1) / kTileKeys);
  const int sms = device_sm_count() > 0 ? device_sm_count() : 1;
  return launch(weights_keys_kernel<D, NMAX>, dim3(unsigned(std::min<long long>(tiles, sms))),
                kThreads, KeysCfg<D, NMAX>::kDynSmem, w.stream, mq, mk, a, N);
}

template <int D>
cudaError_t launch_d(const KeyWeightsArgs& w, KwArgs a) {
  CUtensorMap mk, mq;
  const bool paged = w.block_table != nullptr;
  if (!make_map_bf16_3d(&mk, w.k, D, paged ? w.page_size : w.L,
                        uint64_t(paged ? w.num_pages : w.B) * w.Hkv, a.box_rows))
    return cudaErrorInvalidValue;
  if (a.R <= 64) return launch_keys<D, 64>(mk, w, a);
  if (a.R <= 256) return launch_keys<D, 256>(mk, w, a);
  if (!make_map_bf16_3d(&mq, w.q, D, a.R, uint64_t(a.B) * a.Hkv, kChunk))
    return cudaErrorInvalidValue;
  const int blocks = (a.cap + 2 * kTileKeys - 1) / (2 * kTileKeys);
  const int S = w.splits;
  KwArgs pa = a;
  if (S > 1) pa.out = w.part;
  cudaError_t e = launch(weights_rows_kernel<D>, dim3(unsigned(blocks) * a.B * a.Hkv, S), kThreads,
                         RowsCfg<D>::kDynSmem, w.stream, mq, mk, pa);
  if (e != cudaSuccess || S == 1) return e;
  return launch(weights_join_kernel, dim3((a.cap + 255) / 256, a.B * a.Hkv), 256, 0, w.stream, a,
                static_cast<const float*>(w.part), S);
}

}  // namespace

// Splits of the query rows: none while they stay in shared memory; else as
// many as give four CTAs per SM (their work differs under the causal mask),
// of eight chunks at least.
int key_weights_splits(int B, int Hkv, int R, int cap) {
  if (R <= 256) return 1;
  const long long sms = device_sm_count() > 0 ? device_sm_count() : 152;
  const long long ctas = 1LL * B * Hkv * ((cap + 2 * kTileKeys - 1) / (2 * kTileKeys));
  const long long most = std::max(1, (R + kChunk - 1) / kChunk / 8);
  return int(std::min<long long>(std::min<long long>(most, 64), (4 * sms + ctas - 1) / ctas));
}

cudaError_t launch_key_weights(const KeyWeightsArgs& w) {
  KwArgs a{w.lse, w.prev, w.out, w.seq_lens, w.block_table, w.B, w.Hkv, w.Hq / w.Hkv * w.T, w.T,
           w.len_cap, w.out_len, w.num_pages, w.page_size, w.max_pages, kTileKeys, w.causal,
           w.scale * kLog2e, w.decay};
  // copies of a key tile: whole tiles of a contiguous cache or a single
  // page, else the largest power of two that divides the page size
  if (w.block_table != nullptr && w.max_pages > 1)
    while (w.page_size % a.box_rows != 0) a.box_rows /= 2;
  return w.d == 64 ? launch_d<64>(w, a) : launch_d<128>(w, a);
}

}  // namespace attn
