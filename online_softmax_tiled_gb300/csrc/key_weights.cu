// Attention weight received by each cached key:
//   out[b, g, j] = decay · prev[b, g, j] + Σ_r exp(scale · q_r·k_j - lse_r)
// over the R = G·T query rows r of KV head g (the T query tokens of its G
// heads) that see key j. With the rows' log-sum-exp known the weights need
// no softmax of their own: a matrix product, an exponential per element and
// a sum over one axis.
//
// GB300 mapping. The product is taken transposed, Sᵀ = K Qᵀ: keys are the
// accumulator's rows (TMEM lanes), so that the thread of a key sums its
// weights over the columns in registers and no sum crosses threads. Per (key,
// row) the tensor core spends 2·d flops and the special-function unit one
// exponential (1/32 cycle of an SM each at d = 128): with many rows these two
// bound it, with few the reading of K. A warpgroup reads 128 accumulator
// columns into registers at once and gives the accumulator back before it
// computes, so that products and exponentials overlap. The rows' -lse/scale
// enters the accumulator as one more K = 16 step of the product (a tile of
// ones times three bf16 parts that make up the float32), because a per-column
// read of it from shared memory competes with the product's operands: both
// take about 100 bytes a cycle.
//
//  * At most 256 rows (decode steps, observation windows): the rows of a
//    (request, KV head) stay in shared memory and the keys stream past them
//    in tiles of 128, which the two warpgroups take in turn. One persistent
//    CTA per SM takes an equal share of all key tiles of the batch. Measured:
//    one token of 64 requests (4 rows a KV head, 8 KV heads, 2048 to 4096 keys
//    of 128 in 16-key pages) 72 us, 5.8 TB/s, bound by reading K; 64 tokens
//    over 2 x 16384 keys (256 rows) 22.5 us, 764 TFLOP/s, where a warpgroup
//    takes 2 x 1400 cycles to load and sum a tile's 256 columns and then waits
//    for its next product, 1500 to 1900 cycles from issue to use.
//  * More rows (every token of a prompt as an observer): 256 keys of a
//    (request, KV head) stay in shared memory, 128 per warpgroup, and the
//    rows stream past them in chunks of 128, chunks that see none of the
//    keys left out. A persistent CTA takes an equal share of all (256 keys,
//    128 rows) steps; where a block of keys falls to several CTAs, their
//    partial sums are added in a fixed order by a second kernel. Measured:
//    4096 tokens and keys, causal, 16 heads on 4: 42 us, 818 TFLOP/s of the
//    visible half, exponentials at 0.4 of the special-function unit's rate and
//    the tensor core as busy.
//
// Both forms at 256 rows (2 x 8 heads of 16384 keys): 22.5 us with the rows
// kept, 37 with the keys kept. Past 256 rows the kept rows and a ring of K do
// not fit in shared memory: 260 rows take 45 us, 512 take 49.
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
constexpr int kThreads = 352;     // TMA, MMA and row-data warps; two groups of four for the keys
constexpr float kLog2e = 1.4426950408889634f;

struct KwArgs {
  const float* lse;        // [B, Hkv, R]
  const float* prev;
  float* out;              // [B, Hkv, out_len]
  float* part;             // partial sums [slots][B, Hkv, out_len] (streaming rows)
  const int* seq_lens;
  const int* block_table;
  int B, Hkv, R, T, cap, out_len, num_pages, page_size, max_pages, box_rows;
  int causal, joined;      // joined: key tiles by make_map_bf16_joined's copies
  float c, inv_scale, decay;   // scale · log2 e, 1 / scale
};

// (kEarly: read before the kernel has waited, so from L2)
template <bool kEarly = false>
ATTN_DEVINL int request_len(const KwArgs& a, int b, bool& bad) {
  if (a.seq_lens == nullptr) return a.cap;
  const int n = kEarly ? __ldcg(a.seq_lens + b) : a.seq_lens[b];
  const bool wrong = n < 0 || n > a.cap;
  bad |= wrong;
  return wrong ? 0 : n;
}

// (a 64-bit division takes several hundred cycles)
ATTN_DEVINL long long quotient(long long x, long long y) {
  return (x | y) >> 32 ? x / y : uint32_t(x) / uint32_t(y);
}

// Where the copies of a key tile come from: lane i < boxes has the tile's i-th
// box. The page index is only looked at when the copies are issued, one tile
// later, so that reading it holds nothing up.
struct KeyBox {
  int row, outer, page;        // page: of a paged cache, outer then the KV head
  bool in;
};
ATTN_DEVINL KeyBox find_key_box(const KwArgs& a, int b, int g, int key0, int n, int lane) {
  const int shift = 31 - __clz(a.box_rows);            // box_rows is a power of two
  KeyBox x{0, 0, 0, lane < min(kTileKeys, n - key0 + a.box_rows - 1) >> shift};
  if (x.in) {
    const int key = key0 + lane * a.box_rows;
    if (a.block_table == nullptr) {
      x.row = key;
      x.outer = b * a.Hkv + g;
    } else {
      const int pi = key / a.page_size;
      x.row = key - pi * a.page_size;
      x.outer = g;
      x.page = a.block_table[size_t(b) * a.max_pages + pi];
    }
  }
  return x;
}
// A key tile in shared memory is made of 1024-byte pieces, 8 keys x 64
// elements (128-byte swizzle). Contiguous caches and single pages: one copy of
// 128 keys per 64-column half, the halves one after the other. Pages: one
// copy per page piece that takes both halves (a copy costs its issue, and
// 16-key pages need eight a tile either way), the halves of 8 keys next to
// each other.
struct KeySteps {
  uint32_t group, half;        // bytes from 8 keys to the next, from half to half
};
template <int D> ATTN_DEVINL KeySteps key_steps(const KwArgs& a) {
  return a.joined ? KeySteps{1024 * (D / 64), 1024} : KeySteps{1024, kTileKeys * 128};
}

// The copies of a tile (all lanes of a converged warp); boxes past the
// request's keys or behind a bad page index are left out (their lanes' sums
// are not used).
template <int D>
ATTN_DEVINL void load_key_tile(const KwArgs& a, const KeyBox& x, uint8_t* dst,
                               const CUtensorMap* map, uint64_t* bar, int lane) {
  constexpr int kAtoms = D / 64;
  const bool good = x.in && x.page >= 0 && (a.block_table == nullptr || x.page < a.num_pages);
  const uint32_t live = __ballot_sync(0xffffffffu, good);
  if (lane == 0)
    mbar_arrive_expect_tx(bar, uint32_t(__popc(live)) * a.box_rows * 128 * kAtoms);
  __syncwarp();
  const int outer = x.page * a.Hkv + x.outer;
  if (good) {
    if (a.joined) {
      tc::tma_load_5d(dst + lane * a.box_rows * 128 * kAtoms, map, 0, 0, 0, x.row / 8, outer, bar);
    } else {
#pragma unroll
      for (int at = 0; at < kAtoms; ++at)
        tc::tma_load_3d(dst + at * (kTileKeys * 128) + lane * a.box_rows * 128, map, 64 * at,
                        x.row, outer, bar);
    }
  }
}

// What a row needs besides Q: -lse/scale as three bf16 parts whose sum is the
// float32 value (far below any score where the row counts for nothing: no
// such row, or an infinite lse, as of a row that saw no key), and its token
// (INT_MIN where the row counts for nothing: a Q that is not finite would
// still reach the sum). Returns whether a row of the strip has an infinite
// lse: then every column is to be tested.
//
// The parts are the row's first three columns of a K = 16 operand tile: core
// matrices of 8 rows x 16 bytes, two along K, groups of 8 rows every 256
// bytes; the other columns stay zero.
constexpr int kPartsRow = 32;                 // bytes of a row in the operand tile
constexpr float kFarBelow = -3.0e38f;
// Rows n = lane, lane + 32, ... < 32·kRows of the tile are rows first + n of a
// strip of `length` that begins at row `base` of the head (the reads of all
// rows in flight together).
template <int kRows>
ATTN_DEVINL bool put_rows(const KwArgs& a, int head, int base, int first, int length, int count,
                          uint8_t* parts, int* token, int lane) {
  float l[kRows];
  const float* lse = a.lse + size_t(head) * a.R + base;
#pragma unroll
  for (int u = 0; u < kRows; ++u) l[u] = lse[min(first + u * 32 + lane, length - 1)];
  bool dead = false;
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int n = u * 32 + lane;
    if (n >= count) break;
    const bool in = first + n < length, none = fabsf(l[u]) == INFINITY;
    dead |= in && none;
    float v = -l[u] * a.inv_scale;
    if (!in || none || v < kFarBelow) v = kFarBelow;
    if (v > -kFarBelow) v = -kFarBelow;
    token[n] = in && !none ? (base + first + n) % a.T : INT_MIN;
    const float p0 = __bfloat162float(__float2bfloat16_rn(v));
    const float p1 = __bfloat162float(__float2bfloat16_rn(v - p0));
    *reinterpret_cast<uint4*>(parts + (n >> 3) * 256 + (n & 7) * 16) =
        make_uint4(pack_bf16x2(p0, p1), pack_bf16x2(v - p0 - p1, 0.f), 0u, 0u);
  }
  fence_proxy_async_smem();
  return __any_sync(0xffffffffu, dead);
}
// Ones for the other operand (128 rows x 16), zeros for `bytes` of parts.
ATTN_DEVINL void fill_parts(uint8_t* ones, uint8_t* parts, int bytes, int tid) {
  for (int i = tid; i < kTileKeys * kPartsRow / 16; i += kThreads)
    reinterpret_cast<uint4*>(ones)[i] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u,
                                                   0x3F803F80u);
  for (int i = tid; i < bytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(parts)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
}

// Sᵀ - lse/scale for one key tile against query rows, all lanes of the
// issuing warp: D/16 steps over K and Q (128-byte swizzle; the second half of
// K lies k_half, that of Q q_half descriptor units of 16 bytes on), then the
// parts. The descriptors are the caller's, so that a step costs two additions.
template <int D>
ATTN_DEVINL void issue_product(uint32_t acc, uint64_t k_desc, uint32_t k_half, uint64_t q_desc,
                               uint32_t q_half, uint64_t ones_desc, uint64_t parts_desc,
                               uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    tc::mma_ss_warp(acc, k_desc + (kk / 4) * k_half + (kk % 4) * 2,
                    q_desc + (kk / 4) * q_half + (kk % 4) * 2, idesc, kk > 0);
  tc::mma_ss_warp(acc, ones_desc, parts_desc, idesc, 1u);
}
ATTN_DEVINL uint64_t parts_desc_of(uint32_t addr) {
  return tc::smem_desc(addr, 128, 256, tc::kLayoutNone);
}

ATTN_DEVINL float exp2_unit(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Adds exp2(c·s) over 16 columns. Masked form: a column counts if its token
// is at least `first` (the first token that sees the key).
template <bool kMask>
ATTN_DEVINL void add_columns(const uint32_t* s, const int* token, float c, int first,
                             f2 (&sum)[4]) {
  const f2 c2{c, c};
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    f2 x = mul2(f2{__uint_as_float(s[e]), __uint_as_float(s[e + 1])}, c2);
    f2 y = mul2(f2{__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])}, c2);
    x = f2{exp2_unit(x.x), exp2_unit(x.y)};
    y = f2{exp2_unit(y.x), exp2_unit(y.y)};
    if (kMask) {
      const int4 t = *reinterpret_cast<const int4*>(token + e);
      x.x = t.x >= first ? x.x : 0.f;
      x.y = t.y >= first ? x.y : 0.f;
      y.x = t.z >= first ? y.x : 0.f;
      y.y = t.w >= first ? y.y : 0.f;
    }
    sum[(e / 2) & 3] = add2(sum[(e / 2) & 3], x);
    sum[(e / 2 + 1) & 3] = add2(sum[(e / 2 + 1) & 3], y);
  }
}

// The sum over n columns (a multiple of 16, at most 128) of an accumulator,
// which is given back (an arrival per warp on `empty`, if any) as soon as it
// is in registers.
// masked: every column is tested; otherwise only those past `full`.
ATTN_DEVINL float sum_columns(uint32_t addr, int n, int full, bool masked, const int* token,
                              float c, int first, uint64_t* empty, int lane) {
  uint32_t s[128];
  if (n == 128) {
#pragma unroll
    for (int i = 0; i < 128; i += 32)
      tc::tmem_ld32(addr + i, *reinterpret_cast<uint32_t(*)[32]>(&s[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 128; i += 16)
      if (i < n) tc::tmem_ld16(addr + i, *reinterpret_cast<uint32_t(*)[16]>(&s[i]));
  }
  tc::tmem_ld_wait();
  if (empty != nullptr) {
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(empty);
  }
  f2 sum[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
  if (!masked && n == 128 && full >= 128) {
#pragma unroll
    for (int i = 0; i < 128; i += 16) add_columns<false>(s + i, token + i, c, first, sum);
  } else {
#pragma unroll
    for (int i = 0; i < 128; i += 16)
      if (i < n) {
        if (masked || i + 16 > full)
          add_columns<true>(s + i, token + i, c, first, sum);
        else
          add_columns<false>(s + i, token + i, c, first, sum);
      }
  }
  const f2 t = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
  return t.x + t.y;
}

// What the thread of a key reads for its output, on its way during the sum.
struct KeyOut {
  float prev;
  int page;                    // of a paged cache; checked when the sum is written
};
ATTN_DEVINL KeyOut find_key_out(const KwArgs& a, int b, int g, int j, int n) {
  KeyOut o{0.f, 0};
  if (j < n) {
    if (a.prev != nullptr) o.prev = a.prev[(size_t(b) * a.Hkv + g) * a.out_len + j];
    if (a.block_table != nullptr)
      o.page = a.block_table[size_t(b) * a.max_pages + j / a.page_size];
  }
  return o;
}
ATTN_DEVINL bool page_good(const KwArgs& a, const KeyOut& o) {
  const bool good = a.block_table == nullptr || (o.page >= 0 && o.page < a.num_pages);
  if (!good) attn_flag_error(kErrBadIndex);
  return good;
}
ATTN_DEVINL void write_key(const KwArgs& a, size_t at, const KeyOut& o, float sum) {
  const float kept = a.prev != nullptr ? a.decay * o.prev : 0.f;
  a.out[at] = page_good(a, o) ? kept + sum : kept;
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
  static constexpr int kQBufs = NMAX <= 128 ? 2 : 1;
  static constexpr int kQBytes = NMAX * D * 2;
  static constexpr int kStages = 4 * (128 / D);
  static constexpr int kKOff = kQBufs * kQBytes;
  static constexpr int kOnesOff = kKOff + kStages * kTileBytes;
  static constexpr int kPartsOff = kOnesOff + kTileKeys * kPartsRow;   // of two heads
  static constexpr int kPartsBytes = NMAX * kPartsRow;
  static constexpr int kDynSmem = kPartsOff + 2 * kPartsBytes + 1024;
  // accumulators per warpgroup, of NMAX columns (a product of 256 columns
  // reads 96 bytes of shared memory a cycle, one of 128 columns 128: the limit)
  static constexpr int kTurns = 256 / NMAX;
  static constexpr uint32_t kTmemCols = 512;
};

struct KeysBars {
  uint64_t q_full[2], q_empty[2], k_full[8], k_empty[8], acc_full[2][2], acc_empty[2][2];
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
  __shared__ __align__(16) int row_token[2][NMAX];
  __shared__ int row_dead[2];          // some row has an infinite lse
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    bars.abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.row_full[i], 32);
      mbar_init(&bars.row_empty[i], 8 + 1);   // the key warps and the products
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.acc_full[i >> 1][i & 1], 1);
      mbar_init(&bars.acc_empty[i >> 1][i & 1], 4);
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
  fill_parts(smem + C::kOnesOff, smem + C::kPartsOff, 2 * C::kPartsBytes, tid);
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
    const int first = int(quotient(1LL * total * blockIdx.x, gridDim.x));
    const int last = int(quotient(1LL * total * (blockIdx.x + 1), gridDim.x));
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
    // (the boxes of a tile are looked up one tile ahead of its copies)
    bool ok = true, fresh = true;
    int heads = 0, i = 0;
    KeyBox box{0, 0, 0, false};
    if (count > 0) box = find_key_box(a, w.b, w.g, w.tile * kTileKeys, w.n, lane);
    for (; i < count && ok; ++i) {
      const int head = w.b * a.Hkv + w.g;
      const bool turn = w.next(a);
      KeyBox next{0, 0, 0, false};
      if (i + 1 < count) next = find_key_box(a, w.b, w.g, w.tile * kTileKeys, w.n, lane);
      if (fresh) {
        const int qb = heads % C::kQBufs;
        if (heads >= C::kQBufs)
          ok = mbar_wait_warp(&bars.q_empty[qb], (heads / C::kQBufs - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars.q_full[qb], uint32_t(N) * D * 2);
          for (int at = 0; at < C::kAtoms; ++at)
            tc::tma_load_3d(smem + qb * C::kQBytes + at * (NMAX * 128), &map_q, 64 * at, 0,
                            head, &bars.q_full[qb]);
        }
        __syncwarp();
        ++heads;
      }
      const int st = i % C::kStages;
      if (i >= C::kStages)
        ok = mbar_wait_warp(&bars.k_empty[st], (i / C::kStages - 1) & 1, abort_flag);
      if (!ok) break;
      load_key_tile<D>(a, box, smem + C::kKOff + st * C::kTileBytes, &map_k, &bars.k_full[st],
                       lane);
      box = next;
      fresh = turn;
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
    const KeySteps step = key_steps<D>(a);
    const uint64_t q0 = tc::smem_desc(smem_u32(smem), 16, 1024, tc::kLayoutSW128);
    const uint64_t k0 = tc::smem_desc(smem_u32(smem + C::kKOff), 16, step.group, tc::kLayoutSW128);
    const uint64_t ones = parts_desc_of(smem_u32(smem + C::kOnesOff));
    const uint64_t parts0 = parts_desc_of(smem_u32(smem + C::kPartsOff));
    const uint32_t k_half = step.half / 16, q_half = NMAX * 128 / 16;
    const uint32_t idesc = tc::idesc_bf16_f32(kTileKeys, N, false, false);
    bool ok = true, fresh = true;
    int heads = 0;
    uint64_t q_desc = q0, parts = parts0;
    for (int i = 0; i < count && ok; ++i) {
      if (fresh) {
        ok = mbar_wait_warp(&bars.q_full[heads % C::kQBufs], (heads / C::kQBufs) & 1, abort_flag);
        if (ok) ok = mbar_wait_warp(&bars.row_full[heads & 1], (heads >> 1) & 1, abort_flag);
        q_desc = q0 + (heads % C::kQBufs) * (C::kQBytes / 16);
        parts = parts0 + (heads & 1) * (C::kPartsBytes / 16);
        ++heads;
      }
      const int st = i % C::kStages;
      const int t = i & 1, use = i >> 1, turn = use % C::kTurns;
      if (ok) {
        uint64_t* full = &bars.k_full[st];
        const uint32_t k_phase = (i / C::kStages) & 1;
        ok = use >= C::kTurns
                 ? mbar_wait2_warp(full, k_phase, &bars.acc_empty[t][turn],
                                   (use / C::kTurns - 1) & 1, abort_flag)
                 : mbar_wait_warp(full, k_phase, abort_flag);
      }
      if (!ok) break;
      tc::fence_after_sync();
      issue_product<D>(tmem + (C::kTurns * t + turn) * NMAX, k0 + st * (C::kTileBytes / 16), k_half,
                       q_desc, q_half, ones, parts, idesc);
      tc::mma_commit_warp(&bars.acc_full[t][turn]);
      tc::mma_commit_warp(&bars.k_empty[st]);
      fresh = w.next(a);
      if (fresh) {
        tc::mma_commit_warp(&bars.q_empty[(heads - 1) % C::kQBufs]);
        tc::mma_commit_warp(&bars.row_empty[(heads - 1) & 1]);
      }
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
        if (heads >= 2)
          ok = mbar_wait_warp(&bars.row_empty[rb], ((heads >> 1) - 1) & 1, abort_flag);
        if (!ok) break;
        const bool dead = put_rows<NMAX / 32>(a, w.b * a.Hkv + w.g, 0, 0, a.R, N,
                                              smem + C::kPartsOff + rb * C::kPartsBytes,
                                              row_token[rb], lane);
        if (lane == 0) row_dead[rb] = dead;
        mbar_arrive(&bars.row_full[rb]);
        ++heads;
      }
      fresh = w.next(a);
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    }
  } else {
    // ------------------------------------------------------------ warpgroups of keys
    const int t = (warp - 3) / 4, quarter = warp % 4;    // takes tiles t, t + 2, ...
    const int r = quarter * 32 + lane;                   // key of the tile (TMEM lane)
    const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
    bool ok = true, fresh = true;
    int heads = 0;
    for (int i = 0; i < count && ok; ++i) {
      if (fresh) {
        __syncwarp();
        if (heads > 0 && lane == 0) mbar_arrive(&bars.row_empty[(heads - 1) & 1]);
        ok = mbar_wait_warp(&bars.row_full[heads & 1], (heads >> 1) & 1, abort_flag);
        if (!ok) break;
        ++heads;
      }
      if ((i & 1) == t) {
        const int use = i >> 1, turn = use % C::kTurns;
        const int j = w.tile * kTileKeys + r, first = first_token(a, w.n, j);
        const KeyOut out = find_key_out(a, w.b, w.g, j, w.n);
        ok = mbar_wait_warp(&bars.acc_full[t][turn], (use / C::kTurns) & 1, abort_flag);
        if (!ok) break;
        tc::fence_after_sync();
        // the tile needs its columns tested if the first token misses its last key
        const bool masked = first_token(a, w.n, w.tile * kTileKeys + kTileKeys - 1) > 0 ||
                            row_dead[(heads - 1) & 1];
        const int* token = row_token[(heads - 1) & 1];
        float sum = 0.f;
#pragma unroll 1
        for (int col = 0; col < N; col += 128)
          sum += sum_columns(lanes + (C::kTurns * t + turn) * NMAX + col, min(N - col, 128),
                             a.R - col, masked, token + col, a.c, first,
                             col + 128 < N ? nullptr : &bars.acc_empty[t][turn], lane);
        if (j < w.n) write_key(a, (size_t(w.b) * a.Hkv + w.g) * a.out_len + j, out, sum);
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

constexpr int kChunk = 128;             // query rows per step
constexpr int kBlock = 2 * kTileKeys;   // keys per step

// The R rows of a KV head as strips of `length` rows, cut into chunks of 128
// (the last one of a strip may be short). A strip is all rows, or under a
// causal mask a query head, whose blocks of keys then need the chunks from
// their first token's on only. A step is one chunk against one block of keys;
// a CTA takes `least` steps at least.
struct RowSteps {
  int strips, length, chunks, skip, least;
};
RowSteps row_steps(int R, int T, bool per_head) {
  RowSteps s;
  s.strips = per_head ? R / T : 1;
  s.length = per_head ? T : R;
  s.chunks = (s.length + kChunk - 1) / kChunk;
  s.skip = per_head;
  // about two steps pay for a CTA's start; at most 32 partial sums a key
  const long long all = 1LL * s.strips * s.chunks;
  s.least = int(std::max(4LL, (all + 29) / 30));
  return s;
}
// A strip per head leaves out half the steps of its last T keys, but pays for
// every head's short last chunk: T = 4096 tokens and keys take half the steps,
// 192 tokens of four heads over 2 x 16384 keys 8 instead of 6 (108 us against
// 65 when both were measured).
RowSteps row_steps_for(int R, int T, int causal, int cap) {
  const RowSteps head = row_steps(R, T, true), one = row_steps(R, T, false);
  const double hidden = 0.5 * std::min(T, cap) / cap;
  return causal && head.strips * head.chunks * (1 - hidden) < one.chunks ? head : one;
}
__host__ __device__ inline int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// The first chunk of a strip that sees block k of a request of n keys, and
// the steps of the block.
ATTN_DEVINL int first_chunk(const KwArgs& a, const RowSteps& rs, int n, int k) {
  return rs.skip ? first_token(a, n, k * kBlock) / kChunk : 0;
}
ATTN_DEVINL int steps_of(const KwArgs& a, const RowSteps& rs, int n, int k) {
  return rs.strips * (rs.chunks - first_chunk(a, rs, n, k));
}
// The steps of a head's first k blocks. Block i leaves out max(0, 2 i - c)
// chunks of a strip, c = ceil((n - T) / 128): an arithmetic series from the
// first i with 2 i > c on.
ATTN_DEVINL long long steps_before(const KwArgs& a, const RowSteps& rs, int n, int k) {
  long long s = 1LL * k * rs.chunks;
  if (rs.skip) {
    const int m = n - a.T, c = m >= 0 ? (m + kChunk - 1) / kChunk : -(-m / kChunk);
    const int from = c >= 0 ? c / 2 + 1 : 0;
    if (k > from) s -= 1LL * (k - from) * (k - 1 + from - c);
  }
  return s * rs.strips;
}
ATTN_DEVINL long long steps_of_head(const KwArgs& a, const RowSteps& rs, int n) {
  return steps_before(a, rs, n, blocks_of(n));
}
// Steps per CTA: an equal share, `least` at least.
ATTN_DEVINL long long steps_per_cta(const RowSteps& rs, long long total, int grid) {
  const long long share = quotient(total + grid - 1, grid);
  return share > rs.least ? share : rs.least;
}

template <int D>
struct RowsCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kTileKeys * D * 2;
  static constexpr int kStages = 4;
  static constexpr int kQOff = 2 * kTileBytes;       // two key tiles first
  static constexpr int kOnesOff = kQOff + kStages * kTileBytes;
  static constexpr int kPartsOff = kOnesOff + kTileKeys * kPartsRow;   // of a stage's rows
  static constexpr int kPartsBytes = kChunk * kPartsRow;
  static constexpr int kDynSmem = kPartsOff + kStages * kPartsBytes + 1024;
  static constexpr uint32_t kTmemCols = 512;         // [tile][turn] accumulators of kChunk columns
};

struct RowsBars {
  uint64_t k_full, k_empty, q_full[4], q_empty[4], acc_full[2][2], acc_empty[2][2];
  uint64_t row_full[4], row_empty[4], mma_drain;
  uint32_t tmem_base;
  int abort;
  long long warp_sum[kThreads / 32];
  long long begin, end, each;        // this CTA's steps; the share of a CTA
  int start[3];                      // request, head, block where they begin
  int offset;                        // steps of that block before them
};

// The pieces of a CTA's share: runs of steps of one (request, head, block).
struct PieceWalk {
  int b, g, k, n, blocks;
  int step0, steps;                  // the piece, in steps of the block
  int all;                           // the block's steps
  long long left;
  ATTN_DEVINL void open(const KwArgs& a) {
    bool bad = false;
    n = request_len(a, b, bad);
    blocks = blocks_of(n);
  }
  ATTN_DEVINL void cut(const KwArgs& a, const RowSteps& rs, int from) {
    all = steps_of(a, rs, n, k);
    step0 = from;
    steps = int(min((long long)(all - from), left));
  }
  ATTN_DEVINL void next(const KwArgs& a, const RowSteps& rs) {
    left -= steps;
    if (left <= 0) return;
    if (++k >= blocks) {
      k = 0;
      if (++g >= a.Hkv) {
        g = 0;
        do {
          ++b;
          open(a);
        } while (blocks == 0);
      }
    }
    cut(a, rs, 0);
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
weights_rows_kernel(const __grid_constant__ CUtensorMap map_q,
                    const __grid_constant__ CUtensorMap map_k, KwArgs a, RowSteps rs) {
  using C = RowsCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ RowsBars bars;
  __shared__ __align__(16) int row_token[C::kStages][kChunk];
  __shared__ int row_dead[C::kStages];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    bars.abort = 0;
    mbar_init(&bars.k_full, 2);
    mbar_init(&bars.k_empty, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.row_full[i], 32);
      mbar_init(&bars.row_empty[i], 8 + 1);   // the key warps and the products
    }
    for (int t = 0; t < 2; ++t)
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.acc_full[t][i], 1);
        mbar_init(&bars.acc_empty[t][i], 4);
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
  fill_parts(smem + C::kOnesOff, smem + C::kPartsOff, C::kStages * C::kPartsBytes, tid);
  pdl_wait_primary();
  pdl_launch_dependents();
  // This CTA's share of all steps: thread t counts a run of requests, a scan
  // over the threads gives where each run begins.
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int r0 = min(a.B, tid * per), r1 = min(a.B, r0 + per);
    long long mine = 0;
    bool bad = false;
    for (int b = r0; b < r1; ++b) mine += steps_of_head(a, rs, request_len(a, b, bad)) * a.Hkv;
    if (bad && blockIdx.x == 0) attn_flag_error(kErrBadIndex);
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) bars.warp_sum[warp] = upto;
    __syncthreads();
    long long before = upto - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += bars.warp_sum[w];
      total += bars.warp_sum[w];
    }
    const long long each = steps_per_cta(rs, total, gridDim.x);
    const long long begin = min(total, each * blockIdx.x), end = min(total, begin + each);
    if (tid == 0) {
      bars.begin = begin;
      bars.end = end;
      bars.each = each;
    }
    if (begin < end && before <= begin && begin < before + mine) {
      long long at = before;
      for (int b = r0; b < r1; ++b) {
        const int n = request_len(a, b, bad);
        const long long head = steps_of_head(a, rs, n);
        if (begin < at + head * a.Hkv) {
          const int g = int(quotient(begin - at, head));
          const long long rest = begin - at - g * head;
          int k = 0, over = blocks_of(n);                // the last block that begins at or before
          while (over - k > 1) {
            const int mid = (k + over) / 2;
            if (steps_before(a, rs, n, mid) <= rest)
              k = mid;
            else
              over = mid;
          }
          bars.start[0] = b;
          bars.start[1] = g;
          bars.start[2] = k;
          bars.offset = int(rest - steps_before(a, rs, n, k));
          break;
        }
        at += head * a.Hkv;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = bars.tmem_base;
  volatile int* abort_flag = &bars.abort;
  PieceWalk w{bars.start[0], bars.start[1], bars.start[2], 0, 0, 0, 0, 0, bars.end - bars.begin};
  if (w.left > 0) {
    w.open(a);
    w.cut(a, rs, bars.offset);
  }
  // Step s of a block is chunk (first + s mod per) of strip s / per; and the
  // step after one.
  struct Step {
    int strip, chunk;
  };
  auto step_at = [&](int s) {
    const int c0 = first_chunk(a, rs, w.n, w.k), per = rs.chunks - c0;
    return Step{s / per, c0 + s % per};
  };
  auto advance = [&](Step& s) {
    if (++s.chunk == rs.chunks) {
      s.chunk = first_chunk(a, rs, w.n, w.k);
      ++s.strip;
    }
  };
  // whether tile t of the block has keys, and whether a chunk's last token
  // sees its first one
  auto sees = [&](const Step& s, int t) {
    const int key = w.k * kBlock + t * kTileKeys;
    if (key >= w.n) return false;
    if (!rs.skip) return true;
    return min(rs.length, s.chunk * kChunk + kChunk) > first_token(a, w.n, key);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (the whole warp)
    bool ok = true;
    int i = 0, pieces = 0;                               // chunks and blocks asked for
    for (; w.left > 0 && ok; w.next(a, rs)) {
      KeyBox box[2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
        box[t] = find_key_box(a, w.b, w.g, w.k * kBlock + t * kTileKeys, w.n, lane);
      Step x = step_at(w.step0);
      for (int s = 0; s < w.steps && ok; ++s, ++i, advance(x)) {
        // The keys of the block before leave when its last products are done:
        // meanwhile the first chunks of this one are on their way.
        if (s == min(w.steps, C::kStages - 1) - 1) {
          if (pieces > 0) ok = mbar_wait_warp(&bars.k_empty, (pieces - 1) & 1, abort_flag);
          if (!ok) break;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (w.k * kBlock + t * kTileKeys < w.n)
              load_key_tile<D>(a, box[t], smem + t * C::kTileBytes, &map_k, &bars.k_full, lane);
            else if (lane == 0)
              mbar_arrive(&bars.k_full);
          ++pieces;
        }
        const int st = i % C::kStages;
        if (i >= C::kStages)
          ok = mbar_wait_warp(&bars.q_empty[st], (i / C::kStages - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars.q_full[st], C::kTileBytes);
          for (int at = 0; at < C::kAtoms; ++at)
            tc::tma_load_3d(smem + C::kQOff + st * C::kTileBytes + at * (kChunk * 128), &map_q,
                            64 * at, x.chunk * kChunk,
                            (w.b * a.Hkv + w.g) * rs.strips + x.strip, &bars.q_full[st]);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
      // the loads in flight land before the CTA exits
      if (pieces > 0) mbar_wait_warp(&bars.k_full, (pieces - 1) & 1, nullptr);
      for (int j = max(0, i - C::kStages); j < i; ++j)
        mbar_wait_warp(&bars.q_full[j % C::kStages], (j / C::kStages) & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the whole warp)
    const KeySteps step = key_steps<D>(a);
    const uint64_t k0 = tc::smem_desc(smem_u32(smem), 16, step.group, tc::kLayoutSW128);
    const uint64_t q0 = tc::smem_desc(smem_u32(smem + C::kQOff), 16, 1024, tc::kLayoutSW128);
    const uint64_t ones = parts_desc_of(smem_u32(smem + C::kOnesOff));
    const uint64_t parts0 = parts_desc_of(smem_u32(smem + C::kPartsOff));
    constexpr uint32_t idesc = tc::idesc_bf16_f32(kTileKeys, kChunk, false, false);
    bool ok = true;
    int i = 0, pieces = 0, used[2] = {0, 0};
    for (; w.left > 0 && ok; w.next(a, rs)) {
      ok = mbar_wait_warp(&bars.k_full, pieces & 1, abort_flag);
      ++pieces;
      Step x = step_at(w.step0);
      for (int s = 0; s < w.steps && ok; ++s, ++i, advance(x)) {
        const int st = i % C::kStages;
        ok = mbar_wait2_warp(&bars.q_full[st], (i / C::kStages) & 1, &bars.row_full[st],
                             (i / C::kStages) & 1, abort_flag);
        for (int t = 0; t < 2 && ok; ++t) {
          if (!sees(x, t)) continue;
          const int ab = used[t] & 1;
          if (used[t] >= 2)
            ok = mbar_wait_warp(&bars.acc_empty[t][ab], ((used[t] >> 1) - 1) & 1, abort_flag);
          if (!ok) break;
          tc::fence_after_sync();
          issue_product<D>(tmem + (2 * t + ab) * kChunk, k0 + t * (C::kTileBytes / 16),
                           step.half / 16, q0 + st * (C::kTileBytes / 16), kChunk * 128 / 16, ones,
                           parts0 + st * (C::kPartsBytes / 16), idesc);
          tc::mma_commit_warp(&bars.acc_full[t][ab]);
          ++used[t];
        }
        if (!ok) break;
        tc::mma_commit_warp(&bars.q_empty[st]);
        tc::mma_commit_warp(&bars.row_empty[st]);
      }
      if (ok) tc::mma_commit_warp(&bars.k_empty);
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
    for (; w.left > 0 && ok; w.next(a, rs)) {
      Step x = step_at(w.step0);
      for (int s = 0; s < w.steps; ++s, ++i, advance(x)) {
        const int st = i % C::kStages;
        if (i >= C::kStages)
          ok = mbar_wait_warp(&bars.row_empty[st], (i / C::kStages - 1) & 1, abort_flag);
        if (!ok) break;
        const bool dead = put_rows<kChunk / 32>(
            a, w.b * a.Hkv + w.g, x.strip * rs.length, x.chunk * kChunk, rs.length, kChunk,
            smem + C::kPartsOff + st * C::kPartsBytes, row_token[st], lane);
        if (lane == 0) row_dead[st] = dead;
        mbar_arrive(&bars.row_full[st]);
      }
    }
    if (!ok) {
      if (lane == 0) attn_flag_error(kErrTimeout);
      bars.abort = 1;
    }
  } else {
    // ------------------------------------------------------------ warpgroups of keys
    const int t = (warp - 3) / 4, quarter = warp % 4;
    const int r = quarter * 32 + lane;                   // key of the tile (TMEM lane)
    const uint32_t addr = tmem + (uint32_t(quarter * 32) << 16) + 2 * t * kChunk;
    long long at_step = bars.begin;
    bool ok = true;
    int i = 0, used = 0;
    for (; w.left > 0 && ok; w.next(a, rs)) {
      const int key0 = w.k * kBlock + t * kTileKeys, j = key0 + r;
      const KeyOut out = find_key_out(a, w.b, w.g, j, w.n);
      const int first = first_token(a, w.n, j);
      const int all_from = first_token(a, w.n, key0 + kTileKeys - 1);
      float sum = 0.f;
      Step x = step_at(w.step0);
      for (int s = 0; s < w.steps; ++s, ++i, advance(x)) {
        const int st = i % C::kStages;
        if (sees(x, t)) {
          const int turn = used & 1;
          ok = mbar_wait_warp(&bars.acc_full[t][turn], (used >> 1) & 1, abort_flag);
          if (!ok) break;
          tc::fence_after_sync();
          // tested column by column if the chunk's first token misses a key
          const bool masked =
              (rs.skip ? x.chunk * kChunk : 0) < all_from || row_dead[st];
          sum += sum_columns(addr + turn * kChunk, kChunk, rs.length - x.chunk * kChunk, masked,
                             row_token[st], a.c, first, &bars.acc_empty[t][turn], lane);
          ++used;
        } else {
          // (waited for all the same, so that the arrival below counts for
          // this round of the stage; above, the product has waited for it)
          ok = mbar_wait_warp(&bars.row_full[st], (i / C::kStages) & 1, abort_flag);
          if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.row_empty[st]);
      }
      if (!ok) break;
      const size_t at = (size_t(w.b) * a.Hkv + w.g) * a.out_len + j;
      if (j >= w.n) {
      } else if (w.steps == w.all) {                     // the whole block is this CTA's
        write_key(a, at, out, sum);
      } else {
        // the CTA's place among those of the block
        const int slot = int(blockIdx.x) - int(quotient(at_step - w.step0, bars.each));
        a.part[size_t(slot) * a.B * a.Hkv * a.out_len + at] = page_good(a, out) ? sum : 0.f;
      }
      at_step += w.steps;
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

// out = decay · prev + the partial sums of a block that fell to several CTAs,
// in the order of the CTAs. Grid: x blocks of 256 keys, y (request, KV head).
__global__ void __launch_bounds__(kBlock)
weights_join_kernel(KwArgs a, RowSteps rs, int grid) {
  __shared__ long long sums[2][kBlock / 32];
  const int b = blockIdx.y / a.Hkv, g = blockIdx.y % a.Hkv, k = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  // steps of all requests, and of those before this one
  long long total = 0, before = 0;
  for (int i = tid; i < a.B; i += kBlock) {
    const long long s = steps_of_head(a, rs, request_len<true>(a, i, bad)) * a.Hkv;
    total += s;
    if (i < b) before += s;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, off);
    before += __shfl_xor_sync(0xffffffffu, before, off);
  }
  if (lane == 0) {
    sums[0][tid >> 5] = total;
    sums[1][tid >> 5] = before;
  }
  __syncthreads();
  total = before = 0;
  for (int w = 0; w < kBlock / 32; ++w) {
    total += sums[0][w];
    before += sums[1][w];
  }
  const int n = request_len<true>(a, b, bad), j = k * kBlock + tid;
  const long long first = before + g * steps_of_head(a, rs, n) + steps_before(a, rs, n, k);
  const long long each = steps_per_cta(rs, total, grid);
  const long long last = first + steps_of(a, rs, n, k) - 1;
  const int slots = int(quotient(last, each) - quotient(first, each)) + 1;
  // (Lengths may be read before, from L2: the kernel that made the sums lets this one
  // start only once all that precedes the call is complete.)
  pdl_wait_primary();
  pdl_launch_dependents();
  if (j >= n || slots == 1) return;                      // (one: written where it was summed)
  const size_t at = size_t(blockIdx.y) * a.out_len + j, step = size_t(gridDim.y) * a.out_len;
  float sum = 0.f;
#pragma unroll 4
  for (int s = 0; s < slots; ++s) sum += a.part[s * step + at];
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
  const uint64_t outer = uint64_t(paged ? w.num_pages : w.B) * w.Hkv;
  if (!(a.joined ? make_map_bf16_joined(&mk, w.k, D, w.page_size, outer, a.box_rows)
                 : make_map_bf16_3d(&mk, w.k, D, paged ? w.page_size : w.L, outer, a.box_rows)))
    return cudaErrorInvalidValue;
  // Up to 128 rows there is room for those of the next (request, head) too:
  // 99.7 against 102.7 us for 4 rows and 64 x 4096 keys, 16.7 against 16.9 for
  // 128 rows and 2 x 16384.
  if (a.R <= 128) return launch_keys<D, 128>(mk, w, a);
  if (a.R <= 256) return launch_keys<D, 256>(mk, w, a);
  const RowSteps rs = row_steps_for(a.R, a.T, a.causal, a.cap);
  if (!make_map_bf16_3d(&mq, w.q, D, rs.length, uint64_t(a.B) * a.Hkv * rs.strips, kChunk))
    return cudaErrorInvalidValue;
  const long long most = 1LL * a.B * a.Hkv * blocks_of(a.cap) * rs.strips * rs.chunks;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 1;
  const int grid = int(std::min<long long>(sms, (most + rs.least - 1) / rs.least));
  cudaError_t e = launch(weights_rows_kernel<D>, dim3(grid), kThreads, RowsCfg<D>::kDynSmem,
                         w.stream, mq, mk, a, rs);
  if (e != cudaSuccess) return e;
  return launch(weights_join_kernel, dim3(blocks_of(a.cap), a.B * a.Hkv), 2 * kTileKeys, 0,
                w.stream, a, rs, grid);
}

}  // namespace

int key_weights_slots(int R, int T) {
  if (R <= 256) return 0;
  int most = 0;
  for (const bool per_head : {false, true}) {
    const RowSteps rs = row_steps(R, T, per_head);
    most = std::max(most, (rs.strips * rs.chunks - 1) / rs.least + 2);
  }
  return most;
}

cudaError_t launch_key_weights(const KeyWeightsArgs& w) {
  KwArgs a{w.lse, w.prev, w.out, w.part, w.seq_lens, w.block_table, w.B, w.Hkv,
           w.Hq / w.Hkv * w.T, w.T, w.len_cap, w.out_len, w.num_pages, w.page_size, w.max_pages,
           kTileKeys, w.causal, w.block_table != nullptr && w.max_pages > 1, w.scale * kLog2e,
           1.f / w.scale, w.decay};
  // copies of a key tile: whole tiles of a contiguous cache or a single
  // page, else the largest power of two that divides the page size, both
  // 64-column halves in one copy (issuing a copy takes about 100 cycles: 99.7
  // against 121.9 us for 64 x 4096 keys in 16-key pages)
  if (w.block_table != nullptr && w.max_pages > 1)
    while (w.page_size % a.box_rows != 0) a.box_rows /= 2;
  return w.d == 64 ? launch_d<64>(w, a) : launch_d<128>(w, a);
}

}  // namespace attn
