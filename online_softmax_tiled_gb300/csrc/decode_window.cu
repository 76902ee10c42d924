// Decode of T tokens per request over a paged cache, under a sliding window
// and the first tokens that stay visible, the cache in bf16
// (attn_decode_window) or in 4 bits (attn_decode_cache4).
//
// Mathematics. Softmax attention with the online recurrence: per query row a
// reference m, Σ p and Σ p v of p = 2^(s - m); the reference moves only when a
// score passes it by 8, so p <= 2^8. Partial sums of one row, of warps or of
// teams of warps, are joined exactly on the larger reference.
//
// 4 bits. With K codes k̂ and one scale per group of 32 elements,
// s = Σ_c scale_c (Σ_{i in c} q_i k̂_i): the sums of a group are one pair of
// matrix products on exact float16 values (queries are scaled by a power of two
// per row, which float16 then holds to 2^-33 of the row's largest), scaled and
// added in float32. For V the scale differs per key, the index summed over:
// P·scale_c is what enters the product, in float16 (2^-12 of a probability; bf16
// would lose 2^-9) times a power of two f that follows the largest scale seen,
// so that it stays between 2^-24 and 2^15: the largest that the row itself has seen.
//
// bf16. P enters P·V as two bf16 parts (off by 2^-16 of a probability at most).
//
// Work. Memory bound: 4·D bytes of K and V per key and KV head (4 bits: 9/8·D),
// 4·D flops per (query row, key). A warp takes 16 keys a step (4 bits: 32). Sᵀ = K Qᵀ has the keys as rows of the fragments, so that 8 query rows (the heads
// of a group times the tokens) fill an instruction; P moves into the fragments of Oᵀ =
// Vᵀ Pᵀ by transposes of 8 x 8 within the warp. K and V fragments of a 4-bit row are
// built in registers straight from its bytes (fp4.cuh), at one conversion for two
// values; the tensor instructions are those that take both operands from
// registers, since values unpacked for the ones that read shared memory would be
// written there at four times their size.
//
// Order. All visible keys of all requests and KV heads, in tiles of 16 or 32 of which
// four make a unit, are laid end to end and cut into equal shares, one per team of
// four warps (lengths are read on the device). A team whose share begins or ends inside
// a (request, head) leaves a partial result there, two at most; a dependent launch
// joins them. Calls of so few and short items that the CTAs of one cluster cover
// each one run as clusters instead, which join through distributed shared memory:
// one launch, and no sums over the lengths before it starts. Each warp copies its own
// tiles into a ring of its own, kStages - 1 ahead and across requests, with no barrier
// until the end of a run.
//
// Measured (GB300; Hq 32, Hkv 8, D 128, 16-key pages; of a plain copy's 6.7 TB/s):
// bf16, 64 requests behind a window of 1024, 53-54 us (0.75), 32 requests of 4 tokens behind
// 4096, 98-100 us (0.81); 4 bits, 64 requests of mean 4096 keys, 57-61 us (0.75-0.8), two of
// 131072, 46-50 us (0.67-0.73). About 6 us of each are a chain of latencies: the call before,
// lengths, shares, tables, first copies, the join. Copies alone, nothing computed, take 3
// us less. bf16 shares end 71 to 97 us after the start by the part of the chip that an SM
// is in, the same SMs in every run.

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "fp4.cuh"
#include "launchers.h"

namespace cg = cooperative_groups;

namespace attn {

ATTN_DEFINE_ERROR_WORD(take_error_decode_window)

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kMaxCluster = 8, kMaxTeams = 4, kSmemPerSm = 228 * 1024;
// Keys of a fragment, and runs of them in a step of a warp. (One run a step in 4 bits: 71
// us where two take 63, with blocks of one team; at 16 rows 116 and 98.)
constexpr int kKeys = 16;
template <bool k4> constexpr int kRunsOf = k4 ? 2 : 1;

struct WindowParams {
  const __nv_bfloat16* q;
  const uint8_t *k, *v;                     // pools of bf16 rows, or of codes
  const uint8_t *k_scales, *v_scales;       // 4 bits
  const int *table, *lens;
  __nv_bfloat16* o;
  float* lse;
  float *o_part, *m_part, *l_part;          // [2 · teams][rows of a block][D], [...]
  int B, Hkv, T, R, blocks;                 // R = query rows per KV head, in `blocks` blocks
  int num_pages, page_size, max_pages, cap, left, n_global;
  uint32_t page_mul;                        // key / page_size = umulhi(2 key, mul) >> shift
  int page_shift;
  int teams, block_teams;                   // of warps, in all and in a block
  int cluster;                              // CTAs of an item, 0: shares of all items
  float scale_log2;
};

// The barrier of a team's threads.
ATTN_DEVINL void team_sync(int in_block) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + in_block), "n"(kThreads) : "memory");
}

// ------------------------------------------------------------ division of work

// What a request's tiles are: `global` tiles from key 0 on, then the tiles
// from `first` to the one that holds key n - 1.
struct Tiles {
  int n, lo, global, first, count, units;
  ATTN_DEVINL int at(int i) const { return i < global ? i : i - global + first; }
};
template <int kTile> ATTN_DEVINL Tiles tiles_of(const WindowParams& p, int n) {
  Tiles t;
  t.n = unsigned(n) <= unsigned(p.cap) ? n : 0;
  // first key of the first token's window
  t.lo = p.left < 0 ? 0 : max(0, t.n - p.T - min(p.left, t.n));
  const int end = (t.n + kTile - 1) / kTile;
  t.global = min(end, (min(p.n_global, t.n) + kTile - 1) / kTile);
  t.first = max(t.lo / kTile, t.global);
  t.count = t.global + max(0, end - t.first);
  t.units = (t.count + kWarps - 1) / kWarps;
  return t;
}

// Work is divided by cost: every run of units of one (request, KV head, block of
// rows) counts as kItemCost units more, for its queries, its start and its end. (4 bits,
// 64 requests of mean 4096 keys: 67.4 us at 0, 60.5 at 1, 57.4 at 2, 58.0 at 4.)
// The places of an item are its kItemCost first ones, then one per unit.
constexpr int kItemCost = 2;
ATTN_DEVINL int places_of(int units) { return units > 0 ? units + kItemCost : 0; }

// Sums over the requests of an item's places: of all, and of those before request
// `upto` (all threads of the block get both).
// Lengths come from L2: the join reads them before it waits. (Every block of the join
// reads all B of them: 4 B^2 bytes a run of rows, 16 KB a block at 4096 requests.)
template <int kN, int kTile> struct PlaceSums {
  int total, before;
  ATTN_DEVINL PlaceSums(const WindowParams& p, int upto) {
    __shared__ int part[2][kN / 32];
    int a = 0, b = 0;
    for (int r = threadIdx.x; r < p.B; r += kN) {
      const int u = places_of(tiles_of<kTile>(p, __ldcg(p.lens + r)).units);
      a += u;
      if (r < upto) b += u;
    }
    a = __reduce_add_sync(0xffffffffu, a);
    b = __reduce_add_sync(0xffffffffu, b);
    if (threadIdx.x % 32 == 0) {
      part[0][threadIdx.x / 32] = a;
      part[1][threadIdx.x / 32] = b;
    }
    __syncthreads();
    total = before = 0;
    for (int w = 0; w < kN / 32; ++w) {
      total += part[0][w];
      before += part[1][w];
    }
    __syncthreads();
  }
};

// Share c of `teams` equal ones of `places` (below 2^31): [start(c), start(c + 1)).
ATTN_DEVINL int share_start(int c, int teams, int places) {
  const int q = places / teams, r = places - q * teams;
  return c * q + c * r / teams;                   // (teams below 2^12)
}
// The share that holds a place.
ATTN_DEVINL int share_of(int place, int teams, int places) {
  int c = min(teams - 1, int(float(place) / float(places) * float(teams)));
  while (c + 1 < teams && share_start(c + 1, teams, places) <= place) ++c;
  while (c > 0 && share_start(c, teams, places) > place) --c;
  return c;
}

// A share as units: its first and the one past its last, the request of the first,
// and the units of all requests before that one.
struct Share {
  int begin, end, b, before;
};
// The share of a team, worked out by its threads: each adds up a run of
// requests, the block's running sums find the threads whose requests hold the
// share's ends. Places are counted as units are.
template <int kTile, int kTeams>
ATTN_DEVINL Share find_share(const WindowParams& p, int in_block, int team) {
  __shared__ int team_sums[kTeams][2][kWarps];
  __shared__ Share team_share[kTeams];
  int (&sums)[2][kWarps] = team_sums[in_block];
  Share& share = team_share[in_block];
  const int tid = threadIdx.x % kThreads, lane = tid % 32, warp = tid / 32;
  const int per_request = p.Hkv * p.blocks;
  const int per = (p.B + kThreads - 1) / kThreads, r0 = min(p.B, tid * per),
            r1 = min(p.B, r0 + per);
  int places = 0, units = 0;                      // of the thread's requests
  for (int r = r0; r < r1; ++r) {
    const int n = p.lens[r], u = tiles_of<kTile>(p, n).units;
    if (team == 0 && unsigned(n) > unsigned(p.cap)) attn_flag_error(kErrBadIndex);
    places += places_of(u);
    units += u;
  }
  places *= per_request;
  units *= per_request;
  int at = places, at_u = units;                  // running sums, the thread's included
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, at, off), y = __shfl_up_sync(0xffffffffu, at_u, off);
    if (lane >= off) {
      at += x;
      at_u += y;
    }
  }
  if (lane == 31) {
    sums[0][warp] = at;
    sums[1][warp] = at_u;
  }
  team_sync(in_block);
  int all = 0, all_u = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      at += sums[0][w];
      at_u += sums[1][w];
    }
    all += sums[0][w];
    all_u += sums[1][w];
  }
  const int teams = min(p.teams, all);
  if (team >= teams) return {0, 0, 0, 0};
#pragma unroll
  for (int end = 0; end < 2; ++end) {
    const int place = share_start(team + end, teams, all);
    if (end == 1 && place == all && tid == 0) share.end = all_u;
    if (place < at - places || place >= at) continue;
    int from = at - places, from_u = at_u - units, r = r0, u;
    while (true) {
      u = tiles_of<kTile>(p, p.lens[r]).units;
      if (place < from + places_of(u) * per_request) break;
      from += places_of(u) * per_request;
      from_u += u * per_request;
      ++r;
    }
    const int item = (place - from) / places_of(u);
    const int unit =
        from_u + item * u + max(0, place - from - item * places_of(u) - kItemCost);
    if (end == 1) {
      share.end = unit;
    } else {
      share.begin = unit;
      share.b = r;
      share.before = from_u;
    }
  }
  team_sync(in_block);
  return share;
}

// ------------------------------------------------------------ instructions

template <bool kHalf>
ATTN_DEVINL void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
ATTN_DEVINL void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
               "{%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
ATTN_DEVINL uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
ATTN_DEVINL void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
ATTN_DEVINL void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
ATTN_DEVINL uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two floats as bf16, rounded towards zero; `lo` goes to the low half.
ATTN_DEVINL uint32_t cut_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int kBytes> ATTN_DEVINL void copy_async(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes)
                 : "memory");
}
ATTN_DEVINL void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> ATTN_DEVINL void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// The barrier of a cluster's threads in two halves.
ATTN_DEVINL void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
ATTN_DEVINL void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
ATTN_DEVINL uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
ATTN_DEVINL uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
ATTN_DEVINL uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
ATTN_DEVINL void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
ATTN_DEVINL float max_over_keys(float x) {   // lanes of one t
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
ATTN_DEVINL float sum_over_keys(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
ATTN_DEVINL float pow2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// ------------------------------------------------------------ the tiles

// A warp's ring. A stage holds runs of K rows, V rows and (4 bits) scales of 16
// keys each, then (pages that do not hold whole runs) a word that says which keys
// are there.
template <int D, bool k4, int kRun> struct Ring {
  static constexpr int kRow = k4 ? D / 2 : 2 * D;           // bytes of a row
  static constexpr int kScales = k4 ? D / 16 : 0;           // and of its scales
  static constexpr int kPart = 2 * kKeys * (kRow + kScales);  // bytes of a run
  static constexpr int kInfo = kRun * kPart;
  static constexpr int kStage = kInfo + 16;
  static constexpr int kStages = kRun == 2 ? 2 : 3;
  static constexpr int kBytes = kStages * kStage;
  static constexpr int kPieces = kRow / 16;                 // 16-byte pieces of a row

  // Where piece c of K row r starts in a stage. bf16: pieces of a row are turned
  // by the row, so that the eight rows of an 8 x 8 load lie in different banks.
  // 4 bits: rows as they come; a quarter warp reads two whole rows.
  static ATTN_DEVINL int k_at(int r, int c) {
    return r * kRow + 16 * (k4 ? c : c ^ (r & 7));
  }
  // V. 4 bits: a lane reads rows 2t, 2t + 1, 2t + 8 and 2t + 9, so even rows come
  // first, then odd ones, and every second pair of them is turned by two pieces.
  static ATTN_DEVINL int v_at(int r, int c) {
    if (!k4) return kKeys * kRow + k_at(r, c);
    const int s = r / 2 + (r & 1) * 8;
    return kKeys * kRow + s * kRow + 16 * (D == 128 ? c ^ (s & 2) : c);
  }
  static ATTN_DEVINL int k_scale_at(int r) { return 2 * kKeys * kRow + r * kScales; }
  static ATTN_DEVINL int v_scale_at(int r) { return k_scale_at(r) + kKeys * kScales; }
};

// Teams of a block, which has an SM to itself: as many as registers (4 bits) or rings
// (bf16) leave room for. Blocks of one team start one after the other: 62.3 us for the 64
// requests in 4 bits where blocks of four take 57.9; bf16 alike. In 4 bits at 16 rows two
// teams of D = 128 spill 8 bytes (99 us; three 111); of D = 64, four take 57 us, three 61.
template <int D, bool k4, int NT>
constexpr int kTeamsOf = k4 && (D == 64 || NT == 1) ? 4 : 2;

// Blocks of 16 elements whose sums the warps hand one another at a time, each as
// [32 lanes] of four floats a warp and block of 8 rows: all of them, or (bf16) four at a
// time: at 16 rows those of two teams do not fit beside their rings.
template <int D, bool k4, int NT, bool kTwice>
constexpr int kAtOnce = k4 ? (kTwice ? D / 32 : D / 16) : 4 / NT;

template <int D, bool k4, int NT, bool kTwice>
constexpr int handed_bytes() {                    // (m, l) too
  return kAtOnce<D, k4, NT, kTwice> * NT * kWarps * 512 + kWarps * 8 * NT * 8;
}
template <int D, bool k4, int NT>
constexpr int ring_bytes() { return kWarps * Ring<D, k4, kRunsOf<k4>>::kBytes; }
template <int D, bool k4, int NT, bool kTwice>
constexpr int smem_bytes() {
  return (handed_bytes<D, k4, NT, kTwice>() + ring_bytes<D, k4, NT>() + 127) / 128 * 128;
}
// What the other CTAs of a cluster write into the first one's shared memory, in the
// place of its rings.
template <int D, int NT, bool kTwice>
constexpr int inbox_bytes() {
  return (kMaxCluster - 1) * ((kTwice ? D / 32 : D / 16) * NT * 512 + 8 * NT * 8);
}

// What a tile is: nothing to compute, all keys seen by all tokens, or neither;
// kLacks << r: run r of its keys is not there.
enum : uint32_t { kNone = 0, kFull = 1, kPart = 2, kLacks = 4 };

// NT blocks of 8 query rows at a time (two beyond 8 rows: one would read the keys twice as
// often). kRuns: pages hold whole runs (page_size a multiple of 16), so a run's rows
// are adjacent: one table entry and one address instead of one per row (as per row: 78 us
// where 64 requests behind 1024 keys take 53, 68 where 64 of mean 4096 in 4 bits take
// 57). kTwice (4 bits, up to 4 query rows): the fragments' columns 4 .. 7 hold the rows
// a second time and take the odd groups of 32 elements, columns 0 .. 3 the even
// ones, so that a lane scales half as many sums and probabilities; the unscaled
// halves of columns come out of the products too, and are not read (without it 59.8 us
// instead of 57.4, for two requests of 131072 keys 48.1 instead of 45.8).
template <int D, bool k4, int NT, bool kRuns, bool kTwice>
__global__ void __launch_bounds__(kThreads * kTeamsOf<D, k4, NT>, 1)
window_kernel(const __grid_constant__ WindowParams p) {
  constexpr int kRun = kRunsOf<k4>, kTile = kRun * kKeys;
  using RingT = Ring<D, k4, kRun>;
  constexpr int kStages = RingT::kStages, kRows = 8 * NT, kGroups = D / 32;
  // blocks of 16 elements of a row's sums (kTwice: even and odd groups share theirs)
  constexpr int kM = kTwice ? D / 32 : D / 16, kQ = D / 16;
  // groups that a lane scales
  constexpr int kOwn = kTwice ? kGroups / 2 : kGroups;
  constexpr int kRowMask = kTwice ? 3 : 15;       // of a column's query row
  extern __shared__ __align__(128) uint8_t block_smem[];
  // (uniform, and known to be)
  constexpr int kTeams = kTeamsOf<D, k4, NT>;
  const int warp_ = __shfl_sync(0xffffffffu, int(threadIdx.x) / 32, 0), lane = threadIdx.x % 32;
  const int warp = warp_ % kWarps, in_block = warp_ / kWarps;
  const int team = int(blockIdx.x) * p.block_teams + in_block;
  const int g = lane / 4, t = lane % 4;
  uint8_t* const smem = block_smem + in_block * smem_bytes<D, k4, NT, kTwice>();
  float4* handed = reinterpret_cast<float4*>(smem);
  uint8_t* const rings = smem + handed_bytes<D, k4, NT, kTwice>();
  const uint32_t ring = smem_u32(rings) + warp * RingT::kBytes;
  constexpr int kHand = kAtOnce<D, k4, NT, kTwice>;
  float2* handed_ml = reinterpret_cast<float2*>(handed + kHand * NT * kWarps * 32);

  pdl_wait_primary();
  // (only now: the join reads lengths before it waits for this grid)
  pdl_launch_dependents();
  const int per_request = p.Hkv * p.blocks;
  int b = 0, before = 0, u_begin, u_end;
  if (p.cluster > 0) {
    const int item = int(blockIdx.x) / p.cluster, rank = int(blockIdx.x) % p.cluster;
    b = item / per_request;
    if (unsigned(p.lens[b]) > unsigned(p.cap)) attn_flag_error(kErrBadIndex);
    const int units = tiles_of<kTile>(p, p.lens[b]).units, first = item % per_request * units;
    u_begin = first + share_start(rank, p.cluster, units);
    u_end = first + share_start(rank + 1, p.cluster, units);
  } else {
    if (team >= p.teams) return;
    const Share share = find_share<kTile, kTeams>(p, in_block, team);
    if (share.begin == share.end) return;
    b = share.b;
    before = share.before;
    u_begin = share.begin;
    u_end = share.end;
  }

  // The warp's tile k is its quarter of unit u_begin + k. Tiles 32 i .. 32 i + 31
  // are worked out at once, one per lane, while those before them are computed:
  // `ahead` is the run that follows the one in use.
  struct Tile {
    uint32_t row[kRun];                           // kRuns: of the pool; else the first key
    uint32_t what;
    int b, h;                                     // !kRuns
  } now{}, ahead{};
  int ahead_page[kRun] = {}, ahead_slot[kRun] = {}, pb = b, pbefore = before;
  auto wanted = [&](const Tiles& tl, int key) {   // by any token
    return key < tl.n && (key >= tl.lo || key < p.n_global);
  };
  auto page_of = [&](int key) { return int(__umulhi(2u * uint32_t(key), p.page_mul) >> p.page_shift); };
  auto look_ahead = [&](int k) {                  // of tiles k .. k + 31
    const int u = u_begin + k + lane;
    ahead.what = kNone;
    if (u < u_end) {
      Tiles tl = tiles_of<kTile>(p, p.lens[pb]);
      while (u >= pbefore + tl.units * per_request) {
        pbefore += tl.units * per_request;
        tl = tiles_of<kTile>(p, p.lens[++pb]);
      }
      const int item = (u - pbefore) / tl.units;
      const int i = kWarps * ((u - pbefore) - item * tl.units) + warp;
      if (i < tl.count) {
        const int key0 = kTile * tl.at(i);
        ahead.what = (key0 + kTile - 1 <= tl.n - p.T &&
                      (p.left < 0 || key0 >= tl.n - 1 - p.left)) ||
                             key0 + kTile <= min(p.n_global, tl.n) ? kFull : kPart;
        ahead.b = pb;
        ahead.h = item / p.blocks;
        if constexpr (kRuns) {
#pragma unroll
          for (int r = 0; r < kRun; ++r) {
            // (a run whose first key is not wanted may have none at all, and no page)
            const int key = key0 + r * kKeys;
            const bool any = wanted(tl, key) || wanted(tl, max(key, min(tl.lo, key + kKeys - 1)));
            const int page = page_of(key);
            ahead_slot[r] = key - page * p.page_size;
            ahead_page[r] = any ? p.table[1LL * pb * p.max_pages + page] : 0;
            if (!any) ahead.what |= kLacks << r;
          }
        } else {
          ahead.row[0] = uint32_t(key0);
        }
      }
    }
    pb = __shfl_sync(0xffffffffu, pb, 31);
    pbefore = __shfl_sync(0xffffffffu, pbefore, 31);
  };
  const int n_tiles = u_end - u_begin;
  // !kRuns: a tile's table entries, key lane % kTile's, read a tile before its copies.
  // (Keys that no token sees are not looked up: their pages may be gone.)
  int next_page = 0;
  auto look_up = [&](int k) {
    if (kRuns || k >= n_tiles) return;
    if (k % 32 == 0) {
      now = ahead;
      look_ahead(k + 32);
    }
    if (__shfl_sync(0xffffffffu, now.what, k % 32) == kNone) return;
    const int key = int(__shfl_sync(0xffffffffu, now.row[0], k % 32)) + lane % kTile;
    const int rb = __shfl_sync(0xffffffffu, now.b, k % 32);
    next_page = wanted(tiles_of<kTile>(p, p.lens[rb]), key)
                    ? p.table[1LL * rb * p.max_pages + page_of(key)] : -1;
  };
  // kTwice: picks the low half (columns 0 .. 3) or the high half of two scales, as a float
  const uint32_t own_half = t < 2 ? 0x1044u : 0x3244u;
  const uint32_t low_columns = g < 4 ? 0xffffffffu : 0u;   // of a fragment of Pᵀ
  // the lane's parts of a tile's copies
  const uint8_t* const k_src = p.k + 16 * lane;
  const uint8_t* const v_src = p.v + 16 * lane;
  const uint8_t* const s_src =
      k4 ? (lane < kKeys ? p.k_scales : p.v_scales) + lane % kKeys * RingT::kScales : nullptr;
  constexpr int kPer = 32 / RingT::kPieces;       // rows a step of the copies
  const uint32_t k_dst = ring + RingT::k_at(lane / RingT::kPieces, lane % RingT::kPieces);
  const uint32_t v_dst = ring + RingT::v_at(lane / RingT::kPieces, lane % RingT::kPieces);
  const uint32_t s_dst = ring + (lane < kKeys ? RingT::k_scale_at(lane % kKeys)
                                              : RingT::v_scale_at(lane % kKeys));
  uint32_t whats = 0;                             // of the tiles in the ring, four bits each
  auto issue = [&](int k, uint32_t stage) {       // stage: its offset in the ring
    whats >>= 4;
    if (k < n_tiles) {
      uint32_t what;
      if constexpr (kRuns) {
        if (k % 32 == 0) {
          now = ahead;
#pragma unroll
          for (int r = 0; r < kRun; ++r) {
            // (a pool has fewer than 2^32 rows)
            const bool ok = unsigned(ahead_page[r]) < unsigned(p.num_pages);
            if (!ok && now.what != kNone) {
              attn_flag_error(kErrBadIndex);
              now.what = (now.what & ~kFull) | kPart | kLacks << r;
            }
            now.row[r] = (uint32_t(ok ? ahead_page[r] : 0) * uint32_t(p.Hkv) + uint32_t(now.h)) *
                             uint32_t(p.page_size) + uint32_t(ahead_slot[r]);
          }
        }
        what = __shfl_sync(0xffffffffu, now.what, k % 32);
        if (what != kNone) {
#pragma unroll
          for (int run = 0; run < kRun; ++run) {
            // all 16 rows, of which the page has room for each, seen or not
            const uint32_t row = __shfl_sync(0xffffffffu, now.row[run], k % 32);
            const uint32_t to = stage + run * RingT::kPart;
            const uint8_t* kp = k_src + size_t(row) * RingT::kRow;
            const uint8_t* vp = v_src + size_t(row) * RingT::kRow;
#pragma unroll
            for (int s = 0; s < kKeys / kPer; ++s) {
              // (the swizzles repeat, or turn by a constant)
              const int r = s * kPer + lane / RingT::kPieces, c = lane % RingT::kPieces;
              const uint32_t kd = k4 ? k_dst + s * kPer * RingT::kRow : ring + RingT::k_at(r, c);
              const uint32_t vd = k4 ? v_dst + s * kPer / 2 * RingT::kRow : ring + RingT::v_at(r, c);
              copy_async<16>(kd + to, kp + s * kPer * RingT::kRow);
              copy_async<16>(vd + to, vp + s * kPer * RingT::kRow);
            }
            if constexpr (k4)
              copy_async<RingT::kScales>(s_dst + to, s_src + size_t(row) * RingT::kScales);
          }
        }
        if (k % 32 == 0) look_ahead(k + 32);      // (behind the copies: it takes a while)
      } else {
        what = __shfl_sync(0xffffffffu, now.what, k % 32);
        if (what != kNone) {
          const int key = int(__shfl_sync(0xffffffffu, now.row[0], k % 32)) + lane % kTile;
          const int h = __shfl_sync(0xffffffffu, now.h, k % 32);
          const int rb = __shfl_sync(0xffffffffu, now.b, k % 32);
          const bool ok = unsigned(next_page) < unsigned(p.num_pages);
          if (!ok && wanted(tiles_of<kTile>(p, p.lens[rb]), key)) attn_flag_error(kErrBadIndex);
          const uint32_t row = ok ? (uint32_t(next_page) * uint32_t(p.Hkv) + uint32_t(h)) *
                                            uint32_t(p.page_size) +
                                        uint32_t(key - page_of(key) * p.page_size)
                                  : 0u;
          constexpr uint32_t kAll = kTile == 32 ? 0xffffffffu : 0xffffu;
          const uint32_t there = __ballot_sync(0xffffffffu, ok) & kAll;
#pragma unroll
          for (int run = 0; run < kRun; ++run) {
            const uint32_t to = ring + stage + run * RingT::kPart;
#pragma unroll
            for (int s = 0; s < kKeys / kPer; ++s) {
              const int r = s * kPer + lane / RingT::kPieces, c = lane % RingT::kPieces;
              const size_t off =
                  size_t(__shfl_sync(0xffffffffu, row, run * kKeys + r)) * RingT::kRow + 16 * c;
              copy_async<16>(to + RingT::k_at(r, c), p.k + off);
              copy_async<16>(to + RingT::v_at(r, c), p.v + off);
            }
            if constexpr (k4) {
              const size_t off =
                  size_t(__shfl_sync(0xffffffffu, row, run * kKeys + lane % kKeys)) *
                  RingT::kScales;
              copy_async<RingT::kScales>(
                  s_dst + stage + run * RingT::kPart,
                  (lane < kKeys ? p.k_scales : p.v_scales) + off);
            }
          }
          if (there != kAll) what = there != 0 ? kPart : kNone;
          sts32(ring + stage + RingT::kInfo, there);
        }
      }
      whats |= what << (4 * (kStages - 1));
    }
    copies_commit();
  };
  int k = 0;
  uint32_t stage = 0;                             // of tile k
  bool once = p.cluster > 0;                      // a cluster's CTA takes one run, if empty
  for (int u = u_begin; u < u_end || once;) {
    Tiles tl = tiles_of<kTile>(p, p.lens[b]);
    int item;
    if (once) {
      item = int(blockIdx.x) / p.cluster % per_request;
      once = false;
    } else {
      while (u >= before + tl.units * per_request) {
        before += tl.units * per_request;
        tl = tiles_of<kTile>(p, p.lens[++b]);
      }
      item = (u - before) / tl.units;
    }
    const int local = u - before - item * tl.units;
    const int h = item / p.blocks, r0 = item % p.blocks * kRows;
    const int run = min(tl.units - local, u_end - u);
    const bool whole = p.cluster > 0 || run == tl.units;
    const int rows = min(kRows, p.R - r0);
    const long long q_row0 = (1LL * b * p.Hkv + h) * p.R + r0;

    // Query rows as the fragments of Qᵀ: lane (g, t) holds row g of each block.
    // 4 bits: k-step 2c + s is the elements 32c + 8t + 4s .. + 3; scaled by a power
    // of two that puts the row's largest value into [2^8, 2^9).
    uint32_t qf[kQ][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = (8 * nt + g) & kRowMask;
      const __nv_bfloat16* src = p.q + (q_row0 + row) * D;
      if constexpr (k4) {
#pragma unroll
        for (int c = 0; c < kGroups; ++c) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (row < rows) w = *reinterpret_cast<const uint4*>(src + 32 * c + 8 * t);
          qf[2 * c][nt][0] = w.x; qf[2 * c][nt][1] = w.y;
          qf[2 * c + 1][nt][0] = w.z; qf[2 * c + 1][nt][1] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < kQ; ++j)
#pragma unroll
          for (int s = 0; s < 2; ++s)
            qf[j][nt][s] = row < rows ? *reinterpret_cast<const uint32_t*>(src + 16 * j + 8 * s + 2 * t)
                                      : 0u;
      }
    }
    if (u == u_begin) {                           // the ring begins
      look_ahead(0);
      look_up(0);
#pragma unroll 1
      for (int s = 0; s < kStages - 1; ++s) {
        issue(s, s * RingT::kStage);
        look_up(s + 1);
      }
    }
    float to_log2[NT][2];                         // scores times this, per column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (k4) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kQ; ++j)
#pragma unroll
          for (int s = 0; s < 2; ++s)
            top = max(top, max(qf[j][nt][s] & 0x7fffu, (qf[j][nt][s] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(int(top >> 7) - 127, -100);
        const float up = pow2i(8 - e);
#pragma unroll
        for (int j = 0; j < kQ; ++j)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t w = qf[j][nt][s];
            qf[j][nt][s] =
                kTwice && j / 2 % 2 != g / 4 ? 0u : pack_f16x2(bf16lo(w) * up, bf16hi(w) * up);
          }
        const float down = fmaxf(p.scale_log2 * pow2i(e - 8), 1.17549435e-38f);
        to_log2[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
        to_log2[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
      } else {
        to_log2[nt][0] = to_log2[nt][1] = p.scale_log2;
      }
    }
    // last key of each column's token
    int last[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) last[nt][j] = tl.n - p.T + (r0 + ((8 * nt + 2 * t + j) & kRowMask)) % p.T;

    // m: row maxima, in log2 units, as of the last time that one was passed by 8;
    // limit: 8 above them, as raw sums. Sums are of 2^(s - m + e), e of a column's own:
    // what one token sees and another does not (a key after it, or one that has left
    // its window) may be 2^150 times as large. e is in [-84, 66], the columns' e four
    // bytes of a register; v_limit: the scale of V that the largest of them allows. (With
    // one e for all columns 64.0 us instead of 64.5 at 8 rows, 108.8 instead of 110 at 16,
    // 41.9 instead of 43.5 at 16 behind a window of 1024.)
    float o[kM][NT][4], m[NT][2], limit[NT][2], minus_ref[NT][2], l[NT][2], v_limit = 128.f;
    uint32_t e_packed = 0;
    auto e_of = [&](int nt, int j) { return int(int8_t(e_packed >> (8 * (2 * nt + j)))); };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = limit[nt][j] = -INFINITY;
        l[nt][j] = minus_ref[nt][j] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < kM; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[mt][nt][j] = 0.f;
    }

    for (int i = kWarps * local + warp; i < kWarps * (local + run); i += kWarps, ++k) {
      copies_wait<kStages - 2>();
      __syncwarp();
      // (the copies go into the stage that was used last)
      issue(k + kStages - 1, stage == 0 ? (kStages - 1) * RingT::kStage : stage - RingT::kStage);
      look_up(k + kStages);
      const uint32_t at = ring + stage;
      stage = stage == (kStages - 1) * RingT::kStage ? 0 : stage + RingT::kStage;
      const uint32_t what = whats & 15u;
      if (what == kNone) continue;
      const bool full = what == kFull;

      // Sᵀ: rows are keys g and g + 8 of a run, columns query rows 2t and 2t + 1
      float s[kRun][NT][4];
      float vs[kRun][2][kOwn];                    // 4 bits: scales of V, keys g and g + 8
#pragma unroll
      for (int run_ = 0; run_ < kRun; ++run_) {
        const uint32_t from = at + run_ * RingT::kPart;
        float (&sr)[NT][4] = s[run_];
        if constexpr (k4) {
          uint32_t w[2][D / 32];                  // codes of keys g, g + 8
          float ks[2][kOwn];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = g + 8 * j;
            uint32_t sk[D / 64], sv[D / 64];
            if constexpr (D == 128) {
              const uint4 x = lds128(from + RingT::k_at(r, t));
              w[j][0] = x.x; w[j][1] = x.y; w[j][2] = x.z; w[j][3] = x.w;
              const uint2 y = lds64(from + RingT::k_scale_at(r)),
                          z = lds64(from + RingT::v_scale_at(r));
              sk[0] = y.x; sk[1] = y.y; sv[0] = z.x; sv[1] = z.y;
            } else {
              const uint2 x = lds64(from + RingT::k_at(r, 0) + 8 * t);
              w[j][0] = x.x; w[j][1] = x.y;
              sk[0] = lds32(from + RingT::k_scale_at(r));
              sv[0] = lds32(from + RingT::v_scale_at(r));
            }
#pragma unroll
            for (int c = 0; c < kOwn; ++c) {
              if constexpr (kTwice) {             // the half of the pair that is this lane's
                ks[j][c] = __uint_as_float(__byte_perm(sk[c], 0, own_half));
                vs[run_][j][c] = __uint_as_float(__byte_perm(sv[c], 0, own_half));
              } else {
                ks[j][c] = c % 2 ? bf16hi(sk[c / 2]) : bf16lo(sk[c / 2]);
                vs[run_][j][c] = c % 2 ? bf16hi(sv[c / 2]) : bf16lo(sv[c / 2]);
              }
            }
          }
          float x[NT][4];                         // sums of a group (kTwice: of two)
#pragma unroll
          for (int c = 0; c < kGroups; ++c) {
#pragma unroll
            for (int step = 0; step < 2; ++step) {
              const uint32_t w0 = w[0][step * (D / 64) + c / 2],
                             w1 = w[1][step * (D / 64) + c / 2];
              uint32_t a[4];
              if (c % 2) {
                a[0] = e2m1x2_to_f16x2<2>(w0); a[1] = e2m1x2_to_f16x2<2>(w1);
                a[2] = e2m1x2_to_f16x2<3>(w0); a[3] = e2m1x2_to_f16x2<3>(w1);
              } else {
                a[0] = e2m1x2_to_f16x2<0>(w0); a[1] = e2m1x2_to_f16x2<0>(w1);
                a[2] = e2m1x2_to_f16x2<1>(w0); a[3] = e2m1x2_to_f16x2<1>(w1);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (step == 0 && !(kTwice && c % 2))
                  mma16816_first(x[nt], a, qf[2 * c][nt][0], qf[2 * c][nt][1]);
                else
                  mma16816<true>(x[nt], a, qf[2 * c + step][nt][0], qf[2 * c + step][nt][1]);
              }
            }
            if (kTwice && c % 2 == 0) continue;
            const int o_ = kTwice ? c / 2 : c;    // of the lane's scales
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                sr[nt][j] = o_ == 0 ? x[nt][j] * ks[j / 2][0]
                                    : fmaf(x[nt][j], ks[j / 2][o_], sr[nt][j]);
          }
          if constexpr (kTwice) {                 // even and odd groups together
#pragma unroll
            for (int j = 0; j < 4; ++j) sr[0][j] += __shfl_xor_sync(0xffffffffu, sr[0][j], 2);
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) sr[nt][j] = 0.f;
#pragma unroll
          for (int j = 0; j < kQ; ++j) {
            uint32_t a[4];
            // matrices: keys 0-7, keys 8-15, then the same of the next 8 elements
            ldmatrix4(a, from + RingT::k_at(lane % 16, 2 * j + lane / 16));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(sr[nt], a, qf[j][nt][0], qf[j][nt][1]);
          }
        }
      }

      // the tile's keys below key0 + x, those that are there, and those of them that a
      // token at position `top` sees, a bit each
      auto below = [](int x) {
        return x <= 0 ? 0u : x >= kTile ? 0xffffffffu : (1u << x) - 1u;
      };
      auto present = [&](int key0) {
        uint32_t there = below(tl.n - key0);
        if constexpr (!kRuns) {
          there &= lds32(at + RingT::kInfo);
        } else {
#pragma unroll
          for (int r = 0; r < kRun; ++r)
            if (what & (kLacks << r)) there &= ~(0xffffu << (16 * r));
        }
        return there;
      };
      auto seen_at = [&](int top, int key0, uint32_t there, uint32_t first) {
        const uint32_t near =
            below(top + 1 - key0) & ~(p.left < 0 ? 0u : below(top - p.left - key0));
        return there & (near | first);
      };
      uint32_t hidden[NT][2];                     // !full: a bit a key that a row does not see
      if (!full) {
        const int key0 = kTile * tl.at(i);
        const uint32_t there = present(key0), first = below(p.n_global - key0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            hidden[nt][j] = ~seen_at(last[nt][j], key0, there, first);
#pragma unroll
            for (int r = 0; r < kRun; ++r) {
              if ((hidden[nt][j] >> (16 * r + g)) & 1u) s[r][nt][j] = -INFINITY;
              if ((hidden[nt][j] >> (16 * r + g + 8)) & 1u) s[r][nt][j + 2] = -INFINITY;
            }
          }
      }
      // whether a score passes its row's maximum so far by 8 binary orders, or a
      // scale of V, seen or not, the power of two that P is taken with by 2^7
      auto top_score = [&](int nt, int j) {
        float x = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
        if constexpr (kRun == 2) x = max3(x, s[kRun - 1][nt][j], s[kRun - 1][nt][j + 2]);
        return x;
      };
      bool above = false, scales = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) above |= top_score(nt, j) > limit[nt][j];
      if constexpr (k4) {
        float vmax = 0.f;
#pragma unroll
        for (int r = 0; r < kRun; ++r)
#pragma unroll
          for (int c = 0; c < kOwn; ++c) vmax = max3(vmax, vs[r][0][c], vs[r][1][c]);
        scales = vmax > v_limit;
      }
      if (__any_sync(0xffffffffu, above || scales)) {
        // the references move: everything so far is rescaled
        if constexpr (k4) {
          // (a row that has seen nothing has no sums yet, and takes any e)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) scales |= m[nt][0] == -INFINITY || m[nt][1] == -INFINITY;
          if (__any_sync(0xffffffffu, scales)) {
            // Of a key of the lane its largest scale, as bits. (One that is not finite
            // counts for nothing: its group alone is lost.)
            uint32_t top[kRun][2];
#pragma unroll
            for (int r = 0; r < kRun; ++r)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                top[r][y] = 0;
#pragma unroll
                for (int c = 0; c < kOwn; ++c)
                  if (vs[r][y][c] < INFINITY)
                    top[r][y] = max(top[r][y], __float_as_uint(fmaxf(vs[r][y][c], 0.f)));
              }
            uint32_t all = 0;                     // full: of all keys
            if (full) {
#pragma unroll
              for (int r = 0; r < kRun; ++r) all = max(all, max(top[r][0], top[r][1]));
              all = __reduce_max_sync(0xffffffffu, all);
            }
            int e_top = -128;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t x = all;
                if (!full) {                      // of those that the column's row sees
#pragma unroll
                  for (int r = 0; r < kRun; ++r)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                      if (!((hidden[nt][j] >> (16 * r + g + 8 * y)) & 1u)) x = max(x, top[r][y]);
                  // (the lanes of one t; kTwice: and the lane with the row's other groups)
#pragma unroll
                  for (int off = kTwice ? 2 : 4; off < 32; off *= 2)
                    x = max(x, __shfl_xor_sync(0xffffffffu, x, off));
                }
                const int want = 6 - min(max(int(x >> 23) - 127, -60), 90), e = e_of(nt, j);
                const int e_new = m[nt][j] == -INFINITY || want < e ? want : e;
                const int at_bit = 8 * (2 * nt + j);
                e_packed = (e_packed & ~(0xffu << at_bit)) | uint32_t(e_new & 0xff) << at_bit;
                e_top = max(e_top, e_new);
              }
            v_limit = pow2i(7 - e_top);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float to = fmaxf(m[nt][j], max_over_keys(top_score(nt, j)) * to_log2[nt][j]);
            const float ref = to == -INFINITY ? 0.f : float(e_of(nt, j)) - to;
            // (nothing seen yet: sums of zeros, whatever they are scaled by)
            const float by = m[nt][j] == -INFINITY ? 1.f : fast_exp2(ref - minus_ref[nt][j]);
            m[nt][j] = to;
            limit[nt][j] = to == -INFINITY ? -INFINITY : (to + 8.f) / to_log2[nt][j];
            minus_ref[nt][j] = ref;
            l[nt][j] *= by;
#pragma unroll
            for (int mt = 0; mt < kM; ++mt) {
              o[mt][nt][j] *= by;
              o[mt][nt][j + 2] *= by;
            }
          }
      }
#pragma unroll
      for (int r = 0; r < kRun; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[r][nt][j] =
                fast_exp2(fmaf(s[r][nt][j], to_log2[nt][j % 2], minus_ref[nt][j % 2]));
            l[nt][j % 2] += s[r][nt][j];
          }

      // Oᵀ += Vᵀ Pᵀ
      if constexpr (k4) {
        auto product = [&](auto pick) {
#pragma unroll
          for (int r = 0; r < kRun; ++r) {
            const uint32_t from = at + r * RingT::kPart;
            // codes of keys 2t, 2t + 1 (and + 8): bytes (D/16)·g of their rows, the
            // low halves of a pair of keys in one byte, then the high halves
            uint32_t lo[2][D / 64], hi[2][D / 64];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t x[D / 64], y[D / 64];
              if constexpr (D == 128) {
                const uint2 a = lds64(from + RingT::v_at(2 * t + 8 * j, g / 2) + 8 * (g % 2)),
                            c = lds64(from + RingT::v_at(2 * t + 1 + 8 * j, g / 2) + 8 * (g % 2));
                x[0] = a.x; x[1] = a.y; y[0] = c.x; y[1] = c.y;
              } else {
                x[0] = lds32(from + RingT::v_at(2 * t + 8 * j, g / 4) + 4 * (g % 4));
                y[0] = lds32(from + RingT::v_at(2 * t + 1 + 8 * j, g / 4) + 4 * (g % 4));
              }
#pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                lo[j][c] = (x[c] & 0x0f0f0f0fu) | ((y[c] << 4) & 0xf0f0f0f0u);
                hi[j][c] = ((x[c] >> 4) & 0x0f0f0f0fu) | (y[c] & 0xf0f0f0f0u);
              }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int c = 0; c < kGroups; ++c) {
              const int o_ = kTwice ? c / 2 : c;  // of the lane's scales
              if (!(kTwice && c % 2)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    float a = s[r][nt][2 * j] * vs[r][j][o_], z = s[r][nt][2 * j + 1] * vs[r][j][o_];
                    if constexpr (decltype(pick)::value) {
                      if ((hidden[nt][0] >> (16 * r + g + 8 * j)) & 1u) a = 0.f;
                      if ((hidden[nt][1] >> (16 * r + g + 8 * j)) & 1u) z = 0.f;
                    }
                    pf[nt][j] = transpose8x8(pack_f16x2(a, z));
                  }
              }
              uint32_t b[NT][2];                  // (kTwice: of this group's columns)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  b[nt][j] = !kTwice ? pf[nt][j] : pf[nt][j] & (c % 2 ? ~low_columns : low_columns);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t a[4];
                if (c % 2) {
                  a[0] = y ? e2m1x2_to_f16x2<3>(lo[0][c / 2]) : e2m1x2_to_f16x2<2>(lo[0][c / 2]);
                  a[1] = y ? e2m1x2_to_f16x2<3>(hi[0][c / 2]) : e2m1x2_to_f16x2<2>(hi[0][c / 2]);
                  a[2] = y ? e2m1x2_to_f16x2<3>(lo[1][c / 2]) : e2m1x2_to_f16x2<2>(lo[1][c / 2]);
                  a[3] = y ? e2m1x2_to_f16x2<3>(hi[1][c / 2]) : e2m1x2_to_f16x2<2>(hi[1][c / 2]);
                } else {
                  a[0] = y ? e2m1x2_to_f16x2<1>(lo[0][c / 2]) : e2m1x2_to_f16x2<0>(lo[0][c / 2]);
                  a[1] = y ? e2m1x2_to_f16x2<1>(hi[0][c / 2]) : e2m1x2_to_f16x2<0>(hi[0][c / 2]);
                  a[2] = y ? e2m1x2_to_f16x2<1>(lo[1][c / 2]) : e2m1x2_to_f16x2<0>(lo[1][c / 2]);
                  a[3] = y ? e2m1x2_to_f16x2<1>(hi[1][c / 2]) : e2m1x2_to_f16x2<0>(hi[1][c / 2]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816<true>(o[2 * o_ + y][nt], a, b[nt][0], b[nt][1]);
              }
            }
          }
        };
        // a key that a row does not see may hold anything in its scale
        if (full)
          product(std::false_type{});
        else
          product(std::true_type{});
      } else {
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // The first part is cut off, and the rest gets 2^-23 of P besides, so that both
            // are above 0 wherever P is: an infinite value keeps its sign in their sum.
            const float a = s[0][nt][2 * j], z = s[0][nt][2 * j + 1], up = 1.f + 0x1p-23f;
            const uint32_t x = cut_bf16x2(a, z);
            hi[nt][j] = transpose8x8(x);
            lo[nt][j] = transpose8x8(pack_bf16x2(fmaf(a, up, -bf16lo(x)), fmaf(z, up, -bf16hi(x))));
          }
        // Keys that a row does not see may hold values that are not finite, which would
        // reach it through the product (0 · inf). Those that no row of the block sees
        // enter as zeros; where those that some rows see and others do not are not finite,
        // the tokens' rows go one token after the other, each over the keys that it sees,
        // the others' V as zeros.
        uint32_t some = 0, mixed = 0;             // keys, a bit each
        if (!full) {
          uint32_t all = 0xffffu;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (8 * nt + 2 * t + j < rows) {
                some |= ~hidden[nt][j];
                all &= ~hidden[nt][j];
              }
          some = __reduce_or_sync(0xffffffffu, some);
          mixed = some & 0xffffu & ~__reduce_and_sync(0xffffffffu, all);
        }
        bool spoilt = false;
        if (mixed != 0) {
          for (int c = lane; c < kTile * RingT::kPieces; c += 32) {
            if (!((mixed >> (c / RingT::kPieces)) & 1u)) continue;
            const uint4 x = lds128(at + kTile * RingT::kRow + 16 * c);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              spoilt |= (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
          }
          spoilt = __any_sync(0xffffffffu, spoilt);
        }
        // V of blocks 2 mt and 2 mt + 1 of 8 elements, and of the keys of a mask alone
        auto load_v = [&](uint32_t (&a)[4], int mt) {
          // matrices: elements 0-7 and 8-15 of keys 0-7, then of keys 8-15
          ldmatrix4_trans(a, at + RingT::v_at(lane % 8 + lane / 16 * 8, 2 * mt + lane / 8 % 2));
        };
        auto load_v_of = [&](uint32_t (&a)[4], int mt, uint32_t keys) {
          load_v(a, mt);
#pragma unroll
          for (int j = 0; j < 4; ++j) {           // (a lane holds keys 2t, 2t + 1, and + 8)
            const uint32_t x = keys >> (2 * t + 8 * (j / 2));
            a[j] &= (x & 1u ? 0xffffu : 0u) | (x & 2u ? 0xffff0000u : 0u);
          }
        };
        if (full) {
#pragma unroll
          for (int mt = 0; mt < kM; ++mt) {
            uint32_t a[4];
            load_v(a, mt);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<false>(o[mt][nt], a, lo[nt][0], lo[nt][1]);
              mma16816<false>(o[mt][nt], a, hi[nt][0], hi[nt][1]);
            }
          }
        } else if (!spoilt) {
#pragma unroll
          for (int mt = 0; mt < kM; ++mt) {
            uint32_t a[4];
            load_v_of(a, mt, some);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<false>(o[mt][nt], a, lo[nt][0], lo[nt][1]);
              mma16816<false>(o[mt][nt], a, hi[nt][0], hi[nt][1]);
            }
          }
        } else {
          // (the block's rows, one after the other by token, have as many tokens)
          const int key0 = kTile * tl.at(i), tokens = min(rows, p.T);
          const uint32_t there = present(key0), first = below(p.n_global - key0);
          for (int x0 = 0; x0 < tokens; ++x0) {
            const int tok = (r0 + x0) % p.T;
            const uint32_t keys = seen_at(tl.n - p.T + tok, key0, there, first);
#pragma unroll
            for (int mt = 0; mt < kM; ++mt) {
              uint32_t a[4];
              load_v_of(a, mt, keys);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                // P of this token's rows; others take no part (their sums would
                // be spoilt by what this token sees), so a product of their own
                const bool mine = (r0 + 8 * nt + g) % p.T == tok;
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816<false>(x, a, mine ? lo[nt][0] : 0u, mine ? lo[nt][1] : 0u);
                mma16816<false>(x, a, mine ? hi[nt][0] : 0u, mine ? hi[nt][1] : 0u);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if ((r0 + 8 * nt + 2 * t + j % 2) % p.T == tok) o[mt][nt][j] += x[j];
              }
            }
          }
        }
      }
    }

    // (a cluster's CTA takes one run: its rings are done with, and may be written to)
    if (p.cluster > 1) cluster_arrive();
    // Join the warps' sums, each warp some of the blocks of elements. From here on
    // m is the reference of the sums.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nt][j] = sum_over_keys(l[nt][j]);
        m[nt][j] -= float(e_of(nt, j));           // (-inf stays)
        if (g == 0)
          handed_ml[warp * kRows + 8 * nt + 2 * t + j] = make_float2(m[nt][j], l[nt][j]);
      }
    constexpr int kMine = (kM * NT + kWarps - 1) / kWarps;   // blocks of a warp, at most
    auto mine = [&](int x) { return kM * NT % kWarps == 0 || x * kWarps + warp < kM * NT; };
    float4 sum[kMine];
    // Of `parts` results with (m, l) at ml[part · kRows + row]: what each is
    // scaled by, and the joined m and l.
    auto weigh = [&](auto ml_of, int parts, int nt, int j, float (&w)[kMaxCluster]) {
      float top = -INFINITY, all = 0.f;
      const int row = 8 * nt + 2 * t + j;
#pragma unroll
      for (int x = 0; x < kMaxCluster; ++x)
        if (x < parts) top = fmaxf(top, ml_of(x)[row].x);
#pragma unroll
      for (int x = 0; x < kMaxCluster; ++x)
        if (x < parts) {
          const float2 ml = ml_of(x)[row];
          // (a NaN among the scores is in the sums, not in the references)
          w[x] = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - top);
          all += w[x] * ml.y;
        }
      m[nt][j] = top;
      l[nt][j] = all;
    };
    auto add = [](float4& to, const float4& x, float w0, float w1) {
      to.x += x.x * w0; to.y += x.y * w1; to.z += x.z * w0; to.w += x.w * w1;
    };
    float w[NT][2][kMaxCluster];
#pragma unroll
    for (int m0 = 0; m0 < kM; m0 += kHand) {
#pragma unroll
      for (int mt = 0; mt < kHand; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          handed[((mt * NT + nt) * kWarps + warp) * 32 + lane] = make_float4(
              o[m0 + mt][nt][0], o[m0 + mt][nt][1], o[m0 + mt][nt][2], o[m0 + mt][nt][3]);
      team_sync(in_block);
      if (m0 == 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            weigh([&](int x) { return handed_ml + x * kRows; }, kWarps, nt, j, w[nt][j]);
#pragma unroll
      for (int x = 0; x < (kHand * NT + kWarps - 1) / kWarps; ++x) {
        if (!mine(x)) continue;
        const int at = x * kWarps + warp, nt = NT == 1 ? 0 : warp % NT;
        float4 to = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < kWarps; ++y)
          add(to, handed[(at * kWarps + y) * 32 + lane],
              NT == 1 || nt == 0 ? w[0][0][y] : w[NT - 1][0][y],
              NT == 1 || nt == 0 ? w[0][1][y] : w[NT - 1][1][y]);
        sum[m0 * NT / kWarps + x] = to;
      }
      team_sync(in_block);
    }
    if (p.cluster > 1) {
      // Join the CTAs: the others write into the first one's shared memory.
      cg::cluster_group cluster = cg::this_cluster();
      const int rank = int(cluster.block_rank());
      float4* inbox = reinterpret_cast<float4*>(rings);
      float2* inbox_ml = reinterpret_cast<float2*>(inbox + (kMaxCluster - 1) * kM * NT * 32);
      cluster_wait();
      if (rank > 0) {
        float4* to = cluster.map_shared_rank(inbox, 0) + (rank - 1) * kM * NT * 32 + lane;
#pragma unroll
        for (int x = 0; x < kMine; ++x)
          if (mine(x)) to[(x * kWarps + warp) * 32] = sum[x];
        if (warp == 0 && g == 0) {
          float2* to_ml = cluster.map_shared_rank(inbox_ml, 0) + (rank - 1) * kRows;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) to_ml[8 * nt + 2 * t + j] = make_float2(m[nt][j], l[nt][j]);
        }
      } else if (warp == 0 && g == 0) {           // (its own, for all of its warps)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            handed_ml[8 * nt + 2 * t + j] = make_float2(m[nt][j], l[nt][j]);
      }
      cluster_arrive();
      if (rank > 0) return;
      cluster_wait();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          weigh([&](int x) { return x == 0 ? handed_ml : inbox_ml + (x - 1) * kRows; }, p.cluster,
                nt, j, w[nt][j]);
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        if (!mine(x)) continue;
        const int nt = NT == 1 ? 0 : warp % NT;
        float4 to = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          if (c < p.cluster)
            add(to, c == 0 ? sum[x]
                           : inbox[((c - 1) * kM * NT + x * kWarps + warp) * 32 + lane],
                NT == 1 || nt == 0 ? w[0][0][c] : w[NT - 1][0][c],
                NT == 1 || nt == 0 ? w[0][1][c] : w[NT - 1][1][c]);
        sum[x] = to;
      }
    }
    const int slot = 2 * team + (u == u_begin ? 0 : 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int nt = NT == 1 ? 0 : warp % NT, r = (8 * nt + 2 * t + j) & kRowMask;
      const float lr = NT == 1 || nt == 0 ? l[0][j] : l[NT - 1][j];
      const float by = !whole ? 1.f : lr == 0.f ? 0.f : 1.f / lr;
      if (r >= rows) continue;
      __nv_bfloat16* out = p.o + (q_row0 + r) * D;
      float* part = p.o_part + (1LL * slot * kRows + r) * D;
#pragma unroll
      for (int x = 0; x < kMine; ++x) {
        if (!mine(x)) continue;
        const int mt = (x * kWarps + warp) / NT;
        const float a = (j ? sum[x].y : sum[x].x) * by, z = (j ? sum[x].w : sum[x].z) * by;
        if constexpr (k4) {
          const int e = 32 * (kTwice ? 2 * (mt / 2) + t / 2 : mt / 2) + 4 * g + 2 * (mt % 2);
          if (whole)
            *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(a, z);
          else
            *reinterpret_cast<float2*>(part + e) = make_float2(a, z);
        } else {
          const int e = 16 * mt + g;
          if (whole) {
            out[e] = __float2bfloat16_rn(a);
            out[e + 8] = __float2bfloat16_rn(z);
          } else {
            part[e] = a;
            part[e + 8] = z;
          }
        }
      }
    }
    if (warp == 0 && g == 0 && !(kTwice && t >= 2))
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = (8 * nt + 2 * t + j) & kRowMask;
          if (r >= rows) continue;
          if (!whole) {
            p.m_part[slot * kRows + r] = m[nt][j];
            p.l_part[slot * kRows + r] = l[nt][j];
          } else if (p.lse != nullptr) {
            p.lse[q_row0 + r] = l[nt][j] == 0.f ? -INFINITY
                                                : fmaf(m[nt][j] == -INFINITY ? 0.f : m[nt][j],
                                                       0.693147180559945f, logf(l[nt][j]));
          }
        }
    u += run;
  }
}

// Joins the partial results of rows that more than one team worked on, and
// writes those of requests without keys. kPer warps a row; grid: x over groups of
// kJoinWarps / kPer of the Hkv·R rows of request y. Partial results are fetched
// eight at a time.
// Up to kFewRows rows have many partial results each, over which a block's warps share
// (two requests of 131072 keys, 64 rows: 60 us with a warp a row, 46 with eight); more rows
// fill the SMs a warp each (2048 rows: 59 us with eight warps a row, 53 with one).
constexpr int kJoinWarps = 8, kFewRows = 1024, kClusterUnits = 2;
template <int D, int kRows, int kPer, int kTile>
__global__ void __launch_bounds__(32 * kJoinWarps)
window_join_kernel(const __grid_constant__ WindowParams p) {
  constexpr int kLane = D / 32, kBatch = 8;       // elements of a lane
  // The lengths are read before the wait: this grid starts when every CTA of the
  // one before it has waited for what precedes the call.
  const int b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const PlaceSums<32 * kJoinWarps, kTile> sums(p, b);
  const int row = blockIdx.x * (kJoinWarps / kPer) + warp / kPer;
  const int h = row / p.R, r = row % p.R;
  const Tiles tl = tiles_of<kTile>(p, __ldcg(p.lens + b));
  const long long q_row = 1LL * b * p.Hkv * p.R + row;
  float acc[kLane] = {}, sum = 0.f, top = -INFINITY;
  if (tl.units > 0) {
    const int per_request = p.Hkv * p.blocks, places = sums.total * per_request;
    const int teams = min(p.teams, places);
    const int item = sums.before * per_request +
                     (h * p.blocks + r / kRows) * places_of(tl.units);
    const int u0 = item + kItemCost, u1 = u0 + tl.units - 1;
    const int c0 = share_of(u0, teams, places), c1 = share_of(u1, teams, places);
    // (a share that begins before the item holds a unit of another one first)
    const bool at_start = share_start(c0, teams, places) >= item;
    auto slot_of = [&](int c) {
      return (2 * c + (c == c0 && !at_start ? 1 : 0)) * kRows + r % kRows;
    };
    pdl_wait_primary();
    pdl_launch_dependents();
    if (row >= p.Hkv * p.R || c0 == c1) return;   // (one team alone has written its rows)
    for (int first = c0 + warp % kPer; first <= c1; first += kPer * kBatch) {
      // (one round trip to memory: nothing of a batch depends on the rest of it)
      float x[kBatch][kLane], m[kBatch], l[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = first + i * kPer;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < kLane; ++j) x[i][j] = 0.f;
        if (c > c1) continue;
        const int s = slot_of(c);
        m[i] = p.m_part[s];
        l[i] = p.l_part[s];
        const float* part = p.o_part + 1LL * s * D + kLane * lane;
        if constexpr (kLane == 4) {
          const float4 y = *reinterpret_cast<const float4*>(part);
          x[i][0] = y.x; x[i][1] = y.y; x[i][2] = y.z; x[i][3] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(part);
          x[i][0] = y.x; x[i][1] = y.y;
        }
      }
      float to = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) to = fmaxf(to, m[i]);
      // (a NaN among the scores is in the sums, not in the references)
      const float before = top == -INFINITY ? 1.f : fast_exp2(top - to);
      top = to;
      sum *= before;
#pragma unroll
      for (int j = 0; j < kLane; ++j) acc[j] *= before;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float by = m[i] == -INFINITY ? 1.f : fast_exp2(m[i] - to);
        sum = fmaf(by, l[i], sum);
#pragma unroll
        for (int j = 0; j < kLane; ++j) acc[j] = fmaf(by, x[i][j], acc[j]);
      }
    }
  } else {
    pdl_wait_primary();
    pdl_launch_dependents();
    if (row >= p.Hkv * p.R) return;
  }
  if constexpr (kPer > 1) {
    __shared__ float others[kJoinWarps][D + 2];
#pragma unroll
    for (int j = 0; j < kLane; ++j) others[warp][kLane * lane + j] = acc[j];
    if (lane == 0) {
      others[warp][D] = sum;
      others[warp][D + 1] = top;
    }
    __syncthreads();
    if (warp % kPer != 0) return;
    const float own = top;
#pragma unroll
    for (int w = 1; w < kPer; ++w) top = fmaxf(top, others[warp + w][D + 1]);
    const float by = own == -INFINITY ? 1.f : fast_exp2(own - top);
    sum *= by;
#pragma unroll
    for (int j = 0; j < kLane; ++j) acc[j] *= by;
#pragma unroll
    for (int w = 1; w < kPer; ++w) {
      const float theirs = others[warp + w][D + 1];
      const float with = theirs == -INFINITY ? 1.f : fast_exp2(theirs - top);
      sum += with * others[warp + w][D];
#pragma unroll
      for (int j = 0; j < kLane; ++j) acc[j] += with * others[warp + w][kLane * lane + j];
    }
  }
  const bool empty = sum == 0.f;
  const float inv = empty ? 0.f : 1.f / sum;
  __nv_bfloat16* to = p.o + q_row * D + kLane * lane;
#pragma unroll
  for (int j = 0; j < kLane; j += 2)
    *reinterpret_cast<uint32_t*>(to + j) =
        empty ? 0u : pack_bf16x2(acc[j] * inv, acc[j + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[q_row] =
        empty ? -INFINITY : fmaf(top == -INFINITY ? 0.f : top, 0.693147180559945f, logf(sum));
}

cudaError_t launch_dependent(const void* kernel, dim3 grid, int threads, int smem, int cluster,
                             const WindowParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  void* args[] = {const_cast<WindowParams*>(&p)};
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

// A kernel's shared memory is asked for once per device.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int D, bool k4, int NT, bool kRuns, bool kTwice = false>
cudaError_t launch_t(const WindowArgs& a, WindowParams& p) {
  constexpr int kTile = kKeys * kRunsOf<k4>;
  constexpr int handed = handed_bytes<D, k4, NT, kTwice>(), rings = ring_bytes<D, k4, NT>(),
                inbox = inbox_bytes<D, NT, kTwice>();
  constexpr int smem = smem_bytes<D, k4, NT, kTwice>(), kTeams = kTeamsOf<D, k4, NT>,
                smem_cluster = handed + std::max(rings, inbox);
  static_assert(kTeams <= kMaxTeams, "partial results of all teams have room");
  const void* kernel =
      reinterpret_cast<const void*>(window_kernel<D, k4, NT, kRuns, kTwice>);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(kernel, std::max(kTeams * smem, smem_cluster), allowed);
  if (e != cudaSuccess) return e;
  p.blocks = (p.R + 8 * NT - 1) / (8 * NT);
  // most units that an item can have, by the table and the window
  long long tiles = (p.cap + kTile - 1) / kTile;
  if (p.left >= 0)
    tiles = std::min(tiles, (1LL * p.left + p.T + kTile - 1) / kTile + 1 +
                                (1LL * p.n_global + kTile - 1) / kTile);
  const long long units = (tiles + kWarps - 1) / kWarps, items = 1LL * p.B * p.Hkv * p.blocks;
  const long long slots = 1LL * a.sm_count * kTeams;
  // Clusters, where all of them run at once and a CTA has kClusterUnits at most. (Against
  // shares with a join, 8 items: one unit a CTA 6.0 and 6.9 us in 4 bits, 6.1 and 7.0 in
  // bf16; two 6.9 and 7.6, 6.5 and 7.4; four 8.5 and 8.2, 7.7 and 8.3. 32 items of bf16 in
  // clusters of eight, which then do not all run at once: 10.4 and 8.8.)
  int cluster = 1;
  while (cluster < kMaxCluster && cluster < units) cluster *= 2;
  constexpr int resident = std::min(kTeams, kSmemPerSm / (smem_cluster + 1024));
  if (units <= kClusterUnits * cluster && items * cluster <= 1LL * a.sm_count * resident) {
    p.cluster = cluster;
    p.teams = int(items) * cluster;
    p.block_teams = 1;
    return launch_dependent(kernel, dim3(unsigned(p.teams)), kThreads, smem_cluster, cluster, p,
                            a.stream);
  }
  // Blocks that fill an SM each, or of one team where those are fewer.
  p.teams = int(std::min(items * (units + kItemCost), slots));
  p.block_teams = p.teams == slots ? kTeams : 1;
  e = launch_dependent(kernel, dim3(unsigned(p.teams / p.block_teams)),
                       kThreads * p.block_teams, smem * p.block_teams, 1, p, a.stream);
  if (e != cudaSuccess) return e;
  const int rows = p.Hkv * p.R;
  if (1LL * p.B * rows <= kFewRows)
    return launch_dependent(
        reinterpret_cast<const void*>(window_join_kernel<D, 8 * NT, kJoinWarps, kTile>),
        dim3(unsigned(rows), unsigned(p.B)), 32 * kJoinWarps, 0, 1, p, a.stream);
  return launch_dependent(reinterpret_cast<const void*>(window_join_kernel<D, 8 * NT, 1, kTile>),
                          dim3(unsigned((rows + kJoinWarps - 1) / kJoinWarps), unsigned(p.B)),
                          32 * kJoinWarps, 0, 1, p, a.stream);
}

template <int D, bool k4> cudaError_t launch_d(const WindowArgs& a, WindowParams& p) {
  if (k4 && p.R <= 4)
    return p.page_size % kKeys == 0 ? launch_t<D, k4, 1, true, k4>(a, p)
                                    : launch_t<D, k4, 1, false, k4>(a, p);
  if (p.page_size % kKeys == 0)
    return p.R <= 8 ? launch_t<D, k4, 1, true>(a, p) : launch_t<D, k4, 2, true>(a, p);
  return p.R <= 8 ? launch_t<D, k4, 1, false>(a, p) : launch_t<D, k4, 2, false>(a, p);
}

}  // namespace

int window_partial_rows(int R, int sm_count) {
  // two partial results of 8 or 16 rows a team
  return sm_count * kMaxTeams * 2 * (R <= 8 ? 8 : 16);
}

cudaError_t launch_decode_window(const WindowArgs& a) {
  WindowParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const uint8_t*>(a.k);
  p.v = static_cast<const uint8_t*>(a.v);
  p.k_scales = static_cast<const uint8_t*>(a.k_scales);
  p.v_scales = static_cast<const uint8_t*>(a.v_scales);
  p.table = a.block_table;
  p.lens = a.seq_lens;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.o_part = a.o_part;
  p.m_part = a.m_part;
  p.l_part = a.l_part;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.T = a.T;
  p.R = a.Hq / a.Hkv * a.T;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.cap = a.max_pages * a.page_size;
  // (clamped to the capacity, so that sums of positions stay in 32 bits)
  p.left = a.window_left < 0 ? -1 : std::min(a.window_left, p.cap);
  p.n_global = std::min(a.n_global, p.cap);
  // For d = page_size and 2^s >= d, m = floor(2^(31 + s) / d) + 1 < 2^32 has
  // key·m / 2^(31 + s) = key / d + key·x with 0 < x <= 2^-(31 + s), which is too
  // little to reach the next whole number for key < 2^31.
  int s = 0;
  while ((1LL << s) < a.page_size) ++s;
  p.page_shift = s;
  p.page_mul = uint32_t((1ULL << (31 + s)) / unsigned(a.page_size) + 1);
  p.scale_log2 = float(double(a.scale) * 1.4426950408889634);
  if (a.k_scales != nullptr)
    return a.d == 64 ? launch_d<64, true>(a, p) : launch_d<128, true>(a, p);
  return a.d == 64 ? launch_d<64, false>(a, p) : launch_d<128, false>(a, p);
}

}  // namespace attn
