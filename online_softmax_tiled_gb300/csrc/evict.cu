// Cache eviction: per (request, KV head) keep the first n_sink keys, the last
// n_recent and the best-scored of the others, n_keep in all, and move the
// kept K and V rows, in order, to the front of a new cache.
//
// Selection. The threshold is the want-th largest score of the middle keys,
// want = n_keep - n_sink - n_recent, found exactly by a radix descent over
// the scores mapped to ordered 32-bit integers (11, 11 and 10 bits): each
// pass counts the digits of the scores that share the prefix found so far
// and walks the counts from the top; the last passes fall away where all
// scores of the digit found stay, as where no other score shares 22 bits with
// the threshold. Scores above the threshold are kept,
// those equal to it as long as places remain, lowest index first: the
// result does not depend on the order of the counting atomics.
//
// A row of scores is short (4 bytes a key against 4·d·2 of K and V) but its
// passes depend on each other, so a row is spread over a cluster of up to
// eight CTAs whose counts are summed through distributed shared memory. Up to
// 131072 scores a row stay in registers through all passes; longer rows are
// read again for each (three digits, the count of what is kept, the writing).
//
// Moving the rows is bound by memory: every kept row is read once and
// written once. A thread moves 16-byte pieces, four rows of K and V in
// flight.
//
// Measured: 64 rows of 32768 scores, 4096 kept of d = 128 in bf16, 16-key
// pages: 59.3 us, of which the moving of the rows takes 40 (268 MB read and
// written, 6.6 TB/s) and the selection the rest: 4 to load the scores, 2 a
// pass, a barrier of the cluster between each, 3 to write the indices; none of
// it near a limit, all of it latency. With two CTAs a row; four or eight were
// slower (they share SMs). 6 rows of 1000, 128 kept: 8.8 us, 8.1
// in a CUDA graph.

#include <cooperative_groups.h>

#include "common.cuh"
#include "launchers.h"

namespace cg = cooperative_groups;

namespace attn {

ATTN_DEFINE_ERROR_WORD(take_error_evict)

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kLoads = 16;                // scores a thread has in flight
constexpr int kHeld = 32;                 // most scores a thread keeps in registers

// Ascending integers for ascending scores; NaN ranks as -inf, -0 as +0. Every
// score's key lies between those of -inf and +inf, strictly inside (kAbsent,
// kAlways), in the first and last 11-bit digit even.
constexpr uint32_t kAbsent = 0u, kAlways = 0xffffffffu;
ATTN_DEVINL uint32_t score_key(float s) {
  if (s != s) s = -INFINITY;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u ^ (uint32_t(int(u) >> 31) | 0x80000000u);
}

// The score of a key, where the key tells it (not of held ones, nor where NaN
// or -0 may be meant).
ATTN_DEVINL bool key_has_score(uint32_t key) {
  return key != kAlways && key != 0x007fffffu && key != 0x80000000u;
}
ATTN_DEVINL float score_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

ATTN_DEVINL int length_of(const int* seq_lens, int b, int cap, bool& bad) {
  if (seq_lens == nullptr) return cap;
  const int n = __ldcg(seq_lens + b);
  bad = n < 0 || n > cap;
  return bad ? 0 : n;
}

struct __align__(16) SelectSmem {
  int hist[3][kBins];      // this CTA's digit counts, one table per pass (read by the cluster)
  int part[kSelWarps];
  int sure[kSelWarps], equal[kSelWarps];   // per warp's segment (read by the cluster)
  int found[3];            // digit, how many scores rank above it, how many have it
};

// One cluster per (request, KV head) row; CTA r of C owns the r-th slice of
// the row's scores, warp w the w-th segment of the slice.
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const float* __restrict__ scores, const int* __restrict__ seq_lens,
                    float* __restrict__ scores_out, int* __restrict__ kept,
                    int* __restrict__ new_lens, int Hkv, int score_len, int cap, int cap_out,
                    int n_keep, int n_sink, int n_recent) {
  __shared__ SelectSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), r = int(cluster.block_rank());
  const int row = blockIdx.x / C, b = row / Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < 3 * kBins / 4; i += kSelThreads)
    reinterpret_cast<int4*>(sm.hist)[i] = make_int4(0, 0, 0, 0);
  // (the gathering kernel's start may rely on this wait: it reads the lengths,
  // from L2, before it waits for this kernel)
  pdl_wait_primary();
  pdl_launch_dependents();
  // A barrier over the row's CTAs; a cluster's takes 600 to 1000 cycles, a
  // single CTA's own a few dozen.
  auto row_sync = [&] {
    if (C > 1)
      cluster.sync();
    else
      __syncthreads();
  };

  bool bad = false;
  const int n = length_of(seq_lens, b, cap, bad);
  if (bad && tid == 0 && r == 0) attn_flag_error(kErrBadIndex);
  const int m = min(n, n_keep);
  if (tid == 0 && r == 0 && row % Hkv == 0) new_lens[b] = m;
  int* idx = kept + size_t(row) * n_keep;
  for (int i = m + r * kSelThreads + tid; i < n_keep; i += C * kSelThreads) idx[i] = -1;

  const float* s = scores + size_t(row) * score_len;
  // segments of whole warp reads, the last ones possibly short or empty
  const int seg = ((n + C * kSelWarps - 1) / (C * kSelWarps) + 31) & ~31;
  const int lo = min(n, (r * kSelWarps + warp) * seg), hi = min(n, lo + seg);
  const int mid0 = n_sink, mid1 = n - n_recent;      // the keys that are ranked
  const bool all = n <= n_keep;                      // (the same for the whole cluster)
  const bool held = seg <= 32 * kHeld;
  // Key of score j of this warp's segment (which is not empty): held sinks and
  // recents rank above everything, lanes past the segment below. (Its load is
  // made for every lane, none behind a branch, so that a thread's loads are in
  // flight together.)
  auto key_of = [&](float score, int j) {
    return j >= hi ? kAbsent : j < mid0 || j >= mid1 ? kAlways : score_key(score);
  };
  // The segment in groups of kLoads warp reads; those that fit stay in
  // registers. f(keys of the group, index of the lane's first one).
  uint32_t keys[kHeld];
  auto read = [&](uint32_t* key, int j) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) key[u] = __float_as_uint(s[min(j + u * 32, hi - 1)]);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) key[u] = key_of(__uint_as_float(key[u]), j + u * 32);
  };
  if (held && lo < hi) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) keys[u] = __float_as_uint(s[min(lo + u * 32 + lane, hi - 1)]);
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      keys[u] = key_of(__uint_as_float(keys[u]), lo + u * 32 + lane);
  }
  auto visit = [&](auto&& f) {
    if (held) {
#pragma unroll
      for (int g = 0; g < kHeld; g += kLoads)
        if (lo + g * 32 < hi) f(keys + g, lo + g * 32 + lane);
    } else {
      for (int j = lo; j < hi; j += 32 * kLoads) {
        uint32_t key[kLoads];
        read(key, j + lane);
        f(key, j + lane);
      }
    }
  };

  int need = all ? 0 : n_keep - n_sink - n_recent;   // how many ranked keys stay
  // Threshold: keys above it stay, and `need` of those equal to it.
  uint32_t bar = all ? kAbsent : need == 0 ? kAlways - 1 : 0;
  if (need > 0) {
    __syncthreads();                                 // the tables are zero
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digits = pass == 2 ? 1023 : 2047;
      int* hist = sm.hist[pass];
      const int above_bits = shift + (pass == 2 ? 10 : 11);
      // (in the first pass every lane counts: absent and held ones land in
      // the first and last bin, which no score reaches and the walk ignores)
      visit([&](const uint32_t* key, int) {
        uint32_t low = key[0], high = key[0];
#pragma unroll
        for (int u = 1; u < kLoads; ++u) {
          low = min(low, key[u]);
          high = max(high, key[u]);
        }
        // Scores that were never looked at are all zero: a group that agrees
        // adds once, where every lane would queue for the same counter.
        if (__all_sync(0xffffffffu, low == high) &&
            __reduce_min_sync(0xffffffffu, low) == __reduce_max_sync(0xffffffffu, low)) {
          if (lane == 0 && (pass == 0 || low >> above_bits == bar >> above_bits))
            atomicAdd(&hist[(low >> shift) & digits], 32 * kLoads);
          return;
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
          if (pass == 0 || key[u] >> above_bits == bar >> above_bits)
            atomicAdd(&hist[(key[u] >> shift) & digits], 1);
      });
      row_sync();
      // Thread t owns bins 4t .. 4t + 3 of the cluster's sum (the CTAs'
      // counts as independent 16-byte reads).
      int4 part[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        part[c] = c < C ? reinterpret_cast<const int4*>(
                              cluster.map_shared_rank(&sm, c)->hist[pass])[tid]
                        : make_int4(0, 0, 0, 0);
      int mine[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        mine[0] += part[c].x;
        mine[1] += part[c].y;
        mine[2] += part[c].z;
        mine[3] += part[c].w;
      }
      if (pass == 0 && tid == kBins / 4 - 1) mine[3] = 0;   // the held keys
      const int sum = mine[0] + mine[1] + mine[2] + mine[3];
      int suf = sum;                                 // suffix sums over the warp's lanes
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_down_sync(0xffffffffu, suf, off);
        if (lane + off < 32) suf += x;
      }
      if (lane == 0) sm.part[warp] = suf;
      __syncthreads();
      int above = suf - sum;                         // scores in higher bins
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) above += w > warp ? sm.part[w] : 0;
#pragma unroll
      for (int u = 3; u >= 0; --u) {
        if (above < need && above + mine[u] >= need) {
          sm.found[0] = 4 * tid + u;
          sm.found[1] = above;
          sm.found[2] = mine[u];
        }
        above += mine[u];
      }
      __syncthreads();
      bar |= uint32_t(sm.found[0]) << shift;
      need -= sm.found[1];
      if (need == sm.found[2]) {                     // all of the digit's scores stay
        bar -= 1;                                    // (no score has a zero first digit)
        need = 0;
        break;
      }
    }
  }

  // Keys of this segment that stay for sure, and that equal the threshold.
  int n_sure = 0, n_equal = 0;
  visit([&](const uint32_t* key, int) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      n_sure += key[u] > bar;
      n_equal += key[u] == bar;
    }
  });
  n_sure = __reduce_add_sync(0xffffffffu, n_sure);
  n_equal = __reduce_add_sync(0xffffffffu, n_equal);
  if (lane == 0) {
    sm.sure[warp] = n_sure;
    sm.equal[warp] = n_equal;
  }
  row_sync();
  // How many before this segment: in the warps of the CTAs before this one,
  // then the warps before this one.
  int s0 = 0, e0 = 0;
  for (int i = lane; i < r * kSelWarps + warp; i += 32) {
    const SelectSmem* o = cluster.map_shared_rank(&sm, i / kSelWarps);
    s0 += o->sure[i % kSelWarps];
    e0 += o->equal[i % kSelWarps];
  }
  s0 = __reduce_add_sync(0xffffffffu, s0);
  e0 = __reduce_add_sync(0xffffffffu, e0);
  float* so = scores_out == nullptr ? nullptr : scores_out + size_t(row) * cap_out;
  const uint32_t below = (1u << lane) - 1;
  auto keep = [&](uint32_t key, int at, int j) {
    idx[at] = j;
    if (so != nullptr) so[at] = key_has_score(key) ? score_of(key) : s[j];
  };
  if (need == 0) {
    // (nearly always: no tie is cut; counting bits is what this loop costs)
    visit([&](const uint32_t* key, int j0) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const uint32_t bs = __ballot_sync(0xffffffffu, key[u] > bar);
        if (key[u] > bar) keep(key[u], s0 + __popc(bs & below), j0 + u * 32);
        s0 += __popc(bs);
      }
    });
  } else {
    visit([&](const uint32_t* key, int j0) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const uint32_t bs = __ballot_sync(0xffffffffu, key[u] > bar);
        const uint32_t be = __ballot_sync(0xffffffffu, key[u] == bar);
        const int eq_before = e0 + __popc(be & below);
        if (key[u] > bar || (key[u] == bar && eq_before < need))
          keep(key[u], s0 + __popc(bs & below) + min(eq_before, need), j0 + u * 32);
        s0 += __popc(bs);
        e0 += __popc(be);
      }
    });
  }
  // no CTA leaves while another may still read its counts
  if (C > 1) cluster.sync();
}

struct GatherArgs {
  const uint4* k;
  const uint4* v;
  uint4* k_out;
  uint4* v_out;
  const int* kept;
  const int* seq_lens;
  const int* block_table;       // nullptr: contiguous
  int Hkv, L, len_cap, cap_out, n_keep, page_size, max_pages, num_pages;
};

// Grid: x over runs of kept rows, y over (request, KV head) rows. kPieces =
// 16-byte pieces of a row; a thread moves one piece of U rows, their loads in
// flight together.
template <int kPieces>
__global__ void __launch_bounds__(256) evict_gather_kernel(GatherArgs a) {
  constexpr int U = 4, kRows = 256 / kPieces;
  const int row = blockIdx.y, b = row / a.Hkv, h = row % a.Hkv;
  bool bad = false;
  const int m = min(length_of(a.seq_lens, b, a.len_cap, bad), a.n_keep);
  pdl_wait_primary();
  pdl_launch_dependents();
  const int piece = threadIdx.x % kPieces;
  const int i0 = blockIdx.x * kRows * U + threadIdx.x / kPieces;
  const int* idx = a.kept + size_t(row) * a.n_keep;
  uint4 kk[U], vv[U];
  bool ok[U];
  size_t src[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = i0 + u * kRows;
    ok[u] = i < m;
    if (ok[u]) {
      const int j = idx[i];
      if (a.block_table == nullptr) {
        src[u] = size_t(row) * a.L + j;
      } else {
        const int page = a.block_table[size_t(b) * a.max_pages + j / a.page_size];
        ok[u] = page >= 0 && page < a.num_pages;
        if (!ok[u]) attn_flag_error(kErrBadIndex);
        src[u] = (size_t(page) * a.Hkv + h) * a.page_size + j % a.page_size;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (ok[u]) {
      kk[u] = __ldcs(a.k + src[u] * kPieces + piece);
      vv[u] = __ldcs(a.v + src[u] * kPieces + piece);
    }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (ok[u]) {
      const size_t dst = (size_t(row) * a.cap_out + i0 + u * kRows) * kPieces + piece;
      a.k_out[dst] = kk[u];
      a.v_out[dst] = vv[u];
    }
}

template <int kPieces>
cudaError_t launch_gather(const EvictArgs& a) {
  const GatherArgs g{static_cast<const uint4*>(a.k), static_cast<const uint4*>(a.v),
                     static_cast<uint4*>(a.k_out), static_cast<uint4*>(a.v_out), a.kept,
                     a.seq_lens, a.block_table, a.Hkv, a.L, a.len_cap, a.cap_out, a.n_keep,
                     a.page_size, a.max_pages, a.num_pages};
  constexpr int rows_per_block = 4 * 256 / kPieces;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.n_keep + rows_per_block - 1) / rows_per_block),
                     unsigned(a.B * a.Hkv));
  cfg.blockDim = dim3(256);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_gather_kernel<kPieces>, g);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a) {
  // CTAs per row: as many as hold the row's scores in registers, and more
  // while all rows' CTAs stay within one per SM and keep 2048 scores.
  const int rows = a.B * a.Hkv;
  const long long slots = device_sm_count() > 0 ? device_sm_count() : 1;
  int C = 1;
  while (C < kMaxCluster &&
         (a.len_cap > C * kSelThreads * kHeld ||
          (2LL * C * rows <= slots && a.len_cap / (2 * C) >= 2048)))
    C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(rows * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a.scores, a.seq_lens,
                                     a.scores_out, a.kept, a.new_lens, a.Hkv, a.score_len,
                                     a.len_cap, a.cap_out, a.n_keep, a.n_sink, a.n_recent);
  if (e != cudaSuccess) return e;
  const int pieces = a.d * (a.dt == ATTN_BF16 ? 2 : 4) / 16;
  return pieces == 8 ? launch_gather<8>(a) : pieces == 16 ? launch_gather<16>(a)
                                                          : launch_gather<32>(a);
}

}  // namespace attn
