// Cache eviction: per (request, KV head) keep the first n_sink keys, the last
// n_recent and the best-scored of the others, n_keep in all, and move the
// kept K and V rows, in order, to the front of a new cache.
//
// Selection. The threshold is the want-th largest score of the middle keys,
// want = n_keep - n_sink - n_recent, found exactly by a radix descent over
// the scores mapped to ordered 32-bit integers (11, 11 and 10 bits): each
// pass counts the digits of the scores that share the prefix found so far
// and walks the counts from the top. Scores above the threshold are kept,
// those equal to it as long as places remain, lowest index first: the
// result does not depend on the order of the counting atomics.
//
// A row of scores is short (4 bytes a key against 4·d·2 of K and V) but its
// passes depend on each other, so a row is spread over a cluster of up to
// eight CTAs whose counts are summed through distributed shared memory; the
// scores are read four times, from L2 after the first pass.
//
// Moving the rows is bound by memory: every kept row is read once and
// written once. A thread moves 16-byte pieces, four rows of K and V in
// flight.

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
constexpr int kTile = kSelWarps * 128;    // scores per block-wide compaction step

// Ascending integers for ascending scores; NaN ranks as -inf, -0 as +0.
ATTN_DEVINL uint32_t score_key(float s) {
  if (s != s) s = -INFINITY;
  const uint32_t u = __float_as_uint(s + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

ATTN_DEVINL int length_of(const int* seq_lens, int b, int cap, bool& bad) {
  if (seq_lens == nullptr) return cap;
  const int n = seq_lens[b];
  bad = n < 0 || n > cap;
  return bad ? 0 : n;
}

struct SelectSmem {
  int hist[kBins];         // this CTA's digit counts (read by the cluster)
  int total[kBins];        // the cluster's
  int part[2 * kSelWarps + 2];
  int slice[2];            // kept-for-sure and equal-to-threshold scores of this CTA's slice
  int found[2];            // digit, and how many scores rank above it
};

// One cluster per (request, KV head) row; CTA r of C owns the r-th slice of
// the row's scores.
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const float* __restrict__ scores, const int* __restrict__ seq_lens,
                    float* __restrict__ scores_out, int* __restrict__ kept,
                    int* __restrict__ new_lens, int Hkv, int score_len, int cap, int cap_out,
                    int n_keep, int n_sink, int n_recent) {
  __shared__ SelectSmem sm;
  pdl_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), r = int(cluster.block_rank());
  const int row = blockIdx.x / C, b = row / Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait_primary();

  bool bad = false;
  const int n = length_of(seq_lens, b, cap, bad);
  if (bad && tid == 0 && r == 0) attn_flag_error(kErrBadIndex);
  const int m = min(n, n_keep);
  if (tid == 0 && r == 0 && row % Hkv == 0) new_lens[b] = m;
  int* idx = kept + size_t(row) * n_keep;
  for (int i = m + r * kSelThreads + tid; i < n_keep; i += C * kSelThreads) idx[i] = -1;

  const float* s = scores + size_t(row) * score_len;
  // slices of whole warps' reads, the last ones possibly empty
  const int per = ((n + C - 1) / C + 31) & ~31;
  const int lo = min(n, r * per), hi = min(n, lo + per);
  const int mid0 = n_sink, mid1 = n - n_recent;      // the keys that are ranked
  int need = n_keep - n_sink - n_recent;             // how many of them are kept
  uint32_t prefix = 0;                               // threshold digits found so far

  // (the same for every thread of the cluster)
  const bool all = n <= n_keep;
  if (!all && need > 0) {
    int shift = 21, bits = 11;
    uint32_t fixed = 0;                              // mask of the digits found so far
    for (int pass = 0; pass < 3; ++pass) {
      for (int i = tid; i < kBins; i += kSelThreads) sm.hist[i] = 0;
      __syncthreads();
      const int j0 = max(lo, mid0), j1 = min(hi, mid1);
      for (int base = j0; base < j1; base += 4 * kSelThreads) {
        uint32_t key[4];
        bool in[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = base + u * kSelThreads + tid;
          in[u] = j < j1;
          key[u] = in[u] ? score_key(s[j]) : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool live = in[u] && (key[u] & fixed) == prefix;
          const int digit = live ? int((key[u] >> shift) & ((1u << bits) - 1)) : -1;
          // scores that were never looked at are all zero: one add for a
          // warp that agrees
          int same;
          __match_all_sync(0xffffffffu, digit, &same);
          if (same) {
            if (lane == 0 && live) atomicAdd(&sm.hist[digit], 32);
          } else if (live) {
            atomicAdd(&sm.hist[digit], 1);
          }
        }
      }
      cluster.sync();
      for (int i = tid; i < kBins; i += kSelThreads) {
        int t = 0;
        for (int c = 0; c < C; ++c) t += cluster.map_shared_rank(&sm, c)->hist[i];
        sm.total[i] = t;
      }
      __syncthreads();
      // Thread t owns bins 4t .. 4t + 3; `above` = counts of all higher bins.
      int mine[4], sum = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) sum += mine[u] = sm.total[4 * tid + u];
      int suf = sum;                                 // suffix sums over the warp's lanes
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_down_sync(0xffffffffu, suf, off);
        if (lane + off < 32) suf += x;
      }
      if (lane == 0) sm.part[warp] = suf;
      __syncthreads();
      int above = suf - sum;
      for (int w = warp + 1; w < kSelWarps; ++w) above += sm.part[w];
#pragma unroll
      for (int u = 3; u >= 0; --u) {
        if (above < need && above + mine[u] >= need) {
          sm.found[0] = 4 * tid + u;
          sm.found[1] = above;
        }
        above += mine[u];
      }
      __syncthreads();
      prefix |= uint32_t(sm.found[0]) << shift;
      fixed |= ((1u << bits) - 1) << shift;
      need -= sm.found[1];
      bits = pass == 0 ? 11 : 10;
      shift = pass == 0 ? 10 : 0;
      // every CTA has read this CTA's counts before they are zeroed
      cluster.sync();
    }
  }

  // What becomes of key j: kept for sure, or equal to the threshold.
  auto classify = [&](int j, float& score, bool& sure, bool& equal) {
    const bool in = j < hi;
    score = in ? s[j] : 0.f;
    const bool held = j < mid0 || j >= mid1;
    const uint32_t key = score_key(score);
    sure = in && (all || held || (need > 0 && key > prefix));
    equal = in && !all && !held && need > 0 && key == prefix;
  };
  // (with no ranked key to keep, need is 0 and only held keys stay)
  if (tid < 2) sm.slice[tid] = 0;
  __syncthreads();
  {
    int cs = 0, ce = 0;
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      float score;
      bool sure, equal;
      classify(j, score, sure, equal);
      cs += sure;
      ce += equal;
    }
    cs = __reduce_add_sync(0xffffffffu, cs);
    ce = __reduce_add_sync(0xffffffffu, ce);
    if (lane == 0) {
      atomicAdd(&sm.slice[0], cs);
      atomicAdd(&sm.slice[1], ce);
    }
  }
  cluster.sync();
  int n_sure = 0, n_equal = 0;                       // in the slices before this one
  for (int c = 0; c < r; ++c) {
    n_sure += cluster.map_shared_rank(&sm, c)->slice[0];
    n_equal += cluster.map_shared_rank(&sm, c)->slice[1];
  }
  float* so = scores_out == nullptr ? nullptr : scores_out + size_t(row) * cap_out;
  for (int base = lo; base < hi; base += kTile) {
    float score[4];
    bool sure[4], equal[4];
    int rs[4], re[4], ws = 0, we = 0;                // ranks within the warp's 128 scores
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      classify(base + warp * 128 + u * 32 + lane, score[u], sure[u], equal[u]);
      const uint32_t bs = __ballot_sync(0xffffffffu, sure[u]);
      const uint32_t be = __ballot_sync(0xffffffffu, equal[u]);
      rs[u] = ws + __popc(bs & below);
      re[u] = we + __popc(be & below);
      ws += __popc(bs);
      we += __popc(be);
    }
    if (lane == 0) {
      sm.part[warp] = ws;
      sm.part[kSelWarps + warp] = we;
    }
    __syncthreads();
    int s0 = n_sure, e0 = n_equal, ts = 0, te = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) {
        s0 += sm.part[w];
        e0 += sm.part[kSelWarps + w];
      }
      ts += sm.part[w];
      te += sm.part[kSelWarps + w];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int eq_before = e0 + re[u];
      if (sure[u] || (equal[u] && eq_before < need)) {
        const int at = s0 + rs[u] + min(eq_before, need);
        idx[at] = base + warp * 128 + u * 32 + lane;
        if (so != nullptr) so[at] = score[u];
      }
    }
    n_sure += ts;
    n_equal += te;
    __syncthreads();
  }
  // no CTA leaves while another may still read its counts
  cluster.sync();
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
  pdl_launch_dependents();
  pdl_wait_primary();
  const int row = blockIdx.y, b = row / a.Hkv, h = row % a.Hkv;
  bool bad = false;
  const int m = min(length_of(a.seq_lens, b, a.len_cap, bad), a.n_keep);
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
  // CTAs per row: more while all rows' CTAs stay within two per SM and each
  // keeps 2048 scores (one per thread and load).
  const int rows = a.B * a.Hkv;
  const long long slots = 2LL * (device_sm_count() > 0 ? device_sm_count() : 1);
  int C = 1;
  while (C < 8 && 2LL * C * rows <= slots && a.len_cap / (2 * C) >= 2048) C *= 2;
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
