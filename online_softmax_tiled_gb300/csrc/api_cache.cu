// C ABI entry points around the KV cache (decode behind shared prefixes,
// rotary positions, key weights, eviction): argument validation and dispatch.
// Declarations and their documentation: include/attn.h.

#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "common.cuh"
#include "launchers.h"

using namespace attn;

namespace {

// float32 partials (o, m, l) of `splits` splits per query row
struct PartialLayout {
  size_t m_part, l_part, total;
};
PartialLayout partial_layout(long long rows, int d, long long splits) {
  PartialLayout l;
  const size_t n = size_t(rows) * size_t(splits);
  l.m_part = align256(n * d * sizeof(float));
  l.l_part = l.m_part + align256(n * sizeof(float));
  l.total = l.l_part + align256(n * sizeof(float));
  return l;
}

bool shared_sizes_ok(int B, int Hq, int Hkv, int d, int n_prefix, int prefix_page_size,
                     int max_prefix_pages, int page_size, int max_pages, int prefix_splits,
                     int splits) {
  return B > 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && d > 0 && n_prefix > 0 &&
         prefix_page_size > 0 && max_prefix_pages > 0 && page_size > 0 && max_pages > 0 &&
         prefix_splits >= 0 && splits >= 0;
}

// key positions are 32-bit in the kernels; splits, requests and KV heads are
// grid dimensions
bool shared_sizes_supported(int B, int Hq, int Hkv, int d, int prefix_page_size,
                            int max_prefix_pages, int page_size, int max_pages, int prefix_splits,
                            int splits) {
  const int G = Hq / Hkv;
  return (d == 64 || d == 128) && (G == 1 || G == 2 || G == 4 || G == 8) && B <= 65535 &&
         1LL * Hkv * G <= 65535 && prefix_splits <= 65535 && splits <= 65535 &&
         1LL * prefix_page_size * max_prefix_pages <= (1LL << 30) &&
         1LL * page_size * max_pages <= (1LL << 30) &&
         (max_prefix_pages == 1 || prefix_page_size % 8 == 0);
}

bool key_weights_sizes_ok(int B, int Hq, int Hkv, int T, long long cap, int out_len) {
  return B > 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && T > 0 && cap > 0 && out_len > 0;
}
bool key_weights_sizes_supported(int B, int Hq, int Hkv, int T, long long cap, int out_len) {
  return 1LL * B * Hkv <= 65535 && 1LL * (Hq / Hkv) * T <= (1LL << 30) && cap <= (1LL << 30) &&
         out_len <= (1 << 30) && 1LL * B * Hkv * ((cap + 127) / 128) <= (1LL << 30);
}

}  // namespace

extern "C" {

attn_status attn_rope(const void* q, const attn_strides* q_strides, void* q_out,
                      const attn_strides* q_out_strides, const void* k,
                      const attn_strides* k_strides, void* k_out,
                      const attn_strides* k_out_strides, const int* positions,
                      long long position_batch_stride, const double* inv_freq, int B, int Hq,
                      int Hkv, int N, int d, int rot_dim, int interleaved, float magnitude,
                      int inverse, attn_dtype dt, void* stream) {
  if (B <= 0 || Hq <= 0 || Hkv < 0 || N <= 0 || d <= 0) return ATTN_ERR_INVALID_ARG;
  if (!q || !q_out || !positions || !inv_freq) return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && (!k || !k_out)) return ATTN_ERR_INVALID_ARG;
  if (dt != ATTN_F32 && dt != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (rot_dim < 2 || rot_dim > d || rot_dim % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(magnitude) || position_batch_stride < 0) return ATTN_ERR_INVALID_ARG;
  if (d % 2 != 0 || d > 512) return ATTN_ERR_UNSUPPORTED;
  // tokens and heads are numbered in 32 bits; grid y carries at least 4 heads a block
  if (1LL * B * N > (1LL << 31) - 256 || 1LL * Hq + Hkv > 4 * 65535LL) return ATTN_ERR_UNSUPPORTED;
  const uintptr_t esize = dt == ATTN_BF16 ? 2 : 4;
  if (!aligned_to(q, esize) || !aligned_to(q_out, esize) || !aligned_to(positions, 4) ||
      !aligned_to(inv_freq, 8))
    return ATTN_ERR_MISALIGNED;
  if (Hkv > 0 && (!aligned_to(k, esize) || !aligned_to(k_out, esize))) return ATTN_ERR_MISALIGNED;
  RopeArgs a{q, q_out, k, k_out,
             strides_or_contiguous(q_strides, Hq, N, d),
             strides_or_contiguous(q_out_strides, Hq, N, d),
             strides_or_contiguous(k_strides, Hkv, N, d),
             strides_or_contiguous(k_out_strides, Hkv, N, d),
             positions, position_batch_stride, inv_freq, B, Hq, Hkv, N, d, rot_dim, interleaved,
             magnitude, inverse, dt, static_cast<cudaStream_t>(stream)};
  if (!non_negative(a.qs) || !rows_apart(a.qos, B, Hq, N, d) ||
      (q == q_out && !same_rows(a.qs, a.qos, B, Hq, N)))
    return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && (!non_negative(a.ks) || !rows_apart(a.kos, B, Hkv, N, d) ||
                  (k == k_out && !same_rows(a.ks, a.kos, B, Hkv, N))))
    return ATTN_ERR_INVALID_ARG;
  // blocks run in any order: but for a tensor turned in place, nothing that is
  // written may be read by the call or written twice
  const long long e = static_cast<long long>(esize);
  const RowSet in[] = {row_set(q, a.qs, B, Hq, N, d, e), row_set(k, a.ks, B, Hkv, N, d, e),
                       {positions, 4, {position_batch_stride * 4, 4, 0}, {B, N, 1}},
                       {inv_freq, rot_dim / 2 * 8LL, {0, 0, 0}, {1, 1, 1}}},
               out[] = {row_set(q_out, a.qos, B, Hq, N, d, e),
                        row_set(k_out, a.kos, B, Hkv, N, d, e)};
  for (int i = 0; i < (Hkv > 0 ? 2 : 1); ++i)
    for (int j = 0; j < 4; ++j)
      if ((j != 1 || Hkv > 0) && !(i == j && in[j].base == out[i].base) &&
          RowsMeet::test(in[j], out[i]))
        return ATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && RowsMeet::test(out[0], out[1])) return ATTN_ERR_INVALID_ARG;
  return from_cuda(launch_rope(a));
}

size_t attn_decode_shared_workspace_size(int B, int Hq, int Hkv, int d, int n_prefix,
                                         int prefix_page_size, int max_prefix_pages,
                                         int page_size, int max_pages_per_seq,
                                         int num_prefix_splits, int num_splits) {
  if (!shared_sizes_ok(B, Hq, Hkv, d, n_prefix, prefix_page_size, max_prefix_pages, page_size,
                       max_pages_per_seq, num_prefix_splits, num_splits) ||
      !shared_sizes_supported(B, Hq, Hkv, d, prefix_page_size, max_prefix_pages, page_size,
                              max_pages_per_seq, num_prefix_splits, num_splits))
    return 0;
  const SharedPlan pl = shared_plan(B, Hq, Hkv, d, n_prefix, prefix_page_size, max_prefix_pages,
                                    page_size, max_pages_per_seq, num_prefix_splits, num_splits);
  return partial_layout(1LL * B * Hq, d, 1LL * pl.prefix_splits + pl.own_splits).total;
}

attn_status attn_decode_shared(const void* q, const void* k_prefix, const void* v_prefix,
                               const int* prefix_table, const int* prefix_lens,
                               const int* prefix_start, const void* k_pages, const void* v_pages,
                               const int* block_table, const int* seq_lens, void* o, float* lse,
                               int B, int Hq, int Hkv, int d, int n_prefix, int num_prefix_pages,
                               int prefix_page_size, int max_prefix_pages, int num_pages,
                               int page_size, int max_pages_per_seq, float scale,
                               int num_prefix_splits, int num_splits, void* workspace,
                               size_t ws_bytes, void* stream) {
  if (!shared_sizes_ok(B, Hq, Hkv, d, n_prefix, prefix_page_size, max_prefix_pages, page_size,
                       max_pages_per_seq, num_prefix_splits, num_splits) ||
      num_prefix_pages <= 0 || num_pages <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (!q || !k_prefix || !v_prefix || !prefix_table || !prefix_lens || !prefix_start ||
      !k_pages || !v_pages || !block_table || !seq_lens || !o)
    return ATTN_ERR_INVALID_ARG;
  // (the prefix's kernel takes row maxima before scaling)
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (!shared_sizes_supported(B, Hq, Hkv, d, prefix_page_size, max_prefix_pages, page_size,
                              max_pages_per_seq, num_prefix_splits, num_splits))
    return ATTN_ERR_UNSUPPORTED;
  // rows of the pools: page coordinates of the copies are 32-bit
  if (1LL * num_prefix_pages * Hkv > (1LL << 31) - 1 ||
      1LL * num_pages * Hkv * page_size > (1LL << 40))
    return ATTN_ERR_UNSUPPORTED;
  const void* wide[] = {q, k_prefix, v_prefix, k_pages, v_pages, o};
  for (const void* x : wide)
    if (!aligned_to(x, 16)) return ATTN_ERR_MISALIGNED;
  const void* narrow[] = {prefix_table, prefix_lens, prefix_start, block_table, seq_lens, lse};
  for (const void* x : narrow)
    if (!aligned_to(x, 4)) return ATTN_ERR_MISALIGNED;
  const SharedPlan pl = shared_plan(B, Hq, Hkv, d, n_prefix, prefix_page_size, max_prefix_pages,
                                    page_size, max_pages_per_seq, num_prefix_splits, num_splits);
  // work items are numbered in 32 bits, as are the partial rows
  if (1LL * B * Hq * (1LL * pl.prefix_splits + pl.own_splits) > (1LL << 30))
    return ATTN_ERR_UNSUPPORTED;
  const PartialLayout lay = partial_layout(1LL * B * Hq, d, 1LL * pl.prefix_splits + pl.own_splits);
  if (!workspace || ws_bytes < lay.total) return ATTN_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return ATTN_ERR_MISALIGNED;
  char* ws = static_cast<char*>(workspace);
  SharedArgs a{};
  a.own = DecodeArgs{q, k_pages, v_pages, o, lse, B, Hq, Hkv, 0, d, scale, pl.own_splits,
                     reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + lay.m_part),
                     reinterpret_cast<float*>(ws + lay.l_part), static_cast<cudaStream_t>(stream)};
  a.own.block_table = block_table;
  a.own.seq_lens = seq_lens;
  a.own.num_pages = num_pages;
  a.own.page_size = page_size;
  a.own.max_pages = max_pages_per_seq;
  a.k_prefix = k_prefix;
  a.v_prefix = v_prefix;
  a.prefix_table = prefix_table;
  a.prefix_lens = prefix_lens;
  a.prefix_start = prefix_start;
  a.n_prefix = n_prefix;
  a.num_prefix_pages = num_prefix_pages;
  a.prefix_page_size = prefix_page_size;
  a.max_prefix_pages = max_prefix_pages;
  return from_cuda(launch_decode_shared(a, pl));
}

size_t attn_key_weights_workspace_size(int B, int Hq, int Hkv, int T, int capacity, int out_len) {
  if (!key_weights_sizes_ok(B, Hq, Hkv, T, capacity, out_len) ||
      !key_weights_sizes_supported(B, Hq, Hkv, T, capacity, out_len))
    return 0;
  return align256(size_t(key_weights_slots(Hq / Hkv * T, T)) * B * Hkv * out_len * sizeof(float));
}

attn_status attn_key_weights(const void* q, const void* k, const float* lse, const float* prev,
                             float* out, const int* seq_lens, const int* block_table, int B,
                             int Hq, int Hkv, int T, int L, int num_pages, int page_size,
                             int max_pages_per_seq, int out_len, int d, float scale, float decay,
                             int causal, void* workspace, size_t ws_bytes, void* stream) {
  if (!q || !k || !lse || !out) return ATTN_ERR_INVALID_ARG;
  if (block_table != nullptr &&
      (num_pages <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || !seq_lens))
    return ATTN_ERR_INVALID_ARG;
  const long long cap = block_table != nullptr ? 1LL * max_pages_per_seq * page_size : L;
  if (!key_weights_sizes_ok(B, Hq, Hkv, T, cap, out_len)) return ATTN_ERR_INVALID_ARG;
  if (seq_lens == nullptr && out_len < L) return ATTN_ERR_INVALID_ARG;
  // (1 / scale times a log-sum-exp must stay in range)
  if (!(scale >= 1e-30f) || !std::isfinite(scale) || (prev != nullptr && !std::isfinite(decay)))
    return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (!key_weights_sizes_supported(B, Hq, Hkv, T, cap, out_len)) return ATTN_ERR_UNSUPPORTED;
  if (block_table != nullptr && max_pages_per_seq > 1 && page_size % 8 != 0)
    return ATTN_ERR_UNSUPPORTED;
  // rows of the pool: page coordinates of the copies are 32-bit
  if (block_table != nullptr && 1LL * num_pages * Hkv > (1LL << 31) - 1)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(lse, 4) || !aligned_to(prev, 4) ||
      !aligned_to(out, 4) || !aligned_to(seq_lens, 4) || !aligned_to(block_table, 4))
    return ATTN_ERR_MISALIGNED;
  const size_t n_out = size_t(B) * Hkv * out_len * 4;
  if (prev != out && overlap(prev, n_out, out, n_out)) return ATTN_ERR_INVALID_ARG;
  const size_t rows = size_t(B) * Hq * T, keys = block_table != nullptr
                                                     ? size_t(num_pages) * Hkv * page_size
                                                     : size_t(B) * Hkv * L;
  if (overlap(q, rows * d * 2, out, n_out) || overlap(k, keys * d * 2, out, n_out) ||
      overlap(lse, rows * 4, out, n_out) || overlap(seq_lens, size_t(B) * 4, out, n_out) ||
      overlap(block_table, size_t(B) * max_pages_per_seq * 4, out, n_out))
    return ATTN_ERR_INVALID_ARG;
  const int len_cap = int(std::min<long long>(cap, out_len));
  if (const size_t slots = key_weights_slots(Hq / Hkv * T, T)) {
    if (!workspace || ws_bytes < align256(slots * n_out)) return ATTN_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return ATTN_ERR_MISALIGNED;
  }
  KeyWeightsArgs a{q, k, lse, prev, out, static_cast<float*>(workspace), seq_lens, block_table,
                   B, Hq, Hkv, T, L, num_pages, page_size, max_pages_per_seq, len_cap, out_len, d,
                   causal, scale, decay, static_cast<cudaStream_t>(stream)};
  return from_cuda(launch_key_weights(a));
}

attn_status attn_cache_evict(const void* k, const void* v, const float* scores,
                             const int* seq_lens, const int* block_table, void* k_out,
                             void* v_out, float* scores_out, int* kept, int* new_lens, int B,
                             int Hkv, int L, int num_pages, int page_size, int max_pages_per_seq,
                             int score_len, int d, int n_keep, int n_sink, int n_recent,
                             int out_len, attn_dtype dt, void* stream) {
  if (B <= 0 || Hkv <= 0 || score_len <= 0 || d <= 0) return ATTN_ERR_INVALID_ARG;
  if (!k || !v || !scores || !k_out || !v_out || !kept || !new_lens) return ATTN_ERR_INVALID_ARG;
  if (n_keep < 1 || n_sink < 0 || n_recent < 0 || 1LL * n_sink + n_recent > n_keep ||
      out_len < n_keep)
    return ATTN_ERR_INVALID_ARG;
  if (dt != ATTN_F32 && dt != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  long long cap = L;
  if (block_table != nullptr) {
    if (num_pages <= 0 || page_size <= 0 || max_pages_per_seq <= 0 || !seq_lens)
      return ATTN_ERR_INVALID_ARG;
    cap = 1LL * max_pages_per_seq * page_size;
  } else if (L <= 0 || (seq_lens == nullptr && score_len < L)) {
    return ATTN_ERR_INVALID_ARG;
  }
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  // key positions are 32-bit inside the kernels, (request, head) rows a grid's y
  if (cap > (1LL << 30) || score_len > (1 << 30) || out_len > (1 << 30) ||
      1LL * B * Hkv > 65535)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_out, 16) ||
      !aligned_to(v_out, 16) || !aligned_to(scores, 4) || !aligned_to(scores_out, 4) ||
      !aligned_to(seq_lens, 4) || !aligned_to(block_table, 4) || !aligned_to(kept, 4) ||
      !aligned_to(new_lens, 4))
    return ATTN_ERR_MISALIGNED;
  const size_t row = size_t(d) * (dt == ATTN_BF16 ? 2 : 4), heads = size_t(B) * Hkv;
  const size_t n_in = row * (block_table ? size_t(num_pages) * Hkv * page_size : heads * L);
  struct {
    const void* p;
    size_t n;
  } const in[] = {{k, n_in}, {v, n_in}, {scores, heads * score_len * 4},
                  {seq_lens, size_t(B) * 4},
                  {block_table, size_t(B) * max_pages_per_seq * 4}},
    out[] = {{k_out, heads * out_len * row}, {v_out, heads * out_len * row},
             {scores_out, heads * out_len * 4}, {kept, heads * n_keep * 4},
             {new_lens, size_t(B) * 4}};
  for (int i = 0; i < 5; ++i) {
    for (const auto& x : in)
      if (overlap(x.p, x.n, out[i].p, out[i].n)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[j].p, out[j].n, out[i].p, out[i].n)) return ATTN_ERR_INVALID_ARG;
  }
  EvictArgs a{k, v, scores, k_out, v_out, scores_out, kept, new_lens, seq_lens, block_table,
              num_pages, page_size, max_pages_per_seq, B, Hkv, L, d, score_len,
              int(cap < score_len ? cap : score_len), n_keep, n_sink, n_recent, out_len, dt,
              static_cast<cudaStream_t>(stream)};
  return from_cuda(launch_evict(a));
}

}  // extern "C"
