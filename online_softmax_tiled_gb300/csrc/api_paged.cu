// C ABI entry points of the paged caches (appending with rotation, reading a
// 4-bit cache back, decode under a window and over 4 bits): argument validation
// and dispatch. Declarations and their documentation: include/attn.h.

#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "common.cuh"
#include "launchers.h"

using namespace attn;

namespace {

struct Bytes {
  const void* p;
  size_t n;
};

// Pages of a cache: positions of keys are 32-bit in the kernels, as are the
// rows of a pool.
bool pages_ok(int B, int num_pages, int page_size, int max_pages) {
  return B > 0 && num_pages > 0 && page_size > 0 && max_pages > 0;
}
bool pages_supported(int Hkv, int num_pages, int page_size, int max_pages) {
  return 1LL * page_size * max_pages <= (1LL << 30) &&
         __int128(num_pages) * Hkv * page_size < (__int128(1) << 32);
}

RowSet plain_bytes(const Bytes& b) {
  return {b.p, static_cast<long long>(b.n), {0, 0, 0}, {1, 1, 1}};
}

// Whether any of `out` shares a byte with another of them or with any of `in`.
template <size_t I, size_t O> bool any_overlap(const Bytes (&in)[I], const Bytes (&out)[O]) {
  for (size_t i = 0; i < O; ++i) {
    for (const Bytes& x : in)
      if (overlap(x.p, x.n, out[i].p, out[i].n)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[j].p, out[j].n, out[i].p, out[i].n)) return true;
  }
  return false;
}

attn_status append_common(AppendArgs a, const attn_strides* q_strides,
                          const attn_strides* q_out_strides, const attn_strides* k_strides,
                          const attn_strides* v_strides) {
  if (!pages_ok(a.B, a.num_pages, a.page_size, a.max_pages) || a.Hq < 0 || a.Hkv <= 0 ||
      a.N <= 0 || a.d <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (!a.k || !a.v || !a.k_pool || !a.v_pool || !a.block_table || !a.seq_lens)
    return ATTN_ERR_INVALID_ARG;
  if (a.Hq > 0 && (!a.q || !a.q_out)) return ATTN_ERR_INVALID_ARG;
  if (a.dt != ATTN_F32 && a.dt != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (a.rot < 0 || a.rot > a.d || a.rot % 2 != 0 || (a.rot > 0 && !a.inv_freq))
    return ATTN_ERR_INVALID_ARG;
  if (a.interleaved != 0 && a.interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(a.magnitude) || a.pos_stride < 0) return ATTN_ERR_INVALID_ARG;
  if (a.d != 64 && a.d != 128) return ATTN_ERR_UNSUPPORTED;
  // tokens and heads are numbered in 32 bits
  if (1LL * a.B * a.N > (1LL << 31) - 256 || 1LL * a.Hq + 2LL * a.Hkv > 4 * 65535LL ||
      !pages_supported(a.Hkv, a.num_pages, a.page_size, a.max_pages))
    return ATTN_ERR_UNSUPPORTED;
  const bool four = a.k_scales != nullptr;
  const uintptr_t e = a.dt == ATTN_BF16 ? 2 : 4;
  if ((a.Hq > 0 && (!aligned_to(a.q, e) || !aligned_to(a.q_out, e))) || !aligned_to(a.k, e) ||
      !aligned_to(a.v, e) || !aligned_to(a.k_pool, 16) || !aligned_to(a.v_pool, 16) ||
      !aligned_to(a.k_scales, 16) || !aligned_to(a.v_scales, 16) || !aligned_to(a.block_table, 4) ||
      !aligned_to(a.seq_lens, 4) || !aligned_to(a.new_lens, 4) || !aligned_to(a.positions, 4) ||
      !aligned_to(a.inv_freq, 8))
    return ATTN_ERR_MISALIGNED;
  a.qs = strides_or_contiguous(q_strides, a.Hq, a.N, a.d);
  a.qos = strides_or_contiguous(q_out_strides, a.Hq, a.N, a.d);
  a.ks = strides_or_contiguous(k_strides, a.Hkv, a.N, a.d);
  a.vs = strides_or_contiguous(v_strides, a.Hkv, a.N, a.d);
  if (!non_negative(a.ks) || !non_negative(a.vs)) return ATTN_ERR_INVALID_ARG;
  if (a.Hq > 0 && (!non_negative(a.qs) || !rows_apart(a.qos, a.B, a.Hq, a.N, a.d) ||
                   (a.q == a.q_out && !same_rows(a.qs, a.qos, a.B, a.Hq, a.N))))
    return ATTN_ERR_INVALID_ARG;
  // blocks run in any order: but for queries turned in place, nothing that is
  // written may be read by the call or written twice
  const long long es = static_cast<long long>(e);
  const size_t rows = size_t(a.num_pages) * a.Hkv * a.page_size;
  const size_t row = four ? size_t(a.d) / 2 : size_t(a.d) * e, scale = size_t(a.d) / 16;
  const Bytes pools[] = {{a.k_pool, rows * row}, {a.v_pool, rows * row},
                         {a.k_scales, four ? rows * scale : 0},
                         {a.v_scales, four ? rows * scale : 0}};
  const int n_pools = four ? 4 : 2;
  const long long pos_rows = a.positions ? a.B : 0;
  const RowSet in[] = {
      row_set(a.q, a.qs, a.B, a.Hq, a.N, a.d, es), row_set(a.k, a.ks, a.B, a.Hkv, a.N, a.d, es),
      row_set(a.v, a.vs, a.B, a.Hkv, a.N, a.d, es),
      plain_bytes({a.block_table, size_t(a.B) * a.max_pages * 4}),
      plain_bytes({a.seq_lens, size_t(a.B) * 4}),
      plain_bytes({a.new_lens, a.new_lens ? size_t(a.B) * 4 : 0}),
      {a.positions, a.positions ? 4 : 0, {a.pos_stride * 4, 4, 0}, {pos_rows ? a.B : 1, a.N, 1}},
      plain_bytes({a.inv_freq, size_t(a.rot) / 2 * 8})};
  auto live = [](const RowSet& x) { return x.base != nullptr && x.len > 0; };
  for (int i = 0; i < n_pools; ++i) {
    const RowSet out = plain_bytes(pools[i]);
    for (const RowSet& x : in)
      if (live(x) && RowsMeet::test(x, out)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (RowsMeet::test(plain_bytes(pools[j]), out)) return ATTN_ERR_INVALID_ARG;
  }
  if (a.Hq > 0) {
    const RowSet out = row_set(a.q_out, a.qos, a.B, a.Hq, a.N, a.d, es);
    for (size_t i = 0; i < sizeof(in) / sizeof(in[0]); ++i)
      if (live(in[i]) && !(i == 0 && a.q == a.q_out) && RowsMeet::test(in[i], out))
        return ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < n_pools; ++i)
      if (RowsMeet::test(plain_bytes(pools[i]), out)) return ATTN_ERR_INVALID_ARG;
  }
  const cudaError_t launched = launch_cache_append(a);
  // (more blocks than a grid has: nothing was launched)
  return launched == cudaErrorInvalidConfiguration ? ATTN_ERR_UNSUPPORTED : from_cuda(launched);
}

struct WindowLayout {
  size_t m_part, l_part, total;
};
WindowLayout window_layout(int R, int d, int sm_count) {
  const size_t rows = size_t(window_partial_rows(R, sm_count));
  WindowLayout l;
  l.m_part = align256(rows * d * sizeof(float));
  l.l_part = l.m_part + align256(rows * sizeof(float));
  l.total = l.l_part + align256(rows * sizeof(float));
  return l;
}

bool window_sizes_ok(int B, int Hq, int Hkv, int T, int d) {
  return B > 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && T > 0 && d > 0;
}
// requests are a grid dimension, query rows of a KV head counted in 32 bits
bool window_sizes_supported(int B, int Hq, int Hkv, int T, int d) {
  return (d == 64 || d == 128) && B <= 65535 && 1LL * (Hq / Hkv) * T <= 65536 &&
         1LL * Hq * T <= (1LL << 30);
}

attn_status window_common(WindowArgs a, void* workspace, size_t ws_bytes) {
  if (!window_sizes_ok(a.B, a.Hq, a.Hkv, a.T, a.d) ||
      !pages_ok(a.B, a.num_pages, a.page_size, a.max_pages))
    return ATTN_ERR_INVALID_ARG;
  if (!a.q || !a.k || !a.v || !a.block_table || !a.seq_lens || !a.o) return ATTN_ERR_INVALID_ARG;
  // (a row's maximum is taken before scaling)
  if (!(a.scale > 0.f) || !std::isfinite(a.scale) || a.n_global < 0) return ATTN_ERR_INVALID_ARG;
  if (!window_sizes_supported(a.B, a.Hq, a.Hkv, a.T, a.d) ||
      !pages_supported(a.Hkv, a.num_pages, a.page_size, a.max_pages))
    return ATTN_ERR_UNSUPPORTED;
  // units of 64 keys of all requests and blocks of 8 query rows are counted in 32 bits
  const long long R = 1LL * (a.Hq / a.Hkv) * a.T;
  if (__int128(a.B) * a.Hkv * ((R + 7) / 8) * ((1LL * a.page_size * a.max_pages + 127) / 64) >
      (__int128(1) << 30))
    return ATTN_ERR_UNSUPPORTED;
  const bool four = a.k_scales != nullptr;
  const void* wide[] = {a.q, a.k, a.v, a.k_scales, a.v_scales, a.o};
  for (const void* x : wide)
    if (!aligned_to(x, 16)) return ATTN_ERR_MISALIGNED;
  if (!aligned_to(a.block_table, 4) || !aligned_to(a.seq_lens, 4) || !aligned_to(a.lse, 4))
    return ATTN_ERR_MISALIGNED;
  const size_t rows = size_t(a.num_pages) * a.Hkv * a.page_size, q_rows = size_t(a.B) * a.Hq * a.T;
  const size_t row = four ? size_t(a.d) / 2 : size_t(a.d) * 2, scale = four ? size_t(a.d) / 16 : 0;
  const Bytes in[] = {{a.q, q_rows * a.d * 2}, {a.k, rows * row}, {a.v, rows * row},
                      {a.k_scales, rows * scale}, {a.v_scales, rows * scale},
                      {a.block_table, size_t(a.B) * a.max_pages * 4}, {a.seq_lens, size_t(a.B) * 4}},
              out[] = {{a.o, q_rows * a.d * 2}, {a.lse, q_rows * 4}, {workspace, ws_bytes}};
  if (any_overlap(in, out)) return ATTN_ERR_INVALID_ARG;
  if (!workspace) return ATTN_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return ATTN_ERR_MISALIGNED;
  a.sm_count = device_sm_count();
  if (a.sm_count <= 0) return ATTN_ERR_CUDA;
  const WindowLayout lay = window_layout(int(R), a.d, a.sm_count);
  if (ws_bytes < lay.total) return ATTN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  a.o_part = reinterpret_cast<float*>(ws);
  a.m_part = reinterpret_cast<float*>(ws + lay.m_part);
  a.l_part = reinterpret_cast<float*>(ws + lay.l_part);
  return from_cuda(launch_decode_window(a));
}

}  // namespace

extern "C" {

attn_status attn_cache_append(const void* q, const attn_strides* q_strides, void* q_out,
                              const attn_strides* q_out_strides, const void* k,
                              const attn_strides* k_strides, const void* v,
                              const attn_strides* v_strides, void* k_pages, void* v_pages,
                              const int* block_table, const int* seq_lens, const int* new_lens,
                              const int* positions, long long position_batch_stride,
                              const double* inv_freq, int B, int Hq, int Hkv, int N, int d,
                              int rot_dim, int interleaved, float magnitude, int num_pages,
                              int page_size, int max_pages_per_seq, attn_dtype dt, void* stream) {
  AppendArgs a{q, q_out, k, v, {}, {}, {}, {}, k_pages, v_pages, nullptr, nullptr, block_table,
               seq_lens, new_lens, positions, position_batch_stride, inv_freq, B, Hq, Hkv, N, d,
               rot_dim, interleaved, magnitude, num_pages, page_size, max_pages_per_seq, dt,
               static_cast<cudaStream_t>(stream)};
  return append_common(a, q_strides, q_out_strides, k_strides, v_strides);
}

attn_status attn_cache_append4(const void* q, const attn_strides* q_strides, void* q_out,
                               const attn_strides* q_out_strides, const void* k,
                               const attn_strides* k_strides, const void* v,
                               const attn_strides* v_strides, void* k_codes, void* k_scales,
                               void* v_codes, void* v_scales, const int* block_table,
                               const int* seq_lens, const int* new_lens, const int* positions,
                               long long position_batch_stride, const double* inv_freq, int B,
                               int Hq, int Hkv, int N, int d, int rot_dim, int interleaved,
                               float magnitude, int num_pages, int page_size,
                               int max_pages_per_seq, attn_dtype dt, void* stream) {
  if (!k_scales || !v_scales) return ATTN_ERR_INVALID_ARG;
  AppendArgs a{q, q_out, k, v, {}, {}, {}, {}, k_codes, v_codes, k_scales, v_scales, block_table,
               seq_lens, new_lens, positions, position_batch_stride, inv_freq, B, Hq, Hkv, N, d,
               rot_dim, interleaved, magnitude, num_pages, page_size, max_pages_per_seq, dt,
               static_cast<cudaStream_t>(stream)};
  return append_common(a, q_strides, q_out_strides, k_strides, v_strides);
}

attn_status attn_cache_read4(const void* k_codes, const void* k_scales, const void* v_codes,
                             const void* v_scales, const int* block_table, const int* seq_lens,
                             void* k_out, void* v_out, int B, int Hkv, int L, int num_pages,
                             int page_size, int max_pages_per_seq, int d, void* stream) {
  if (!pages_ok(B, num_pages, page_size, max_pages_per_seq) || Hkv <= 0 || L <= 0 || d <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (!k_codes || !k_scales || !v_codes || !v_scales || !block_table || !seq_lens || !k_out ||
      !v_out)
    return ATTN_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || !pages_supported(Hkv, num_pages, page_size, max_pages_per_seq) ||
      1LL * B * Hkv > 65535 || L > (1 << 30))
    return ATTN_ERR_UNSUPPORTED;
  const void* wide[] = {k_codes, k_scales, v_codes, v_scales, k_out, v_out};
  for (const void* x : wide)
    if (!aligned_to(x, 16)) return ATTN_ERR_MISALIGNED;
  if (!aligned_to(block_table, 4) || !aligned_to(seq_lens, 4)) return ATTN_ERR_MISALIGNED;
  const size_t rows = size_t(num_pages) * Hkv * page_size, n_out = size_t(B) * Hkv * L * d * 2;
  const Bytes in[] = {{k_codes, rows * d / 2}, {v_codes, rows * d / 2}, {k_scales, rows * d / 16},
                      {v_scales, rows * d / 16}, {block_table, size_t(B) * max_pages_per_seq * 4},
                      {seq_lens, size_t(B) * 4}},
              out[] = {{k_out, n_out}, {v_out, n_out}};
  if (any_overlap(in, out)) return ATTN_ERR_INVALID_ARG;
  Read4Args a{k_codes, k_scales, v_codes, v_scales, block_table, seq_lens, k_out, v_out, B, Hkv, L,
              d, num_pages, page_size, max_pages_per_seq, static_cast<cudaStream_t>(stream)};
  return from_cuda(launch_cache_read4(a));
}

size_t attn_decode_window_workspace_size(int B, int Hq, int Hkv, int T, int d) {
  if (!window_sizes_ok(B, Hq, Hkv, T, d) || !window_sizes_supported(B, Hq, Hkv, T, d)) return 0;
  const int sms = device_sm_count();
  return sms > 0 ? window_layout(Hq / Hkv * T, d, sms).total : 0;
}

attn_status attn_decode_window(const void* q, const void* k_pages, const void* v_pages,
                               const int* block_table, const int* seq_lens, void* o, float* lse,
                               int B, int Hq, int Hkv, int T, int num_pages, int page_size,
                               int max_pages_per_seq, int d, float scale, int window_left,
                               int n_global, void* workspace, size_t ws_bytes, void* stream) {
  WindowArgs a{q, k_pages, v_pages, nullptr, nullptr, block_table, seq_lens, o, lse, nullptr,
               nullptr, nullptr, B, Hq, Hkv, T, num_pages, page_size, max_pages_per_seq, d,
               window_left, n_global, 0, scale, static_cast<cudaStream_t>(stream)};
  return window_common(a, workspace, ws_bytes);
}

attn_status attn_decode_cache4(const void* q, const void* k_codes, const void* k_scales,
                               const void* v_codes, const void* v_scales, const int* block_table,
                               const int* seq_lens, void* o, float* lse, int B, int Hq, int Hkv,
                               int T, int num_pages, int page_size, int max_pages_per_seq, int d,
                               float scale, int window_left, int n_global, void* workspace,
                               size_t ws_bytes, void* stream) {
  if (!k_scales || !v_scales) return ATTN_ERR_INVALID_ARG;
  WindowArgs a{q, k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, o, lse, nullptr,
               nullptr, nullptr, B, Hq, Hkv, T, num_pages, page_size, max_pages_per_seq, d,
               window_left, n_global, 0, scale, static_cast<cudaStream_t>(stream)};
  return window_common(a, workspace, ws_bytes);
}

}  // extern "C"
