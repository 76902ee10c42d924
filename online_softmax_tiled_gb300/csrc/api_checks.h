// Checks of arguments that entry points share: alignment, strided rows, and
// whether bytes that a call writes are read or written by it elsewhere.
#pragma once

#include <stdint.h>

#include <algorithm>

#include <cuda_runtime.h>

#include "attn.h"

namespace attn {

inline attn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

inline attn_strides strides_or_contiguous(const attn_strides* s, int H, int N, int d) {
  if (s != nullptr) return *s;
  return attn_strides{1LL * H * N * d, 1LL * N * d, d};
}

// Whether the rows of a [B, H, N, d] tensor are apart: each dimension (by
// growing stride) steps over all that the ones before it cover.
inline bool rows_apart(const attn_strides& s, int B, int H, int N, int d) {
  struct Dim {
    long long stride;
    int n;
  } dims[3] = {{s.batch, B}, {s.head, H}, {s.token, N}};
  std::sort(dims, dims + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  long long covered = d;
  for (const Dim& x : dims) {
    if (x.n == 1) continue;
    if (x.stride < covered) return false;
    covered += x.stride * (x.n - 1);
  }
  return true;
}

inline bool non_negative(const attn_strides& s) { return s.batch >= 0 && s.head >= 0 && s.token >= 0; }

inline bool same_rows(const attn_strides& a, const attn_strides& b, int B, int H, int N) {
  return (B == 1 || a.batch == b.batch) && (H == 1 || a.head == b.head) &&
         (N == 1 || a.token == b.token);
}

// Rows of `len` bytes at base + i·stride0 + j·stride1 + k·stride2 (bytes;
// strides >= 0).
struct RowSet {
  const void* base;
  long long len;
  long long stride[3];
  int n[3];
  __int128 first() const { return __int128(reinterpret_cast<uintptr_t>(base)); }
  __int128 last() const {      // of its bytes
    __int128 at = first() + len - 1;
    for (int i = 0; i < 3; ++i) at += __int128(stride[i]) * (n[i] - 1);
    return at;
  }
};
inline RowSet row_set(const void* p, const attn_strides& s, int B, int H, int N, int d, long long esize) {
  return {p, d * esize, {s.batch * esize, s.head * esize, s.token * esize}, {B, H, N}};
}

// Whether a byte belongs to rows of both sets. With the strides of both as
// one list, the row starts lie a.base - b.base + Σ stride·x apart, each x in a
// range of its own (equal strides joined), and two rows meet where that is in
// [-(a.len - 1), b.len - 1]. The x are tried from the largest stride down,
// those only from which the smaller strides can still reach: one or two each
// for sets that lie apart or inside each other's gaps. Sets that would take
// long to tell count as meeting.
struct RowsMeet {
  using Wide = __int128;
  Wide stride[6], lo[6], hi[6], rest_lo[7], rest_hi[7];
  Wide from, to;               // distances at which rows meet
  int dims = 0, left = 4096;   // distances still to be tried

  void add(long long s, long long first, long long last) {
    if (s == 0 || first == last) return;
    int i = 0;
    while (i < dims && stride[i] > s) ++i;
    if (i < dims && stride[i] == s) {
      lo[i] += first;
      hi[i] += last;
      return;
    }
    for (int k = dims++; k > i; --k) {
      stride[k] = stride[k - 1];
      lo[k] = lo[k - 1];
      hi[k] = hi[k - 1];
    }
    stride[i] = s;
    lo[i] = first;
    hi[i] = last;
  }
  static Wide floor_div(Wide x, Wide y) { return x / y - (x % y < 0); }
  bool search(int k, Wide at) {
    if (--left < 0) return true;
    if (k == dims) return at >= from && at <= to;
    const Wide s = stride[k];
    const Wide x0 = std::max(lo[k], -floor_div(at + rest_hi[k + 1] - from, s));
    const Wide x1 = std::min(hi[k], floor_div(to - at - rest_lo[k + 1], s));
    for (Wide x = x0; x <= x1; ++x)
      if (search(k + 1, at + s * x)) return true;
    return false;
  }
  static bool test(const RowSet& a, const RowSet& b) {
    if (a.first() > b.last() || b.first() > a.last()) return false;
    RowsMeet m;
    for (int i = 0; i < 3; ++i) {
      m.add(a.stride[i], 0, a.n[i] - 1);
      m.add(b.stride[i], -(b.n[i] - 1LL), 0);
    }
    m.rest_lo[m.dims] = m.rest_hi[m.dims] = 0;
    for (int k = m.dims - 1; k >= 0; --k) {
      m.rest_lo[k] = m.rest_lo[k + 1] + m.stride[k] * m.lo[k];
      m.rest_hi[k] = m.rest_hi[k + 1] + m.stride[k] * m.hi[k];
    }
    m.from = -(a.len - 1);
    m.to = b.len - 1;
    return m.search(0, a.first() - b.first());
  }
};

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}

}  // namespace attn
