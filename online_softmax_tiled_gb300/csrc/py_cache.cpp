// Python calls of the cache operators (attn_rope, attn_decode_shared,
// attn_key_weights, attn_cache_evict, attn_cache_append, attn_cache_append4,
// attn_cache_read4, attn_decode_window, attn_decode_cache4): checks of the
// tensors, their pointers, shapes and strides, the current stream, and the C
// call. The operators run
// for a few microseconds; the same checks written in Python took two to five
// times as long as the kernels of a small call.
//
// Every function takes its arguments by position, None for an absent tensor,
// and raises ValueError or TypeError before anything is launched; a status of
// the C call other than ATTN_OK raises the class given to set_error().

#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "attn.h"

namespace {

PyObject* g_error = nullptr;   // AttnError(status, what)

struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void refuse_value(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
[[noreturn]] void refuse_type(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
struct Failed {
  int status;
  const char* what;
};

using Opt = std::optional<at::Tensor>;

at::Tensor tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
Opt optional_tensor(PyObject* o, const char* name) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, name);
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse_type("expected a whole number");
  }
  return v;
}
int small_int(PyObject* o) {
  const long long v = integer(o);
  if (v < -(1LL << 31) || v >= (1LL << 31)) refuse_value("number out of range");
  return int(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse_type("expected a number");
  }
  return float(v);
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse_type("expected a truth value");
  }
  return v;
}
int size(const at::Tensor& t, int i) {
  const int64_t n = t.size(i);
  if (n >= (1LL << 31)) refuse_value("dimension too large");
  return int(n);
}

// All tensors of a call are on one GPU, which the call makes current.
struct Device {
  int index = -1;
  explicit Device(const at::Tensor& t) {
    if (!t.is_cuda()) refuse_value("tensors must be on the GPU (device pointers)");
    index = t.get_device();
  }
  void on(const at::Tensor& t) const {
    if (!t.is_cuda() || t.get_device() != index)
      refuse_value("all tensors of a call must be on one GPU");
  }
  // the address of a contiguous tensor of type `dtype` on this device
  void* data(const at::Tensor& t, at::ScalarType dtype) const {
    on(t);
    if (t.scalar_type() != dtype)
      refuse_type(std::string("expected ") + c10::toString(dtype) + ", got " +
                  c10::toString(t.scalar_type()));
    if (!t.is_contiguous()) refuse_value("tensors must be contiguous");
    return t.data_ptr();
  }
  void* data(const Opt& t, at::ScalarType dtype) const {
    return t ? data(*t, dtype) : nullptr;
  }
  void* stream(PyObject* o) const {
    if (o != Py_None) return reinterpret_cast<void*>(integer(o));
    return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(index)).stream();
  }
};

// A new contiguous tensor on the current device (straight from the allocator's
// factory: the way through the dispatcher takes about as long again).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType dtype, const Device& dev) {
  return at::Tensor(at::detail::empty_cuda(
      sizes, dtype, c10::Device(c10::kCUDA, c10::DeviceIndex(dev.index)), std::nullopt));
}

attn_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return ATTN_BF16;
  if (t.scalar_type() == at::kFloat) return ATTN_F32;
  refuse_type(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) +
              ": float32 or bfloat16");
}

void check(attn_status st, const char* what) {
  if (st != ATTN_OK) throw Failed{int(st), what};
}

bool same_shape(const at::Tensor& a, const at::Tensor& b) { return a.sizes() == b.sizes(); }

template <typename F> PyObject* guarded(Py_ssize_t given, Py_ssize_t want, F&& f) {
  try {
    if (given != want) refuse_type("wrong number of arguments");
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const Failed& e) {
    PyObject* x = g_error == nullptr ? nullptr
                                     : PyObject_CallFunction(g_error, "is", e.status, e.what);
    if (x != nullptr) {
      PyErr_SetObject(g_error, x);
      Py_DECREF(x);
    } else if (!PyErr_Occurred()) {
      PyErr_SetString(PyExc_RuntimeError, e.what);
    }
  } catch (...) {
    // an allocation's or the runtime's: as torch itself raises it
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

PyObject* pair(const at::Tensor& a, const Opt& b) {
  PyObject* t = PyTuple_New(2);
  if (t == nullptr) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, b ? THPVariable_Wrap(*b) : (Py_INCREF(Py_None), Py_None));
  return t;
}

// attn_strides of a [B, H, N, d] or [B, H, d] tensor
attn_strides strides_of(const at::Tensor& t) {
  const auto st = t.strides();
  const auto n = st.size();
  if (st[n - 1] != 1 && t.size(int64_t(n) - 1) != 1)
    refuse_value("the last dimension must be contiguous");
  return attn_strides{st[0], st[1], n == 4 ? st[2] : 0};
}

// Positions of the tokens of a [B, H, N, d] (or [B, H, d]) tensor: [B, N], or [N]
// or [1, N] for all requests; of one token also [B]. Gives the stride between
// requests.
int64_t position_stride(const at::Tensor& pos, int64_t B, int64_t N) {
  const int64_t rows = pos.dim() == 2 ? pos.size(0) : pos.dim() == 1 && N == 1 ? pos.size(0) : 1;
  const int64_t cols = pos.dim() == 2 || (pos.dim() == 1 && N > 1) ? pos.size(-1) : 1;
  if (pos.dim() < 1 || pos.dim() > 2 || cols != N || (rows != B && rows != 1))
    refuse_value("positions must be [B, N], or [N] for all requests");
  return rows == B ? N : 0;
}

// q, k, positions, inv_freq, interleaved, magnitude, inverse, q_out, k_out, stream
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor q = tensor(a[0], "q"), pos = tensor(a[2], "positions"),
                     freq = tensor(a[3], "inv_freq");
    const Opt k = optional_tensor(a[1], "k");
    Opt q_out = optional_tensor(a[7], "q_out"), k_out = optional_tensor(a[8], "k_out");
    const Device dev(q);
    const int64_t dims = q.dim();
    if (dims != 3 && dims != 4) refuse_value("q must be [B, Hq, N, d] or [B, Hq, d]");
    const int B = size(q, 0), Hq = size(q, 1), N = dims == 4 ? size(q, 2) : 1,
              d = size(q, int(dims) - 1);
    const attn_dtype dt = dtype_of(q);
    c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev.index)};
    int Hkv = 0;
    if (k) {
      dev.on(*k);
      if (k->dim() != dims || k->size(0) != B || k->sizes().slice(2) != q.sizes().slice(2))
        refuse_value("k must be like q but for the number of heads");
      if (k->scalar_type() != q.scalar_type()) refuse_type("q and k must have one dtype");
      Hkv = size(*k, 1);
    } else if (k_out) {
      refuse_value("k and k_out go together");
    }
    if (!q_out) {
      q_out = fresh(q.sizes(), q.scalar_type(), dev);
      if (k && !k_out) k_out = fresh(k->sizes(), q.scalar_type(), dev);
    }
    if (k.has_value() != k_out.has_value()) refuse_value("k and k_out go together");
    for (const auto& p : {std::make_pair(&q, &q_out), std::make_pair(k ? &*k : nullptr, &k_out)}) {
      if (p.first == nullptr) continue;
      dev.on(**p.second);
      if (!same_shape(*p.first, **p.second) || (*p.second)->scalar_type() != q.scalar_type())
        refuse_value("outputs must be like q and k");
    }
    const int64_t pos_stride = position_stride(pos, B, N);
    if (freq.dim() != 1) refuse_value("inv_freq must be [rot_dim / 2]");
    const void* pp = dev.data(pos, at::kInt);
    const void* pw = dev.data(freq, at::kDouble);
    const attn_strides qs = strides_of(q), qos = strides_of(*q_out);
    attn_strides ks{}, kos{};
    if (k) {
      ks = strides_of(*k);
      kos = strides_of(*k_out);
    }
    check(attn_rope(q.data_ptr(), &qs, q_out->data_ptr(), &qos, k ? k->data_ptr() : nullptr,
                    k ? &ks : nullptr, k ? k_out->data_ptr() : nullptr, k ? &kos : nullptr,
                    static_cast<const int*>(pp), pos_stride,
                    static_cast<const double*>(pw), B, Hq, Hkv, N, d, 2 * size(freq, 0),
                    truth(a[4]), real(a[5]), truth(a[6]), dt, dev.stream(a[9])),
          "attn_rope");
    return pair(*q_out, k_out);
  });
}

// q, k_prefix, v_prefix, prefix_table, prefix_lens, prefix_start, k_pages,
// v_pages, block_table, seq_lens, o, lse, scale, num_prefix_splits,
// num_splits, workspace, allocate, stream
PyObject* py_decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&]() -> PyObject* {
    const at::Tensor q = tensor(a[0], "q"), kp = tensor(a[1], "k_prefix"),
                     vp = tensor(a[2], "v_prefix"), pt = tensor(a[3], "prefix_table"),
                     pl = tensor(a[4], "prefix_lens"), ps = tensor(a[5], "prefix_start"),
                     kk = tensor(a[6], "k_pages"), vv = tensor(a[7], "v_pages"),
                     bt = tensor(a[8], "block_table"), sl = tensor(a[9], "seq_lens");
    Opt o = optional_tensor(a[10], "o"), lse = optional_tensor(a[11], "lse"),
        ws = optional_tensor(a[15], "workspace");
    const Device dev(q);
    if (q.dim() != 3 || kp.dim() != 4 || kk.dim() != 4 || pt.dim() != 2 || bt.dim() != 2)
      refuse_value("shapes do not go together (see attn_decode_shared)");
    const int B = size(q, 0), Hq = size(q, 1), d = size(q, 2), Hkv = size(kp, 1),
              n_prefix = size(pt, 0);
    if (!same_shape(kp, vp) || !same_shape(kk, vv) || kp.size(3) != d || kk.size(3) != d ||
        kk.size(1) != Hkv || pl.dim() != 1 || pl.size(0) != n_prefix || ps.dim() != 1 ||
        ps.size(0) != n_prefix + 1 || bt.size(0) != B || sl.dim() != 1 || sl.size(0) != B)
      refuse_value("shapes do not go together (see attn_decode_shared)");
    const void* in[10] = {
        dev.data(q, at::kBFloat16),  dev.data(kp, at::kBFloat16), dev.data(vp, at::kBFloat16),
        dev.data(pt, at::kInt),      dev.data(pl, at::kInt),      dev.data(ps, at::kInt),
        dev.data(kk, at::kBFloat16), dev.data(vv, at::kBFloat16), dev.data(bt, at::kInt),
        dev.data(sl, at::kInt)};
    c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev.index)};
    const float scale = real(a[12]);
    const int sp = small_int(a[13]), so = small_int(a[14]);
    c10::DataPtr own_ws;
    size_t own_bytes = 0;
    if (truth(a[16])) {
      o = fresh(q.sizes(), at::kBFloat16, dev);
      lse = fresh({B, Hq}, at::kFloat, dev);
      if (!ws) {
        // (freed when the call returns, to be handed out again on its stream)
        own_bytes = attn_decode_shared_workspace_size(B, Hq, Hkv, d, n_prefix, size(kp, 2),
                                                      size(pt, 1), size(kk, 2), size(bt, 1), sp,
                                                      so);
        own_ws = c10::cuda::CUDACachingAllocator::get()->allocate(own_bytes);
      }
    }
    if (!o || (!ws && !truth(a[16]))) refuse_value("o and workspace are needed");
    if (!same_shape(*o, q) || (lse && (lse->dim() != 2 || lse->size(0) != B || lse->size(1) != Hq)))
      refuse_value("shapes do not go together (see attn_decode_shared)");
    if (ws) {
      dev.on(*ws);
      if (!ws->is_contiguous()) refuse_value("tensors must be contiguous");
    }
    auto ints = [](const void* p) { return static_cast<const int*>(p); };
    check(attn_decode_shared(in[0], in[1], in[2], ints(in[3]), ints(in[4]), ints(in[5]), in[6],
                             in[7], ints(in[8]), ints(in[9]), dev.data(*o, at::kBFloat16),
                             static_cast<float*>(dev.data(lse, at::kFloat)), B, Hq, Hkv, d,
                             n_prefix, size(kp, 0), size(kp, 2), size(pt, 1), size(kk, 0),
                             size(kk, 2), size(bt, 1), scale, sp, so,
                             ws ? ws->data_ptr() : own_ws.get(),
                             ws ? size_t(ws->nbytes()) : own_bytes, dev.stream(a[17])),
          "attn_decode_shared");
    return pair(*o, lse);
  });
}

// q, k, lse, prev, out, scale, decay, causal, seq_lens, block_table,
// workspace, allocate, stream
PyObject* py_key_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor q = tensor(a[0], "q"), k = tensor(a[1], "k"), lse = tensor(a[2], "lse");
    const Opt prev = optional_tensor(a[3], "prev"), sl = optional_tensor(a[8], "seq_lens"),
              bt = optional_tensor(a[9], "block_table");
    Opt out = optional_tensor(a[4], "out"), ws = optional_tensor(a[10], "workspace");
    const bool allocate = truth(a[11]);
    const Device dev(q);
    const int64_t dims = q.dim();
    if ((dims != 3 && dims != 4) || k.dim() != 4 || (bt && bt->dim() != 2))
      refuse_value("shapes do not go together (see attn_key_weights)");
    const int B = size(q, 0), Hq = size(q, 1), T = dims == 4 ? size(q, 2) : 1,
              d = size(q, int(dims) - 1), Hkv = size(k, 1), L = size(k, 2);
    const int max_pages = bt ? size(*bt, 1) : 0;
    const void* pq = dev.data(q, at::kBFloat16);
    const void* pk = dev.data(k, at::kBFloat16);
    const void* pl = dev.data(lse, at::kFloat);
    c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev.index)};
    const int64_t cap = bt ? int64_t(max_pages) * L : L;
    if (!out && allocate) {
      out = sl ? at::zeros({B, Hkv, cap}, k.options().dtype(at::kFloat))
               : fresh({B, Hkv, cap}, at::kFloat, dev);
    }
    if (!out) refuse_value("out is needed");
    if (out->dim() != 3 || out->size(0) != B || out->size(1) != Hkv || k.size(3) != d ||
        lse.sizes() != q.sizes().slice(0, dims - 1) || (bt ? bt->size(0) : k.size(0)) != B ||
        (prev && !same_shape(*prev, *out)) || (sl && (sl->dim() != 1 || sl->size(0) != B)))
      refuse_value("shapes do not go together (see attn_key_weights)");
    const int out_len = size(*out, 2);
    if (!ws && allocate && Hkv > 0 && int64_t(T) * Hq > 256LL * Hkv && cap < (1LL << 31)) {
      const size_t need = attn_key_weights_workspace_size(B, Hq, Hkv, T, int(cap), out_len);
      if (need > 0) ws = fresh({int64_t(need)}, at::kByte, dev);
    }
    if (ws) {
      dev.on(*ws);
      if (!ws->is_contiguous()) refuse_value("tensors must be contiguous");
    }
    check(attn_key_weights(pq, pk, static_cast<const float*>(pl),
                           static_cast<const float*>(dev.data(prev, at::kFloat)),
                           static_cast<float*>(dev.data(*out, at::kFloat)),
                           static_cast<const int*>(dev.data(sl, at::kInt)),
                           static_cast<const int*>(dev.data(bt, at::kInt)), B, Hq, Hkv, T, L,
                           size(k, 0), L, max_pages, out_len, d, real(a[5]), real(a[6]),
                           truth(a[7]), ws ? ws->data_ptr() : nullptr,
                           ws ? size_t(ws->nbytes()) : 0, dev.stream(a[12])),
          "attn_key_weights");
    return THPVariable_Wrap(*out);
  });
}

// k, v, scores, k_out, v_out, scores_out, kept, new_lens, n_sink, n_recent,
// seq_lens, block_table, stream
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor k = tensor(a[0], "k"), v = tensor(a[1], "v"), s = tensor(a[2], "scores"),
                     ko = tensor(a[3], "k_out"), vo = tensor(a[4], "v_out"),
                     kept = tensor(a[6], "kept"), len = tensor(a[7], "new_lens");
    const Opt so = optional_tensor(a[5], "scores_out"), sl = optional_tensor(a[10], "seq_lens"),
              bt = optional_tensor(a[11], "block_table");
    const Device dev(k);
    const attn_dtype dt = dtype_of(k);
    const auto type = k.scalar_type();
    if (k.dim() != 4 || kept.dim() != 3 || s.dim() != 3 || ko.dim() != 4 || len.dim() != 1 ||
        (so && so->dim() != 3) || (sl && sl->dim() != 1) || (bt && bt->dim() != 2))
      refuse_value("shapes do not go together (see attn_cache_evict)");
    const int B = size(kept, 0), Hkv = size(kept, 1), n_keep = size(kept, 2), d = size(k, 3),
              out_len = size(ko, 2);
    if (!same_shape(k, v) || k.size(1) != Hkv || s.size(0) != B || s.size(1) != Hkv ||
        ko.size(0) != B || ko.size(1) != Hkv || ko.size(3) != d || !same_shape(ko, vo) ||
        len.size(0) != B || (so && so->sizes() != ko.sizes().slice(0, 3)) ||
        (sl && sl->size(0) != B) || (bt ? bt->size(0) : k.size(0)) != B)
      refuse_value("shapes do not go together (see attn_cache_evict)");
    c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev.index)};
    check(attn_cache_evict(
              dev.data(k, type), dev.data(v, type), static_cast<float*>(dev.data(s, at::kFloat)),
              static_cast<int*>(dev.data(sl, at::kInt)), static_cast<int*>(dev.data(bt, at::kInt)),
              dev.data(ko, type), dev.data(vo, type), static_cast<float*>(dev.data(so, at::kFloat)),
              static_cast<int*>(dev.data(kept, at::kInt)),
              static_cast<int*>(dev.data(len, at::kInt)), B, Hkv, size(k, 2), size(k, 0),
              size(k, 2), bt ? size(*bt, 1) : 0, size(s, 2), d, n_keep, small_int(a[8]),
              small_int(a[9]), out_len, dt, dev.stream(a[12])),
          "attn_cache_evict");
    Py_RETURN_NONE;
  });
}

// The pools of a paged cache: [num_pages, Hkv, page_size, d] rows, or codes
// [.., d / 2] and scales [.., d / 32].
struct Pools {
  at::Tensor k, v;
  Opt ks, vs;
  int pages, Hkv, page, d;
  void *kp, *vp, *ksp = nullptr, *vsp = nullptr;
  Pools(PyObject* const* a, const Device& dev, at::ScalarType rows, bool four)
      : k(tensor(a[0], four ? "k_codes" : "k_pages")), v(tensor(a[four ? 2 : 1], "v")) {
    if (k.dim() != 4 || !same_shape(k, v)) refuse_value("pools must be alike, [pages, Hkv, page, d]");
    pages = size(k, 0);
    Hkv = size(k, 1);
    page = size(k, 2);
    d = size(k, 3) * (four ? 2 : 1);
    const at::ScalarType type = four ? at::kByte : rows;
    kp = dev.data(k, type);
    vp = dev.data(v, type);
    if (!four) return;
    ks = tensor(a[1], "k_scales");
    vs = tensor(a[3], "v_scales");
    if (ks->dim() != 4 || !same_shape(*ks, *vs) || ks->sizes().slice(0, 3) != k.sizes().slice(0, 3) ||
        ks->size(3) * 32 != d)
      refuse_value("scales must be [pages, Hkv, page, d / 32]");
    ksp = dev.data(*ks, at::kBFloat16);
    vsp = dev.data(*vs, at::kBFloat16);
  }
};

// Block table [B, max_pages] and lengths [B] of a call's requests.
struct Requests {
  const int *table, *lens;
  int max_pages;
  Requests(const at::Tensor& t, const at::Tensor& l, int64_t B, const Device& dev) {
    if (t.dim() != 2 || t.size(0) != B || l.dim() != 1 || l.size(0) != B)
      refuse_value("block_table must be [B, max_pages], seq_lens [B]");
    table = static_cast<const int*>(dev.data(t, at::kInt));
    lens = static_cast<const int*>(dev.data(l, at::kInt));
    max_pages = size(t, 1);
  }
};

// q, k, v, 2 (rows) or 4 (4 bits) pools, block_table, seq_lens, inv_freq,
// positions, new_lens, interleaved, magnitude, q_out, allocate, stream
template <bool kFour> PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kPools = kFour ? 4 : 2;
  return guarded(n, 13 + kPools, [&]() -> PyObject* {
    const Opt q = optional_tensor(a[0], "q");
    const at::Tensor k = tensor(a[1], "k"), v = tensor(a[2], "v");
    PyObject* const* r = a + 3 + kPools;
    const Opt freq = optional_tensor(r[2], "inv_freq"), pos = optional_tensor(r[3], "positions"),
              fresh_lens = optional_tensor(r[4], "new_lens");
    Opt q_out = optional_tensor(r[7], "q_out");
    const Device dev(k);
    const int64_t dims = k.dim();
    if (dims != 3 && dims != 4) refuse_value("k must be [B, Hkv, N, d] or [B, Hkv, d]");
    const attn_dtype dt = dtype_of(k);
    const int B = size(k, 0), Hkv = size(k, 1), N = dims == 4 ? size(k, 2) : 1,
              d = size(k, int(dims) - 1);
    dev.on(v);
    if (!same_shape(k, v) || v.scalar_type() != k.scalar_type())
      refuse_value("k and v must be alike");
    c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev.index)};
    const Pools pools(a + 3, dev, k.scalar_type(), kFour);
    if (pools.Hkv != Hkv || pools.d != d) refuse_value("pools must have the heads and d of k");
    const Requests req(tensor(r[0], "block_table"), tensor(r[1], "seq_lens"), B, dev);
    int Hq = 0;
    if (q) {
      dev.on(*q);
      if (q->dim() != dims || q->size(0) != B || q->sizes().slice(2) != k.sizes().slice(2) ||
          q->scalar_type() != k.scalar_type())
        refuse_value("q must be like k but for the number of heads");
      Hq = size(*q, 1);
      if (!q_out && truth(r[8])) q_out = fresh(q->sizes(), q->scalar_type(), dev);
      if (!q_out) refuse_value("q_out is needed");
      dev.on(*q_out);
      if (!same_shape(*q, *q_out) || q_out->scalar_type() != q->scalar_type())
        refuse_value("q_out must be like q");
    } else if (q_out) {
      refuse_value("q and q_out go together");
    }
    if (freq && freq->dim() != 1) refuse_value("inv_freq must be [rot_dim / 2]");
    if (fresh_lens && (fresh_lens->dim() != 1 || fresh_lens->size(0) != B))
      refuse_value("new_lens must be [B]");
    attn_strides qs{}, qos{};
    if (q) {
      qs = strides_of(*q);
      qos = strides_of(*q_out);
    }
    const attn_strides ks = strides_of(k), vs = strides_of(v);
    const int rot = freq ? 2 * size(*freq, 0) : 0;
    auto ints = [&](const Opt& t) { return static_cast<const int*>(dev.data(t, at::kInt)); };
    const double* fp = static_cast<const double*>(dev.data(freq, at::kDouble));
    const int64_t stride = pos ? position_stride(*pos, B, N) : 0;
    const void* qp = q ? q->data_ptr() : nullptr;
    void* qop = q ? q_out->data_ptr() : nullptr;
    if constexpr (kFour)
      check(attn_cache_append4(qp, &qs, qop, &qos, k.data_ptr(), &ks, v.data_ptr(), &vs, pools.kp,
                               pools.ksp, pools.vp, pools.vsp, req.table, req.lens,
                               ints(fresh_lens), ints(pos), stride, fp, B, Hq, Hkv, N, d, rot,
                               truth(r[5]), real(r[6]), pools.pages, pools.page, req.max_pages, dt,
                               dev.stream(r[9])),
            "attn_cache_append4");
    else
      check(attn_cache_append(qp, &qs, qop, &qos, k.data_ptr(), &ks, v.data_ptr(), &vs, pools.kp,
                              pools.vp, req.table, req.lens, ints(fresh_lens), ints(pos), stride,
                              fp, B, Hq, Hkv, N, d, rot, truth(r[5]), real(r[6]), pools.pages,
                              pools.page, req.max_pages, dt, dev.stream(r[9])),
            "attn_cache_append");
    if (!q) Py_RETURN_NONE;
    return THPVariable_Wrap(*q_out);
  });
}

// 4 pools, block_table, seq_lens, k_out, v_out, stream
PyObject* py_read4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor ko = tensor(a[6], "k_out"), vo = tensor(a[7], "v_out");
    const Device dev(ko);
    if (ko.dim() != 4 || !same_shape(ko, vo)) refuse_value("outputs must be [B, Hkv, L, d]");
    const int B = size(ko, 0);
    c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev.index)};
    const Pools pools(a, dev, at::kByte, true);
    if (ko.size(1) != pools.Hkv || ko.size(3) != pools.d)
      refuse_value("outputs must have the heads and d of the pools");
    const Requests req(tensor(a[4], "block_table"), tensor(a[5], "seq_lens"), B, dev);
    check(attn_cache_read4(pools.kp, pools.ksp, pools.vp, pools.vsp, req.table, req.lens,
                           dev.data(ko, at::kBFloat16), dev.data(vo, at::kBFloat16), B, pools.Hkv,
                           size(ko, 2), pools.pages, pools.page, req.max_pages, pools.d,
                           dev.stream(a[8])),
          "attn_cache_read4");
    return pair(ko, vo);
  });
}

// q, 2 (bf16) or 4 (4 bits) pools, block_table, seq_lens, o, lse, scale,
// window_left, n_global, workspace, allocate, stream
template <bool kFour> PyObject* py_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kPools = kFour ? 4 : 2;
  return guarded(n, 11 + kPools, [&]() -> PyObject* {
    const at::Tensor q = tensor(a[0], "q");
    PyObject* const* r = a + 1 + kPools;
    Opt o = optional_tensor(r[2], "o"), lse = optional_tensor(r[3], "lse");
    const Opt ws = optional_tensor(r[7], "workspace");
    const bool allocate = truth(r[8]);
    const Device dev(q);
    const int64_t dims = q.dim();
    if (dims != 3 && dims != 4) refuse_value("q must be [B, Hq, T, d] or [B, Hq, d]");
    const int B = size(q, 0), Hq = size(q, 1), T = dims == 4 ? size(q, 2) : 1,
              d = size(q, int(dims) - 1);
    const void* qp = dev.data(q, at::kBFloat16);
    c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev.index)};
    const Pools pools(a + 1, dev, at::kBFloat16, kFour);
    if (pools.d != d) refuse_value("pools must have the d of q");
    const Requests req(tensor(r[0], "block_table"), tensor(r[1], "seq_lens"), B, dev);
    c10::DataPtr own_ws;
    size_t own_bytes = 0;
    if (allocate) {
      o = fresh(q.sizes(), at::kBFloat16, dev);
      lse = fresh(q.sizes().slice(0, dims - 1), at::kFloat, dev);
      if (!ws) {
        // (freed when the call returns, to be handed out again on its stream)
        own_bytes = attn_decode_window_workspace_size(B, Hq, pools.Hkv, T, d);
        own_ws = c10::cuda::CUDACachingAllocator::get()->allocate(own_bytes);
      }
    }
    if (!o || (!ws && !allocate)) refuse_value("o and workspace are needed");
    if (!same_shape(*o, q) || (lse && lse->sizes() != q.sizes().slice(0, dims - 1)))
      refuse_value("o must be like q, lse like q without d");
    if (ws) {
      dev.on(*ws);
      if (!ws->is_contiguous()) refuse_value("tensors must be contiguous");
    }
    void* op = dev.data(*o, at::kBFloat16);
    float* lp = static_cast<float*>(dev.data(lse, at::kFloat));
    void* wp = ws ? ws->data_ptr() : own_ws.get();
    const size_t wn = ws ? size_t(ws->nbytes()) : own_bytes;
    const float scale = real(r[4]);
    const int left = small_int(r[5]), global = small_int(r[6]);
    if constexpr (kFour)
      check(attn_decode_cache4(qp, pools.kp, pools.ksp, pools.vp, pools.vsp, req.table, req.lens,
                               op, lp, B, Hq, pools.Hkv, T, pools.pages, pools.page, req.max_pages,
                               d, scale, left, global, wp, wn, dev.stream(r[9])),
            "attn_decode_cache4");
    else
      check(attn_decode_window(qp, pools.kp, pools.vp, req.table, req.lens, op, lp, B, Hq,
                               pools.Hkv, T, pools.pages, pools.page, req.max_pages, d, scale, left,
                               global, wp, wn, dev.stream(r[9])),
            "attn_decode_window");
    return pair(*o, lse);
  });
}

PyObject* py_set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define FAST(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST("rope", py_rope),
                           FAST("decode_shared", py_decode_shared),
                           FAST("key_weights", py_key_weights),
                           FAST("evict", py_evict),
                           FAST("append", py_append<false>),
                           FAST("append4", py_append<true>),
                           FAST("read4", py_read4),
                           FAST("window", py_window<false>),
                           FAST("cache4", py_window<true>),
                           {"set_error", py_set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cache_calls", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_calls() { return PyModule_Create(&g_module); }
