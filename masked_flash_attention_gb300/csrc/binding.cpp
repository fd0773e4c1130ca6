// binding.cpp -- the host side of the short calls (fa_rope, fa_qk_norm_rope,
// fa_kvcache_append, fa_fwd_chunk and the forms for a cache in 8 bits) as a CPython module: reads torch tensors, allocates outputs on
// the call's stream, fills the C ABI's structures and calls it.  One token's
// rotation runs 3 us on the device; through ctypes its call took 28 us on the
// host.  Arguments come positionally from the Python functions of the same
// names, which hold the signatures, defaults and documentation; a non-zero
// status comes back as an int, to be raised there.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <optional>

#include "fa.h"

namespace {

struct Refused {};  // the arguments do not reach the C ABI: FA_ERR_INVALID_ARG
struct Raised {};   // a Python exception is set

// One call's arguments, structures and stream.
struct Call {
  PyObject* const* args;
  const bool on_device;  // false: host-only (plans)
  mutable int device = -1;  // the current CUDA device, asked for with the first tensor
  fa_tensor descs[20];
  int n_descs = 0;
  fa_opts opts;
  std::optional<c10::cuda::CUDAStreamGuard> guard;

  Call(PyObject* const* a, bool on_dev) : args(a), on_device(on_dev) { memset(&opts, 0, sizeof(opts)); }

  // The tensor argument i (null for None), on the current device.
  const at::Tensor* tensor(int i) const {
    PyObject* o = args[i];
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (on_device) {
      if (!t.is_cuda()) throw Refused();
      if (device < 0) device = c10::cuda::current_device();
      if (t.get_device() != device) throw Refused();
    }
    return &t;
  }
  const at::Tensor& required(int i) const {
    const at::Tensor* t = tensor(i);
    if (!t) throw Refused();
    return *t;
  }
  int32_t i32(int i, bool optional = false) const {
    if (optional && args[i] == Py_None) return 0;
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(args[i], &over);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    if (over || v < INT32_MIN || v > INT32_MAX) throw Refused();
    return (int32_t)v;
  }
  float f32(int i, bool optional = false) const {
    if (optional && args[i] == Py_None) return 0.f;
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return (float)v;
  }
  int32_t truth(int i) const {
    const int v = PyObject_IsTrue(args[i]);
    if (v < 0) throw Raised();
    return v;
  }
  void* pointer(int i) const {
    if (args[i] == Py_None) return nullptr;
    void* v = PyLong_AsVoidPtr(args[i]);
    if (!v && PyErr_Occurred()) throw Raised();
    return v;
  }

  // A view of t for the C ABI (null for null).
  const fa_tensor* describe(const at::Tensor* t) {
    if (!t) return nullptr;
    fa_tensor& d = descs[n_descs++];
    memset(&d, 0, sizeof(d));
    if (t->dim() > 4) throw Refused();
    // an empty tensor may have no storage: a dummy non-null pointer (never read)
    void* ptr = t->numel() ? t->data_ptr() : nullptr;
    d.data = ptr ? ptr : reinterpret_cast<void*>(16);
    switch (t->scalar_type()) {
      case at::kBFloat16: d.dtype = FA_DTYPE_BF16; break;
      case at::kFloat: d.dtype = FA_DTYPE_F32; break;
      case at::kInt: d.dtype = FA_DTYPE_I32; break;
      case at::kHalf: d.dtype = FA_DTYPE_F16; break;
      case at::kDouble: d.dtype = FA_DTYPE_F64; break;
      case at::kFloat8_e4m3fn: d.dtype = FA_DTYPE_E4M3; break;
      default: d.dtype = 0;
    }
    d.ndim = (int32_t)t->dim();
    for (int i = 0; i < d.ndim; ++i) {
      d.shape[i] = t->size(i);
      d.stride[i] = t->stride(i);
    }
    return &d;
  }

  // The call's stream: argument i (a raw handle), or the current one.  What the
  // call allocates belongs to it.
  void use_stream(int i) {
    const cudaStream_t current = c10::cuda::getCurrentCUDAStream(device).stream();
    opts.stream = current;
    if (args[i] == Py_None) return;
    opts.stream = pointer(i);
    if (opts.stream != current)
      guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(opts.stream), device));
  }
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)device), std::nullopt));
  }
  // Workspace argument t, or a new one whose first 256 bytes are zero-filled.
  at::Tensor workspace(const at::Tensor* t, size_t bytes) {
    at::Tensor ws;
    if (t) {
      if (!t->is_contiguous()) throw Refused();  // (its bytes would not be those behind its pointer)
      ws = *t;
    } else {
      ws = empty({(int64_t)(bytes < 256 ? 256 : bytes)}, at::kByte);
      if (cudaMemsetAsync(ws.data_ptr(), 0, 256, static_cast<cudaStream_t>(opts.stream)) != cudaSuccess) {
        cudaGetLastError();
        throw Refused();
      }
    }
    opts.workspace = ws.data_ptr();
    opts.workspace_bytes = ws.nbytes();
    return ws;
  }
};

PyObject* wrap(const at::Tensor* t) {
  if (!t || !t->defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}

PyObject* result(const at::Tensor* a, const at::Tensor* b, const at::Tensor* c) {
  PyObject* o[3] = {wrap(a), wrap(b), wrap(c)};
  PyObject* r = (o[0] && o[1] && o[2]) ? PyTuple_Pack(3, o[0], o[1], o[2]) : nullptr;
  for (PyObject* x : o) Py_XDECREF(x);
  return r;
}

// Runs f; C++ exceptions end here.
template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F f) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, have);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused&) {
    return PyLong_FromLong(FA_ERR_INVALID_ARG);
  } catch (const Raised&) {
    return nullptr;
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// q, k, q_out, k_out, positions, inv_freq, mscale, interleaved, inverse, stream, event_begin, event_end
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    Call c(a, true);
    const at::Tensor &q = c.required(0), *k = c.tensor(1), *pos = c.tensor(4), &f = c.required(5);
    const at::Tensor *qo = c.tensor(2), *ko = c.tensor(3);
    if (!k && ko) throw Refused();
    c.use_stream(9);
    at::Tensor q_new, k_new;
    if (!qo) qo = &(q_new = c.empty(q.sizes(), q.scalar_type()));
    if (k && !ko) ko = &(k_new = c.empty(k->sizes(), k->scalar_type()));
    c.opts.event_begin = c.pointer(10);
    c.opts.event_end = c.pointer(11);
    const fa_tensor *dq = c.describe(&q), *dk = c.describe(k), *dqo = c.describe(qo), *dko = c.describe(ko);
    const int rc = fa_rope(dq, dk, dqo, dko, c.describe(pos), c.describe(&f), c.f32(6), c.truth(7), c.truth(8), &c.opts);
    return rc ? PyLong_FromLong(rc) : result(qo, ko, nullptr);
  });
}

// k_new, v_new, k_cache, v_cache, cache_seqlens, q, q_out, cu_seqlens_q, block_table, positions, inv_freq, mscale,
// interleaved, seqlens_out, workspace, stream, event_begin, event_end
PyObject* kvcache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&]() -> PyObject* {
    Call c(a, true);
    const at::Tensor &k = c.required(0), &v = c.required(1), &kc = c.required(2), &vc = c.required(3), &len = c.required(4);
    const at::Tensor *q = c.tensor(5), *qo = c.tensor(6), *cu = c.tensor(7), *bt = c.tensor(8), *pos = c.tensor(9),
                     *f = c.tensor(10), *lo = c.tensor(13), *ws = c.tensor(14);
    if (!q && qo) throw Refused();
    c.use_stream(15);
    at::Tensor q_new, l_new;
    if (q && !qo) qo = &(q_new = c.empty(q->sizes(), q->scalar_type()));
    if (!lo) lo = &(l_new = c.empty(len.sizes(), at::kInt));
    const at::Tensor w = c.workspace(ws, FA_KVCACHE_APPEND_WORKSPACE_BYTES);
    c.opts.event_begin = c.pointer(16);
    c.opts.event_end = c.pointer(17);
    const fa_tensor *dq = c.describe(q), *dqo = c.describe(qo), *dk = c.describe(&k), *dv = c.describe(&v);
    const fa_tensor *dkc = c.describe(&kc), *dvc = c.describe(&vc), *dcu = c.describe(cu), *dl = c.describe(&len);
    const fa_tensor *db = c.describe(bt), *dp = c.describe(pos), *df = c.describe(f), *dlo = c.describe(lo);
    const int rc =
        fa_kvcache_append(dq, dqo, dk, dv, dkc, dvc, dcu, dl, db, dp, df, c.f32(11), c.truth(12), dlo, &c.opts);
    return rc ? PyLong_FromLong(rc) : result(qo, lo, &w);
  });
}

// The arguments that fa_fwd_chunk and its plan share: q, k_cache, v_cache, out, lse, cu_seqlens_q, seqlens_k,
// block_table, prefix_lens, window_left, window_right, softcap, scale, causal, max_seqlen_q, max_seqlen_k, debug_flags
struct ChunkArgs {
  const fa_tensor *q, *kc, *vc, *out, *lse, *cu, *len, *bt, *pre;
  int32_t wl, wr, causal;
  float softcap, scale;

  ChunkArgs(Call& c, const at::Tensor& out_t, const at::Tensor& lse_t) {
    q = c.describe(&c.required(0));
    kc = c.describe(&c.required(1));
    vc = c.describe(&c.required(2));
    out = c.describe(&out_t);
    lse = c.describe(&lse_t);
    cu = c.describe(c.tensor(5));
    len = c.describe(&c.required(6));
    bt = c.describe(c.tensor(7));
    pre = c.describe(c.tensor(8));
    wl = c.i32(9);
    wr = c.i32(10);
    softcap = c.f32(11);
    scale = c.f32(12, true);
    causal = c.truth(13);
    c.opts.max_seqlen_q = c.i32(14, true);
    if (c.args[15] == Py_None) throw Refused();
    c.opts.max_seqlen_k = c.i32(15);
    c.opts.debug_flags = (uint32_t)c.i32(16);
  }
  int plan(const Call& c, fa_plan* pl) const {
    return fa_fwd_chunk_plan(q, kc, vc, out, lse, cu, len, bt, pre, wl, wr, softcap, scale, causal, &c.opts, pl);
  }
};

// [Hq, total_q] or [B, Hq, Sq]; empty when q has another rank (the C ABI then refuses the call)
c10::SmallVector<int64_t, 3> lse_shape(const at::Tensor& q, bool packed) {
  if (packed && q.dim() == 3) return {q.size(1), q.size(0)};
  if (!packed && q.dim() == 4) return {q.size(0), q.size(2), q.size(1)};
  throw Refused();
}

// ... stream, workspace, alibi_slopes, event_begin, event_attn_end, event_end
PyObject* fwd_chunk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 23, [&]() -> PyObject* {
    Call c(a, true);
    const at::Tensor &q = c.required(0), *out = c.tensor(3), *lse = c.tensor(4), *ws = c.tensor(18), *al = c.tensor(19);
    c.use_stream(17);
    at::Tensor o_new, l_new;
    if (!out) out = &(o_new = c.empty(q.sizes(), q.scalar_type()));
    if (!lse) lse = &(l_new = c.empty(lse_shape(q, a[5] != Py_None), at::kFloat));
    if (al) {
      if (al->scalar_type() != at::kFloat || al->dim() != 1 || q.dim() < 2 || al->size(0) != q.size(q.dim() - 2) ||
          !al->is_contiguous())
        throw Refused();
      c.opts.alibi_slopes = al->data_ptr();
    }
    c.opts.event_begin = c.pointer(20);
    c.opts.event_attn_end = c.pointer(21);
    c.opts.event_end = c.pointer(22);
    const ChunkArgs x(c, *out, *lse);
    size_t bytes = 0;
    if (!ws) {
      fa_plan pl;
      const int rc = x.plan(c, &pl);
      if (rc) return PyLong_FromLong(rc);
      bytes = pl.workspace_bytes;
    }
    const at::Tensor w = c.workspace(ws, bytes);
    const int rc = fa_fwd_chunk(x.q, x.kc, x.vc, x.out, x.lse, x.cu, x.len, x.bt, x.pre, x.wl, x.wr, x.softcap, x.scale,
                                x.causal, &c.opts);
    return rc ? PyLong_FromLong(rc) : result(out, lse, &w);
  });
}

// The shared arguments (out and lse given) and the address of an fa_plan; host-only.
PyObject* fwd_chunk_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&]() -> PyObject* {
    Call c(a, false);
    const ChunkArgs x(c, c.required(3), c.required(4));
    return PyLong_FromLong(x.plan(c, static_cast<fa_plan*>(c.pointer(17))));
  });
}

// q, k, q_weight, k_weight, q_out, k_out, positions, inv_freq, eps, mscale, interleaved, stream, event_begin, event_end
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    Call c(a, true);
    const at::Tensor &q = c.required(0), *k = c.tensor(1), *qw = c.tensor(2), *kw = c.tensor(3), *qo = c.tensor(4),
                     *ko = c.tensor(5), *pos = c.tensor(6), *f = c.tensor(7);
    if (!k && ko) throw Refused();
    c.use_stream(11);
    at::Tensor q_new, k_new;
    if (!qo) qo = &(q_new = c.empty(q.sizes(), q.scalar_type()));
    if (k && !ko) ko = &(k_new = c.empty(k->sizes(), k->scalar_type()));
    c.opts.event_begin = c.pointer(12);
    c.opts.event_end = c.pointer(13);
    const fa_tensor *dq = c.describe(&q), *dk = c.describe(k), *dqw = c.describe(qw), *dkw = c.describe(kw);
    const fa_tensor *dqo = c.describe(qo), *dko = c.describe(ko), *dp = c.describe(pos), *df = c.describe(f);
    const int rc = fa_qk_norm_rope(dq, dk, dqw, dkw, dqo, dko, dp, df, c.f32(8), c.f32(9), c.truth(10), &c.opts);
    return rc ? PyLong_FromLong(rc) : result(qo, ko, nullptr);
  });
}

// dq_out, dk_out, q, k, q_weight, k_weight, dq, dk, dq_weight, dk_weight, positions, inv_freq, eps, mscale, interleaved,
// workspace, stream, event_begin, event_end
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 19, [&]() -> PyObject* {
    Call c(a, true);
    const at::Tensor &gq = c.required(0), *gk = c.tensor(1), &q = c.required(2), *k = c.tensor(3), *qw = c.tensor(4),
                     *kw = c.tensor(5), *dq = c.tensor(6), *dk = c.tensor(7), *dqw = c.tensor(8), *dkw = c.tensor(9),
                     *pos = c.tensor(10), *f = c.tensor(11), *ws = c.tensor(15);
    if (!k && (gk || dk || dkw)) throw Refused();
    c.use_stream(16);
    at::Tensor t[4];
    const auto d = [](const at::Tensor& x) { return x.dim() ? x.size(x.dim() - 1) : 0; };
    if (!dq) dq = &(t[0] = c.empty(q.sizes(), q.scalar_type()));
    if (k && !dk) dk = &(t[1] = c.empty(k->sizes(), k->scalar_type()));
    if (qw && !dqw) dqw = &(t[2] = c.empty({d(q)}, at::kFloat));
    if (k && kw && !dkw) dkw = &(t[3] = c.empty({d(*k)}, at::kFloat));
    at::Tensor w;
    if (ws || dqw || dkw) w = c.workspace(ws, FA_QK_NORM_ROPE_BWD_WORKSPACE_BYTES);
    c.opts.event_begin = c.pointer(17);
    c.opts.event_end = c.pointer(18);
    const fa_tensor *xgq = c.describe(&gq), *xgk = c.describe(gk), *xq = c.describe(&q), *xk = c.describe(k);
    const fa_tensor *xqw = c.describe(qw), *xkw = c.describe(kw), *xdq = c.describe(dq), *xdk = c.describe(dk);
    const fa_tensor *xdqw = c.describe(dqw), *xdkw = c.describe(dkw), *xp = c.describe(pos), *xf = c.describe(f);
    const int rc = fa_qk_norm_rope_bwd(xgq, xgk, xq, xk, xqw, xkw, xdq, xdk, xdqw, xdkw, xp, xf, c.f32(12), c.f32(13),
                                       c.truth(14), &c.opts);
    if (rc) return PyLong_FromLong(rc);
    const at::Tensor* o[5] = {dq, dk, dqw, dkw, &w};
    PyObject* r = PyTuple_New(5);
    for (int i = 0; r && i < 5; ++i) {
      PyObject* x = wrap(o[i]);
      if (!x) {
        Py_DECREF(r);
        return nullptr;
      }
      PyTuple_SET_ITEM(r, i, x);
    }
    return r;
  });
}

// k_new, v_new, k_cache, v_cache, k_scale, v_scale, cache_seqlens, q, q_out, cu_seqlens_q, block_table, positions, inv_freq,
// mscale, interleaved, q_weight, k_weight, eps, seqlens_out, workspace, stream, event_begin, event_end
PyObject* kvcache_append_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 23, [&]() -> PyObject* {
    Call c(a, true);
    const at::Tensor &k = c.required(0), &v = c.required(1), &kc = c.required(2), &vc = c.required(3), &ks = c.required(4),
                     &vs = c.required(5), &len = c.required(6);
    const at::Tensor *q = c.tensor(7), *qo = c.tensor(8), *cu = c.tensor(9), *bt = c.tensor(10), *pos = c.tensor(11),
                     *f = c.tensor(12), *qw = c.tensor(15), *kw = c.tensor(16), *lo = c.tensor(18), *ws = c.tensor(19);
    if (!q && qo) throw Refused();
    c.use_stream(20);
    at::Tensor q_new, l_new;
    if (q && !qo) qo = &(q_new = c.empty(q->sizes(), q->scalar_type()));
    if (!lo) lo = &(l_new = c.empty(len.sizes(), at::kInt));
    const at::Tensor w = c.workspace(ws, FA_KVCACHE_APPEND_WORKSPACE_BYTES);
    c.opts.event_begin = c.pointer(21);
    c.opts.event_end = c.pointer(22);
    const fa_tensor *dq = c.describe(q), *dqo = c.describe(qo), *dk = c.describe(&k), *dv = c.describe(&v);
    const fa_tensor *dkc = c.describe(&kc), *dvc = c.describe(&vc), *dks = c.describe(&ks), *dvs = c.describe(&vs);
    const fa_tensor *dcu = c.describe(cu), *dl = c.describe(&len), *db = c.describe(bt), *dp = c.describe(pos);
    const fa_tensor *df = c.describe(f), *dqw = c.describe(qw), *dkw = c.describe(kw), *dlo = c.describe(lo);
    const int rc = fa_kvcache_append_q8(dq, dqo, dk, dv, dkc, dvc, dks, dvs, dcu, dl, db, dp, df, c.f32(13), c.truth(14), dqw,
                                        dkw, c.f32(17, true), dlo, &c.opts);
    return rc ? PyLong_FromLong(rc) : result(qo, lo, &w);
  });
}

// k_cache, v_cache, k_scale, v_scale, cu_seqlens_k, seqlens_k, block_table, k_out, v_out, rows (of an output that is
// allocated: in all, or per sequence), f16, workspace, stream, event_begin, event_end
PyObject* kvcache_read_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    Call c(a, true);
    const at::Tensor &kc = c.required(0), &vc = c.required(1), &ks = c.required(2), &vs = c.required(3);
    const at::Tensor *cu = c.tensor(4), *len = c.tensor(5), *bt = c.tensor(6), *ko = c.tensor(7), *vo = c.tensor(8),
                     *ws = c.tensor(11);
    c.use_stream(12);
    at::Tensor t[2];
    if (!ko || !vo) {
      if (a[9] == Py_None || kc.dim() != 4 || (!cu && (!len || len->dim() != 1))) throw Refused();
      const int64_t rows = c.i32(9);
      if (rows < 0) throw Refused();
      c10::SmallVector<int64_t, 4> shape;
      if (!cu) shape.push_back(len->size(0));
      shape.push_back(rows);
      shape.push_back(kc.size(2));
      shape.push_back(kc.size(3));
      const at::ScalarType type = c.truth(10) ? at::kHalf : at::kBFloat16;
      if (!ko) ko = &(t[0] = c.empty(shape, vo ? vo->scalar_type() : type));
      if (!vo) vo = &(t[1] = c.empty(shape, ko->scalar_type()));
    }
    const at::Tensor w = c.workspace(ws, FA_KVCACHE_APPEND_WORKSPACE_BYTES);
    c.opts.event_begin = c.pointer(13);
    c.opts.event_end = c.pointer(14);
    const fa_tensor *dkc = c.describe(&kc), *dvc = c.describe(&vc), *dks = c.describe(&ks), *dvs = c.describe(&vs);
    const fa_tensor *dcu = c.describe(cu), *dl = c.describe(len), *db = c.describe(bt), *dko = c.describe(ko), *dvo = c.describe(vo);
    const int rc = fa_kvcache_read_q8(dkc, dvc, dks, dvs, dcu, dl, db, dko, dvo, &c.opts);
    return rc ? PyLong_FromLong(rc) : result(ko, vo, &w);
  });
}

// The arguments that fa_fwd_chunk_q8 and its plan share: q, k_cache, v_cache, k_scale, v_scale, out, lse, cu_seqlens_q,
// seqlens_k, block_table, prefix_lens, sink_keys, window_left, window_right, softcap, scale, causal, max_seqlen_q,
// max_seqlen_k, debug_flags
struct ChunkQ8Args {
  const fa_tensor* t[11];
  int32_t sinks, wl, wr, causal;
  float softcap, scale;

  ChunkQ8Args(Call& c, const at::Tensor& out_t, const at::Tensor& lse_t) {
    for (int i = 0; i < 11; ++i)
      t[i] = i == 5 ? c.describe(&out_t) : i == 6 ? c.describe(&lse_t) : i < 5 || i == 8 ? c.describe(&c.required(i)) : c.describe(c.tensor(i));
    sinks = c.i32(11);
    wl = c.i32(12);
    wr = c.i32(13);
    softcap = c.f32(14);
    scale = c.f32(15, true);
    causal = c.truth(16);
    c.opts.max_seqlen_q = c.i32(17, true);
    if (c.args[18] == Py_None) throw Refused();
    c.opts.max_seqlen_k = c.i32(18);
    c.opts.debug_flags = (uint32_t)c.i32(19);
  }
  int plan(const Call& c, fa_plan* pl) const {
    return fa_fwd_chunk_q8_plan(t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7], t[8], t[9], t[10], sinks, wl, wr, softcap, scale,
                                causal, &c.opts, pl);
  }
};

// ... stream, workspace, alibi_slopes, event_begin, event_attn_end, event_end
PyObject* fwd_chunk_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 26, [&]() -> PyObject* {
    Call c(a, true);
    const at::Tensor &q = c.required(0), *out = c.tensor(5), *lse = c.tensor(6), *ws = c.tensor(21), *al = c.tensor(22);
    c.use_stream(20);
    at::Tensor o_new, l_new;
    if (!out) out = &(o_new = c.empty(q.sizes(), q.scalar_type()));
    if (!lse) lse = &(l_new = c.empty(lse_shape(q, a[7] != Py_None), at::kFloat));
    if (al) {
      if (al->scalar_type() != at::kFloat || al->dim() != 1 || q.dim() < 2 || al->size(0) != q.size(q.dim() - 2) ||
          !al->is_contiguous())
        throw Refused();
      c.opts.alibi_slopes = al->data_ptr();
    }
    c.opts.event_begin = c.pointer(23);
    c.opts.event_attn_end = c.pointer(24);
    c.opts.event_end = c.pointer(25);
    const ChunkQ8Args x(c, *out, *lse);
    size_t bytes = 0;
    if (!ws) {
      fa_plan pl;
      const int rc = x.plan(c, &pl);
      if (rc) return PyLong_FromLong(rc);
      bytes = pl.workspace_bytes;
    }
    const at::Tensor w = c.workspace(ws, bytes);
    const int rc = fa_fwd_chunk_q8(x.t[0], x.t[1], x.t[2], x.t[3], x.t[4], x.t[5], x.t[6], x.t[7], x.t[8], x.t[9], x.t[10],
                                   x.sinks, x.wl, x.wr, x.softcap, x.scale, x.causal, &c.opts);
    return rc ? PyLong_FromLong(rc) : result(out, lse, &w);
  });
}

// The shared arguments (out and lse given) and the address of an fa_plan; host-only.
PyObject* fwd_chunk_q8_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 21, [&]() -> PyObject* {
    Call c(a, false);
    const ChunkQ8Args x(c, c.required(5), c.required(6));
    return PyLong_FromLong(x.plan(c, static_cast<fa_plan*>(c.pointer(20))));
  });
}

#define FAST(name) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"rope", FAST(rope)},
                         {"kvcache_append", FAST(kvcache_append)},
                         {"fwd_chunk", FAST(fwd_chunk)},
                         {"fwd_chunk_plan", FAST(fwd_chunk_plan)},
                         {"qk_norm_rope", FAST(qk_norm_rope)},
                         {"qk_norm_rope_bwd", FAST(qk_norm_rope_bwd)},
                         {"kvcache_append_q8", FAST(kvcache_append_q8)},
                         {"kvcache_read_q8", FAST(kvcache_read_q8)},
                         {"fwd_chunk_q8", FAST(fwd_chunk_q8)},
                         {"fwd_chunk_q8_plan", FAST(fwd_chunk_q8_plan)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* m = PyModule_Create(&module);
  // what the module was compiled against: the package checks both before it uses it
  if (m && (PyModule_AddIntConstant(m, "ABI_VERSION", FA_ABI_VERSION) < 0 ||
            PyModule_AddStringConstant(m, "TORCH_VERSION", MFA_TORCH_VERSION) < 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
