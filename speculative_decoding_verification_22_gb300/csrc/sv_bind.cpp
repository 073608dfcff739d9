// sv_bind.cpp -- argument marshalling of the target-layer operators for
// Python: checks of torch tensors, allocation of missing outputs, and the call
// of the C entry points of include/spec_target.h and include/spec_layer.h.
//
// A call on a few tokens takes the GPU 2 to 10 us, and reading the tensors'
// attributes from Python alone took the host 5 to 8; here it takes well under
// one.  Bad arguments raise ValueError, an entry point's error the exception
// class given to set_error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <stdexcept>
#include <string>

#include "spec_layer.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr;      // SpecVerifyError(code, what)
PyObject *g_raw = nullptr;        // "_raw": the handle's address, or None
PyObject *g_index = nullptr;      // "_index": the number of the handle's device
PyObject *g_stream = nullptr;     // "cuda_stream"

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python error is set

void need(bool ok, const char *what) {
  if (!ok) throw Bad(what);
}

const Tensor &tensor(PyObject *o, const char *what) {
  if (!THPVariable_Check(o)) throw Bad(std::string(what) + ": a tensor is expected");
  return THPVariable_Unpack(o);
}
bool given(PyObject *o) { return o != Py_None; }

int code_of(at::ScalarType t, const char *what) {
  switch (t) {
    case at::kBFloat16: return SV_BF16;
    case at::kHalf: return SV_FP16;
    case at::kFloat: return SV_FP32;
    default:
      throw Bad(std::string(what) + ": bfloat16, float16 or float32 expected");
  }
}

// E4M3 values, or their bytes.
bool e4m3(const Tensor &t) {
  return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte;
}

long long integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
// A size in 32 bits; beyond them the nearest, so that none turns into another's
// value (a window of 2^32 + 5 keys is one of all keys, -2^32 is still negative).
int32_t size32(PyObject *o) {
  return static_cast<int32_t>(
      std::clamp<long long>(integer(o), INT32_MIN, INT32_MAX));
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

spec_target_t *handle(PyObject *self) {
  PyObject *o = PyObject_GetAttr(self, g_raw);
  if (!o) throw Raised();
  spec_target_t *h = nullptr;
  if (o != Py_None) h = static_cast<spec_target_t *>(PyLong_AsVoidPtr(o));
  Py_DECREF(o);
  return h;
}

// The device of the handle, the only one whose memory its kernels may be given.
class Device {
 public:
  explicit Device(PyObject *self) : self_(self) {}
  bool has(const Tensor &t) {
    if (!t.is_cuda()) return false;
    if (index_ < 0) {
      PyObject *o = PyObject_GetAttr(self_, g_index);
      if (!o) throw Raised();
      index_ = integer(o);
      Py_DECREF(o);
    }
    return t.get_device() == index_;
  }
  template <class... More>
  bool has(const Tensor &t, const More &...more) {
    return has(t) && has(more...);
  }

 private:
  PyObject *self_;
  long long index_ = -1;
};

// The stream of a call: the one given (an object with cuda_stream, or its
// number), else the current one of the tensor's device.  While it lives the
// given stream is the current one, so that new outputs come from its memory.
class Stream {
 public:
  Stream(PyObject *o, const Tensor &x) {
    const c10::DeviceIndex dev = x.get_device();
    if (!given(o)) {
      stream_ = c10::cuda::getCurrentCUDAStream(dev).stream();
      return;
    }
    void *p;
    if (PyLong_Check(o)) {
      p = PyLong_AsVoidPtr(o);
    } else {
      PyObject *n = PyObject_GetAttr(o, g_stream);
      if (!n) throw Raised();
      p = PyLong_AsVoidPtr(n);
      Py_DECREF(n);
    }
    if (PyErr_Occurred()) throw Raised();
    stream_ = static_cast<cudaStream_t>(p);
    guard_.reset_stream(p ? c10::cuda::getStreamFromExternal(stream_, dev)
                          : c10::cuda::getDefaultCUDAStream(dev));
  }
  void *get() const { return stream_; }

 private:
  cudaStream_t stream_ = nullptr;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};

Tensor empty(at::IntArrayRef sizes, at::ScalarType t, const Tensor &like) {
  return at::detail::empty_cuda(sizes, t, like.device(), std::nullopt);
}

void check(int code, const char *what) {
  if (code == SV_OK) return;
  PyObject *e = g_error ? PyObject_CallFunction(g_error, "is", code, what) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// Row stride of a 2-D tensor whose rows are dense.
int64_t row_stride(const Tensor &t, const char *what) {
  need(t.dim() == 2, what);
  if (t.stride(1) != 1 && t.size(1) != 1)
    throw Bad(std::string(what) + ": rows must be dense");
  return t.stride(0);
}

// The caller's output if there is one (a new reference), else `made`.
PyObject *result(PyObject *o, const Tensor &made) {
  if (given(o)) {
    Py_INCREF(o);
    return o;
  }
  return THPVariable_Wrap(made);
}

template <class F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F &&f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised &) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "call failed");
  } catch (const Bad &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// norm(self, x, weight, eps, residual, group, out, scale, residual_out, stream);
// group: None for the rows' type, 0 or 128 for E4M3.
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    const Tensor &x = tensor(a[1], "rms_norm: x"), &w = tensor(a[2], "rms_norm: weight");
    const at::ScalarType dt = x.scalar_type();
    const int code = code_of(dt, "rms_norm");
    need(x.dim() == 2 && w.dim() == 1 && w.size(0) == x.size(1),
         "rms_norm: x [rows, d] and weight [d]");
    need(w.scalar_type() == dt && w.is_contiguous(),
         "rms_norm: weight must be dense and of x's type");
    Device device(a[0]);
    need(device.has(x, w), "rms_norm: tensors must be on the GPU of the handle");
    const Stream stream(a[9], x);
    const int64_t rows = x.size(0), d = x.size(1), xs = row_stride(x, "x");
    auto like_x = [&](const Tensor &t) {
      return t.dim() == 2 && t.size(0) == rows && t.size(1) == d && t.scalar_type() == dt &&
             device.has(t);
    };
    const void *res = nullptr;
    int64_t rs = 0, ros = 0;
    Tensor made_res;
    void *ro = nullptr;
    if (given(a[4])) {
      const Tensor &r = tensor(a[4], "rms_norm: residual");
      need(like_x(r), "rms_norm: residual must have x's shape, type and device");
      res = r.data_ptr();
      rs = row_stride(r, "residual");
    }
    const bool second = given(a[4]) || given(a[8]);
    if (given(a[8])) {
      const Tensor &r = tensor(a[8], "rms_norm: residual_out");
      need(like_x(r), "rms_norm: residual_out must have x's shape, type and device");
      ro = r.data_ptr();
      ros = row_stride(r, "residual_out");
    } else if (res) {
      made_res = empty({rows, d}, dt, x);
      ro = made_res.data_ptr();
      ros = d;
    }
    const bool quant = given(a[5]);
    const int group = quant ? size32(a[5]) : 0;
    const float eps = static_cast<float>(number(a[3]));
    Tensor made, made_scale;
    void *out;
    int64_t os = d;
    if (given(a[6])) {
      const Tensor &o = tensor(a[6], "rms_norm: out");
      if (quant)
        need(o.dim() == 2 && o.size(0) == rows && o.size(1) == d && e4m3(o) &&
                 o.is_contiguous() && device.has(o),
             "rms_norm_fp8: out must be dense float8_e4m3fn (or uint8) of x's shape");
      else
        need(like_x(o), "rms_norm: out must have x's shape, type and device");
      out = o.data_ptr();
      os = row_stride(o, "out");
    } else {
      made = empty({rows, d}, quant ? at::kFloat8_e4m3fn : dt, x);
      out = made.data_ptr();
    }
    if (!quant) {
      check(spec_target_rms_norm(handle(a[0]), x.data_ptr(), xs, res, rs, w.data_ptr(), eps, rows,
                                 d, code, out, os, ro, ros, stream.get()),
            "spec_target_rms_norm");
      PyObject *list = PyList_New(second ? 2 : 1);
      PyList_SET_ITEM(list, 0, result(a[6], made));
      if (second) PyList_SET_ITEM(list, 1, result(a[8], made_res));
      return list;
    }
    const int64_t groups = (d + SV_SCALE_BLOCK - 1) / SV_SCALE_BLOCK;
    float *scale;
    if (given(a[7])) {
      const Tensor &s = tensor(a[7], "rms_norm_fp8: scale");
      need(s.scalar_type() == at::kFloat && s.is_contiguous() && device.has(s) &&
               s.dim() == (group ? 2 : 1) && s.size(0) == rows && (!group || s.size(1) == groups),
           "rms_norm_fp8: scale must be float32 [rows, ceil(d/128)] or [rows]");
      scale = s.data_ptr<float>();
    } else {
      made_scale = group ? empty({rows, groups}, at::kFloat, x) : empty({rows}, at::kFloat, x);
      scale = made_scale.data_ptr<float>();
    }
    check(spec_target_rms_norm_fp8(handle(a[0]), x.data_ptr(), xs, res, rs, w.data_ptr(), eps,
                                   rows, d, code, group, out, scale, ro, ros, stream.get()),
          "spec_target_rms_norm_fp8");
    PyObject *list = PyList_New(second ? 3 : 2);
    PyList_SET_ITEM(list, 0, result(a[6], made));
    PyList_SET_ITEM(list, 1, result(a[7], made_scale));
    if (second) PyList_SET_ITEM(list, 2, result(a[8], made_res));
    return list;
  });
}

// matmul(self, a8, a_scale, w8, w_scale, out_dtype code, out, stream)
PyObject *matmul(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    const Tensor &x = tensor(a[1], "matmul_fp8: a8"), &sx = tensor(a[2], "matmul_fp8: a_scale");
    const Tensor &w = tensor(a[3], "matmul_fp8: w8"), &sw = tensor(a[4], "matmul_fp8: w_scale");
    need(x.dim() == 2 && w.dim() == 2 && x.size(1) == w.size(1),
         "matmul_fp8: a8 [M, K] and w8 [N, K]");
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0);
    const int64_t kb = (K + SV_SCALE_BLOCK - 1) / SV_SCALE_BLOCK;
    need(e4m3(x) && e4m3(w), "matmul_fp8: a8 and w8 must be float8_e4m3fn (or its bytes, uint8)");
    need(sx.scalar_type() == at::kFloat && sw.scalar_type() == at::kFloat && sx.dim() == 2 &&
             sw.dim() == 2 && sx.size(0) == M && sx.size(1) == kb &&
             sw.size(0) == (N + SV_SCALE_BLOCK - 1) / SV_SCALE_BLOCK && sw.size(1) == kb,
         "matmul_fp8: float32 scales [M, ceil(K/128)] and [ceil(N/128), ceil(K/128)]");
    need(x.is_contiguous() && w.is_contiguous() && sx.is_contiguous() && sw.is_contiguous(),
         "tensors must be contiguous");
    Device device(a[0]);
    need(device.has(x, w, sx, sw), "matmul_fp8: tensors must be on the GPU of the handle");
    const Stream stream(a[7], x);
    Tensor made;
    void *out;
    int64_t os = N;
    int code;
    if (given(a[6])) {
      const Tensor &o = tensor(a[6], "matmul_fp8: out");
      need(o.dim() == 2 && o.size(0) == M && o.size(1) == N && device.has(o),
           "matmul_fp8: out must be [M, N] on the GPU of the handle");
      code = code_of(o.scalar_type(), "matmul_fp8: out");
      os = row_stride(o, "out");
      out = o.data_ptr();
    } else {
      code = static_cast<int>(integer(a[5]));
      made = empty({M, N}, code == SV_BF16 ? at::kBFloat16 : code == SV_FP16 ? at::kHalf
                                                                             : at::kFloat, x);
      out = made.data_ptr();
    }
    check(spec_target_matmul_fp8(handle(a[0]), x.data_ptr(), sx.data_ptr<float>(), w.data_ptr(),
                                 sw.data_ptr<float>(), M, N, K, code, out, os,
                                 stream.get()),
          "spec_target_matmul_fp8");
    return result(a[6], made);
  });
}

// rope(self, q, k, v, positions, slots, freqs, k_cache, v_cache, interleaved,
//      magnitude, q_out, stream)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    const Tensor &q = tensor(a[1], "rope_append: q"), &k = tensor(a[2], "rope_append: k");
    const Tensor &v = tensor(a[3], "rope_append: v");
    const Tensor &pos = tensor(a[4], "rope_append: positions");
    const Tensor &slots = tensor(a[5], "rope_append: slots");
    const Tensor &f = tensor(a[6], "rope_append: freqs");
    const Tensor &kc = tensor(a[7], "rope_append: k_cache");
    const Tensor &vc = tensor(a[8], "rope_append: v_cache");
    need(q.dim() == 3 && k.dim() == 3 && k.size(0) == q.size(0) && k.size(2) == q.size(2) &&
             v.sizes() == k.sizes(),
         "rope_append: q [T, Hq, D], k and v [T, Hkv, D]");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
    need(kc.dim() == 4 && kc.size(2) == Hkv && kc.size(3) == D && vc.sizes() == kc.sizes(),
         "rope_append: caches must be [pages, page_size, Hkv, D]");
    const at::ScalarType dt = q.scalar_type();
    const int code = code_of(dt, "rope_append");
    need(k.scalar_type() == dt && v.scalar_type() == dt && kc.scalar_type() == dt &&
             vc.scalar_type() == dt,
         "rope_append: q, k, v and the caches must have one type");
    need(pos.scalar_type() == at::kLong && slots.scalar_type() == at::kLong &&
             pos.numel() == T && slots.numel() == T && pos.is_contiguous() &&
             slots.is_contiguous(),
         "rope_append: positions and slots are int64 [T]");
    need(f.scalar_type() == at::kDouble && f.is_contiguous(),
         "rope_append: freqs is float64 [rot_dim/2]");
    Device device(a[0]);
    need(device.has(q, k, v, pos, slots, f, kc, vc),
         "rope_append: tensors must be on the GPU of the handle");
    const Stream stream(a[12], q);
    Tensor made;
    if (given(a[11])) {
      const Tensor &o = tensor(a[11], "rope_append: q_out");
      need(o.sizes() == q.sizes() && o.scalar_type() == dt && device.has(o),
           "rope_append: q_out must have q's shape, type and device");
    } else {
      made = empty({T, Hq, D}, dt, q);
    }
    const Tensor &qo = given(a[11]) ? THPVariable_Unpack(a[11]) : made;
    need(D == 1 || (q.stride(2) == 1 && k.stride(2) == 1 && v.stride(2) == 1 &&
                    qo.stride(2) == 1 && kc.stride(3) == 1 && vc.stride(3) == 1),
         "rope_append: heads must be dense");
    need(T <= INT32_MAX && kc.size(1) <= INT32_MAX, "rope_append: too many tokens");
    sv_rope_append_t r{};
    r.q = q.data_ptr();
    r.k = k.data_ptr();
    r.v = v.data_ptr();
    r.q_token = q.stride(0);
    r.q_head = q.stride(1);
    r.k_token = k.stride(0);
    r.k_head = k.stride(1);
    r.v_token = v.stride(0);
    r.v_head = v.stride(1);
    r.positions = pos.data_ptr<int64_t>();
    r.slots = slots.data_ptr<int64_t>();
    r.freqs = f.data_ptr<double>();
    r.q_out = qo.data_ptr();
    r.qo_token = qo.stride(0);
    r.qo_head = qo.stride(1);
    r.k_cache = kc.data_ptr();
    r.v_cache = vc.data_ptr();
    r.kc_page = kc.stride(0);
    r.kc_token = kc.stride(1);
    r.kc_head = kc.stride(2);
    r.vc_page = vc.stride(0);
    r.vc_token = vc.stride(1);
    r.vc_head = vc.stride(2);
    r.num_pages = kc.size(0);
    r.page_size = static_cast<int32_t>(kc.size(1));
    r.T = static_cast<int32_t>(T);
    r.Hq = static_cast<int32_t>(Hq);
    r.Hkv = static_cast<int32_t>(Hkv);
    r.D = static_cast<int32_t>(D);
    r.rot_dim = static_cast<int32_t>(2 * f.numel());
    r.interleaved = PyObject_IsTrue(a[9]) == 1;
    r.dtype = code;
    r.magnitude = static_cast<float>(number(a[10]));
    check(spec_target_rope_append(handle(a[0]), &r, stream.get()),
          "spec_target_rope_append");
    return result(a[11], made);
  });
}

// attention(self, q, k_cache, v_cache, page_table, q_start, kv_len, scale,
//           window, tree_mask, out, lse, stream)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    const Tensor &q = tensor(a[1], "attention: q"), &kc = tensor(a[2], "attention: k_cache");
    const Tensor &vc = tensor(a[3], "attention: v_cache");
    const Tensor &table = tensor(a[4], "attention: page_table");
    const Tensor &qs = tensor(a[5], "attention: q_start"), &kl = tensor(a[6], "attention: kv_len");
    need(q.dim() == 3, "attention: q must be [T, Hq, D]");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    need(kc.dim() == 4 && kc.size(3) == D && vc.sizes() == kc.sizes(),
         "attention: caches must be [pages, page_size, Hkv, D]");
    const at::ScalarType dt = q.scalar_type();
    const int code = code_of(dt, "attention");
    need(kc.scalar_type() == dt && vc.scalar_type() == dt,
         "attention: q and the caches must have one type");
    need(table.dim() == 2 && table.scalar_type() == at::kInt && qs.scalar_type() == at::kInt &&
             kl.scalar_type() == at::kInt && qs.numel() == table.size(0) + 1 &&
             kl.numel() == table.size(0) && qs.is_contiguous() && kl.is_contiguous(),
         "attention: int32 page_table [B, max_pages], q_start [B+1], kv_len [B]");
    Device device(a[0]);
    need(device.has(q, kc, vc, table, qs, kl),
         "attention: tensors must be on the GPU of the handle");
    need(T <= INT32_MAX && table.size(0) <= INT32_MAX && table.size(1) <= INT32_MAX &&
             kc.size(1) <= INT32_MAX,
         "attention: sizes");
    const Stream stream(a[12], q);
    sv_attention_t r{};
    if (given(a[9])) {
      const Tensor &m = tensor(a[9], "attention: tree_mask");
      // (a mask without words has no address, and would be taken for none)
      need(m.dim() == 2 && m.size(0) == T && m.size(1) >= 1 && m.scalar_type() == at::kInt &&
               m.is_contiguous() && device.has(m),
           "attention: tree_mask must be int32 [T, words], with a word at least");
      r.tree_mask = m.data_ptr<int32_t>();
      r.tree_words = static_cast<int32_t>(m.size(1));
    }
    if (given(a[11])) {
      const Tensor &l = tensor(a[11], "attention: lse");
      need(l.dim() == 2 && l.size(0) == T && l.size(1) == Hq && l.scalar_type() == at::kFloat &&
               l.is_contiguous() && device.has(l),
           "attention: lse must be float32 [T, Hq]");
      r.lse = l.data_ptr<float>();
    }
    Tensor made;
    if (given(a[10])) {
      const Tensor &o = tensor(a[10], "attention: out");
      need(o.sizes() == q.sizes() && o.scalar_type() == dt && device.has(o),
           "attention: out must have q's shape, type and device");
    } else {
      made = empty({T, Hq, D}, dt, q);
    }
    const Tensor &out = given(a[10]) ? THPVariable_Unpack(a[10]) : made;
    need(D == 1 || (q.stride(2) == 1 && out.stride(2) == 1 && kc.stride(3) == 1 &&
                    vc.stride(3) == 1),
         "attention: heads must be dense");
    r.q = q.data_ptr();
    r.k_cache = kc.data_ptr();
    r.v_cache = vc.data_ptr();
    r.page_table = table.data_ptr<int32_t>();
    r.q_start = qs.data_ptr<int32_t>();
    r.kv_len = kl.data_ptr<int32_t>();
    r.out = out.data_ptr();
    r.q_token = q.stride(0);
    r.q_head = q.stride(1);
    r.o_token = out.stride(0);
    r.o_head = out.stride(1);
    r.kc_page = kc.stride(0);
    r.kc_token = kc.stride(1);
    r.kc_head = kc.stride(2);
    r.vc_page = vc.stride(0);
    r.vc_token = vc.stride(1);
    r.vc_head = vc.stride(2);
    r.table_stride = row_stride(table, "page_table");
    r.num_pages = kc.size(0);
    r.T = static_cast<int32_t>(T);
    r.B = static_cast<int32_t>(table.size(0));
    r.Hq = static_cast<int32_t>(Hq);
    r.Hkv = static_cast<int32_t>(kc.size(2));
    r.D = static_cast<int32_t>(D);
    r.page_size = static_cast<int32_t>(kc.size(1));
    r.max_pages = static_cast<int32_t>(table.size(1));
    r.window = size32(a[8]);
    r.dtype = code;
    r.scale = static_cast<float>(given(a[7]) ? number(a[7])
                                             : 1.0 / std::sqrt(static_cast<double>(D)));
    check(spec_target_attention(handle(a[0]), &r, stream.get()), "spec_target_attention");
    return result(a[10], made);
  });
}

// The weight, bias and output of the products.
void check_weight(const Tensor &w, const Tensor &x, int64_t N, const char *what) {
  need(w.dim() == 2 && w.size(0) == N && w.size(1) == x.size(1) &&
           w.scalar_type() == x.scalar_type(),
       what);
}
const void *bias_of(PyObject *o, const Tensor &x, int64_t N, Device &device, const char *what) {
  if (!given(o)) return nullptr;
  const Tensor &b = tensor(o, what);
  need(b.dim() == 1 && b.size(0) == N && b.scalar_type() == x.scalar_type() &&
           (b.is_contiguous()) && device.has(b),
       what);
  return b.data_ptr();
}
// The type named by its code, or x's where the code is -1.
at::ScalarType out_type(long long code, const Tensor &x) {
  return code == SV_BF16   ? at::kBFloat16
         : code == SV_FP16 ? at::kHalf
         : code == SV_FP32 ? at::kFloat
                           : x.scalar_type();
}

// linear(self, x, w, bias, activation code, residual, out type code or -1, out,
//        stream)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    const Tensor &x = tensor(a[1], "linear: x"), &w = tensor(a[2], "linear: weight");
    need(x.dim() == 2 && w.dim() == 2, "linear: x [M, K] and weight [N, K]");
    sv_linear_t r{};
    r.M = x.size(0);
    r.K = x.size(1);
    r.N = w.size(0);
    r.dtype = code_of(x.scalar_type(), "linear: x");
    check_weight(w, x, r.N, "linear: weight must be [N, K] of x's type");
    Device device(a[0]);
    need(device.has(x, w), "linear: tensors must be on the GPU of the handle");
    r.bias = bias_of(a[3], x, r.N, device, "linear: bias must be dense [N] of x's type");
    const Stream stream(a[8], x);
    Tensor made;
    if (given(a[7])) {
      const Tensor &o = tensor(a[7], "linear: out");
      need(o.dim() == 2 && o.size(0) == r.M && o.size(1) == r.N && device.has(o),
           "linear: out must be [M, N] on the GPU of the handle");
    } else {
      made = empty({r.M, r.N}, out_type(integer(a[6]), x), x);
    }
    const Tensor &out = given(a[7]) ? THPVariable_Unpack(a[7]) : made;
    r.out_dtype = code_of(out.scalar_type(), "linear: out");
    if (given(a[5])) {
      const Tensor &res = tensor(a[5], "linear: residual");
      need(res.dim() == 2 && res.size(0) == r.M && res.size(1) == r.N &&
               res.scalar_type() == out.scalar_type() && device.has(res),
           "linear: residual must be [M, N] of the output's type");
      r.residual = res.data_ptr();
      r.residual_stride = row_stride(res, "linear: residual");
    }
    r.x = x.data_ptr();
    r.w = w.data_ptr();
    r.out = out.data_ptr();
    r.x_stride = row_stride(x, "linear: x");
    r.w_stride = row_stride(w, "linear: weight");
    r.out_stride = row_stride(out, "linear: out");
    r.activation = size32(a[4]);
    check(spec_layer_linear(handle(a[0]), &r, stream.get()), "spec_layer_linear");
    return result(a[7], made);
  });
}

// gated(self, x, w_gate, w_up, bias_gate, bias_up, activation code, out type
//       code or -1, out, stream)
PyObject *gated(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    const Tensor &x = tensor(a[1], "gated_linear: x"), &g = tensor(a[2], "gated_linear: w_gate");
    const Tensor &u = tensor(a[3], "gated_linear: w_up");
    need(x.dim() == 2 && g.dim() == 2, "gated_linear: x [M, K], w_gate and w_up [N, K]");
    sv_gated_linear_t r{};
    r.M = x.size(0);
    r.K = x.size(1);
    r.N = g.size(0);
    r.dtype = code_of(x.scalar_type(), "gated_linear: x");
    check_weight(g, x, r.N, "gated_linear: w_gate must be [N, K] of x's type");
    check_weight(u, x, r.N, "gated_linear: w_up must be [N, K] of x's type");
    Device device(a[0]);
    need(device.has(x, g, u), "gated_linear: tensors must be on the GPU of the handle");
    r.bias_gate = bias_of(a[4], x, r.N, device, "gated_linear: bias_gate must be dense [N]");
    r.bias_up = bias_of(a[5], x, r.N, device, "gated_linear: bias_up must be dense [N]");
    const Stream stream(a[9], x);
    Tensor made;
    if (given(a[8])) {
      const Tensor &o = tensor(a[8], "gated_linear: out");
      need(o.dim() == 2 && o.size(0) == r.M && o.size(1) == r.N && device.has(o),
           "gated_linear: out must be [M, N] on the GPU of the handle");
    } else {
      made = empty({r.M, r.N}, out_type(integer(a[7]), x), x);
    }
    const Tensor &out = given(a[8]) ? THPVariable_Unpack(a[8]) : made;
    r.out_dtype = code_of(out.scalar_type(), "gated_linear: out");
    r.x = x.data_ptr();
    r.w_gate = g.data_ptr();
    r.w_up = u.data_ptr();
    r.out = out.data_ptr();
    r.x_stride = row_stride(x, "gated_linear: x");
    r.gate_stride = row_stride(g, "gated_linear: w_gate");
    r.up_stride = row_stride(u, "gated_linear: w_up");
    r.out_stride = row_stride(out, "gated_linear: out");
    r.activation = size32(a[6]);
    check(spec_layer_gated_linear(handle(a[0]), &r, stream.get()), "spec_layer_gated_linear");
    return result(a[8], made);
  });
}

// block_norm(self, x, residual, weight, post_weight, gate, branch_scale, eps,
//            group, out, scale, residual_out, stream); group: None for the
// rows' type, 0 or 128 for E4M3.
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    const Tensor &x = tensor(a[1], "block_norm: x"), &res = tensor(a[2], "block_norm: residual");
    const Tensor &w = tensor(a[3], "block_norm: weight");
    const at::ScalarType dt = x.scalar_type();
    sv_block_norm_t r{};
    r.dtype = code_of(dt, "block_norm");
    need(x.dim() == 2, "block_norm: x must be [rows, d]");
    Device device(a[0]);
    need(device.has(x), "block_norm: tensors must be on the GPU of the handle");
    r.rows = x.size(0);
    r.d = x.size(1);
    auto like_x = [&](const Tensor &t) {
      return t.dim() == 2 && t.size(0) == r.rows && t.size(1) == r.d && t.scalar_type() == dt &&
             device.has(t);
    };
    auto column = [&](const Tensor &t) {
      return t.dim() == 1 && t.size(0) == r.d && t.scalar_type() == dt && t.is_contiguous() &&
             device.has(t);
    };
    need(like_x(res), "block_norm: residual must have x's shape, type and device");
    need(column(w), "block_norm: weight must be dense [d] of x's type and device");
    if (given(a[4])) {
      const Tensor &p = tensor(a[4], "block_norm: post_weight");
      need(column(p), "block_norm: post_weight must be dense [d] of x's type and device");
      r.post_weight = p.data_ptr();
    }
    if (given(a[5])) {
      const Tensor &g = tensor(a[5], "block_norm: gate");
      const int64_t dim = g.dim();
      need((dim == 1 || dim == 2) && g.scalar_type() == dt && device.has(g),
           "block_norm: gate must be [d], [1, d], [rows, 1] or [rows, d] of x's type and device");
      const int64_t rows = dim == 2 ? g.size(0) : 1, cols = g.size(dim - 1);
      need((rows == 1 || rows == r.rows) && (cols == 1 || cols == r.d),
           "block_norm: gate must be [d], [1, d], [rows, 1] or [rows, d]");
      r.gate = g.data_ptr();
      r.gate_row = rows == 1 ? 0 : g.stride(0);
      r.gate_col = cols == 1 ? 0 : g.stride(dim - 1);
      need(r.gate_col <= 1, "block_norm: the gate's rows must be dense");
    }
    const Stream stream(a[12], x);
    const bool quant = given(a[8]);
    r.group = quant ? size32(a[8]) : -1;
    need(!quant || r.group == 0 || r.group == SV_SCALE_BLOCK, "block_norm: group must be 0 or 128");
    r.branch_scale = static_cast<float>(number(a[6]));
    r.eps = static_cast<float>(number(a[7]));
    Tensor made, made_scale, made_res;
    if (given(a[9])) {
      const Tensor &o = tensor(a[9], "block_norm: out");
      if (quant)
        need(o.dim() == 2 && o.size(0) == r.rows && o.size(1) == r.d && e4m3(o) &&
                 o.is_contiguous() && device.has(o),
             "block_norm_fp8: out must be dense float8_e4m3fn (or uint8) of x's shape");
      else
        need(like_x(o), "block_norm: out must have x's shape, type and device");
    } else {
      made = empty({r.rows, r.d}, quant ? at::kFloat8_e4m3fn : dt, x);
    }
    const Tensor &out = given(a[9]) ? THPVariable_Unpack(a[9]) : made;
    if (quant) {
      const int64_t groups = (r.d + SV_SCALE_BLOCK - 1) / SV_SCALE_BLOCK;
      if (given(a[10])) {
        const Tensor &s = tensor(a[10], "block_norm_fp8: scale");
        need(s.scalar_type() == at::kFloat && s.is_contiguous() && device.has(s) &&
                 s.dim() == (r.group ? 2 : 1) && s.size(0) == r.rows &&
                 (!r.group || s.size(1) == groups),
             "block_norm_fp8: scale must be float32 [rows, ceil(d/128)] or [rows]");
        r.scale = s.data_ptr<float>();
      } else {
        made_scale = r.group ? empty({r.rows, groups}, at::kFloat, x)
                             : empty({r.rows}, at::kFloat, x);
        r.scale = made_scale.data_ptr<float>();
      }
    }
    if (given(a[11])) {
      need(like_x(tensor(a[11], "block_norm: residual_out")),
           "block_norm: residual_out must have x's shape, type and device");
    } else {
      made_res = empty({r.rows, r.d}, dt, x);
    }
    const Tensor &ro = given(a[11]) ? THPVariable_Unpack(a[11]) : made_res;
    r.x = x.data_ptr();
    r.residual = res.data_ptr();
    r.weight = w.data_ptr();
    r.out = out.data_ptr();
    r.residual_out = ro.data_ptr();
    r.x_stride = row_stride(x, "block_norm: x");
    r.residual_stride = row_stride(res, "block_norm: residual");
    r.out_stride = row_stride(out, "block_norm: out");
    r.residual_out_stride = row_stride(ro, "block_norm: residual_out");
    check(spec_layer_block_norm(handle(a[0]), &r, stream.get()), "spec_layer_block_norm");
    PyObject *list = PyList_New(quant ? 3 : 2);
    if (!list) throw Raised();
    PyList_SET_ITEM(list, 0, result(a[9], made));
    if (quant) PyList_SET_ITEM(list, 1, result(a[10], made_scale));
    PyList_SET_ITEM(list, quant ? 2 : 1, result(a[11], made_res));
    return list;
  });
}

// log_probs(self, logits, tokens, top, temperature, out, stream); out: None or
// the sequence of tensors that is returned otherwise
PyObject *log_probs(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject * {
    const Tensor &x = tensor(a[1], "log_probs: logits");
    need(x.dim() == 2, "log_probs: logits must be [rows, V]");
    sv_log_probs_t r{};
    r.dtype = code_of(x.scalar_type(), "log_probs");
    r.rows = x.size(0);
    r.V = x.size(1);
    Device device(a[0]);
    need(device.has(x), "log_probs: tensors must be on the GPU of the handle");
    if (given(a[2])) {
      const Tensor &t = tensor(a[2], "log_probs: tokens");
      need(t.dim() == 2 && t.size(0) == r.rows && t.scalar_type() == at::kInt &&
               t.is_contiguous() && t.size(1) <= INT32_MAX && device.has(t),
           "log_probs: tokens must be dense int32 [rows, n]");
      r.tokens = t.data_ptr<int32_t>();
      r.n = static_cast<int32_t>(t.size(1));
    }
    r.top = size32(a[3]);
    need(r.top >= 0 && r.top <= SV_MAX_TOP && r.top <= std::max<int64_t>(r.V, 0),
         "log_probs: top must be from 0 to 64 and at most V");
    r.temperature = static_cast<float>(number(a[4]));
    const Stream stream(a[6], x);
    Tensor outs[4];
    const int count = r.top ? 4 : 2;
    if (given(a[5])) {
      PyObject *seq = PySequence_Fast(a[5], "log_probs: out must be a sequence of tensors");
      if (!seq) throw Raised();
      struct Held {
        PyObject *o;
        ~Held() { Py_DECREF(o); }
      } held{seq};
      need(PySequence_Fast_GET_SIZE(seq) == count, "log_probs: out must hold two tensors, or four with top");
      for (int i = 0; i < count; ++i)
        outs[i] = tensor(PySequence_Fast_GET_ITEM(seq, i), "log_probs: out");
      const int64_t cols[4] = {r.n, 1, r.top, r.top};
      for (int i = 0; i < count; ++i)
        need(outs[i].scalar_type() == (i == 2 ? at::kInt : at::kFloat) &&
                 outs[i].is_contiguous() && device.has(outs[i]) &&
                 outs[i].dim() == (i == 1 ? 1 : 2) && outs[i].size(0) == r.rows &&
                 (i == 1 || outs[i].size(1) == cols[i]),
             "log_probs: out must be float32 [rows, n], [rows], int32 and float32 [rows, top]");
    } else {
      outs[0] = empty({r.rows, r.n}, at::kFloat, x);
      outs[1] = empty({r.rows}, at::kFloat, x);
      if (r.top) {
        outs[2] = empty({r.rows, r.top}, at::kInt, x);
        outs[3] = empty({r.rows, r.top}, at::kFloat, x);
      }
    }
    r.logits = x.data_ptr();
    r.stride = row_stride(x, "log_probs: logits");
    r.log_probs = outs[0].data_ptr<float>();
    r.entropy = outs[1].data_ptr<float>();
    if (r.top) {
      r.top_ids = outs[2].data_ptr<int32_t>();
      r.top_log_probs = outs[3].data_ptr<float>();
    }
    check(spec_layer_log_probs(handle(a[0]), &r, stream.get()), "spec_layer_log_probs");
    PyObject *list = PyList_New(count);
    if (!list) throw Raised();
    for (int i = 0; i < count; ++i) PyList_SET_ITEM(list, i, THPVariable_Wrap(outs[i]));
    return list;
  });
}

PyObject *set_error(PyObject *, PyObject *cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&norm)), METH_FASTCALL,
     "rms_norm and rms_norm_fp8"},
    {"matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&matmul)), METH_FASTCALL,
     "matmul_fp8"},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&rope)), METH_FASTCALL,
     "rope_append"},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&attention)),
     METH_FASTCALL, "attention"},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&linear)), METH_FASTCALL,
     "linear"},
    {"gated", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&gated)), METH_FASTCALL,
     "gated_linear"},
    {"block_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&block_norm)),
     METH_FASTCALL, "block_norm and block_norm_fp8"},
    {"log_probs", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&log_probs)),
     METH_FASTCALL, "log_probs"},
    {"set_error", set_error, METH_O, "the class raised for an entry point's error"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_target_bind", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__target_bind() {
  g_raw = PyUnicode_InternFromString("_raw");
  g_index = PyUnicode_InternFromString("_index");
  g_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&g_module);
}
