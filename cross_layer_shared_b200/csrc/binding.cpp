// Marshalling of the 8-bit cache calls for Python.
//
// A decode step's calls run for 2 to 10 microseconds on the GPU.  Checking a
// dozen tensors from Python and handing them to ctypes takes 5 to 6 more than
// the launch itself; here they are read directly (under 1).  Only checks and
// argument order live here: the work is libsa's, whose entry points bind()
// receives as addresses, and whose status each call returns.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/sa.h"

namespace {

decltype(&sa_cache_append_q8) g_append = nullptr;
decltype(&sa_cache_read_q8) g_read = nullptr;
decltype(&sa_index_score_q8) g_index = nullptr;
decltype(&sa_decode_attn_q8) g_attn = nullptr;

constexpr int64_t kBlock = 64;

struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void bad(const char* name, const std::string& what) { throw BadArgument(std::string(name) + what); }

std::string describe(const at::Tensor& t) {
  std::ostringstream s;
  s << t.scalar_type() << " " << t.sizes() << " on " << t.device();
  return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(name, " must be a tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor* tensor_or_none(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

// the kernels run on the current GPU: the first tensor has to be there, the others beside it
int gpu_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
    bad(name, " must be on the current GPU, not " + describe(t));
  return (int)t.get_device();
}

void* address(const at::Tensor& t, int64_t n, at::ScalarType type, int dev, const char* name) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() || t.numel() != n) {
    std::ostringstream s;
    s << " must be a contiguous tensor of " << n << " elements of " << type << " on GPU " << dev << ", not "
      << describe(t);
    bad(name, s.str());
  }
  return t.data_ptr();
}

int64_t integer(PyObject* o, const char* name, int64_t lo, int64_t hi) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(name, " must be an integer");
  }
  if (v < lo || v > hi) bad(name, "=" + std::to_string(v) + " is out of range");
  return v;
}
int int32_of(PyObject* o, const char* name) { return (int)integer(o, name, INT32_MIN, INT32_MAX); }

void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  return reinterpret_cast<void*>(integer(o, "stream", INT64_MIN, INT64_MAX));
}

sa_dtype float_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return SA_BF16;
  if (t.scalar_type() == at::kFloat) return SA_F32;
  bad(name, " must be bfloat16 or float32, not " + describe(t));
}

struct Cache {
  void *K, *Ks, *V = nullptr, *Vs = nullptr;
  int64_t n_tokens;
};

// codes [.., d] and one scale for each 64 rows of them, of K and (unless V is None) of V
Cache cache(PyObject* const* args, int64_t Hkv, int64_t d, int dev, bool pair) {
  const at::Tensor& k = tensor(args[0], "K8");
  Cache c;
  const int64_t n = k.numel();
  if (Hkv < 1 || d < 1 || n % (kBlock * Hkv * d) || k.dim() < 1 || k.size(-1) != d)
    bad("K8", " must be [.., " + std::to_string(d) + "] with a multiple of 64 token places of " + std::to_string(Hkv) +
                  " heads, not " + describe(k));
  const int64_t n_scales = n / (d * kBlock);
  c.n_tokens = n / (Hkv * d);
  c.K = address(k, n, at::kFloat8_e4m3fn, dev, "K8");
  c.Ks = address(tensor(args[1], "K_scale"), n_scales, at::kFloat, dev, "K_scale");
  if (!pair) return c;
  const at::Tensor *v = tensor_or_none(args[2], "V8"), *vs = tensor_or_none(args[3], "V_scale");
  if (!v != !vs) bad("V8", " and V_scale go together");
  if (v) {
    c.V = address(*v, n, at::kFloat8_e4m3fn, dev, "V8");
    c.Vs = address(*vs, n_scales, at::kFloat, dev, "V_scale");
  }
  return c;
}

struct Seqs {
  const int64_t* off;
  const int32_t* len;
  int64_t B;
};
Seqs seqs(PyObject* off, PyObject* len, int dev) {
  const at::Tensor &o = tensor(off, "seq_off"), &l = tensor(len, "seq_len");
  const int64_t B = l.numel();
  if (B > INT32_MAX) bad("seq_len", " is too long");
  return {(const int64_t*)address(o, B + 1, at::kLong, dev, "seq_off"),
          (const int32_t*)address(l, B, at::kInt, dev, "seq_len"), B};
}

// new tokens' rows [n, Hkv, d], each row of heads contiguous; returns the rows' stride
int64_t new_rows(const at::Tensor& x, int dev, const char* name) {
  if (x.dim() != 3 || !x.is_cuda() || x.get_device() != dev ||
      (x.numel() && ((x.size(2) > 1 && x.stride(2) != 1) || (x.size(1) > 1 && x.stride(1) != x.size(2))))) {
    std::ostringstream s;
    s << " must be [n, Hkv, d] on GPU " << dev << " with each token's [Hkv, d] contiguous, not " << describe(x)
      << " with strides " << x.strides();
    bad(name, s.str());
  }
  return x.size(0) > 1 ? x.stride(0) : x.size(1) * x.size(2);
}

struct Workspace {
  void* p;
  size_t n;
};
Workspace workspace(PyObject* o, int dev) {
  const at::Tensor& t = tensor(o, "ws");
  return {address(t, t.numel(), at::kByte, dev, "ws"), (size_t)t.numel()};
}

// runs f with the interpreter released and returns its status as an int
template <typename F>
PyObject* status(F f) {
  sa_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return PyLong_FromLong((long)st);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, bool bound, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  if (!bound) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  try {
    return f();
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// bind(address of sa_cache_append_q8, .._read_q8, sa_index_score_q8, sa_decode_attn_q8)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, true, [&]() -> PyObject* {
    g_append = reinterpret_cast<decltype(g_append)>(integer(a[0], "address", INT64_MIN, INT64_MAX));
    g_read = reinterpret_cast<decltype(g_read)>(integer(a[1], "address", INT64_MIN, INT64_MAX));
    g_index = reinterpret_cast<decltype(g_index)>(integer(a[2], "address", INT64_MIN, INT64_MAX));
    g_attn = reinterpret_cast<decltype(g_attn)>(integer(a[3], "address", INT64_MIN, INT64_MAX));
    Py_RETURN_NONE;
  });
}

// (new_K, new_V, K8, K_scale, V8, V_scale, seq_off, seq_len, new_off, max_new, ws, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, g_append != nullptr, [&] {
    const at::Tensor& k = tensor(a[0], "new_K");
    const at::Tensor* v = tensor_or_none(a[1], "new_V");
    const int dev = gpu_of(k, "new_K");
    const sa_dtype type = float_type(k, "new_K");
    const int64_t sk = new_rows(k, dev, "new_K"), rows = k.size(0), Hkv = k.size(1), d = k.size(2);
    int64_t sv = 0;
    if (!v != (a[4] == Py_None)) bad("new_V", " and V8 go together");
    if (v) {
      if (v->sizes() != k.sizes() || v->scalar_type() != k.scalar_type())
        bad("new_V", " must have new_K's shape and dtype, not " + describe(*v));
      sv = new_rows(*v, dev, "new_V");
    }
    const Cache c = cache(a + 2, Hkv, d, dev, true);
    const Seqs s = seqs(a[6], a[7], dev);
    const int64_t* off = nullptr;
    int64_t max_new = 1;
    if (const at::Tensor* t = tensor_or_none(a[8], "new_off")) {
      off = (const int64_t*)address(*t, s.B + 1, at::kLong, dev, "new_off");
      max_new = a[9] == Py_None ? rows : integer(a[9], "max_new", INT32_MIN, INT32_MAX);
      if (max_new > INT32_MAX) bad("new_K", " has too many rows");
    } else if (rows != s.B) {
      bad("new_K", " must have one row per sequence without new_off: " + std::to_string(s.B) + ", not " +
                       std::to_string(rows));
    }
    const Workspace w = workspace(a[10], dev);
    void* stream = stream_of(a[11], dev);
    return status([&] {
      return g_append(k.data_ptr(), sk, v ? v->data_ptr() : nullptr, sv, type, rows, off, (int)max_new, c.K,
                      (float*)c.Ks, c.V, (float*)c.Vs, s.off, s.len, (int)s.B, c.n_tokens, (int)Hkv, (int)d, w.p, w.n,
                      stream);
    });
  });
}

// (K8, K_scale, V8, V_scale, seq_off, seq_len, S_max, Hkv, idx, out_off, n_out, K, V, ws, stream)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, g_read != nullptr, [&] {
    const at::Tensor& k8 = tensor(a[0], "K8");
    const int dev = gpu_of(k8, "K8");
    const int64_t d = k8.dim() ? k8.size(-1) : 0;
    const int Hkv = int32_of(a[7], "Hkv");
    const Cache c = cache(a, Hkv, d, dev, true);
    const Seqs s = seqs(a[4], a[5], dev);
    const at::Tensor *idx = tensor_or_none(a[8], "idx"), *off = tensor_or_none(a[9], "out_off");
    const at::Tensor& K = tensor(a[11], "K");
    const at::Tensor* V = tensor_or_none(a[12], "V");
    if (!V != (a[2] == Py_None)) bad("V", " and V8 go together");
    if (!idx == !off) bad("idx", " (picked rows) or out_off (whole sequences): give one of them");
    int64_t k = 0, n_out = 0, rows;
    const int32_t* idxp = nullptr;
    const int64_t* offp = nullptr;
    if (idx) {
      if (idx->dim() != 2) bad("idx", " must be [B, k], not " + describe(*idx));
      k = idx->size(1);
      if (k > INT32_MAX) bad("idx", " is too wide");
      idxp = (const int32_t*)address(*idx, s.B * k, at::kInt, dev, "idx");
      rows = s.B * Hkv * k;
    } else {
      offp = (const int64_t*)address(*off, s.B + 1, at::kLong, dev, "out_off");
      n_out = integer(a[10], "n_out", 0, INT32_MAX);
      rows = n_out * Hkv;
    }
    const sa_dtype type = float_type(K, "K");
    void* Kp = address(K, rows * d, K.scalar_type(), dev, "K");
    void* Vp = V ? address(*V, rows * d, K.scalar_type(), dev, "V") : nullptr;
    const int S_max = int32_of(a[6], "S_max");
    const Workspace w = workspace(a[13], dev);
    void* stream = stream_of(a[14], dev);
    return status([&] {
      return g_read(c.K, (float*)c.Ks, c.V, (float*)c.Vs, s.off, s.len, (int)s.B, c.n_tokens, S_max, Hkv, (int)d, idxp,
                    (int)k, offp, n_out, Kp, Vp, type, w.p, w.n, stream);
    });
  });
}

// (qI, w, KI8, KI_scale, seq_off, seq_len, S_max, scores, ws, stream)
PyObject* index(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, g_index != nullptr, [&] {
    const at::Tensor& q = tensor(a[0], "qI");
    const int dev = gpu_of(q, "qI");
    if (q.dim() != 3) bad("qI", " must be [B, H_I, d_I], not " + describe(q));
    const int64_t B = q.size(0), H = q.size(1), d = q.size(2);
    if (H > INT32_MAX || d > INT32_MAX) bad("qI", " is too large");
    const Cache c = cache(a + 2, 1, d, dev, false);
    const Seqs s = seqs(a[4], a[5], dev);
    if (s.B != B) bad("seq_len", " must have " + std::to_string(B) + " entries, not " + std::to_string(s.B));
    const int S_max = int32_of(a[6], "S_max");
    const at::Tensor& scores = tensor(a[7], "scores");
    if (scores.dim() != 2 || scores.size(1) < S_max)
      bad("scores", " must be [" + std::to_string(B) + ", >= " + std::to_string(S_max) + "], not " + describe(scores));
    const int64_t ld = scores.size(1);
    void* qp = address(q, B * H * d, at::kBFloat16, dev, "qI");
    void* wp = address(tensor(a[1], "w"), B * H, at::kFloat, dev, "w");
    void* sp = address(scores, B * ld, at::kFloat, dev, "scores");
    const Workspace w = workspace(a[8], dev);
    void* stream = stream_of(a[9], dev);
    return status([&] {
      return g_index(qp, (const float*)wp, c.K, (const float*)c.Ks, s.off, s.len, (int)B, c.n_tokens, S_max, (int)H,
                     (int)d, (float*)sp, ld, w.p, w.n, stream);
    });
  });
}

// (Q, K8, K_scale, V8, V_scale, seq_off, seq_len, S_max, Hkv, scale, idx, O, ws, stream)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, g_attn != nullptr, [&] {
    const at::Tensor& q = tensor(a[0], "Q");
    const int dev = gpu_of(q, "Q");
    if (q.dim() != 4) bad("Q", " must be [L, B, Hq, d], not " + describe(q));
    const int64_t L = q.size(0), B = q.size(1), Hq = q.size(2), d = q.size(3);
    if (L > INT32_MAX || Hq > INT32_MAX || d > INT32_MAX) bad("Q", " is too large");
    const int Hkv = int32_of(a[8], "Hkv");
    const Cache c = cache(a + 1, Hkv, d, dev, true);
    if (a[3] == Py_None) bad("V8", " is missing");
    const Seqs s = seqs(a[5], a[6], dev);
    if (s.B != B) bad("seq_len", " must have " + std::to_string(B) + " entries, not " + std::to_string(s.B));
    const int S_max = int32_of(a[7], "S_max");
    const double scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      bad("scale", " must be a number");
    }
    const at::Tensor* idx = tensor_or_none(a[10], "idx");
    int64_t k = 0;
    const int32_t* idxp = nullptr;
    if (idx) {
      if (idx->dim() != 2) bad("idx", " must be [B, k], not " + describe(*idx));
      k = idx->size(1);
      if (k > INT32_MAX) bad("idx", " is too wide");
      idxp = (const int32_t*)address(*idx, B * k, at::kInt, dev, "idx");
    }
    const at::Tensor& O = tensor(a[11], "O");
    const sa_dtype type = float_type(O, "O");
    if (O.sizes() != q.sizes()) bad("O", " must have Q's shape, not " + describe(O));
    void* qp = address(q, q.numel(), at::kBFloat16, dev, "Q");
    void* op = address(O, q.numel(), O.scalar_type(), dev, "O");
    const Workspace w = workspace(a[12], dev);
    void* stream = stream_of(a[13], dev);
    return status([&] {
      return g_attn(qp, c.K, (const float*)c.Ks, c.V, (const float*)c.Vs, s.off, s.len, idxp, (int)L, (int)B,
                    c.n_tokens, S_max, (int)Hq, Hkv, (int)d, (int)k, (float)scale, op, type, w.p, w.n, stream);
    });
  });
}

PyMethodDef kMethods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, "libsa's entry points, as addresses"},
    {"cache_append_q8", (PyCFunction)(void (*)(void))append, METH_FASTCALL, "sa_cache_append_q8; returns its status"},
    {"cache_read_q8", (PyCFunction)(void (*)(void))read, METH_FASTCALL, "sa_cache_read_q8; returns its status"},
    {"index_score_q8", (PyCFunction)(void (*)(void))index, METH_FASTCALL, "sa_index_score_q8; returns its status"},
    {"decode_attn_q8", (PyCFunction)(void (*)(void))attn, METH_FASTCALL, "sa_decode_attn_q8; returns its status"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", "Marshalling of libsa's 8-bit cache calls", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
