// Argument marshalling of the calls around the layer for the Python binding: the checks that the binding would make in
// Python take longer there than the smallest kernels (a norm of one token: 7.5 us of 10.5 a call, here 0.4).
//
// Each function takes its Python counterpart's arguments in order and returns the C call's status, or None where an
// argument is not what it should be: the binding's own checks then find the reason, and raise.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace {

struct Calls {
  decltype(&moe_rms_norm) rms_norm;
  decltype(&moe_rms_norm_backward) rms_norm_backward;
  decltype(&moe_select) select;
  decltype(&moe_select_backward) select_backward;
  decltype(&moe_pack_rows8) pack_rows8;
  decltype(&moe_linear_backward8) linear_backward8;
} calls = {};

// The arguments of one call; `ok` ends up false where one of them is not what it should be.
struct Args {
  PyObject* const* a;
  bool ok;
  int device = -1;
  void* stream = nullptr;
  at::ScalarType type = at::kFloat;       // of the call's rows
  moe_dtype dt = MOE_F32;

  Args(PyObject* const* a_, Py_ssize_t n, Py_ssize_t want) : a(a_), ok(n == want) {
    if (!ok) return;
    const auto s = c10::cuda::getCurrentCUDAStream();
    device = s.device_index();
    stream = s.stream();
  }
  const at::Tensor* tensor(PyObject* o) {
    if (ok && THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.is_cuda() && t.get_device() == device && t.layout() == at::kStrided) return &t;
    }
    ok = false;
    return nullptr;
  }
  static bool dtype_of(const at::Tensor& t, moe_dtype* d) {
    switch (t.scalar_type()) {
      case at::kBFloat16: *d = MOE_BF16; return true;
      case at::kHalf: *d = MOE_F16; return true;
      case at::kFloat: *d = MOE_F32; return true;
      default: return false;
    }
  }
  // The sizes of matrix argument i, whose type the call's rows have.
  void shape(int i, int* n, int* c) {
    const at::Tensor* t = tensor(a[i]);
    if (!t) return;
    ok = t->dim() == 2 && t->size(0) <= INT_MAX && t->size(1) <= INT_MAX && dtype_of(*t, &dt);
    if (!ok) return;
    type = t->scalar_type();
    *n = static_cast<int>(t->size(0));
    *c = static_cast<int>(t->size(1));
  }
  moe_rows matrix(PyObject* o, at::ScalarType want, int64_t n, int64_t c) {
    if (o == Py_None) return {nullptr, 0};
    const at::Tensor* t = tensor(o);
    if (!t) return {nullptr, 0};
    int64_t ld = 0;
    ok = t->scalar_type() == want && t->dim() == 2 && t->size(0) == n && t->size(1) == c;
    if (ok) {
      ld = n <= 1 ? (c + 7) / 8 * 8 : t->stride(0);       // (one row: the pitch is never used)
      ok = (c <= 1 || t->stride(1) == 1) && ld >= c;
    }
    if (!ok) return {nullptr, 0};
    return {t->data_ptr(), ld};
  }
  moe_rows rows(int i, int64_t n, int64_t c) { return matrix(a[i], type, n, c); }
  moe_rows8 rows8(int i, int64_t n, int64_t c) {
    if (a[i] == Py_None) return {nullptr, nullptr, 0, 0};
    if (!ok || !PyTuple_Check(a[i]) || PyTuple_GET_SIZE(a[i]) != 2) {
      ok = false;
      return {nullptr, nullptr, 0, 0};
    }
    const moe_rows q = matrix(PyTuple_GET_ITEM(a[i], 0), at::kByte, n, c);
    const moe_rows s = matrix(PyTuple_GET_ITEM(a[i], 1), at::kByte, n, (c + 127) / 128);
    ok = ok && q.ptr && s.ptr;
    return {static_cast<uint8_t*>(q.ptr), static_cast<uint8_t*>(s.ptr), q.ld, s.ld};
  }
  // A contiguous tensor of these sizes.
  void* full(int i, at::ScalarType want, std::initializer_list<int64_t> sizes) {
    if (a[i] == Py_None) return nullptr;
    const at::Tensor* t = tensor(a[i]);
    if (!t) return nullptr;
    ok = t->scalar_type() == want && t->sizes() == at::IntArrayRef(sizes) && t->is_contiguous();
    return ok ? t->data_ptr() : nullptr;
  }
  void* workspace(int i, size_t* bytes) {
    *bytes = 0;
    if (a[i] == Py_None) return nullptr;
    const at::Tensor* t = tensor(a[i]);
    if (!t) return nullptr;
    ok = t->scalar_type() == at::kByte && t->is_contiguous();
    *bytes = static_cast<size_t>(t->numel());
    return t->data_ptr();
  }
  int integer(int i) {
    if (!ok) return 0;
    int over = 0;
    const long v = PyLong_Check(a[i]) ? PyLong_AsLongAndOverflow(a[i], &over) : (over = 1);
    ok = !over && v >= INT_MIN && v <= INT_MAX;
    return static_cast<int>(v);
  }
  float number(int i) {
    if (!ok) return 0.f;
    if (PyFloat_Check(a[i])) return static_cast<float>(PyFloat_AS_DOUBLE(a[i]));
    return static_cast<float>(integer(i));
  }
};

// Runs a call's body: its status as a Python number, None where its arguments were not in order.
template <class F>
PyObject* run(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, F&& body) {
  try {
    Args x(a, n, want);
    if (x.ok) {
      const int status = body(x);
      if (x.ok) return PyLong_FromLong(status);
    }
  } catch (...) {
    // (a tensor without storage, a machine without a GPU)
  }
  Py_RETURN_NONE;
}
// The C call itself, outside Python's lock.
template <class F>
int enqueue(F&& call) {
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = call();
  Py_END_ALLOW_THREADS;
  return status;
}

// x, weight, eps, residual, sum_out, y, y8
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(a, n, 7, [](Args& x) {
    int T = 0, H = 0;
    x.shape(0, &T, &H);
    const moe_rows in = x.rows(0, T, H), res = x.rows(3, T, H), sum = x.rows(4, T, H), y = x.rows(5, T, H);
    const float* w = static_cast<const float*>(x.full(1, at::kFloat, {H}));
    const moe_rows8 y8 = x.rows8(6, T, H);
    const float eps = x.number(2);
    if (!x.ok) return 0;
    return enqueue([&] { return calls.rms_norm(x.dt, in, res, w, eps, T, H, sum, y, y8, x.stream); });
  });
}

// dy, x, weight, eps, dx, ws, dweight, dsum
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(a, n, 8, [](Args& x) {
    int T = 0, H = 0;
    size_t bytes;
    x.shape(0, &T, &H);
    const moe_rows dy = x.rows(0, T, H), in = x.rows(1, T, H), dx = x.rows(4, T, H), ds = x.rows(7, T, H);
    const float* w = static_cast<const float*>(x.full(2, at::kFloat, {H}));
    float* dw = static_cast<float*>(x.full(6, at::kFloat, {H}));
    void* ws = x.workspace(5, &bytes);
    const float eps = x.number(3);
    if (!x.ok) return 0;
    return enqueue([&] { return calls.rms_norm_backward(x.dt, dy, in, w, eps, ds, T, H, dx, dw, ws, bytes, x.stream); });
  });
}

// logits, topk_ids, topk_w, e_score_bias, fn, n_groups, topk_groups, group_best, renormalize, scale
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(a, n, 10, [](Args& x) {
    int T = 0, E = 0;
    x.shape(0, &T, &E);
    const moe_rows logits = x.rows(0, T, E);
    const at::Tensor* ids = x.tensor(x.a[1]);
    if (!ids || ids->dim() != 2) return x.ok = false, 0;
    const int64_t K = ids->size(1);
    int32_t* id = static_cast<int32_t*>(x.full(1, at::kInt, {T, K}));
    float* w = static_cast<float*>(x.full(2, at::kFloat, {T, K}));
    const float* bias = static_cast<const float*>(x.full(3, at::kFloat, {E}));
    moe_select_rule r;
    r.fn = static_cast<moe_score_fn>(x.integer(4));
    r.n_groups = x.integer(5);
    r.topk_groups = x.integer(6);
    r.group_best = x.integer(7);
    r.renormalize = x.integer(8);
    r.scale = x.number(9);
    if (!x.ok || K > INT_MAX) return x.ok = false, 0;
    return enqueue([&] { return calls.select(x.dt, logits, bias, T, E, static_cast<int>(K), r, id, w, x.stream); });
  });
}

// logits, topk_ids, topk_w, dtopk_w, dlogits, ws, fn, renormalize, scale
PyObject* select_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(a, n, 9, [](Args& x) {
    int T = 0, E = 0;
    size_t bytes;
    x.shape(0, &T, &E);
    const moe_rows logits = x.rows(0, T, E);
    const at::Tensor *ids = x.tensor(x.a[1]), *out = x.tensor(x.a[4]);
    moe_dtype gdt;
    if (!x.ok || ids->dim() != 2 || !Args::dtype_of(*out, &gdt)) return x.ok = false, 0;
    const int64_t K = ids->size(1);
    const int32_t* id = static_cast<const int32_t*>(x.full(1, at::kInt, {T, K}));
    const float* w = static_cast<const float*>(x.full(2, at::kFloat, {T, K}));
    const float* dw = static_cast<const float*>(x.full(3, at::kFloat, {T, K}));
    const moe_rows dl = x.matrix(x.a[4], out->scalar_type(), T, E);
    void* ws = x.workspace(5, &bytes);
    const moe_score_fn fn = static_cast<moe_score_fn>(x.integer(6));
    const int renorm = x.integer(7);
    const float scale = x.number(8);
    if (!x.ok || K > INT_MAX) return x.ok = false, 0;
    return enqueue([&] {
      return calls.select_backward(x.dt, logits, id, w, dw, T, E, static_cast<int>(K), fn, renorm, scale, gdt, dl, ws, bytes,
                                   x.stream);
    });
  });
}

// x, x8, expert_counts, align, ws
PyObject* pack_rows8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(a, n, 5, [](Args& x) {
    int rows = 0, cols = 0, E = 0;
    size_t bytes;
    x.shape(0, &rows, &cols);
    const moe_rows in = x.rows(0, rows, cols);
    const moe_rows8 x8 = x.rows8(1, rows, cols);
    const int32_t* counts = nullptr;
    if (x.ok && x.a[2] != Py_None) {
      const at::Tensor* c = x.tensor(x.a[2]);
      if (!c || c->dim() != 1 || c->size(0) < 1 || c->size(0) > INT_MAX) return x.ok = false, 0;
      E = static_cast<int>(c->size(0));
      counts = static_cast<const int32_t*>(x.full(2, at::kInt, {E}));
    }
    const int align = x.integer(3);
    void* ws = x.workspace(4, &bytes);
    if (!x.ok) return 0;
    return enqueue([&] { return calls.pack_rows8(x.dt, in, counts, rows, cols, E, align, x8, ws, bytes, x.stream); });
  });
}

// dy, w, ws, x, x8, z, z8, x_ids, x_div, dx, dw, dbias, act, dx_residual, expert_counts, align
PyObject* linear_backward8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(a, n, 16, [](Args& x) {
    int rows = 0, cols = 0;
    size_t bytes;
    x.shape(0, &rows, &cols);
    const at::Tensor* w = x.tensor(x.a[1]);
    const bool experts = x.a[14] != Py_None;
    if (!w || w->dim() != (experts ? 3 : 2) || w->scalar_type() != x.type || !w->is_contiguous()) return x.ok = false, 0;
    const int64_t E = experts ? w->size(0) : 0, N = w->size(-2), K = w->size(-1);
    if (E > INT_MAX || N > INT_MAX || K > INT_MAX || (experts && E < 1)) return x.ok = false, 0;
    const int act = x.integer(12);
    if (cols != (act == MOE_ACT_SWIGLU ? N / 2 : N)) return x.ok = false, 0;
    const moe_rows dy = x.rows(0, rows, cols), in = x.rows(3, rows, K), z = x.rows(5, rows, N), dx = x.rows(9, rows, K),
                   res = x.rows(13, rows, K);
    int64_t src = rows;
    if (x.ok && x.a[7] != Py_None && x.a[4] != Py_None) {
      if (!PyTuple_Check(x.a[4]) || PyTuple_GET_SIZE(x.a[4]) != 2) return x.ok = false, 0;
      const at::Tensor* q = x.tensor(PyTuple_GET_ITEM(x.a[4], 0));
      if (!q || q->dim() != 2 || q->size(0) > INT_MAX) return x.ok = false, 0;
      src = q->size(0);
    }
    const moe_rows8 x8 = x.rows8(4, src, K), z8 = x.rows8(6, rows, N);
    const int32_t* ids = static_cast<const int32_t*>(x.full(7, at::kInt, {rows}));
    const int div = x.integer(8), align = x.integer(15);
    const int32_t* counts = static_cast<const int32_t*>(x.full(14, at::kInt, {E}));
    void* dw = experts ? x.full(10, x.type, {E, N, K}) : x.full(10, x.type, {N, K});
    float* db = static_cast<float*>(experts ? x.full(11, at::kFloat, {E, N}) : x.full(11, at::kFloat, {N}));
    void* ws = x.workspace(2, &bytes);
    if (!x.ok) return 0;
    return enqueue([&] {
      return calls.linear_backward8(x.dt, dy, in, x8, ids, div, static_cast<int>(src), w->data_ptr(), z, z8,
                                    static_cast<moe_act>(act), counts, rows, static_cast<int>(N), static_cast<int>(K),
                                    static_cast<int>(E), align, res, dx, dw, db, ws, bytes, x.stream);
    });
  });
}

// Takes the C calls from the library at this path.
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!lib) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
  const auto take = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(lib, name));
    if (!f) PyErr_Format(PyExc_RuntimeError, "%s has no %s", p, name);
    return f != nullptr;
  };
  if (!take(calls.rms_norm, "moe_rms_norm") || !take(calls.rms_norm_backward, "moe_rms_norm_backward") ||
      !take(calls.select, "moe_select") || !take(calls.select_backward, "moe_select_backward") ||
      !take(calls.pack_rows8, "moe_pack_rows8") || !take(calls.linear_backward8, "moe_linear_backward8"))
    return nullptr;
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"rms_norm", fast(rms_norm), METH_FASTCALL, nullptr},
                         {"rms_norm_backward", fast(rms_norm_backward), METH_FASTCALL, nullptr},
                         {"select", fast(select), METH_FASTCALL, nullptr},
                         {"select_backward", fast(select_backward), METH_FASTCALL, nullptr},
                         {"pack_rows8", fast(pack_rows8), METH_FASTCALL, nullptr},
                         {"linear_backward8", fast(linear_backward8), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
