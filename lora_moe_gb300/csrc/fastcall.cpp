// fastcall.cpp -- the serving operators' calls from Python without ctypes: a
// decode step's small kernels run for 1 to 8 us, and marshalling a call with
// Python code and ctypes takes 4 to 6 us, here under 1.
//
// Each function takes the operator's tensors, on their own current stream, and
// returns the library's status; or None where anything is not as it should be
// (another type, device or shape, uneven rows), for binding.py to treat or to
// refuse with its message.  bind() gets the library's 8-bit entry points, bind16()
// those of the router and the bf16 products.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_lora.h"

namespace {

decltype(&moe_add_rms_norm_fp8) norm_fn;
decltype(&moe_silu_mul_fp8) act_fn;
decltype(&moe_fp8_matmul) matmul_fn;
decltype(&moe_fp8_grouped_matmul) grouped_fn;
decltype(&moe_fp8_grouped_matmul_naive) naive_fn;
decltype(&moe_fp8_grouped_workspace_bytes) space_fn;
decltype(&moe_route) route_fn;
decltype(&moe_bf16_matmul) matmul16_fn;
decltype(&moe_bf16_grouped_matmul) grouped16_fn;
decltype(&moe_bf16_grouped_matmul_naive) naive16_fn;
decltype(&moe_bf16_grouped_workspace_bytes) space16_fn;

constexpr int64_t kIntMax = 0x7FFFFFFF;

int64_t groups(int64_t n) { return (n + 127) / 128; }

// One call's arguments: `ok` falls where one is not as it should be.
struct Args {
  PyObject *const *args;
  bool ok = true;
  int device = -1;

  const at::Tensor *tensor(int i, at::ScalarType type, bool optional = false) {
    if (optional && args[i] == Py_None) return nullptr;
    if (!THPVariable_Check(args[i])) {
      ok = false;
      return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    // an ordinary strided CUDA tensor, on the device of the others
    if (!t.is_cuda() || t.layout() != at::kStrided || t.scalar_type() != type || t.is_neg() || t.is_conj()) {
      ok = false;
      return nullptr;
    }
    if (device < 0) device = t.get_device();
    if (t.get_device() != device) ok = false;
    return &t;
  }
  // Address of a contiguous tensor of `numel` elements (any number: -1).
  template <typename T>
  T *dense(int i, at::ScalarType type, int64_t numel, bool optional = false) {
    const at::Tensor *t = tensor(i, type, optional);
    if (!t) return nullptr;
    if ((numel >= 0 && t->numel() != numel) || !t->is_contiguous()) ok = false;
    return static_cast<T *>(t->data_ptr());
  }
  // Address and leading dimension of `rows` evenly spaced rows of `columns`.
  template <typename T>
  T *rows(int i, at::ScalarType type, int64_t rows, int64_t columns, long long *ld, bool optional = false) {
    *ld = columns;
    const at::Tensor *t = tensor(i, type, optional);
    if (!t) return nullptr;
    const int64_t dim = t->dim();
    if (dim < 1 || t->size(dim - 1) != columns || t->numel() != rows * columns ||
        (columns > 1 && t->stride(dim - 1) != 1)) {
      ok = false;
      return nullptr;
    }
    if (rows == 1) {
      *ld = (columns + 15) / 16 * 16;   // one row: any leading dimension will do
    } else if (!t->is_contiguous()) {
      int64_t step = -1;
      for (int64_t d = dim - 2; d >= 0; --d) {
        if (t->size(d) == 1) continue;
        if (step < 0) step = *ld = t->stride(d);
        if (t->stride(d) != step) ok = false;
        step *= t->size(d);
      }
    }
    return static_cast<T *>(t->data_ptr());
  }
  // type of argument i, bf16 or fp32; ok falls for any other.  None: bf16
  at::ScalarType either(int i) {
    if (args[i] == Py_None) return at::kBFloat16;
    if (!THPVariable_Check(args[i])) {
      ok = false;
      return at::kBFloat16;
    }
    const at::ScalarType t = THPVariable_Unpack(args[i]).scalar_type();
    if (t != at::kBFloat16 && t != at::kFloat) ok = false;
    return t;
  }
  // argument i as an int
  int integer(int i) {
    if (!PyLong_Check(args[i])) {
      ok = false;
      return 0;
    }
    const long v = PyLong_AsLong(args[i]);
    if ((v == -1 && PyErr_Occurred()) || v < -kIntMax || v > kIntMax) {
      PyErr_Clear();
      ok = false;
      return 0;
    }
    return (int)v;
  }
  // sizes of argument i, which has `dim` dimensions that fit an int
  const int64_t *sizes(int i, int64_t dim) {
    if (!THPVariable_Check(args[i])) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    if (t.dim() != dim) return nullptr;
    for (int64_t d = 0; d < dim; ++d)
      if (t.size(d) > kIntMax) return nullptr;
    return t.sizes().data();
  }
  void *stream() { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
  // The library works on the current device.
  bool ready() { return ok && device >= 0 && device == c10::cuda::current_device(); }
};

constexpr at::ScalarType kBf = at::kBFloat16, kF8 = at::kFloat8_e4m3fn, kF32 = at::kFloat, kI32 = at::kInt;

PyObject *none() { Py_RETURN_NONE; }

// x, weight, q, scales, residual, residual_out, normed, eps
PyObject *norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 8 || !PyFloat_Check(args[7])) return none();
  Args a{args};
  const int64_t *q = a.sizes(2, 2);
  if (!q) return none();
  const int64_t M = q[0], H = q[1];
  const at::Tensor *x = a.tensor(0, kBf);
  if (!x || x->dim() < 2 || x->dim() > 3 || x->size(0) != M || x->size(-1) != H || (H > 1 && x->stride(-1) != 1))
    return none();
  const int64_t parts = x->dim() == 3 ? x->size(1) : 1;
  const long long ldx = M > 1 ? x->stride(0) : H, ld_part = parts > 1 ? x->stride(1) : 0;
  if (parts < 1 || parts > kIntMax) return none();
  long long ldr, ldo, ldn, ldq;
  auto *res = a.rows<moe_lora_bf16>(4, kBf, M, H, &ldr, true);
  auto *out = a.rows<moe_lora_bf16>(5, kBf, M, H, &ldo, true);
  auto *normed = a.rows<moe_lora_bf16>(6, kBf, M, H, &ldn, true);
  auto *qp = a.rows<moe_lora_fp8>(2, kF8, M, H, &ldq);
  auto *weight = a.dense<moe_lora_bf16>(1, kBf, H);
  auto *scales = a.dense<float>(3, kF32, M * groups(H));
  if (!a.ready()) return none();
  return PyLong_FromLong(norm_fn(static_cast<const moe_lora_bf16 *>(x->data_ptr()), ldx, ld_part, (int)parts, res, ldr,
                                 weight, (float)PyFloat_AS_DOUBLE(args[7]), out, ldo, normed, ldn, qp, ldq, scales,
                                 (int)M, (int)H, a.stream()));
}

// x, q, scales, act
PyObject *act(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 4) return none();
  Args a{args};
  const at::Tensor *q = a.tensor(1, kF8);
  if (!q || q->dim() < 1 || q->numel() == 0) return none();
  const int64_t I = q->size(-1), rows = q->numel() / I;
  if (I > kIntMax || rows > kIntMax) return none();
  long long ldx, lda, ldq;
  auto *x = a.rows<moe_lora_bf16>(0, kBf, rows, 2 * I, &ldx);
  auto *qp = a.rows<moe_lora_fp8>(1, kF8, rows, I, &ldq);
  auto *scales = a.dense<float>(2, kF32, rows * groups(I));
  auto *out = a.rows<moe_lora_bf16>(3, kBf, rows, I, &lda, true);
  if (!a.ready()) return none();
  return PyLong_FromLong(act_fn(x, ldx, out, lda, qp, ldq, scales, (int)rows, (int)I, a.stream()));
}

// x, x_scales, w, w_scales, y, err_flag
PyObject *matmul(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 6) return none();
  Args a{args};
  const int64_t *y = a.sizes(4, 2), *x = a.sizes(0, 2);
  if (!y || !x) return none();
  const int64_t M = y[0], N = y[1], K = x[1];
  long long ldx, ldw, ldy;
  auto *xp = a.rows<moe_lora_fp8>(0, kF8, M, K, &ldx);
  auto *xs = a.dense<float>(1, kF32, M * groups(K));
  auto *w = a.rows<moe_lora_fp8>(2, kF8, N, K, &ldw);
  auto *ws = a.dense<float>(3, kF32, groups(N) * groups(K));
  auto *yp = a.rows<moe_lora_bf16>(4, kBf, M, N, &ldy);
  auto *err = a.dense<int32_t>(5, kI32, -1, true);
  if (!a.ready()) return none();
  return PyLong_FromLong(
      matmul_fn(xp, ldx, xs, w, ldw, ws, yp, ldy, (int)M, (int)N, (int)K, err, a.stream()));
}

// What both grouped calls share: x, x_scales, w, w_scales, y, topk_weights, x_per_pair, err_flag
struct Grouped {
  int64_t M, topk, N, E, K;
  int per_pair;
  long long ldx, ldw, ldy;
  const moe_lora_fp8 *x, *w;
  const float *xs, *ws, *weights;
  moe_lora_bf16 *y;
  int32_t *err;
  bool take(Args &a) {
    const int64_t *ys = a.sizes(4, 3), *wsz = a.sizes(2, 3);
    if (!ys || !wsz || !PyBool_Check(a.args[6])) return false;
    M = ys[0], topk = ys[1], N = ys[2], E = wsz[0], K = wsz[2];
    if (wsz[1] != N || M * topk > kIntMax) return false;
    per_pair = a.args[6] == Py_True;
    const int64_t rows = per_pair ? M * topk : M;
    x = a.rows<moe_lora_fp8>(0, kF8, rows, K, &ldx);
    xs = a.dense<float>(1, kF32, rows * groups(K));
    w = a.rows<moe_lora_fp8>(2, kF8, E * N, K, &ldw);
    ws = a.dense<float>(3, kF32, E * groups(N) * groups(K));
    y = a.rows<moe_lora_bf16>(4, kBf, M * topk, N, &ldy);
    weights = a.dense<float>(5, kF32, M * topk, true);
    err = a.dense<int32_t>(7, kI32, -1, true);
    return a.ok;
  }
};

// .., topk_ids
PyObject *naive(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 9) return none();
  Args a{args};
  Grouped g;
  if (!g.take(a)) return none();
  auto *ids = a.dense<int32_t>(8, kI32, g.M * g.topk);
  if (!a.ready()) return none();
  return PyLong_FromLong(naive_fn(g.x, g.per_pair, g.ldx, g.xs, g.w, g.ldw, g.ws, g.y, g.ldy, g.weights, ids, (int)g.M,
                                  (int)g.topk, (int)g.E, (int)g.K, (int)g.N, g.err, a.stream()));
}

// .., sorted_token_ids, expert_ids, num_tokens_post_padded, block_size; the workspace, where the call needs one, from
// torch's allocator (freed when the call has been enqueued: its next use is ordered behind it on this stream)
PyObject *grouped(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 12 || !PyLong_Check(args[11])) return none();
  Args a{args};
  Grouped g;
  if (!g.take(a)) return none();
  const long block = PyLong_AsLong(args[11]);
  if (block == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  if (block < 1 || block > 1024) return none();
  auto *sorted = a.dense<int32_t>(8, kI32, -1);
  auto *experts = a.dense<int32_t>(9, kI32, -1);
  auto *padded = a.dense<int32_t>(10, kI32, -1);
  if (!a.ready()) return none();
  const int64_t cap = THPVariable_Unpack(args[8]).numel(), capb = THPVariable_Unpack(args[9]).numel();
  if (cap > kIntMax || capb > kIntMax || THPVariable_Unpack(args[10]).numel() < 1) return none();
  const size_t need = space_fn((int)g.M, (int)g.topk, (int)g.E, (int)g.K, (int)g.N, (int)block);
  at::Tensor space;
  if (need) space = at::empty({(int64_t)need}, THPVariable_Unpack(args[4]).options().dtype(at::kByte));
  return PyLong_FromLong(grouped_fn(g.x, g.per_pair, g.ldx, g.xs, g.w, g.ldw, g.ws, g.y, g.ldy, g.weights, sorted,
                                    experts, padded, (int)g.M, (int)g.topk, (int)g.E, (int)g.K, (int)g.N, (int)block,
                                    (int)cap, (int)capb, need ? space.data_ptr() : nullptr, need, g.err, a.stream()));
}

// logits, topk_ids, topk_weights, bias, scoring, renormalize, scale, num_groups, topk_groups, group_best
PyObject *route(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 10 || !PyBool_Check(args[5]) || !PyFloat_Check(args[6])) return none();
  Args a{args};
  const int64_t *l = a.sizes(0, 2), *i = a.sizes(1, 2);
  if (!l || !i || i[0] != l[0]) return none();
  const int64_t M = l[0], E = l[1], topk = i[1];
  const at::ScalarType type = a.either(0);
  if (!a.ok) return none();
  long long ld;
  auto *logits = a.rows<void>(0, type, M, E, &ld);
  auto *ids = a.dense<int32_t>(1, kI32, M * topk);
  auto *weights = a.dense<float>(2, kF32, M * topk);
  auto *bias = a.dense<float>(3, kF32, E, true);
  const int scoring = a.integer(4), groups = a.integer(7), topk_groups = a.integer(8), best = a.integer(9);
  if (!a.ready()) return none();
  return PyLong_FromLong(route_fn(logits, type == kF32, ld, bias, scoring, args[5] == Py_True,
                                  (float)PyFloat_AS_DOUBLE(args[6]), groups, topk_groups, best, ids, weights, (int)M,
                                  (int)E, (int)topk, a.stream()));
}

// x, w, y, bias, residual, activation, err_flag
PyObject *matmul16(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 7) return none();
  Args a{args};
  const int64_t *y = a.sizes(2, 2), *x = a.sizes(0, 2);
  if (!y || !x) return none();
  const int64_t M = y[0], N = y[1], K = x[1];
  const at::ScalarType type = a.either(2), bias_type = a.either(3);
  if (!a.ok) return none();
  long long ldx, ldw, ldy, ldr;
  auto *xp = a.rows<moe_lora_bf16>(0, kBf, M, K, &ldx);
  auto *w = a.rows<moe_lora_bf16>(1, kBf, N, K, &ldw);
  auto *yp = a.rows<void>(2, type, M, N, &ldy);
  auto *bias = a.dense<void>(3, bias_type, N, true);
  auto *res = a.rows<void>(4, type, M, N, &ldr, true);
  const int act = a.integer(5);
  auto *err = a.dense<int32_t>(6, kI32, -1, true);
  if (!a.ready()) return none();
  return PyLong_FromLong(matmul16_fn(xp, ldx, w, ldw, bias, bias_type == kF32, res, ldr, yp, ldy, type == kF32, act,
                                     (int)M, (int)N, (int)K, err, a.stream()));
}

// What both grouped bf16 calls share: x, w, y, bias, activation, topk_weights, x_per_pair, err_flag
struct Grouped16 {
  int64_t M, topk, N, E, K;
  int per_pair, act, bias_f32;
  long long ldx, ldw, ldy;
  const moe_lora_bf16 *x, *w;
  const void *bias;
  const float *weights;
  moe_lora_bf16 *y;
  int32_t *err;
  bool take(Args &a) {
    const int64_t *ys = a.sizes(2, 3), *wsz = a.sizes(1, 3);
    if (!ys || !wsz || !PyBool_Check(a.args[6])) return false;
    M = ys[0], topk = ys[1], N = ys[2], E = wsz[0], K = wsz[2];
    if (wsz[1] != N || M * topk > kIntMax) return false;
    per_pair = a.args[6] == Py_True;
    const at::ScalarType bias_type = a.either(3);
    if (!a.ok) return false;
    bias_f32 = bias_type == kF32;
    x = a.rows<moe_lora_bf16>(0, kBf, per_pair ? M * topk : M, K, &ldx);
    w = a.rows<moe_lora_bf16>(1, kBf, E * N, K, &ldw);
    y = a.rows<moe_lora_bf16>(2, kBf, M * topk, N, &ldy);
    bias = a.dense<void>(3, bias_type, E * N, true);
    act = a.integer(4);
    weights = a.dense<float>(5, kF32, M * topk, true);
    err = a.dense<int32_t>(7, kI32, -1, true);
    return a.ok;
  }
};

// .., topk_ids
PyObject *naive16(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 9) return none();
  Args a{args};
  Grouped16 g;
  if (!g.take(a)) return none();
  auto *ids = a.dense<int32_t>(8, kI32, g.M * g.topk);
  if (!a.ready()) return none();
  return PyLong_FromLong(naive16_fn(g.x, g.per_pair, g.ldx, g.w, g.ldw, g.bias, g.bias_f32, g.y, g.ldy, g.act, g.weights,
                                    ids, (int)g.M, (int)g.topk, (int)g.E, (int)g.K, (int)g.N, g.err, a.stream()));
}

// .., sorted_token_ids, expert_ids, num_tokens_post_padded, block_size; the workspace as in grouped()
PyObject *grouped16(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 12) return none();
  Args a{args};
  Grouped16 g;
  if (!g.take(a)) return none();
  const int block = a.integer(11);
  auto *sorted = a.dense<int32_t>(8, kI32, -1);
  auto *experts = a.dense<int32_t>(9, kI32, -1);
  auto *padded = a.dense<int32_t>(10, kI32, -1);
  if (!a.ready()) return none();
  const int64_t cap = THPVariable_Unpack(args[8]).numel(), capb = THPVariable_Unpack(args[9]).numel();
  if (cap > kIntMax || capb > kIntMax || THPVariable_Unpack(args[10]).numel() < 1) return none();
  const size_t need = space16_fn((int)g.M, (int)g.topk, (int)g.E, (int)g.K, (int)g.N, block);
  at::Tensor space;
  if (need) space = at::empty({(int64_t)need}, THPVariable_Unpack(args[2]).options().dtype(at::kByte));
  return PyLong_FromLong(grouped16_fn(g.x, g.per_pair, g.ldx, g.w, g.ldw, g.bias, g.bias_f32, g.y, g.ldy, g.act,
                                      g.weights, sorted, experts, padded, (int)g.M, (int)g.topk, (int)g.E, (int)g.K,
                                      (int)g.N, block, (int)cap, (int)capb, need ? space.data_ptr() : nullptr, need,
                                      g.err, a.stream()));
}

// n addresses, none of them null
bool addresses(PyObject *const *args, Py_ssize_t n, void **p) {
  for (Py_ssize_t i = 0; i < n; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry point");
      return false;
    }
  }
  return true;
}

// the entry points' addresses, in the order of the declarations above
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind() takes six addresses");
    return nullptr;
  }
  if (!addresses(args, n, p)) return nullptr;
  norm_fn = reinterpret_cast<decltype(norm_fn)>(p[0]);
  act_fn = reinterpret_cast<decltype(act_fn)>(p[1]);
  matmul_fn = reinterpret_cast<decltype(matmul_fn)>(p[2]);
  grouped_fn = reinterpret_cast<decltype(grouped_fn)>(p[3]);
  naive_fn = reinterpret_cast<decltype(naive_fn)>(p[4]);
  space_fn = reinterpret_cast<decltype(space_fn)>(p[5]);
  return none();
}

PyObject *bind16(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[5];
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind16() takes five addresses");
    return nullptr;
  }
  if (!addresses(args, n, p)) return nullptr;
  route_fn = reinterpret_cast<decltype(route_fn)>(p[0]);
  matmul16_fn = reinterpret_cast<decltype(matmul16_fn)>(p[1]);
  grouped16_fn = reinterpret_cast<decltype(grouped16_fn)>(p[2]);
  naive16_fn = reinterpret_cast<decltype(naive16_fn)>(p[3]);
  space16_fn = reinterpret_cast<decltype(space16_fn)>(p[4]);
  return none();
}

// No C++ exception leaves a call: torch's accessors may throw on tensors of other kinds.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guard(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (...) {
    return none();
  }
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guard<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind), ENTRY(norm), ENTRY(act), ENTRY(matmul), ENTRY(grouped), ENTRY(naive), ENTRY(bind16),
                         ENTRY(route), ENTRY(matmul16), ENTRY(grouped16), ENTRY(naive16),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fastcall(void) { return PyModule_Create(&module); }
