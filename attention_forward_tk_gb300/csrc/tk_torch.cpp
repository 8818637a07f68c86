// tk_torch.cpp -- the torch helpers of a decoder's serving calls, compiled.
//
// A decoder makes these calls for every layer of every token, and at one token
// a sequence a kernel takes a few microseconds.  Reading some thirty tensor
// attributes from Python and marshalling the C call through ctypes took 11 to 27 us
// (GB300's host cores); here the checks, the allocations and the call take 3 to
// 9.  Every function checks its tensors (ValueError), makes their device
// current, allocates through torch what it is not given, enqueues on torch's
// current stream of that device through the C ABI, and returns the results, or
// the C call's status where it is not 0.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <sstream>

#include "tk_attn.h"

namespace {

using at::Tensor;
using Shape = c10::IntArrayRef;

struct Refused : std::exception {};

[[noreturn]] void refuse(const Tensor &t, const char *name, const std::string &want) {
  std::ostringstream s;
  s << name << " must be " << want << ", not " << t.scalar_type() << ' ' << t.sizes()
    << " with strides " << t.strides() << " on " << t.device();
  PyErr_SetString(PyExc_ValueError, s.str().c_str());
  throw Refused();
}

[[noreturn]] void refuse(const std::string &what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string words(at::ScalarType dtype, Shape shape, int dev) {
  std::ostringstream s;
  s << "a contiguous " << dtype << " tensor " << shape << " on cuda:" << dev;
  return s.str();
}

// t is contiguous, of this type and shape, on CUDA device dev.
const Tensor &want(const Tensor &t, const char *name, at::ScalarType dtype, Shape shape, int dev) {
  if (t.scalar_type() != dtype || !t.sizes().equals(shape) || !t.is_contiguous() || !t.is_cuda() ||
      t.get_device() != dev)
    refuse(t, name, words(dtype, shape, dev));
  return t;
}

// t is a bf16 [B, H, N, D] tensor of this shape, its last dimension contiguous.
const Tensor &want_rows(const Tensor &t, const char *name, Shape shape, int dev) {
  if (t.scalar_type() != at::kBFloat16 || !t.sizes().equals(shape) || t.stride(3) != 1 ||
      !t.is_cuda() || t.get_device() != dev) {
    std::ostringstream s;
    s << "a bfloat16 tensor " << shape << " with a contiguous last dimension on cuda:" << dev;
    refuse(t, name, s.str());
  }
  return t;
}

struct Strides {
  long long s[3];
  explicit Strides(const Tensor &t) : s{t.stride(0), t.stride(1), t.stride(2)} {}
};

tk_attn_stream_t stream_of(int dev) {
  return reinterpret_cast<tk_attn_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
}

Tensor make(Shape shape, at::ScalarType dtype, const Tensor &like) {
  return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
}

// What the C calls take of each argument.
int size32(int64_t x) {
  if (x > 0x7fffffff) refuse("a dimension is larger than 2^31 - 1");
  return (int)x;
}

int truth(PyObject *o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw Refused();  // (its exception is set)
  return t;
}

PyObject *wrap2(const Tensor &a, const Tensor &b) {
  PyObject *t = PyTuple_New(2);
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

void count_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("wrong number of arguments");
}

// ------------------------------------------------------------------ norm and rotation

struct NormRope {
  const Tensor &q, &k, &qw, &kw;
  const unsigned long long *turns = nullptr;
  const int *pos = nullptr;
  int dev, B, H, Hk, N, D, rot = 0, f32;

  // a[0..5]: q, k, q_weight, k_weight, turns, positions
  explicit NormRope(PyObject *const *a)
      : q(tensor(a[0], "q")), k(tensor(a[1], "k")), qw(tensor(a[2], "q_weight")),
        kw(tensor(a[3], "k_weight")) {
    if (q.dim() != 4 || k.dim() != 4 || q.size(0) != k.size(0) || q.size(2) != k.size(2) ||
        q.size(3) != k.size(3))
      refuse("q must be [B, H, N, D] and k [B, Hk, N, D]");
    if (!q.is_cuda()) refuse("q must be a CUDA tensor");
    dev = q.get_device();
    want_rows(q, "q", q.sizes(), dev);
    want_rows(k, "k", k.sizes(), dev);
    const auto wt = qw.scalar_type();
    f32 = wt == at::kFloat;
    if (!f32 && wt != at::kBFloat16) refuse("q_weight and k_weight must be bfloat16 or float32");
    const int64_t d = q.size(3);
    want(qw, "q_weight", wt, {d}, dev);
    want(kw, "k_weight", wt, {d}, dev);
    if (a[4] != Py_None) {
      const Tensor &t = tensor(a[4], "turns");
      want(t, "turns", at::kLong, {t.numel()}, dev);
      rot = size32(2 * t.numel());
      turns = static_cast<const unsigned long long *>(t.const_data_ptr());
    }
    if (a[5] != Py_None)
      pos = want(tensor(a[5], "positions"), "positions", at::kInt, {q.size(0), q.size(2)}, dev)
                .const_data_ptr<int>();
    B = size32(q.size(0));
    H = size32(q.size(1));
    Hk = size32(k.size(1));
    N = size32(q.size(2));
    D = size32(d);
  }
};

// (q, k, q_weight, k_weight, turns, positions, eps, interleaved, out_q, out_k)
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 10);
    const NormRope c(a);
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const int inter = truth(a[7]);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const Tensor oq = a[8] == Py_None
                          ? make(c.q.sizes(), at::kBFloat16, c.q)
                          : want(tensor(a[8], "out_q"), "out_q", at::kBFloat16, c.q.sizes(), c.dev);
    const Tensor ok = a[9] == Py_None
                          ? make(c.k.sizes(), at::kBFloat16, c.q)
                          : want(tensor(a[9], "out_k"), "out_k", at::kBFloat16, c.k.sizes(), c.dev);
    const Strides qs(c.q), ks(c.k);
    const int st = tk_attn_qk_norm_rope(
        c.q.const_data_ptr(), qs.s, c.k.const_data_ptr(), ks.s, c.qw.const_data_ptr(),
        c.kw.const_data_ptr(), c.f32, c.turns, c.pos, oq.data_ptr(), ok.data_ptr(), c.B, c.H, c.Hk,
        c.N, c.D, c.rot, inter, (float)eps, stream_of(c.dev));
    return st ? PyLong_FromLong(st) : wrap2(oq, ok);
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (q, k, q_weight, k_weight, turns, positions, eps, interleaved, dq_out, dk_out,
//  dq, dk, workspace)
PyObject *norm_rope_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 13);
    const NormRope c(a);
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const int inter = truth(a[7]);
    const Tensor &gq = want_rows(tensor(a[8], "dq_out"), "dq_out", c.q.sizes(), c.dev);
    const Tensor &gk = want_rows(tensor(a[9], "dk_out"), "dk_out", c.k.sizes(), c.dev);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const Tensor dq = a[10] == Py_None ? at::empty_like(c.q).detach() : tensor(a[10], "dq");
    const Tensor dk = a[11] == Py_None ? at::empty_like(c.k).detach() : tensor(a[11], "dk");
    want_rows(dq, "dq", c.q.sizes(), c.dev);
    want_rows(dk, "dk", c.k.sizes(), c.dev);
    const Tensor dw = make({2, c.D}, at::kFloat, c.q);
    const Tensor ws =
        a[12] == Py_None
            ? make({(int64_t)tk_attn_qk_norm_rope_bwd_workspace_bytes(c.D)}, at::kByte, c.q)
            : tensor(a[12], "workspace");
    if (!ws.is_cuda() || ws.get_device() != c.dev || !ws.is_contiguous())
      refuse("the workspace must be contiguous and on the tensors' device");
    const Strides qs(c.q), ks(c.k), gqs(gq), gks(gk), dqs(dq), dks(dk);
    float *w = dw.data_ptr<float>();
    const int st = tk_attn_qk_norm_rope_bwd(
        c.q.const_data_ptr(), qs.s, c.k.const_data_ptr(), ks.s, c.qw.const_data_ptr(),
        c.kw.const_data_ptr(), c.f32, c.turns, c.pos, gq.const_data_ptr(), gqs.s,
        gk.const_data_ptr(), gks.s, dq.data_ptr(), dqs.s, dk.data_ptr(), dks.s, w, w + c.D, c.B,
        c.H, c.Hk, c.N, c.D, c.rot, inter, (float)eps, ws.data_ptr(), ws.nbytes(),
        stream_of(c.dev));
    if (st) return PyLong_FromLong(st);
    PyObject *t = PyTuple_New(4);
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(dq));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(dk));
    PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(dw.select(0, 0)));
    PyTuple_SET_ITEM(t, 3, THPVariable_Wrap(dw.select(0, 1)));
    return t;
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ the 8-bit paged cache

struct Kv8 {
  int dev, P, H, page, D, max_pages, stride, B;
  void *k, *v, *ke, *ve;
  const int *table;
  int64_t b;  // sequences

  Kv8(PyObject *cache, PyObject *tab) {
    if (!PyTuple_Check(cache) || PyTuple_GET_SIZE(cache) != 4)
      refuse("the cache must be a Kv8Cache");
    const Tensor &tk = tensor(PyTuple_GET_ITEM(cache, 0), "the cache's k");
    if (tk.dim() != 4 || tk.scalar_type() != at::kFloat8_e4m3fn || !tk.is_cuda() ||
        !tk.is_contiguous())
      refuse(tk, "the cache's k", "a contiguous float8_e4m3fn CUDA tensor [pages, heads, page, D]");
    dev = tk.get_device();
    const Shape s = tk.sizes();
    const Tensor &tv = want(tensor(PyTuple_GET_ITEM(cache, 1), "the cache's v"), "the cache's v",
                            at::kFloat8_e4m3fn, s, dev);
    const Tensor &tke = want(tensor(PyTuple_GET_ITEM(cache, 2), "the cache's k_exp"),
                             "the cache's k_exp", at::kChar, s.slice(0, 2), dev);
    const Tensor &tve = want(tensor(PyTuple_GET_ITEM(cache, 3), "the cache's v_exp"),
                             "the cache's v_exp", at::kChar, s.slice(0, 2), dev);
    const Tensor &t = tensor(tab, "page_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1) ||
        !t.is_cuda() || t.get_device() != dev)
      refuse(t, "page_table", "an int32 tensor [B, pages] with contiguous rows on the cache's device");
    b = t.size(0);
    P = size32(s[0]);
    H = size32(s[1]);
    page = size32(s[2]);
    D = size32(s[3]);
    B = size32(b);
    max_pages = size32(t.size(1));
    // (one sequence's table has no row stride of its own)
    if (b > 1 && t.stride(0) < t.size(1)) refuse(t, "page_table", "rows that do not overlap");
    stride = b > 1 ? size32(t.stride(0)) : max_pages;
    k = tk.data_ptr();
    v = tv.data_ptr();
    ke = tke.data_ptr();
    ve = tve.data_ptr();
    table = t.const_data_ptr<int>();
  }

  // An int32 [B] tensor on the cache's device.
  const int *per_sequence(PyObject *o, const char *name) const {
    return want(tensor(o, name), name, at::kInt, {b}, dev).const_data_ptr<int>();
  }
};

// (cache, k, v, page_table, start, counts)
PyObject *kv8_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 6);
    const Kv8 c(a[0], a[3]);
    const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    if (k.dim() != 4) refuse("k must be [B, Hkv, N, D]");
    const std::array<int64_t, 4> shape = {c.b, c.H, k.size(2), c.D};
    want_rows(k, "k", shape, c.dev);
    want_rows(v, "v", shape, c.dev);
    const int *start = c.per_sequence(a[4], "start");
    const int *counts = a[5] == Py_None ? nullptr : c.per_sequence(a[5], "counts");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const Strides ks(k), vs(v);
    const int st = tk_attn_kv8_write(k.const_data_ptr(), ks.s, v.const_data_ptr(), vs.s, c.k, c.v,
                                     c.ke, c.ve, c.table, start, counts, c.B, c.H,
                                     size32(k.size(2)), c.D, c.P, c.page, c.max_pages, c.stride,
                                     stream_of(c.dev));
    return PyLong_FromLong(st);
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (cache, page_table, lengths, n, out_k, out_v)
PyObject *kv8_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 6);
    const Kv8 c(a[0], a[1]);
    const int *lengths = c.per_sequence(a[2], "lengths");
    int64_t rows;
    if (a[3] != Py_None) {
      rows = PyLong_AsLongLong(a[3]);
      if (rows == -1 && PyErr_Occurred()) return nullptr;
    } else {
      PyObject *given = a[4] != Py_None ? a[4] : a[5];
      if (given == Py_None) refuse("give n, or out_k and out_v");
      const Tensor &t = tensor(given, "out_k");
      if (t.dim() != 4) refuse(t, "out_k", "[B, Hkv, n, D]");
      rows = t.size(2);
    }
    if (rows <= 0) refuse("n must be positive");
    const std::array<int64_t, 4> shape = {c.b, c.H, rows, c.D};
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const auto like = at::TensorOptions().dtype(at::kBFloat16).device(at::kCUDA, c.dev);
    const Tensor k = a[4] == Py_None ? at::zeros(shape, like)
                                     : want(tensor(a[4], "out_k"), "out_k", at::kBFloat16, shape,
                                            c.dev);
    const Tensor v = a[5] == Py_None ? at::zeros(shape, like)
                                     : want(tensor(a[5], "out_v"), "out_v", at::kBFloat16, shape,
                                            c.dev);
    const int st = tk_attn_kv8_read(c.k, c.v, c.ke, c.ve, c.table, lengths, k.data_ptr(),
                                    v.data_ptr(), c.B, c.H, size32(rows), c.D, c.P, c.page,
                                    c.max_pages, c.stride, stream_of(c.dev));
    return st ? PyLong_FromLong(st) : wrap2(k, v);
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (q, cache, page_table, lengths, counts, causal, scale, out, lse, workspace)
PyObject *kv8_attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count_args(n, 10);
    const Kv8 c(a[1], a[2]);
    const Tensor &q = tensor(a[0], "q");
    if (q.dim() != 4 || q.scalar_type() != at::kBFloat16 || !q.is_cuda() || !q.is_contiguous() ||
        q.get_device() != c.dev || q.size(0) != c.b || q.size(3) != c.D || c.H == 0 ||
        q.size(1) % c.H)
      refuse(q, "q",
             "a contiguous bfloat16 tensor [B, H, Nq, D] on the cache's device, with the page "
             "table's B, the cache's D and a multiple of its heads");
    const int *lengths = c.per_sequence(a[3], "lengths");
    const int *counts = a[4] == Py_None ? nullptr : c.per_sequence(a[4], "counts");
    const int causal = truth(a[5]);
    double scale = 1.0 / std::sqrt((double)c.D);
    if (a[6] != Py_None) {
      scale = PyFloat_AsDouble(a[6]);
      if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    }
    const int H = size32(q.size(1)), Nq = size32(q.size(2));
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const Shape ls = q.sizes().slice(0, 3);
    const Tensor o = a[7] == Py_None
                         ? make(q.sizes(), at::kBFloat16, q)
                         : want(tensor(a[7], "out"), "out", at::kBFloat16, q.sizes(), c.dev);
    const Tensor lse = a[8] == Py_None ? make(ls, at::kFloat, q)
                                       : want(tensor(a[8], "lse"), "lse", at::kFloat, ls, c.dev);
    const Tensor ws =
        a[9] == Py_None
            ? make({(int64_t)tk_attn_fwd_kv8_workspace_bytes(c.B, H, c.H, Nq, c.D)}, at::kByte, q)
            : tensor(a[9], "workspace");
    if (!ws.is_cuda() || ws.get_device() != c.dev || !ws.is_contiguous())
      refuse("the workspace must be contiguous and on the tensors' device");
    const int st = tk_attn_fwd_kv8(
        q.const_data_ptr(), c.k, c.v, c.ke, c.ve, c.table, lengths, counts, o.data_ptr(),
        lse.data_ptr<float>(), c.B, H, c.H, Nq, c.D, c.P, c.page, c.max_pages, c.stride,
        (float)scale, causal, ws.data_ptr(), ws.nbytes(), stream_of(c.dev));
    return st ? PyLong_FromLong(st) : wrap2(o, lse);
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define TK_FUNCTION(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), \
                        METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TK_FUNCTION(norm_rope), TK_FUNCTION(norm_rope_bwd),
                         TK_FUNCTION(kv8_write), TK_FUNCTION(kv8_read), TK_FUNCTION(kv8_attend),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tk_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tk_torch(void) { return PyModule_Create(&module); }
