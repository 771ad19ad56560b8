/*
 * The tensor calls of operators.py: checks, output and workspace allocation and the launch on the current stream of
 * the tensors' device, in one native call each.
 *
 * A decoding step makes these calls once per layer and its kernels take 3 to 10 us.  The same checks and allocations
 * made from Python with the C entry points through ctypes took 19 (norm), 12 (cache write) and 23 us (attention) a
 * call, so the host bound the step; from here they take 4.9, 2.2 and 8.9 us, most of it the launches (two in the
 * attention).  PyTorch supplies memory and streams only.
 */
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <stdexcept>
#include <string>

#include "fa.h"

namespace {

using at::Tensor;
using Strides = long long[3];

struct Failed { /* a status of the library, raised as FAError by the package's own check() */
  fa_status status;
  const char* what;
};

[[noreturn]] void refuse(const std::string& why) { throw std::invalid_argument(why); }

int size32(int64_t n) {
  if (n > INT_MAX) refuse("a size of 2^31 or more");
  return (int)n;
}

const Tensor* opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw torch::TypeError(std::string(name) + ": expected a tensor");
  return &THPVariable_Unpack(o);
}

const Tensor& need(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw torch::TypeError(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}

bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x != 0;
}

/* Address of a tensor's elements; NULL for no tensor and for an empty one. */
const void* ptr(const Tensor* t) { return t && t->numel() ? t->const_data_ptr() : nullptr; }
const void* ptr(const Tensor& t) { return ptr(&t); }
void* out(const Tensor& t) { return t.numel() ? t.mutable_data_ptr() : nullptr; }

/* bf16 CUDA tensor [B,H,N,d] with contiguous rows; its strides between batches, heads and rows. */
void rows_of(const Tensor& t, const char* name, Strides st) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 4 || !t.is_cuda())
    refuse(std::string(name) + ": expected a bf16 CUDA tensor of shape [B, H, N, d]");
  if (t.size(3) > 1 && t.stride(3) != 1 && t.numel())
    refuse(std::string(name) + ": the elements of a row must be contiguous");
  for (int i = 0; i < 3; ++i) st[i] = t.stride(i);
}

void ints(const Tensor& t, const char* name, at::IntArrayRef shape, int device) {
  if (t.scalar_type() != at::kInt || t.sizes() != shape || !t.is_cuda() || t.get_device() != device ||
      !t.is_contiguous()) {
    std::string s = std::string(name) + ": expected a contiguous int32 tensor of shape (";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    refuse(s + ") on cuda:" + std::to_string(device));
  }
}

/* Runs `call` with the tensors' device current and without the interpreter's lock. */
template <typename F>
void launch(const char* what, int device, F call) {
  c10::cuda::CUDAGuard guard(device);
  const fa_stream_t stream = (fa_stream_t)c10::cuda::getCurrentCUDAStream(device).stream();
  PyThreadState* state = PyEval_SaveThread();
  const fa_status status = call(stream);
  PyEval_RestoreThread(state);
  if (status != FA_OK) throw Failed{status, what};
}

/* The caller's workspace if it is large enough, else a new one. */
Tensor workspace_of(PyObject* o, size_t bytes, const Tensor& like) {
  if (const Tensor* t = opt(o, "workspace"))
    if (t->device() == like.device() && t->is_contiguous() && t->nbytes() >= bytes && t->nbytes()) return *t;
  return at::empty({(int64_t)(bytes ? bytes : 16)}, like.options().dtype(at::kByte));
}

PyObject* pack(std::initializer_list<const Tensor*> ts) {
  PyObject* tuple = PyTuple_New((Py_ssize_t)ts.size());
  if (!tuple) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = t->defined() ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(tuple);
      throw python_error();
    }
    PyTuple_SET_ITEM(tuple, i++, o);
  }
  return tuple;
}

/* ---------------------------------------------------------------- norm and rotation */

struct Norm {
  const Tensor &q, &k;
  const Tensor *qw, *kw, *cos, *sin, *pos;
  Strides sq, sk;
  int device, bf16 = 0, rope = 0, table_rows = 0, B, H, Hk, N, d;

  Norm(PyObject* oq, PyObject* ok, PyObject* const* rest)
      : q(need(oq, "q")), k(need(ok, "k")), qw(opt(rest[0], "q_weight")), kw(opt(rest[1], "k_weight")),
        cos(opt(rest[2], "cos")), sin(opt(rest[3], "sin")), pos(opt(rest[4], "positions")) {
    rows_of(q, "q", sq);
    rows_of(k, "k", sk);
    device = q.get_device();
    if (k.size(0) != q.size(0) || k.size(2) != q.size(2) || k.size(3) != q.size(3) || k.get_device() != device)
      refuse("k must be [B, Hk, N, d] with the B, N and d of q, on its device");
    B = size32(q.size(0)), H = size32(q.size(1)), Hk = size32(k.size(1)), N = size32(q.size(2)), d = size32(q.size(3));
    for (const Tensor* w : {qw, kw}) {
      if (!w) continue;
      const auto type = w->scalar_type();
      if (w->dim() != 1 || w->size(0) != d || (type != at::kFloat && type != at::kBFloat16) || !w->is_cuda() ||
          w->get_device() != device || !w->is_contiguous())
        refuse("weights must be contiguous fp32 or bf16 tensors [d] on q's device");
      bf16 = type == at::kBFloat16;
    }
    if (qw && kw && qw->scalar_type() != kw->scalar_type()) refuse("both weights must have one type");
    if (!cos != !sin) refuse("cos and sin come together");
    if (cos) {
      for (const Tensor* t : {cos, sin})
        if (t->scalar_type() != at::kFloat || t->dim() != 2 || t->sizes() != cos->sizes() || !t->is_cuda() ||
            t->get_device() != device || !t->is_contiguous())
          refuse("cos and sin must be contiguous fp32 tensors [positions, rope / 2] on q's device");
      table_rows = size32(cos->size(0));
      rope = size32(2 * cos->size(1));
    }
    if (pos) {
      if (!cos) refuse("positions need the cos and sin tables");
      ints(*pos, "positions", {B, N}, device);
    }
    /* no rows and no positions: tables without an address */
    if (cos && !cos->size(0) && (!B || !N)) cos = sin = pos = nullptr, rope = 0;
  }
};

PyObject* qk_norm_rope(PyObject* const* a) { /* q k qw kw cos sin positions eps interleaved */
  const Norm n(a[0], a[1], a + 2);
  const double eps = number(a[7]);
  const int interleaved = truth(a[8]);
  Tensor qo = at::empty({n.B, n.H, n.N, n.d}, n.q.options()), ko = at::empty({n.B, n.Hk, n.N, n.d}, n.q.options());
  launch("fa_qk_norm_rope", n.device, [&](fa_stream_t s) {
    return fa_qk_norm_rope(ptr(n.q), ptr(n.k), out(qo), out(ko), n.sq, n.sk, ptr(n.qw), ptr(n.kw), n.bf16,
                           (const float*)ptr(n.cos), (const float*)ptr(n.sin), n.rope, n.table_rows, interleaved,
                           (const int*)ptr(n.pos), n.B, n.H, n.Hk, n.N, n.d, (float)eps, s);
  });
  return pack({&qo, &ko});
}

PyObject* qk_norm_rope_backward(PyObject* const* a) { /* q k dq_out dk_out qw kw cos sin positions eps interleaved ws */
  const Norm n(a[0], a[1], a + 4);
  const Tensor &gq = need(a[2], "dq_out"), &gk = need(a[3], "dk_out");
  Strides sgq, sgk, sdq, sdk;
  rows_of(gq, "dq_out", sgq);
  rows_of(gk, "dk_out", sgk);
  if (gq.sizes() != n.q.sizes() || gq.get_device() != n.device) refuse("dq_out: expected the shape and device of q");
  if (gk.sizes() != n.k.sizes() || gk.get_device() != n.device) refuse("dk_out: expected the shape and device of k");
  const double eps = number(a[9]);
  const int interleaved = truth(a[10]);
  Tensor dq = at::empty_like(n.q), dk = at::empty_like(n.k), dqw, dkw, ws;
  if (n.qw) dqw = at::empty_like(*n.qw);
  if (n.kw) dkw = at::empty_like(*n.kw);
  if (n.qw || n.kw) {
    const size_t bytes = fa_qk_norm_rope_bwd_workspace_size(n.B, n.H, n.Hk, n.N, n.d);
    if (bytes == (size_t)-1) throw Failed{FA_ERR_UNSUPPORTED, "fa_qk_norm_rope_bwd_workspace_size"};
    ws = workspace_of(a[11], bytes, n.q);
  }
  rows_of(dq, "dq", sdq);
  rows_of(dk, "dk", sdk);
  launch("fa_qk_norm_rope_bwd", n.device, [&](fa_stream_t s) {
    return fa_qk_norm_rope_bwd(ptr(n.q), ptr(n.k), ptr(gq), ptr(gk), out(dq), out(dk), n.sq, n.sk, sgq, sgk, sdq, sdk,
                               ptr(n.qw), ptr(n.kw), n.qw ? out(dqw) : nullptr, n.kw ? out(dkw) : nullptr, n.bf16,
                               (const float*)ptr(n.cos), (const float*)ptr(n.sin), n.rope, n.table_rows, interleaved,
                               (const int*)ptr(n.pos), n.B, n.H, n.Hk, n.N, n.d, (float)eps,
                               ws.defined() ? ws.mutable_data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, s);
  });
  return pack({&dq, &dk, &dqw, &dkw});
}

/* ---------------------------------------------------------------- the cache */

struct Cache {
  fa_cache c;
  int device;

  explicit Cache(PyObject* const* a) { /* k v k_exp v_exp */
    const Tensor &k = need(a[0], "a cache's k"), &v = need(a[1], "a cache's v");
    const auto type = k.scalar_type();
    if ((type != at::kBFloat16 && type != at::kFloat8_e4m3fn) || v.scalar_type() != type || k.dim() != 4 ||
        k.sizes() != v.sizes() || !k.is_cuda() || v.device() != k.device() || !k.is_contiguous() || !v.is_contiguous())
      refuse("a cache's k and v must be contiguous bf16 or float8_e4m3fn CUDA tensors [pages, Hk, page_size, d] of one "
             "type and device");
    const bool fp8 = type == at::kFloat8_e4m3fn;
    const Tensor* e[2] = {opt(a[2], "a cache's k_exp"), opt(a[3], "a cache's v_exp")};
    for (const Tensor* t : e) {
      if ((t != nullptr) != fp8) refuse("an e4m3 cache has exponent bytes k_exp and v_exp, a bf16 cache has none");
      if (fp8 && (t->scalar_type() != at::kByte || t->sizes() != k.sizes().slice(0, 3) || t->device() != k.device() ||
                  !t->is_contiguous()))
        refuse("exponent bytes must be contiguous uint8 tensors [pages, Hk, page_size] on the cache's device");
    }
    c = fa_cache{out(k), out(v), fp8 ? (unsigned char*)out(*e[0]) : nullptr, fp8 ? (unsigned char*)out(*e[1]) : nullptr,
                 fp8 ? FA_CACHE_E4M3 : FA_CACHE_BF16, size32(k.size(0)), size32(k.size(1)), size32(k.size(2)),
                 size32(k.size(3))};
    device = k.get_device();
  }
};

struct Table {
  const int *table, *lens, *n_new = nullptr;
  int B, cols;
  long long stride;

  Table(const Cache& c, PyObject* ot, PyObject* ol, PyObject* on) {
    const Tensor &t = need(ot, "table"), &l = need(ol, "lens");
    if (t.dim() != 2 || t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != c.device ||
        (t.size(1) > 1 && t.stride(1) != 1))
      refuse("the page table must be an int32 tensor [B, columns] on the cache's device, rows contiguous");
    B = size32(t.size(0)), cols = size32(t.size(1)), stride = t.stride(0);
    ints(l, "lens", {B}, c.device);
    table = (const int*)ptr(t), lens = (const int*)ptr(l);
    if (const Tensor* n = on ? opt(on, "n_new") : nullptr) {
      ints(*n, "n_new", {B}, c.device);
      n_new = (const int*)ptr(n);
    }
  }
};

PyObject* cache_write(PyObject* const* a) { /* ck cv ke ve k v table lens n_new */
  const Tensor &k = need(a[4], "k"), &v = need(a[5], "v");
  Strides sk, sv;
  rows_of(k, "k", sk);
  rows_of(v, "v", sv);
  const Cache c(a);
  const Table t(c, a[6], a[7], a[8]);
  if (v.sizes() != k.sizes() || k.get_device() != c.device || v.get_device() != c.device || k.size(0) != t.B ||
      k.size(1) != c.c.Hk || k.size(3) != c.c.d)
    refuse("k and v must be [B, Hk, T, d] with the table's B and the cache's Hk and d, on its device");
  const int T = size32(k.size(2));
  launch("fa_cache_write", c.device, [&](fa_stream_t s) {
    return fa_cache_write(&c.c, ptr(k), ptr(v), sk, sv, t.B, T, t.table, t.cols, t.stride, t.lens, t.n_new, s);
  });
  Py_RETURN_NONE;
}

PyObject* cache_read(PyObject* const* a) { /* ck cv ke ve table lens length */
  const Cache c(a);
  const Table t(c, a[4], a[5], nullptr);
  const long long length = PyLong_AsLongLong(a[6]);
  if (length == -1 && PyErr_Occurred()) throw python_error();
  if (length < 0) refuse("length must not be negative");
  const int n = size32(length);
  const auto opts = THPVariable_Unpack(a[0]).options().dtype(at::kBFloat16);
  Tensor k = at::empty({t.B, c.c.Hk, n, c.c.d}, opts), v = at::empty({t.B, c.c.Hk, n, c.c.d}, opts);
  launch("fa_cache_read", c.device, [&](fa_stream_t s) {
    return fa_cache_read(&c.c, out(k), out(v), t.B, n, t.table, t.cols, t.stride, t.lens, s);
  });
  return pack({&k, &v});
}

/* ---------------------------------------------------------------- attention of drafted tokens */

PyObject* attention_tree(PyObject* const* a) { /* q ck cv ke ve table lens tree n_new scale workspace */
  const Tensor& q = need(a[0], "q");
  if (q.scalar_type() != at::kBFloat16 || q.dim() != 4 || !q.is_cuda() || !q.is_contiguous())
    refuse("q: expected a contiguous bf16 CUDA tensor of shape [B, H, T, d]");
  const Cache c(a + 1);
  const Table t(c, a[5], a[6], a[8]);
  const int H = size32(q.size(1)), T = size32(q.size(2)), d = c.c.d;
  if (q.size(0) != t.B || q.size(3) != d || q.get_device() != c.device)
    refuse("q must be [B, H, T, d] with the table's B and the cache's d, on its device");
  if (H && (c.c.Hk == 0 || H % c.c.Hk)) refuse("the heads of q must be a multiple of the cache's");
  const Tensor* tree = opt(a[7], "tree");
  long long stride = 0;
  if (tree) {
    const int64_t W = ((int64_t)T + 63) / 64, batched[3] = {t.B, T, W};
    const at::IntArrayRef shape(batched);
    if (tree->scalar_type() != at::kLong || !tree->is_cuda() || tree->get_device() != c.device ||
        !tree->is_contiguous() || (tree->sizes() != shape && tree->sizes() != shape.slice(1)))
      refuse("tree must be a contiguous int64 tensor [B, T, W] or [T, W], W = ceil(T / 64), on q's device");
    stride = tree->dim() == 3 ? T * W : 0;
  }
  const double scale = a[9] == Py_None ? 1.0 / std::sqrt((double)d) : number(a[9]);
  size_t bytes = fa_fwd_tree_workspace_size(t.B, H, c.c.Hk, T, d);
  if (bytes == (size_t)-1) bytes = 0; /* sizes that the call below refuses, with its own status */
  const Tensor ws = workspace_of(a[10], bytes, q);
  Tensor o = at::empty(q.sizes(), q.options()), l = at::empty({t.B, H, T}, q.options().dtype(at::kFloat));
  launch("fa_fwd_tree", c.device, [&](fa_stream_t s) {
    return fa_fwd_tree(ptr(q), &c.c, out(o), (float*)out(l), t.B, H, T, t.table, t.cols, t.stride, t.lens, t.n_new,
                       (const unsigned long long*)ptr(tree), stride, (float)scale, ws.mutable_data_ptr(), ws.nbytes(),
                       s);
  });
  return pack({&o, &l});
}

/* ---------------------------------------------------------------- the module */

void raise_status(const Failed& f) {
  PyObject* package = PyImport_ImportModule(FA_PACKAGE);
  PyObject* r = package ? PyObject_CallMethod(package, "check", "is", (int)f.status, f.what) : nullptr;
  Py_XDECREF(r);
  Py_XDECREF(package);
}

template <PyObject* (*Call)(PyObject* const*), int Args>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != Args) throw torch::TypeError("expected " + std::to_string(Args) + " arguments");
  try {
    return Call(args);
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Failed& f) {
    raise_status(f);
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name, args) {#name, (PyCFunction)(void*)entry<name, args>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(qk_norm_rope, 9), ENTRY(qk_norm_rope_backward, 12), ENTRY(cache_write, 9),
                         ENTRY(cache_read, 7),   ENTRY(attention_tree, 11),        {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "tensor_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_tensor_calls() { return PyModule_Create(&module); }
