// Argument checks of the binding's latency-bound calls, next to PyTorch's tensors: a decode step calls
// them by the dozen, and reading a tensor's shape, type, strides and address from Python costs more
// than the launch (half a microsecond a tensor; a few nanoseconds here).  Each function checks its
// tensors, calls the entry point of libmsa.so with their addresses and returns its status; what does
// not fit raises ValueError before the library is called.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/msa.h"
#include "overlap.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  throw Refused(buf);
}

struct Entry {
  decltype(&msa_rotate) rotate;
  decltype(&msa_head_norm_rotate) head_norm_rotate;
  decltype(&msa_head_norm_append) head_norm_append;
  decltype(&msa_head_norm_rotate_grad) head_norm_rotate_grad;
  decltype(&msa_tree_plan) tree_plan;
  decltype(&msa_tree_attend) tree_attend;
  decltype(&msa_tree_commit) tree_commit;
} entry;

std::string text(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// what the tensors of a call share
struct Call {
  c10::Device dev;
  explicit Call(const at::Tensor& t) : dev(t.device()) {}
  // checked last, so that a host tensor of the wrong shape is told its shape
  void on_current_device(const char* name) const {
    if (!dev.is_cuda()) refuse("%s: expected a CUDA tensor, got one on %s", name, dev.str().c_str());
    if (dev.index() != c10::cuda::current_device())
      refuse("%s: on %s, but the current device is cuda:%d", name, dev.str().c_str(), (int)c10::cuda::current_device());
  }
  void* stream(PyObject* o) const {  // None: the current stream; else its handle
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw Refused("");
    return reinterpret_cast<void*>(v);
  }
  void* flat(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type) const {
    if (t.sizes() != shape || t.scalar_type() != type || t.device() != dev || !t.is_contiguous())
      refuse("%s: expected a contiguous %s tensor of shape %s on %s, got %s %s on %s%s", name, c10::toString(type),
             text(shape).c_str(), dev.str().c_str(), c10::toString(t.scalar_type()), text(t.sizes()).c_str(),
             t.device().str().c_str(), t.is_contiguous() ? "" : ", not contiguous");
    return t.data_ptr();
  }
  void* flat(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type) const {
    return flat(tensor(o, name), name, shape, type);
  }
  void* flat_or_null(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type) const {
    return o == Py_None ? nullptr : flat(tensor(o, name), name, shape, type);
  }
  // heads [rows, heads, head_dim] with any strides but contiguous elements, and their output (or none)
  msa_heads heads(const at::Tensor& x, const at::Tensor* out, const char* name, int64_t rows, int64_t head_dim,
                  at::ScalarType type) const {
    if (x.dim() != 3 || x.size(0) != rows || x.size(2) != head_dim || x.size(1) < 1 || x.scalar_type() != type ||
        x.device() != dev || x.stride(2) != 1)
      refuse("%s: expected [%lld, heads, %lld] %s on %s with contiguous head elements, got %s %s on %s, strides %s", name,
             (long long)rows, (long long)head_dim, c10::toString(type), dev.str().c_str(), text(x.sizes()).c_str(),
             c10::toString(x.scalar_type()), x.device().str().c_str(), text(x.strides()).c_str());
    if (x.size(1) > INT32_MAX) refuse("%s: expected fewer than 2^31 heads, got %lld", name, (long long)x.size(1));
    msa_heads h{};
    h.in = x.data_ptr();
    h.in_row = x.stride(0);
    h.in_head = x.stride(1);
    h.heads = (int32_t)x.size(1);
    if (out) {
      if (out->sizes() != x.sizes() || out->scalar_type() != type || out->device() != dev || out->stride(2) != 1)
        refuse("the output of %s: expected %s %s on %s with contiguous head elements, got %s %s on %s, strides %s", name,
               text(x.sizes()).c_str(), c10::toString(type), dev.str().c_str(), text(out->sizes()).c_str(),
               c10::toString(out->scalar_type()), out->device().str().c_str(), text(out->strides()).c_str());
      h.out = out->data_ptr();
      h.out_row = out->stride(0);
      h.out_head = out->stride(1);
    }
    return h;
  }
};

msa_dtype dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MSA_BF16;
    case at::kHalf: return MSA_FP16;
    case at::kFloat: return MSA_FP32;
    default: refuse("%s: expected BFloat16, Half or Float, got %s", name, c10::toString(t.scalar_type()));
  }
}

// What the tensors of one call may share: an output nothing with another output or input (but with its
// own input in place, which the library checks).  Kernels of many CTAs would read what others have written.
struct Place : msa::Blocks {  // and the bytes that it reaches over (a tensor lies in one allocation: 64 bits hold them)
  uintptr_t end;
  Place(const void* p, int64_t rows, int64_t heads, int64_t row, int64_t head, int64_t width)
      : Blocks{reinterpret_cast<uintptr_t>(p), rows, heads, row, head, width},
        end(p && rows > 0 ? base + (rows - 1) * row + (heads - 1) * head + width : base) {}
};
struct Apart {
  int64_t rows, head_dim, size;
  Place in(const msa_heads& h) const {
    return {h.in, rows, h.heads, h.in_row * size, h.in_head * size, head_dim * size};
  }
  Place out(const msa_heads& h) const {
    return {h.out, rows, h.heads, h.out_row * size, h.out_head * size, head_dim * size};
  }
  static Place vec(const void* p, int64_t bytes) { return {p, 1, 1, 0, 0, bytes}; }  // nothing where p is null
  static void check(const Place& written, const char* name, const Place& other, const char* other_name) {
    if (written.base < other.end && other.base < written.end && msa::share_bytes(written, other))
      refuse("%s and %s overlap: expected tensors apart", name, other_name);
  }
  // an output against the small inputs of the call
  void small(const Place& written, const char* name, const void* positions, const void* q_weight,
             const void* k_weight) const {
    check(written, name, vec(positions, rows * 4), "positions");
    check(written, name, vec(q_weight, head_dim * size), "q_weight");
    check(written, name, vec(k_weight, head_dim * size), "k_weight");
  }
  // the outputs of the query and key heads (k.heads == 0: none)
  void pair(const msa_heads& q, const msa_heads& k, const void* positions, const void* q_weight, const void* k_weight) const {
    const Place q_out = out(q);
    small(q_out, "out", positions, q_weight, k_weight);
    if (!k.heads) return;
    const Place k_out = out(k);
    small(k_out, "k_out", positions, q_weight, k_weight);
    check(q_out, "out", in(k), "k");
    check(k_out, "k_out", in(q), "q");
    check(q_out, "out", k_out, "k_out");
  }
};

// a ctypes structure by its buffer
template <typename S>
struct Struct {
  Py_buffer b{};
  explicit Struct(PyObject* o) {
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Refused("");
    if (b.len != (Py_ssize_t)sizeof(S)) {
      PyBuffer_Release(&b);
      refuse("a structure of %zu bytes was expected, got %zd", sizeof(S), b.len);
    }
  }
  ~Struct() { PyBuffer_Release(&b); }
  Struct(const Struct&) = delete;
  const S* operator->() const { return static_cast<const S*>(b.buf); }
  const S* get() const { return static_cast<const S*>(b.buf); }
};

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused("");
  return v;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused("");
  return v;
}

// The library's call without the interpreter's lock: a launch may have to wait (for a place in the
// stream's queue, for the first load of a kernel), and what the queue waits for may be a host function that
// needs the interpreter.  Nothing of Python is touched meanwhile: the arguments are read before.
template <typename F, typename... A>
long unlocked(F f, A... a) {
  PyThreadState* state = PyEval_SaveThread();
  const msa_status st = f(a...);
  PyEval_RestoreThread(state);
  return st;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused("");
  return v != 0;
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// the parts that the rotation and norm calls share: rows, positions, dtype
struct Rows {
  const at::Tensor& q;
  Call call;
  msa_dtype code;
  at::ScalarType type;
  int64_t rows;
  const int32_t* pos;
  Rows(PyObject* q_, PyObject* positions, const msa_rotary* rot)
      : q(tensor(q_, "q")), call(q), code(dtype_of(q, "q")), type(q.scalar_type()) {
    if (q.dim() != 3) refuse("q: expected [rows, heads, %d], got %s", rot->head_dim, text(q.sizes()).c_str());
    rows = q.size(0);
    pos = static_cast<const int32_t*>(call.flat(positions, "positions", {rows}, at::kInt));
  }
};

// rotate(rot, q, positions, k, grad, out, k_out, stream)
PyObject* py_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    Struct<msa_rotary> rot(a[0]);
    Rows r(a[1], a[2], rot.get());
    const int D = rot->head_dim;
    const msa_heads q = r.call.heads(r.q, &tensor(a[5], "out"), "q", r.rows, D, r.type);
    msa_heads k{};
    if (a[3] != Py_None) k = r.call.heads(tensor(a[3], "k"), &tensor(a[6], "k_out"), "k", r.rows, D, r.type);
    const bool grad = truth(a[4]);
    Apart{r.rows, D, r.q.element_size()}.pair(q, k, r.pos, nullptr, nullptr);
    r.call.on_current_device("q");
    return unlocked(entry.rotate, rot.get(), r.code, &q, a[3] != Py_None ? &k : nullptr, r.rows, r.pos, (int32_t)grad,
                    r.call.stream(a[7]));
  });
}

// head_norm_rotate(rot, q, k, q_weight, k_weight, positions, eps, weight_offset, out, k_out, stream)
PyObject* py_head_norm_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    Struct<msa_rotary> rot(a[0]);
    Rows r(a[1], a[5], rot.get());
    const int D = rot->head_dim;
    const msa_heads q = r.call.heads(r.q, &tensor(a[8], "out"), "q", r.rows, D, r.type);
    msa_heads k{};
    if (a[2] != Py_None) k = r.call.heads(tensor(a[2], "k"), &tensor(a[9], "k_out"), "k", r.rows, D, r.type);
    const void* wq = r.call.flat_or_null(a[3], "q_weight", {D}, r.type);
    const void* wk = r.call.flat_or_null(a[4], "k_weight", {D}, r.type);
    const float eps = (float)number(a[6]), off = (float)number(a[7]);
    Apart{r.rows, D, r.q.element_size()}.pair(q, k, r.pos, wq, wk);
    r.call.on_current_device("q");
    return unlocked(entry.head_norm_rotate, rot.get(), r.code, &q, a[2] != Py_None ? &k : nullptr, r.rows, wq, wk, off,
                    eps, r.pos, r.call.stream(a[10]));
  });
}

// head_norm_append(rot, q, k, v, q_weight, k_weight, positions, slots, K_loc, V_loc, eps, weight_offset, out, stream)
PyObject* py_head_norm_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    Struct<msa_rotary> rot(a[0]);
    Rows r(a[1], a[6], rot.get());
    const int D = rot->head_dim;
    const msa_heads q = r.call.heads(r.q, &tensor(a[12], "out"), "q", r.rows, D, r.type);
    const at::Tensor &kt = tensor(a[2], "k"), &vt = tensor(a[3], "v"), &kc = tensor(a[8], "K_loc");
    const msa_heads k = r.call.heads(kt, nullptr, "k", r.rows, D, r.type);
    const msa_heads v = r.call.heads(vt, nullptr, "v", r.rows, D, r.type);
    if (vt.size(1) != kt.size(1)) refuse("v: expected k's shape %s, got %s", text(kt.sizes()).c_str(), text(vt.sizes()).c_str());
    const void* wq = r.call.flat_or_null(a[4], "q_weight", {D}, r.type);
    const void* wk = r.call.flat_or_null(a[5], "k_weight", {D}, r.type);
    const auto* slots = static_cast<const int32_t*>(r.call.flat(a[7], "slots", {r.rows}, at::kInt));
    if (kc.dim() != 4) refuse("K_loc: expected [B, t_loc_max, n_kv, head_dim], got %s", text(kc.sizes()).c_str());
    const int64_t cache[4] = {kc.size(0), kc.size(1), kt.size(1), D};
    void* K = r.call.flat(kc, "K_loc", cache, r.type);
    void* V = r.call.flat(a[9], "V_loc", cache, r.type);
    const float eps = (float)number(a[10]), off = (float)number(a[11]);
    const Apart t{r.rows, D, r.q.element_size()};
    const Place q_in = t.in(q), k_in = t.in(k), v_in = t.in(v), q_out = t.out(q), at = t.vec(slots, r.rows * 4);
    t.small(q_out, "out", r.pos, wq, wk);
    t.check(q_out, "out", at, "slots");
    t.check(q_out, "out", k_in, "k");
    t.check(q_out, "out", v_in, "v");
    for (int i = 0; i < 2; ++i) {
      const char* name = i ? "V_loc" : "K_loc";
      const Place c = t.vec(i ? V : K, kc.nbytes());
      t.small(c, name, r.pos, wq, wk);
      t.check(c, name, at, "slots");
      t.check(c, name, q_in, "q");
      t.check(c, name, k_in, "k");
      t.check(c, name, v_in, "v");
      t.check(c, name, q_out, "out");
    }
    r.call.on_current_device("q");
    return unlocked(entry.head_norm_append, rot.get(), r.code, &q, &k, &v, r.rows, wq, wk, off, eps, r.pos, slots, K, V,
                    (int32_t)cache[0], (int32_t)cache[1], r.call.stream(a[13]));
  });
}

// a workspace tensor: its 256-byte aligned address and the bytes from there
void workspace(PyObject* o, void** ws, size_t* bytes) {
  const at::Tensor& t = tensor(o, "ws");
  if (!t.is_contiguous()) refuse("ws: expected a contiguous tensor, got strides %s", text(t.strides()).c_str());
  const size_t p = reinterpret_cast<size_t>(t.data_ptr()), at = (p + 255) & ~size_t(255);
  const size_t have = t.nbytes();
  *ws = reinterpret_cast<void*>(at);
  *bytes = have > at - p ? have - (at - p) : 0;
}

// head_norm_rotate_grad(rot, q, k, q_weight, k_weight, positions, dq, dk, eps, weight_offset, gq, gk, gwq, gwk, ws, stream)
PyObject* py_head_norm_rotate_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    Struct<msa_rotary> rot(a[0]);
    Rows r(a[1], a[5], rot.get());
    const int D = rot->head_dim;
    const bool has_k = a[2] != Py_None;
    if (has_k != (a[7] != Py_None)) refuse("k and dk go together: expected both or neither");
    const msa_heads q = r.call.heads(r.q, nullptr, "q", r.rows, D, r.type);
    const at::Tensor& dqt = tensor(a[6], "dq");
    const msa_heads dq = r.call.heads(dqt, &tensor(a[10], "out[0]"), "dq", r.rows, D, r.type);
    if (dqt.size(1) != r.q.size(1)) refuse("dq: expected q's shape %s, got %s", text(r.q.sizes()).c_str(), text(dqt.sizes()).c_str());
    msa_heads k{}, dk{};
    if (has_k) {
      const at::Tensor &kt = tensor(a[2], "k"), &dkt = tensor(a[7], "dk");
      k = r.call.heads(kt, nullptr, "k", r.rows, D, r.type);
      dk = r.call.heads(dkt, &tensor(a[11], "out[1]"), "dk", r.rows, D, r.type);
      if (dkt.size(1) != kt.size(1)) refuse("dk: expected k's shape %s, got %s", text(kt.sizes()).c_str(), text(dkt.sizes()).c_str());
    }
    const void* wq = r.call.flat_or_null(a[3], "q_weight", {D}, r.type);
    const void* wk = r.call.flat_or_null(a[4], "k_weight", {D}, r.type);
    auto* gwq = static_cast<float*>(r.call.flat_or_null(a[12], "out[2]", {D}, at::kFloat));
    auto* gwk = static_cast<float*>(r.call.flat_or_null(a[13], "out[3]", {D}, at::kFloat));
    const float eps = (float)number(a[8]), off = (float)number(a[9]);
    void* ws;
    size_t bytes;
    workspace(a[14], &ws, &bytes);
    if (tensor(a[14], "ws").device() != r.call.dev) refuse("ws: expected on %s", r.call.dev.str().c_str());
    const Apart t{r.rows, D, r.q.element_size()};
    const Place q_in = t.in(q), gq = t.out(dq), sums[2] = {t.vec(gwq, D * 4), t.vec(gwk, D * 4)};
    t.small(gq, "out[0]", r.pos, wq, wk);
    if (!msa::same_blocks(gq, q_in)) t.check(gq, "out[0]", q_in, "q");  // in place: a lane reads its elements of both first
    if (has_k) {
      const Place k_in = t.in(k), gk = t.out(dk);
      t.small(gk, "out[1]", r.pos, wq, wk);
      if (!msa::same_blocks(gk, k_in)) t.check(gk, "out[1]", k_in, "k");
      t.check(gq, "out[0]", k_in, "k");
      t.check(gq, "out[0]", t.in(dk), "dk");
      t.check(gk, "out[1]", q_in, "q");
      t.check(gk, "out[1]", t.in(dq), "dq");
      t.check(gq, "out[0]", gk, "out[1]");
      for (const Place& w : sums) t.check(w, "a weight's gradient", gk, "out[1]");
    }
    for (const Place& w : sums) t.check(w, "a weight's gradient", gq, "out[0]");
    t.check(sums[0], "out[2]", sums[1], "out[3]");
    r.call.on_current_device("q");
    return unlocked(entry.head_norm_rotate_grad, rot.get(), r.code, &q, has_k ? &k : nullptr, &dq,
                    has_k ? &dk : nullptr, r.rows, wq, wk, off, eps, r.pos, gwq, gwk, ws, bytes, r.call.stream(a[15]));
  });
}

// tree_plan(parents, loc_len, pos_offset, n_draft, mask, positions, stream)
PyObject* py_tree_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const at::Tensor& parents = tensor(a[0], "parents");
    Call c(parents);
    if (parents.dim() != 2) refuse("parents: expected [B, M], got %s", text(parents.sizes()).c_str());
    const int64_t B = parents.size(0), M = parents.size(1);
    const auto* par = static_cast<const int32_t*>(c.flat(parents, "parents", {B, M}, at::kInt));
    const auto* loc = static_cast<const int32_t*>(c.flat(a[1], "loc_len", {B}, at::kInt));
    const auto* nd = static_cast<const int32_t*>(c.flat_or_null(a[3], "n_draft", {B}, at::kInt));
    auto* mask = static_cast<int32_t*>(c.flat(a[4], "out[0]", {B, M, (M + 31) / 32}, at::kInt));
    auto* pos = static_cast<int32_t*>(c.flat(a[5], "out[1]", {B, M}, at::kInt));
    const long long off = integer(a[2]);
    if (off < 0 || off > INT32_MAX) refuse("pos_offset: expected an int32 >= 0, got %lld", off);
    c.on_current_device("parents");
    return unlocked(entry.tree_plan, par, nd, loc, (int32_t)B, (int32_t)M, (int32_t)off, mask, pos, c.stream(a[6]));
  });
}

// tree_attend(dims, q, K_draft, V_draft, mask, K_loc, V_loc, loc_len, n_draft, K_bar, V_bar, chunk_off, topk_idx,
//             softmax_scale, out, ws, stream)
PyObject* py_tree_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    Struct<msa_dims> d(a[0]);
    const at::Tensor& q = tensor(a[1], "q");
    Call c(q);
    if (q.dim() != 4) refuse("q: expected [B, M, n_q, head_dim], got %s", text(q.sizes()).c_str());
    const int64_t B = q.size(0), M = q.size(1), n_kv = d->n_kv, D = d->head_dim;
    const int64_t rows[4] = {B, M, d->n_q, D}, drafts[4] = {B, M, n_kv, D};
    const auto bf = at::kBFloat16, i32 = at::kInt;
    const void* qp = c.flat(q, "q", rows, bf);
    const void *kd = c.flat(a[2], "K_draft", drafts, bf), *vd = c.flat(a[3], "V_draft", drafts, bf);
    const auto* mask = static_cast<const int32_t*>(c.flat(a[4], "mask", {B, M, (M + 31) / 32}, i32));
    const auto* loc = static_cast<const int32_t*>(c.flat(a[7], "loc_len", {B}, i32));
    const auto* nd = static_cast<const int32_t*>(c.flat_or_null(a[8], "n_draft", {B}, i32));
    if ((a[5] == Py_None) != (a[6] == Py_None)) refuse("K_loc and V_loc go together: expected both or neither");
    int64_t t_loc = 0;
    const void *kl = nullptr, *vl = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& K = tensor(a[5], "K_loc");
      t_loc = K.dim() == 4 ? K.size(1) : -1;
      const int64_t cache[4] = {B, t_loc, n_kv, D};
      kl = c.flat(K, "K_loc", cache, bf);
      vl = c.flat(a[6], "V_loc", cache, bf);
      if (t_loc == 0) kl = vl = nullptr;
    }
    int given = 0;
    for (int i = 9; i < 13; ++i) given += a[i] != Py_None;
    if (given != 0 && given != 4) refuse("K_bar, V_bar, chunk_off and topk_idx go together: expected all or none");
    int64_t k = 0, n_docs = 0, n_chunks = 0;
    const void *kb = nullptr, *vb = nullptr;
    const int32_t *co = nullptr, *top = nullptr;
    if (given) {
      const at::Tensor &K = tensor(a[9], "K_bar"), &off = tensor(a[11], "chunk_off"), &idx = tensor(a[12], "topk_idx");
      if (K.dim() != 3 || idx.dim() != 2 || off.dim() != 1)
        refuse("expected K_bar [n_chunks, n_kv, head_dim], chunk_off [n_docs + 1], topk_idx [B, k]");
      k = idx.size(1);
      n_docs = off.size(0) - 1;
      n_chunks = K.size(0);
      const int64_t memory[3] = {n_chunks, n_kv, D};
      kb = c.flat(K, "K_bar", memory, bf);
      vb = c.flat(a[10], "V_bar", memory, bf);
      co = static_cast<const int32_t*>(c.flat(off, "chunk_off", {n_docs + 1}, i32));
      top = static_cast<const int32_t*>(c.flat(idx, "topk_idx", {B, k}, i32));
      if (n_chunks > INT32_MAX) refuse("K_bar: expected fewer than 2^31 pooled rows");
      if (k == 0) {
        kb = vb = nullptr;
        co = top = nullptr;
      }
    }
    if (B > INT32_MAX || M > INT32_MAX || t_loc > INT32_MAX) refuse("expected sizes below 2^31");
    void* out = c.flat(a[14], "out", rows, bf);
    const float scale = (float)number(a[13]);
    void* ws;
    size_t bytes;
    workspace(a[15], &ws, &bytes);
    if (tensor(a[15], "ws").device() != c.dev) refuse("ws: expected on %s", c.dev.str().c_str());
    c.on_current_device("q");
    return unlocked(entry.tree_attend, d.get(), qp, kd, vd, mask, nd, (int32_t)B, (int32_t)M, kl, vl, loc,
                    (int32_t)t_loc, kb, vb, co, (int32_t)n_docs, (int32_t)n_chunks, top, (int32_t)k, scale, out, ws,
                    bytes, c.stream(a[16]));
  });
}

// tree_commit(K_draft, V_draft, path, n_path, K_loc, V_loc, loc_len, out, stream)
PyObject* py_tree_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const at::Tensor &kd = tensor(a[0], "K_draft"), &path = tensor(a[2], "path"), &kl = tensor(a[4], "K_loc");
    Call c(kd);
    if (kd.dim() != 4 || kl.dim() != 4 || path.dim() != 2)
      refuse("expected K_draft [B, M, n_kv, head_dim], K_loc [B, t_loc_max, n_kv, head_dim], path [B, A]");
    const int64_t B = kd.size(0), M = kd.size(1), n_kv = kd.size(2), D = kd.size(3), T = kl.size(1), A = path.size(1);
    const int64_t drafts[4] = {B, M, n_kv, D}, cache[4] = {B, T, n_kv, D};
    const auto bf = at::kBFloat16, i32 = at::kInt;
    if (B > INT32_MAX || M > INT32_MAX || T > INT32_MAX || n_kv > INT32_MAX || D > INT32_MAX) refuse("expected sizes below 2^31");
    const void *kp = c.flat(kd, "K_draft", drafts, bf), *vp = c.flat(a[1], "V_draft", drafts, bf);
    const auto* pp = static_cast<const int32_t*>(c.flat(path, "path", {B, A}, i32));
    const auto* np = static_cast<const int32_t*>(c.flat(a[3], "n_path", {B}, i32));
    void *K = c.flat(kl, "K_loc", cache, bf), *V = c.flat(a[5], "V_loc", cache, bf);
    const auto* loc = static_cast<const int32_t*>(c.flat(a[6], "loc_len", {B}, i32));
    auto* out = static_cast<int32_t*>(c.flat(a[7], "out", {B}, i32));
    c.on_current_device("K_draft");
    msa_dims d{};  // of which only the KV heads matter
    d.hidden = 64;
    d.n_q = d.n_kv = (int32_t)n_kv;
    d.head_dim = (int32_t)D;
    d.n_r = 1;
    d.d_r = d.chunk = 64;
    d.rope_base = 1e6f;
    return unlocked(entry.tree_commit, &d, kp, vp, pp, np, (int32_t)B, (int32_t)M, (int32_t)A, K, V, loc, (int32_t)T,
                    out, c.stream(a[8]));
  });
}

// bind(path): the entry points of the library at path
PyObject* py_bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return nullptr;
  }
  bool ok = true;
  auto get = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(h, name));
    ok = ok && f;
  };
  get(entry.rotate, "msa_rotate");
  get(entry.head_norm_rotate, "msa_head_norm_rotate");
  get(entry.head_norm_append, "msa_head_norm_append");
  get(entry.head_norm_rotate_grad, "msa_head_norm_rotate_grad");
  get(entry.tree_plan, "msa_tree_plan");
  get(entry.tree_attend, "msa_tree_attend");
  get(entry.tree_commit, "msa_tree_commit");
  if (!ok) {
    PyErr_SetString(PyExc_ImportError, "libmsa.so lacks an entry point");
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rotate), FAST(head_norm_rotate), FAST(head_norm_append), FAST(head_norm_rotate_grad),
                         FAST(tree_plan), FAST(tree_attend), FAST(tree_commit), {"bind", py_bind, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", "argument checks and calls of libmsa.so", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&module); }
