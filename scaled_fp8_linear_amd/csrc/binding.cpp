// CPython binding of the row operators (layer norm, router, expert exchange, activation) and of the
// experts' products: the checks of tensors, their addresses, and the call of the C entry point, in
// one native call. For one token the kernels take 3 us and their launch 2.7 us of host time; the
// same checks in Python took 3.4 us more. Entry points come in as addresses (bind), so the library
// is loaded once, elsewhere.
//
// Every function raises ValueError before anything is enqueued if a tensor does not fit, and
// the binding's own error for a status other than 0. Outputs that are None and wanted are
// allocated by torch in the call, in the pool of the stream that writes them: as at::empty does on
// the current stream, by the caller's function (bind's "new") on one that was passed.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/Allocator.h>
#include <c10/core/TensorImpl.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/fp8lin.h"

namespace {

// ------------------------------------------------------------------------- entry points

struct Entries {
  decltype(&fp8_layernorm_fwd) layernorm_fwd;
  decltype(&fp8_layernorm_bwd) layernorm_bwd;
  decltype(&fp8_layernorm_bwd_workspace) layernorm_bwd_workspace;
  decltype(&fp8_moe_rows) moe_rows;
  decltype(&fp8_moe_sort_workspace) moe_sort_workspace;
  decltype(&fp8_moe_sort) moe_sort;
  decltype(&fp8_moe_dispatch) moe_dispatch;
  decltype(&fp8_moe_dispatch_bwd) moe_dispatch_bwd;
  decltype(&fp8_moe_combine) moe_combine;
  decltype(&fp8_moe_combine_bwd) moe_combine_bwd;
  decltype(&fp8_moe_route_workspace) moe_route_workspace;
  decltype(&fp8_moe_route) moe_route;
  decltype(&fp8_moe_route_bwd) moe_route_bwd;
  decltype(&fp8_act_quantize) act_quantize;
  decltype(&fp8_act_quantize_bwd) act_quantize_bwd;
  decltype(&fp8_grouped_linear_fwd) grouped_linear_fwd;
  decltype(&fp8_grouped_linear_dgrad) grouped_linear_dgrad;
  decltype(&fp8_grouped_linear_wgrad) grouped_linear_wgrad;
} entry;
// new(shape, dtype, device, stream); check(name, status); current_device(); raw_stream(device)
PyObject *py_new, *py_check, *py_device, *py_raw_stream;

struct Raised {};                                  // a Python error is set
[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

struct Ref {                                       // an owned reference
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {
    if (!o) throw Raised();
  }
  Ref(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* release() { PyObject* o = p; p = nullptr; return o; }
};

long to_long(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int32_t to_i32(PyObject* o, const char* name) {
  const long v = to_long(o);
  if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}
bool to_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

void check(const char* fn, int status) {
  if (status == FP8_OK) return;
  Ref r(PyObject_CallFunction(py_check, "si", fn, status));   // raises
}

// ------------------------------------------------------------------------- tensors

using Shape = std::initializer_list<int64_t>;

std::string str(at::IntArrayRef s) {
  std::ostringstream o;
  o << '(';
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}
template <typename V> std::string str(const V& v) {
  std::ostringstream o;
  o << v;
  return o.str();
}
std::string str(at::ScalarType t) { return at::toString(t); }

int dt_code(at::ScalarType t) {
  return t == at::kBFloat16 ? FP8_DT_BF16 : t == at::kHalf ? FP8_DT_F16 : FP8_DT_F32;
}

// A tensor argument; null for None.
struct Arg {
  const at::Tensor* t = nullptr;
  const char* name;
  Arg(PyObject* o, const char* n) : name(n) {
    if (o == Py_None) return;
    if (!THPVariable_Check(o)) bad(std::string(n) + " must be a tensor");
    t = &THPVariable_Unpack(o);
  }
  explicit operator bool() const { return t != nullptr; }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
  const at::Tensor& need() const {
    if (!t) bad(std::string(name) + " is needed");
    return *t;
  }
};

std::string one_of(std::initializer_list<at::ScalarType> types) {
  std::string s;
  for (auto d : types) s += (s.empty() ? "" : " or ") + str(d);
  return s;
}

// dtype, exact shape, contiguity, device.
void fits(const Arg& a, at::IntArrayRef shape, std::initializer_list<at::ScalarType> types,
          at::Device dev) {
  if (!a) return;
  const at::Tensor& t = *a.t;
  bool type_ok = false;
  for (auto d : types) type_ok |= t.scalar_type() == d;
  if (type_ok && t.sizes() == shape && t.is_contiguous() && t.device() == dev) return;
  const std::string n = a.name;
  if (!type_ok) bad(n + " has dtype " + str(t.scalar_type()) + ", expected " + one_of(types));
  if (t.sizes() != shape) bad(n + " has shape " + str(t.sizes()) + ", expected " + str(shape));
  if (!t.is_contiguous()) bad(n + " must be contiguous (row-major)");
  bad(n + " is on " + str(t.device()) + ", the operands on " + str(dev));
}

// A [rows, cols] input whose rows may be a cut out of a wider tensor: its row stride in
// elements, at least the width (tensors of up to one row may have any).
int64_t row_stride(const Arg& a) {
  const at::Tensor& t = a.need();
  const std::string n = a.name;
  const auto d = t.scalar_type();
  if (d != at::kBFloat16 && d != at::kHalf && d != at::kFloat)
    bad(n + " has dtype " + str(d) + ", expected bfloat16, float16 or float32");
  if (t.dim() != 2) bad(n + " must be 2-D [rows, cols], got shape " + str(t.sizes()));
  const int64_t r = t.size(0), c = t.size(1), ld = t.stride(0);
  if (c > 1 && t.stride(1) != 1)
    bad(n + ": the columns of a row must be contiguous, stride " + str(t.stride(1)));
  if (r <= 1) return ld > c ? ld : c;
  if (ld < c) bad(n + ": rows overlap (stride " + str(ld) + ", " + str(c) + " columns)");
  return ld;
}
int64_t row_stride(const Arg& a, int64_t rows, int64_t cols, at::ScalarType dtype,
                   at::Device dev) {
  const int64_t ld = row_stride(a);
  const at::Tensor& t = *a.t;
  const std::string n = a.name;
  if (t.size(0) != rows || t.size(1) != cols)
    bad(n + " has shape " + str(t.sizes()) + ", expected " + str(at::IntArrayRef({rows, cols})));
  if (t.scalar_type() != dtype)
    bad(n + " has dtype " + str(t.scalar_type()) + ", expected " + str(dtype));
  if (t.device() != dev) bad(n + " is on " + str(t.device()) + ", the operands on " + str(dev));
  return ld;
}

// The common dtype of parameters [cols]: the rows' or float32; `none` without any.
at::ScalarType param_type(at::ScalarType rows, int64_t cols, at::Device dev, at::ScalarType none,
                          std::initializer_list<const Arg*> params) {
  bool have = false;
  at::ScalarType d = none;
  for (const Arg* a : params) {
    if (!*a) continue;
    if (!have) {
      d = a->t->scalar_type();
      if (d != rows && d != at::kFloat)
        bad(std::string(a->name) + " has dtype " + str(d) + ", expected " + str(rows) +
            " or float32");
      have = true;
    }
    fits(*a, {cols}, {d}, dev);
  }
  return d;
}

// The handle of the stream that the call goes to; the operands must be on the current device
// (kernels go to the current device's streams).
void* launch_stream(const at::Tensor& t, PyObject* stream) {
  if (!t.is_cuda()) bad("fp8lin takes device tensors");
  Ref cur(PyObject_CallNoArgs(py_device));
  const long dev = to_long(cur.p);
  if (t.device().index() != dev)
    bad("the operands are on " + str(t.device()) + ", the current device is cuda:" + str(dev));
  if (stream == Py_None) {
    Ref h(PyObject_CallOneArg(py_raw_stream, cur.p));
    void* p = PyLong_AsVoidPtr(h.p);
    if (!p && PyErr_Occurred()) throw Raised();
    return p;
  }
  Ref d(PyObject_GetAttrString(stream, "device")), i(PyObject_GetAttrString(d.p, "index"));
  if (to_long(i.p) != dev)
    bad("the stream is on cuda:" + str(to_long(i.p)) + ", the current device is cuda:" + str(dev));
  Ref h(PyObject_GetAttrString(stream, "cuda_stream"));
  void* p = PyLong_AsVoidPtr(h.p);
  if (!p && PyErr_Occurred()) throw Raised();
  return p;
}

// A dense tensor of `storage`, at `offset` bytes.
at::Tensor in_storage(c10::Storage storage, int64_t offset, at::IntArrayRef shape,
                      at::ScalarType dtype) {
  const auto type = c10::scalarTypeToTypeMeta(dtype);
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA), type);
  t.unsafeGetTensorImpl()->set_storage_offset(offset / (int64_t)type.itemsize());
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}
at::Tensor torch_empty(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like) {
  return at::empty(shape, like.options().dtype(dtype).requires_grad(false));
}
// Whether at::empty would take memory from torch's allocator and do nothing else: no mode or
// transform stands before it, and it would not fill the memory.
bool plain_empty(const at::Tensor& like) {
  const auto on = c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set;
  const auto& ctx = at::globalContext();
  return on.empty() && !like.unsafeGetTensorImpl()->is_python_dispatch() &&
         !(ctx.deterministicAlgorithms() && ctx.deterministicFillUninitializedMemory());
}
// That allocator, which torch settles before its first device tensor, as a plain one names it; null
// if that one does not.
c10::Allocator* device_allocator(const at::Tensor& like) {
  static c10::Allocator* known = nullptr;          // under the interpreter's lock
  if (!known) {
    const at::Tensor t = torch_empty({1}, at::kByte, like);
    if (!t.unsafeGetTensorImpl()->is_python_dispatch() && t.device() == like.device() &&
        t.storage().device() == t.device())
      known = t.storage().allocator();
  }
  return known;
}
// `bytes` of device memory: as at::empty gives them, without torch's dispatcher (0.4 us instead of 0.8
// to 1 of host time) where that makes no difference; else a null storage.
c10::Storage new_storage(int64_t bytes, const at::Tensor& like) {
  if (!plain_empty(like)) return c10::Storage();
  c10::Allocator* const a = device_allocator(like);
  if (!a) return c10::Storage();
  return c10::Storage(c10::Storage::use_byte_size_t(), (size_t)bytes, a->allocate((size_t)bytes), a,
                      /*resizable=*/true);
}
int64_t bytes_of(at::IntArrayRef shape, at::ScalarType dtype) {
  int64_t n = (int64_t)c10::elementSize(dtype);
  for (int64_t s : shape) n *= s;
  return n;
}

// An output or workspace of the call: the caller's tensor, or a new one in the memory pool of
// the stream that will write it, so that a call on a stream other than the current one never
// reuses memory in use on the latter.
struct Out {
  PyObject* o;                                     // owned
  void* ptr = nullptr;
  explicit Out(PyObject* given) : o(Py_NewRef(given)) {}
  Out(const Out&) = delete;
  ~Out() { Py_XDECREF(o); }
  void hold(PyObject* n) {
    if (!n) throw Raised();
    Py_DECREF(o);
    o = n;
  }
  void make(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like, PyObject* stream,
            bool wanted = true) {
    if (o == Py_None && wanted) {
      if (stream == Py_None) {
        c10::Storage mem = new_storage(bytes_of(shape, dtype), like);
        hold(THPVariable_Wrap(mem ? in_storage(std::move(mem), 0, shape, dtype)
                                  : torch_empty(shape, dtype, like)));
      } else {
        Ref sh(PyTuple_New((Py_ssize_t)shape.size()));
        for (size_t i = 0; i < shape.size(); ++i)
          PyTuple_SET_ITEM(sh.p, (Py_ssize_t)i, PyLong_FromLongLong(shape[i]));
        Ref like_o(THPVariable_Wrap(like)), dev(PyObject_GetAttrString(like_o.p, "device"));
        hold(PyObject_CallFunction(py_new, "OsOO", sh.p, at::toString(dtype), dev.p, stream));
      }
    }
    if (o != Py_None) ptr = THPVariable_Unpack(o).data_ptr();
  }
  PyObject* take() { PyObject* r = o; o = nullptr; return r; }
};

// New outputs in one allocation, or, where the caller gave one of them, its stream or more than
// `most` bytes, in one each. An allocation is 0.4 us of host time: of a small call's time the outputs
// are a good part, and share one up to kShared bytes in all. Larger ones do not, so that keeping one
// of them does not keep the others' memory.
constexpr int64_t kShared = 32 * 1024;
struct Wanted {
  Out* out;
  std::array<int64_t, 2> shape;
  int dims;
  at::ScalarType dtype;
  bool wanted = true;
  at::IntArrayRef sizes() const { return {shape.data(), (size_t)dims}; }
};
bool make_shared(std::initializer_list<Wanted> outs, const at::Tensor& like, PyObject* stream,
                 int64_t most) {
  constexpr int64_t kAlign = 64;
  auto room = [](const Wanted& w) {
    return w.wanted ? (bytes_of(w.sizes(), w.dtype) + kAlign - 1) / kAlign * kAlign : 0;
  };
  int64_t total = 0;
  bool all = stream == Py_None;
  for (const Wanted& w : outs) all = all && w.out->o == Py_None, total += room(w);
  if (!all || total > most) return false;
  const c10::Storage mem = new_storage(total, like);
  if (!mem) return false;
  char* const base = static_cast<char*>(mem.mutable_data());
  int64_t at = 0;
  for (const Wanted& w : outs) {
    if (!w.wanted) continue;
    w.out->hold(THPVariable_Wrap(in_storage(mem, at, w.sizes(), w.dtype)));
    w.out->ptr = base + at;
    at += room(w);
  }
  return true;
}
void make_all(std::initializer_list<Wanted> outs, const at::Tensor& like, PyObject* stream,
              int64_t most = kShared) {
  if (make_shared(outs, like, stream, most)) return;
  for (const Wanted& w : outs) w.out->make(w.sizes(), w.dtype, like, stream, w.wanted);
}

// A uint8 workspace of at least `bytes`.
int64_t workspace(Out& w, int64_t bytes, const at::Tensor& like, PyObject* stream) {
  if (w.o == Py_None) {
    w.make({bytes}, at::kByte, like, stream, bytes > 0);
    return bytes;
  }
  const Arg a(w.o, "workspace");
  if (a.t->scalar_type() != at::kByte || !a.t->is_contiguous() || a.t->device() != like.device())
    bad("workspace must be a contiguous uint8 tensor on " + str(like.device()));
  if (a.t->numel() < bytes)
    bad("workspace holds " + str(a.t->numel()) + " bytes, needs " + str(bytes));
  w.ptr = a.t->data_ptr();
  return a.t->numel();
}

PyObject* tuple(std::initializer_list<Out*> outs) {
  Ref t(PyTuple_New((Py_ssize_t)outs.size()));
  Py_ssize_t i = 0;
  for (Out* o : outs) PyTuple_SET_ITEM(t.p, i++, o->take());
  return t.release();
}

// ------------------------------------------------------------------------- operators

// x, gamma, beta, eps, y, mean, rstd, want_stats, stream
PyObject* layernorm_fwd(PyObject* const* p) {
  const Arg x(p[0], "x"), gamma(p[1], "gamma"), beta(p[2], "beta");
  const int64_t ld = row_stride(x), rows = x.t->size(0), cols = x.t->size(1);
  const auto dev = x.t->device();
  const auto dt = x.t->scalar_type();
  const auto pdt = param_type(dt, cols, dev, dt, {&gamma, &beta});
  const double eps = PyFloat_AsDouble(p[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw Raised();
  fits(Arg(p[4], "y"), {rows, cols}, {dt}, dev);
  fits(Arg(p[5], "mean"), {rows}, {at::kFloat}, dev);
  fits(Arg(p[6], "rstd"), {rows}, {at::kFloat}, dev);
  const bool stats = to_bool(p[7]);
  void* s = launch_stream(*x.t, p[8]);
  Out y(p[4]), mean(p[5]), rstd(p[6]);
  y.make({rows, cols}, dt, *x.t, p[8]);
  mean.make({rows}, at::kFloat, *x.t, p[8], stats);
  rstd.make({rows}, at::kFloat, *x.t, p[8], stats);
  check("fp8_layernorm_fwd",
        entry.layernorm_fwd(x.ptr(), ld, gamma.ptr(), beta.ptr(), rows, cols, dt_code(dt),
                            dt_code(pdt), (float)eps, y.ptr, static_cast<float*>(mean.ptr),
                            static_cast<float*>(rstd.ptr), s));
  return tuple({&y, &mean, &rstd});
}

// dy, x, mean, rstd, gamma, dx, dgamma, dbeta, want_dx, want_dgamma, want_dbeta, params_f32
// (the parameters' type without any: None the rows'), workspace, stream
PyObject* layernorm_bwd(PyObject* const* p) {
  const Arg dy(p[0], "dy"), x(p[1], "x"), mean(p[2], "mean"), rstd(p[3], "rstd");
  const Arg gamma(p[4], "gamma"), adg(p[6], "dgamma"), adb(p[7], "dbeta");
  const int64_t ld = row_stride(x), rows = x.t->size(0), cols = x.t->size(1);
  const auto dev = x.t->device();
  const auto dt = x.t->scalar_type();
  const int64_t lddy = row_stride(dy, rows, cols, dt, dev);
  fits(mean, {rows}, {at::kFloat}, dev);
  fits(rstd, {rows}, {at::kFloat}, dev);
  if (!mean || !rstd) bad("mean and rstd of the forward are needed");
  const auto pdt = param_type(dt, cols, dev, to_bool(p[11]) ? at::kFloat : dt,
                              {&gamma, &adg, &adb});
  fits(Arg(p[5], "dx"), {rows, cols}, {dt}, dev);
  void* s = launch_stream(*x.t, p[13]);
  Out dx(p[5]), dgamma(p[6]), dbeta(p[7]), ws(p[12]);
  dx.make({rows, cols}, dt, *x.t, p[13], to_bool(p[8]));
  dgamma.make({cols}, pdt, *x.t, p[13], to_bool(p[9]));
  dbeta.make({cols}, pdt, *x.t, p[13], to_bool(p[10]));
  int64_t bytes = 0;
  if (dgamma.o != Py_None || dbeta.o != Py_None) {
    check("fp8_layernorm_bwd_workspace", entry.layernorm_bwd_workspace(rows, cols, &bytes));
    bytes = workspace(ws, bytes, *x.t, p[13]);
  }
  check("fp8_layernorm_bwd",
        entry.layernorm_bwd(dy.ptr(), lddy, x.ptr(), ld, static_cast<float*>(mean.ptr()),
                            static_cast<float*>(rstd.ptr()), gamma.ptr(), rows, cols, dt_code(dt),
                            dt_code(pdt), dx.ptr, dgamma.ptr, dbeta.ptr, ws.ptr, bytes, s));
  return tuple({&dx, &dgamma, &dbeta});
}

// expert_idx, experts, multiple, slot, source, counts, offsets, workspace, stream
PyObject* moe_sort(PyObject* const* p) {
  const Arg idx(p[0], "expert_idx");
  if (idx.need().dim() != 2)
    bad("expert_idx must be 2-D [tokens, topk], got " + str(idx.t->sizes()));
  const int64_t tokens = idx.t->size(0), topk = idx.t->size(1);
  const auto dev = idx.t->device();
  fits(idx, {tokens, topk}, {at::kInt, at::kLong}, dev);
  if (topk > INT32_MAX) bad("expert_idx: too many choices");
  const int32_t experts = to_i32(p[1], "experts"), multiple = to_i32(p[2], "multiple");
  int64_t rows = 0, bytes = 0;
  check("fp8_moe_rows", entry.moe_rows(tokens, (int32_t)topk, experts, multiple, &rows));
  fits(Arg(p[3], "slot"), {tokens, topk}, {at::kInt}, dev);
  fits(Arg(p[4], "source"), {rows}, {at::kInt}, dev);
  fits(Arg(p[5], "counts"), {experts}, {at::kInt}, dev);
  fits(Arg(p[6], "offsets"), {(int64_t)experts + 1}, {at::kInt}, dev);
  void* s = launch_stream(*idx.t, p[8]);
  Out slot(p[3]), source(p[4]), counts(p[5]), offsets(p[6]), ws(p[7]);
  slot.make({tokens, topk}, at::kInt, *idx.t, p[8]);
  source.make({rows}, at::kInt, *idx.t, p[8]);
  counts.make({experts}, at::kInt, *idx.t, p[8]);
  offsets.make({(int64_t)experts + 1}, at::kInt, *idx.t, p[8]);
  check("fp8_moe_sort_workspace", entry.moe_sort_workspace(tokens, (int32_t)topk, experts, &bytes));
  bytes = workspace(ws, bytes, *idx.t, p[8]);
  check("fp8_moe_sort",
        entry.moe_sort(idx.ptr(), (int)idx.t->element_size(), tokens, (int32_t)topk, experts,
                       multiple, static_cast<int32_t*>(slot.ptr), static_cast<int32_t*>(source.ptr),
                       static_cast<int32_t*>(counts.ptr), static_cast<int32_t*>(offsets.ptr),
                       ws.ptr, bytes, s));
  return tuple({&slot, &source, &counts, &offsets});
}

// The index tensors of a sort.
struct Plan {
  Arg slot, source;
  int64_t tokens, topk, rows = 0;
  Plan(PyObject* sl, PyObject* so, at::Device dev) : slot(sl, "slot"), source(so, "source") {
    if (slot.need().dim() != 2)
      bad("slot must be 2-D [tokens, topk], got " + str(slot.t->sizes()));
    fits(slot, slot.t->sizes(), {at::kInt}, dev);
    tokens = slot.t->size(0);
    topk = slot.t->size(1);
    if (topk > INT32_MAX) bad("slot: too many choices");
    if (!source) return;
    if (source.t->dim() != 1) bad("source must be 1-D [rows], got " + str(source.t->sizes()));
    fits(source, source.t->sizes(), {at::kInt}, dev);
    rows = source.t->size(0);
  }
  const int32_t* slots() const { return static_cast<const int32_t*>(slot.ptr()); }
  const int32_t* sources() const { return static_cast<const int32_t*>(source.ptr()); }
};

// x, slot, source, xs, stream
PyObject* moe_dispatch(PyObject* const* p) {
  const Arg x(p[0], "x");
  const int64_t ld = row_stride(x), cols = x.t->size(1);
  const auto dev = x.t->device();
  const auto dt = x.t->scalar_type();
  const Plan k(p[1], p[2], dev);
  k.source.need();
  if (x.t->size(0) != k.tokens)
    bad("x has " + str(x.t->size(0)) + " rows, slot is for " + str(k.tokens) + " tokens");
  fits(Arg(p[3], "xs"), {k.rows, cols}, {dt}, dev);
  void* s = launch_stream(*x.t, p[4]);
  Out xs(p[3]);
  xs.make({k.rows, cols}, dt, *x.t, p[4]);
  check("fp8_moe_dispatch",
        entry.moe_dispatch(x.ptr(), ld, k.slots(), k.sources(), k.tokens, (int32_t)k.topk, k.rows,
                           cols, dt_code(dt), xs.ptr, s));
  return xs.take();
}

// dxs, slot, dx, stream
PyObject* moe_dispatch_bwd(PyObject* const* p) {
  const Arg dxs(p[0], "dxs");
  const int64_t ld = row_stride(dxs), rows = dxs.t->size(0), cols = dxs.t->size(1);
  const auto dev = dxs.t->device();
  const auto dt = dxs.t->scalar_type();
  const Plan k(p[1], Py_None, dev);
  fits(Arg(p[2], "dx"), {k.tokens, cols}, {dt}, dev);
  void* s = launch_stream(*dxs.t, p[3]);
  Out dx(p[2]);
  dx.make({k.tokens, cols}, dt, *dxs.t, p[3]);
  check("fp8_moe_dispatch_bwd",
        entry.moe_dispatch_bwd(dxs.ptr(), ld, k.slots(), k.tokens, (int32_t)k.topk, rows, cols,
                               dt_code(dt), dx.ptr, s));
  return dx.take();
}

// ys, slot, weights, y, stream
PyObject* moe_combine(PyObject* const* p) {
  const Arg ys(p[0], "ys"), w(p[2], "weights");
  const int64_t ld = row_stride(ys), rows = ys.t->size(0), cols = ys.t->size(1);
  const auto dev = ys.t->device();
  const auto dt = ys.t->scalar_type();
  const Plan k(p[1], Py_None, dev);
  w.need();
  fits(w, {k.tokens, k.topk}, {at::kFloat}, dev);
  fits(Arg(p[3], "y"), {k.tokens, cols}, {dt}, dev);
  void* s = launch_stream(*ys.t, p[4]);
  Out y(p[3]);
  y.make({k.tokens, cols}, dt, *ys.t, p[4]);
  check("fp8_moe_combine",
        entry.moe_combine(ys.ptr(), ld, k.slots(), static_cast<const float*>(w.ptr()), k.tokens,
                          (int32_t)k.topk, rows, cols, dt_code(dt), y.ptr, s));
  return y.take();
}

// dy, ys, slot, source, weights, dys, dw, stream
PyObject* moe_combine_bwd(PyObject* const* p) {
  const Arg dy(p[0], "dy"), ys(p[1], "ys"), w(p[4], "weights");
  const int64_t ldys = row_stride(ys), cols = ys.t->size(1);
  const auto dev = ys.t->device();
  const auto dt = ys.t->scalar_type();
  const Plan k(p[2], p[3], dev);
  k.source.need();
  if (ys.t->size(0) != k.rows)
    bad("ys has " + str(ys.t->size(0)) + " rows, source " + str(k.rows));
  const int64_t lddy = row_stride(dy, k.tokens, cols, dt, dev);
  w.need();
  fits(w, {k.tokens, k.topk}, {at::kFloat}, dev);
  fits(Arg(p[5], "dys"), {k.rows, cols}, {dt}, dev);
  fits(Arg(p[6], "dw"), {k.tokens, k.topk}, {at::kFloat}, dev);
  void* s = launch_stream(*ys.t, p[7]);
  Out dys(p[5]), dw(p[6]);
  dys.make({k.rows, cols}, dt, *ys.t, p[7]);
  dw.make({k.tokens, k.topk}, at::kFloat, *ys.t, p[7]);
  check("fp8_moe_combine_bwd",
        entry.moe_combine_bwd(dy.ptr(), lddy, ys.ptr(), ldys, k.slots(), k.sources(),
                              static_cast<const float*>(w.ptr()), k.tokens, (int32_t)k.topk, k.rows,
                              cols, dt_code(dt), dys.ptr, static_cast<float*>(dw.ptr), s));
  return tuple({&dys, &dw});
}

// ------------------------------------------------------------------------- the router

// A count of valid rows: all of them for None.
int64_t valid_rows(PyObject* o, int64_t rows, const char* name) {
  const int64_t v = o == Py_None ? rows : to_long(o);
  if (v < 0 || v > rows)
    bad(std::string(name) + "=" + str(v) + " outside [0, " + str(rows) + "]");
  return v;
}

// logits, topk, tokens_valid, normalize, expert_idx, weights, lse, counts, losses, workspace, stream
PyObject* moe_route(PyObject* const* p) {
  const Arg x(p[0], "logits");
  const int64_t ld = row_stride(x), tokens = x.t->size(0), experts = x.t->size(1);
  const auto dev = x.t->device();
  const auto dt = x.t->scalar_type();
  const int32_t topk = to_i32(p[1], "topk");
  if (topk < 1) bad("topk=" + str(topk) + " must be positive");
  const int64_t valid = valid_rows(p[2], tokens, "tokens_valid");
  const bool normalize = to_bool(p[3]);
  if (experts > INT32_MAX) bad("logits: too many experts");
  fits(Arg(p[4], "expert_idx"), {tokens, topk}, {at::kInt}, dev);
  fits(Arg(p[5], "weights"), {tokens, topk}, {at::kFloat}, dev);
  fits(Arg(p[6], "lse"), {tokens}, {at::kFloat}, dev);
  fits(Arg(p[7], "counts"), {experts}, {at::kInt}, dev);
  fits(Arg(p[8], "losses"), {2}, {at::kFloat}, dev);
  PyObject* const stream = p[10];
  void* s = launch_stream(*x.t, stream);
  int64_t bytes = 0;
  check("fp8_moe_route_workspace", entry.moe_route_workspace(tokens, (int32_t)experts, &bytes));
  Out idx(p[4]), weights(p[5]), lse(p[6]), counts(p[7]), losses(p[8]), ws(p[9]);
  make_all({{&idx, {tokens, topk}, 2, at::kInt}, {&weights, {tokens, topk}, 2, at::kFloat},
            {&lse, {tokens, 0}, 1, at::kFloat}, {&counts, {experts, 0}, 1, at::kInt},
            {&losses, {2, 0}, 1, at::kFloat}}, *x.t, stream);
  bytes = workspace(ws, bytes, *x.t, stream);
  check("fp8_moe_route",
        entry.moe_route(x.ptr(), ld, tokens, valid, (int32_t)experts, topk, dt_code(dt), normalize,
                        static_cast<int32_t*>(idx.ptr), static_cast<float*>(weights.ptr),
                        static_cast<float*>(lse.ptr), static_cast<int32_t*>(counts.ptr),
                        static_cast<float*>(losses.ptr), ws.ptr, bytes, s));
  return tuple({&idx, &weights, &lse, &counts, &losses});
}

// logits, lse, expert_idx, weights, counts, dweights, dlosses, tokens_valid, normalize, dlogits,
// stream
PyObject* moe_route_bwd(PyObject* const* p) {
  const Arg x(p[0], "logits"), lse(p[1], "lse"), idx(p[2], "expert_idx"), w(p[3], "weights");
  const Arg counts(p[4], "counts"), dw(p[5], "dweights"), dl(p[6], "dlosses");
  const int64_t ld = row_stride(x), tokens = x.t->size(0), experts = x.t->size(1);
  const auto dev = x.t->device();
  const auto dt = x.t->scalar_type();
  if (idx.need().dim() != 2)
    bad("expert_idx must be 2-D [tokens, topk], got " + str(idx.t->sizes()));
  const int64_t topk = idx.t->size(1);
  if (topk > INT32_MAX || experts > INT32_MAX) bad("expert_idx: too many choices");
  lse.need(), w.need(), counts.need();
  fits(idx, {tokens, topk}, {at::kInt}, dev);
  fits(lse, {tokens}, {at::kFloat}, dev);
  fits(w, {tokens, topk}, {at::kFloat}, dev);
  fits(counts, {experts}, {at::kInt}, dev);
  fits(dw, {tokens, topk}, {at::kFloat}, dev);
  fits(dl, {2}, {at::kFloat}, dev);
  const int64_t valid = valid_rows(p[7], tokens, "tokens_valid");
  const bool normalize = to_bool(p[8]);
  fits(Arg(p[9], "dlogits"), {tokens, experts}, {dt}, dev);
  void* s = launch_stream(*x.t, p[10]);
  Out out(p[9]);
  out.make({tokens, experts}, dt, *x.t, p[10]);
  check("fp8_moe_route_bwd",
        entry.moe_route_bwd(x.ptr(), ld, static_cast<float*>(lse.ptr()),
                            static_cast<int32_t*>(idx.ptr()), static_cast<float*>(w.ptr()),
                            static_cast<int32_t*>(counts.ptr()), static_cast<float*>(dw.ptr()),
                            static_cast<float*>(dl.ptr()), tokens, valid, (int32_t)experts,
                            (int32_t)topk, dt_code(dt), normalize, out.ptr, s));
  return out.take();
}

// ------------------------------------------------------------------------- activation

constexpr int64_t kTile = 128;               // codes per scale
constexpr std::initializer_list<at::ScalarType> kCodes = {at::kByte, at::kFloat8_e4m3fn};

// Codes [r, c] and their scales [r, c / 128], of which both or none are given.
void fits_pair(const Arg& q, const Arg& scale, int64_t r, int64_t c, at::Device dev) {
  if (bool(q) != bool(scale))
    bad(std::string(q.name) + " and " + scale.name + " must both be given or both be None");
  fits(q, {r, c}, kCodes, dev);
  fits(scale, {r, c / kTile}, {at::kFloat}, dev);
}
// Codes and their scales, which are used together and so share an allocation of any size.
struct OutPair {
  Out q, scale;
  OutPair(PyObject* a, PyObject* b) : q(a), scale(b) {}
  Wanted codes(int64_t r, int64_t c, bool wanted) { return {&q, {r, c}, 2, at::kByte, wanted}; }
  Wanted scaling(int64_t r, int64_t c, bool wanted) {
    return {&scale, {r, c / kTile}, 2, at::kFloat, wanted};
  }
  void make(int64_t r, int64_t c, const at::Tensor& like, PyObject* stream, bool wanted) {
    make_all({codes(r, c, wanted), scaling(r, c, wanted)}, like, stream, INT64_MAX);
  }
  float* scales() const { return static_cast<float*>(scale.ptr); }
};

// h, act, gated, rows_valid, q, scale, q_t, scale_t, hq, hscale, want_q, want_q_t,
// want_checkpoint, stream
PyObject* act_quantize(PyObject* const* p) {
  const Arg h(p[0], "h");
  const int64_t ld = row_stride(h), rows = h.t->size(0), width = h.t->size(1);
  const auto dev = h.t->device();
  const int32_t act = to_i32(p[1], "act");
  const bool gated = to_bool(p[2]);
  if (gated && width % 2) bad("h [rows, 2 cols] has an odd width " + str(width));
  const int64_t cols = gated ? width / 2 : width;
  if (cols < 1 || cols % kTile) bad("h: cols=" + str(cols) + " must be a positive multiple of 128");
  const int64_t valid = valid_rows(p[3], rows, "rows_valid");
  const bool want_q = to_bool(p[10]), want_t = to_bool(p[11]), want_h = to_bool(p[12]);
  fits_pair(Arg(p[4], "q"), Arg(p[5], "scale"), rows, cols, dev);
  fits_pair(Arg(p[6], "q_t"), Arg(p[7], "scale_t"), cols, rows, dev);
  fits_pair(Arg(p[8], "hq"), Arg(p[9], "hscale"), rows, width, dev);
  if ((want_t || p[6] != Py_None) && rows % kTile)
    bad("q_t needs rows to be a multiple of 128, got " + str(rows));
  void* s = launch_stream(*h.t, p[13]);
  OutPair q(p[4], p[5]), t(p[6], p[7]), c(p[8], p[9]);
  if (!make_shared({q.codes(rows, cols, want_q), q.scaling(rows, cols, want_q),
                    t.codes(cols, rows, want_t), t.scaling(cols, rows, want_t),
                    c.codes(rows, width, want_h), c.scaling(rows, width, want_h)},
                   *h.t, p[13], kShared)) {
    q.make(rows, cols, *h.t, p[13], want_q);
    t.make(cols, rows, *h.t, p[13], want_t);
    c.make(rows, width, *h.t, p[13], want_h);
  }
  check("fp8_act_quantize",
        entry.act_quantize(h.ptr(), ld, rows, valid, cols, act, gated,
                           dt_code(h.t->scalar_type()), q.q.ptr, q.scales(), t.q.ptr, t.scales(),
                           c.q.ptr, c.scales(), s));
  return tuple({&q.q, &q.scale, &t.q, &t.scale, &c.q, &c.scale});
}

// da, hq, hscale, act, gated, rows_valid, q, scale, q_t, scale_t, dh, want_q, want_q_t, want_dh,
// stream
PyObject* act_quantize_bwd(PyObject* const* p) {
  const Arg da(p[0], "da"), hq(p[1], "hq"), hscale(p[2], "hscale");
  const int64_t ld = row_stride(da), rows = da.t->size(0), cols = da.t->size(1);
  const auto dev = da.t->device();
  const auto dt = da.t->scalar_type();
  const int32_t act = to_i32(p[3], "act");
  const bool gated = to_bool(p[4]);
  if (cols < 1 || cols % kTile) bad("da: cols=" + str(cols) + " must be a positive multiple of 128");
  const int64_t width = gated ? 2 * cols : cols;
  const int64_t valid = valid_rows(p[5], rows, "rows_valid");
  hq.need(), hscale.need();
  fits_pair(hq, hscale, rows, width, dev);
  fits_pair(Arg(p[6], "q"), Arg(p[7], "scale"), rows, width, dev);
  fits_pair(Arg(p[8], "q_t"), Arg(p[9], "scale_t"), width, rows, dev);
  fits(Arg(p[10], "dh"), {rows, width}, {dt}, dev);
  const bool want_q = to_bool(p[11]), want_t = to_bool(p[12]), want_dh = to_bool(p[13]);
  if ((want_t || p[8] != Py_None) && rows % kTile)
    bad("q_t needs rows to be a multiple of 128, got " + str(rows));
  void* s = launch_stream(*da.t, p[14]);
  OutPair q(p[6], p[7]), t(p[8], p[9]);
  Out dh(p[10]);
  if (!make_shared({q.codes(rows, width, want_q), q.scaling(rows, width, want_q),
                    t.codes(width, rows, want_t), t.scaling(width, rows, want_t),
                    {&dh, {rows, width}, 2, dt, want_dh}},
                   *da.t, p[14], kShared)) {
    q.make(rows, width, *da.t, p[14], want_q);
    t.make(width, rows, *da.t, p[14], want_t);
    dh.make({rows, width}, dt, *da.t, p[14], want_dh);
  }
  check("fp8_act_quantize_bwd",
        entry.act_quantize_bwd(da.ptr(), ld, hq.ptr(), static_cast<float*>(hscale.ptr()), rows,
                               valid, cols, act, gated, dt_code(dt), q.q.ptr, q.scales(), t.q.ptr,
                               t.scales(), dh.ptr, s));
  return tuple({&q.q, &q.scale, &t.q, &t.scale, &dh});
}

// ------------------------------------------------------------------------- experts' products

// Rows of codes and their scales, dense: [rows, cols], cols a positive multiple of 128.
void code_rows(const Arg& q, const Arg& scale, int64_t& rows, int64_t& cols) {
  if (q.need().dim() != 2)
    bad(std::string(q.name) + " must be 2-D [rows, cols], got " + str(q.t->sizes()));
  scale.need();
  rows = q.t->size(0), cols = q.t->size(1);
  fits_pair(q, scale, rows, cols, q.t->device());
}

// The experts' matrices [experts, r, c], each with contiguous rows; any expert and row strides.
void stacked(const Arg& a, int64_t e, int64_t r, int64_t c, std::initializer_list<at::ScalarType> types,
             at::Device dev, int64_t& ld, int64_t& stride) {
  const at::Tensor& t = a.need();
  const std::string n = a.name;
  bool type_ok = false;
  for (auto d : types) type_ok |= t.scalar_type() == d;
  if (!type_ok) bad(n + " has dtype " + str(t.scalar_type()) + ", expected " + one_of(types));
  if (t.sizes() != at::IntArrayRef({e, r, c}))
    bad(n + " has shape " + str(t.sizes()) + ", expected " + str(at::IntArrayRef({e, r, c})));
  if (t.device() != dev) bad(n + " is on " + str(t.device()) + ", the operands on " + str(dev));
  if (c > 1 && t.stride(2) != 1) bad(n + ": its rows must be contiguous, stride " + str(t.stride(2)));
  ld = r > 1 ? t.stride(1) : c;
  stride = e > 1 ? t.stride(0) : 0;
  if (ld < c) bad(n + ": rows overlap (stride " + str(ld) + ", " + str(c) + " columns)");
}

struct Groups {
  Arg offsets, counts;
  int64_t experts;
  Groups(PyObject* o, PyObject* c, at::Device dev) : offsets(o, "offsets"), counts(c, "counts") {
    if (counts.need().dim() != 1) bad("counts must be 1-D [experts], got " + str(counts.t->sizes()));
    experts = counts.t->size(0);
    if (experts > INT32_MAX - 1) bad("counts: too many experts");
    fits(counts, {experts}, {at::kInt}, dev);
    offsets.need();
    fits(offsets, {experts + 1}, {at::kInt}, dev);
  }
  const int32_t* off() const { return static_cast<const int32_t*>(offsets.ptr()); }
  const int32_t* cnt() const { return static_cast<const int32_t*>(counts.ptr()); }
};

// dgrad, x, w, sx, sw, offsets, counts, y, max_rows, stream
PyObject* grouped_linear(PyObject* const* p) {
  const bool dgrad = to_bool(p[0]);
  const Arg x(p[1], dgrad ? "qg" : "qx"), w(p[2], dgrad ? "qw_t" : "qw");
  const Arg sx(p[3], dgrad ? "sg" : "sx"), sw(p[4], dgrad ? "sw_t" : "sw");
  int64_t rows, in, ldw, stride_w, ldsw, stride_sw;
  code_rows(x, sx, rows, in);
  const auto dev = x.t->device();
  const Groups g(p[5], p[6], dev);
  if (w.need().dim() != 3)
    bad(std::string(w.name) + " must be 3-D [experts, out, in], got " + str(w.t->sizes()));
  const int64_t out = w.t->size(1);
  stacked(w, g.experts, out, in, kCodes, dev, ldw, stride_w);
  stacked(sw, g.experts, out / kTile, in / kTile, {at::kFloat}, dev, ldsw, stride_sw);
  fits(Arg(p[7], dgrad ? "dx" : "y"), {rows, out}, {at::kBFloat16}, dev);
  const int64_t most = p[8] == Py_None ? rows : to_long(p[8]);
  if (most < 0) bad("max_rows=" + str(most) + " is negative");
  void* s = launch_stream(*x.t, p[9]);
  Out y(p[7]);
  y.make({rows, out}, at::kBFloat16, *x.t, p[9]);
  const float *fx = static_cast<float*>(sx.ptr()), *fw = static_cast<float*>(sw.ptr());
  if (dgrad)
    check("fp8_grouped_linear_dgrad",
          entry.grouped_linear_dgrad(x.ptr(), w.ptr(), ldw, stride_w, fx, fw, ldsw, stride_sw,
                                     g.off(), g.cnt(), (int32_t)g.experts, rows, in, out, most,
                                     y.ptr, s));
  else
    check("fp8_grouped_linear_fwd",
          entry.grouped_linear_fwd(x.ptr(), w.ptr(), ldw, stride_w, fx, fw, ldsw, stride_sw,
                                   g.off(), g.cnt(), (int32_t)g.experts, rows, out, in, most, y.ptr,
                                   s));
  return y.take();
}

// qg_t, qx_t, sg_t, sx_t, offsets, counts, dw, stream
PyObject* grouped_wgrad(PyObject* const* p) {
  const Arg g(p[0], "qg_t"), x(p[1], "qx_t"), sg(p[2], "sg_t"), sx(p[3], "sx_t");
  int64_t n, k, rows, rows_x;
  code_rows(g, sg, n, rows);
  code_rows(x, sx, k, rows_x);
  const auto dev = g.t->device();
  if (rows_x != rows)
    bad("qg_t has " + str(rows) + " rows of tokens, qx_t " + str(rows_x));
  if (x.t->device() != dev) bad("qx_t is on " + str(x.t->device()) + ", qg_t on " + str(dev));
  const Groups e(p[4], p[5], dev);
  fits(Arg(p[6], "dw"), {e.experts, n, k}, {at::kBFloat16}, dev);
  void* s = launch_stream(*g.t, p[7]);
  Out dw(p[6]);
  dw.make({e.experts, n, k}, at::kBFloat16, *g.t, p[7]);
  check("fp8_grouped_linear_wgrad",
        entry.grouped_linear_wgrad(g.ptr(), x.ptr(), static_cast<float*>(sg.ptr()),
                                   static_cast<float*>(sx.ptr()), e.off(), e.cnt(),
                                   (int32_t)e.experts, rows, n, k, dw.ptr, s));
  return dw.take();
}

// ------------------------------------------------------------------------- the module

template <PyObject* (*F)(PyObject* const*), int NARGS>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != NARGS) return PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", NARGS, n);
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "fp8lin binding failed");
  }
  return nullptr;
}

// bind(addresses by entry point name, new, check, current_device, raw_stream)
PyObject* bind(PyObject* const* p) {
  auto take = [&](const char* name, auto& fn) {
    PyObject* a = PyDict_GetItemString(p[0], name);
    if (!a) bad(std::string("no entry point ") + name);
    void* v = PyLong_AsVoidPtr(a);
    if (!v) bad(std::string("no address for ") + name);
    fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(v);
  };
  take("fp8_layernorm_fwd", entry.layernorm_fwd);
  take("fp8_layernorm_bwd", entry.layernorm_bwd);
  take("fp8_layernorm_bwd_workspace", entry.layernorm_bwd_workspace);
  take("fp8_moe_rows", entry.moe_rows);
  take("fp8_moe_sort_workspace", entry.moe_sort_workspace);
  take("fp8_moe_sort", entry.moe_sort);
  take("fp8_moe_dispatch", entry.moe_dispatch);
  take("fp8_moe_dispatch_bwd", entry.moe_dispatch_bwd);
  take("fp8_moe_combine", entry.moe_combine);
  take("fp8_moe_combine_bwd", entry.moe_combine_bwd);
  take("fp8_moe_route_workspace", entry.moe_route_workspace);
  take("fp8_moe_route", entry.moe_route);
  take("fp8_moe_route_bwd", entry.moe_route_bwd);
  take("fp8_act_quantize", entry.act_quantize);
  take("fp8_act_quantize_bwd", entry.act_quantize_bwd);
  take("fp8_grouped_linear_fwd", entry.grouped_linear_fwd);
  take("fp8_grouped_linear_dgrad", entry.grouped_linear_dgrad);
  take("fp8_grouped_linear_wgrad", entry.grouped_linear_wgrad);
  PyObject** const held[] = {&py_new, &py_check, &py_device, &py_raw_stream};
  for (int i = 0; i < 4; ++i) {
    PyObject* old = *held[i];
    *held[i] = Py_NewRef(p[1 + i]);
    Py_XDECREF(old);
  }
  return Py_NewRef(Py_None);
}

#define FP8LIN_FN(name, nargs)                                                                   \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<name, nargs>)),       \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FP8LIN_FN(bind, 5),          FP8LIN_FN(layernorm_fwd, 9),
                         FP8LIN_FN(layernorm_bwd, 14), FP8LIN_FN(moe_sort, 9),
                         FP8LIN_FN(moe_dispatch, 5),   FP8LIN_FN(moe_dispatch_bwd, 4),
                         FP8LIN_FN(moe_combine, 5),    FP8LIN_FN(moe_combine_bwd, 8),
                         FP8LIN_FN(moe_route, 11),     FP8LIN_FN(moe_route_bwd, 11),
                         FP8LIN_FN(act_quantize, 14),  FP8LIN_FN(act_quantize_bwd, 15),
                         FP8LIN_FN(grouped_linear, 10), FP8LIN_FN(grouped_wgrad, 8),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
