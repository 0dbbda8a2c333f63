// Python module of the row operators over the ranks: checks the tensors of a
// call, collects their addresses and calls the C ABI (include/hbmcoll.h).
//
// A decode step's operator runs for about 5 us, and a call names up to 40
// tensors.  The norms' of 8 ranks: 28 us for the checks in Python and 1.5 us for
// the whole call here, on one host; one row's call 19.1 and 5.6 us on an MI355X's.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <string>
#include <vector>

#include "hbmcoll.h"

namespace {

constexpr int kMaxRanks = 64;

// Thrown where a Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised();
}

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: a tensor is needed, got %.80s", what, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

int dtype_code(const at::Tensor& t, const char* what) {
  switch (t.scalar_type()) {
    case at::kFloat: return HBMC_FP32;
    case at::kHalf: return HBMC_FP16;
    case at::kBFloat16: return HBMC_BF16;
    default: raise(PyExc_TypeError, "%s: unsupported tensor dtype %s", what, c10::toString(t.scalar_type()));
  }
}

int id_bytes(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kInt) return 4;
  if (t.scalar_type() == at::kLong) return 8;
  raise(PyExc_TypeError, "%s: ids are int32 or int64, got %s", what, c10::toString(t.scalar_type()));
}

// The tensors of one call: P ranks, all on device `dev`.
struct Call {
  int P, dev;

  void* address(const at::Tensor& t, at::ScalarType dtype, at::IntArrayRef shape, const char* what, int rank = -1) const {
    if (t.scalar_type() != dtype || t.get_device() != dev || t.sizes() != shape || !t.is_contiguous()) {
      const std::string of = rank < 0 ? "" : " of rank " + std::to_string(rank);
      raise(PyExc_ValueError, "%s%s: a contiguous %s tensor of shape %s on device %d is needed, got %s%s %s on device %d", what,
            of.c_str(), c10::toString(dtype), text(shape).c_str(), dev, t.is_contiguous() ? "" : "non-contiguous ",
            c10::toString(t.scalar_type()), text(t.sizes()).c_str(), static_cast<int>(t.get_device()));
    }
    return t.data_ptr();
  }
  void* address(PyObject* o, at::ScalarType dtype, at::IntArrayRef shape, const char* what) const {
    return address(tensor(o, what), dtype, shape, what);
  }
  void* optional(PyObject* o, at::ScalarType dtype, at::IntArrayRef shape, const char* what) const {
    return o == Py_None ? nullptr : address(o, dtype, shape, what);
  }
};

// The ranks' tensors of one argument: a list or tuple of P, or one tensor whose
// first dimension is the rank.
class Ranks {
 public:
  Ranks(PyObject* o, const Call& c, const char* what) : call_(c), what_(what) {
    if (THPVariable_Check(o)) {
      whole_ = &THPVariable_Unpack(o);
      if (whole_->dim() < 1 || whole_->size(0) != c.P) raise(PyExc_ValueError, "%s: [%d, ...] is needed for %d ranks", what, c.P, c.P);
      sizes_ = whole_->sizes().slice(1);
      dtype_ = whole_->scalar_type();
      return;
    }
    if (!PyList_Check(o) && !PyTuple_Check(o))
      raise(PyExc_TypeError, "%s: a list of tensors is needed, got %.80s", what, Py_TYPE(o)->tp_name);
    if (PySequence_Fast_GET_SIZE(o) != c.P)
      raise(PyExc_ValueError, "%s: %d tensors are needed, got %d", what, c.P, static_cast<int>(PySequence_Fast_GET_SIZE(o)));
    items_ = PySequence_Fast_ITEMS(o);
    const at::Tensor& first = tensor(items_[0], what);
    sizes_ = first.sizes();
    dtype_ = first.scalar_type();
  }
  at::ScalarType dtype() const { return dtype_; }
  // Sizes of rank r's tensor, without checks of anything else.
  at::IntArrayRef sizes(int r) const { return items_ ? tensor(items_[r], what_).sizes() : sizes_; }
  int64_t size(int r, int dim, int dims) const {
    const at::IntArrayRef s = sizes(r);
    if (static_cast<int>(s.size()) != dims) raise(PyExc_ValueError, "%s: %d dimensions are needed, got %s", what_, dims, text(s).c_str());
    return s[dim];
  }
  const at::Tensor& first() const { return whole_ ? *whole_ : THPVariable_Unpack(items_[0]); }
  // Addresses of the ranks' tensors, rank r of shape [rows(r), columns(r)] (one
  // dimension where `flat`).
  template <typename Rows, typename Columns>
  void addresses(at::ScalarType dtype, Rows&& rows, Columns&& columns, bool flat, void** to) const {
    if (whole_) {
      const int64_t shape[3] = {call_.P, rows(0), columns(0)};
      for (int r = 1; r < call_.P; ++r)
        if (rows(r) != shape[1] || columns(r) != shape[2])
          raise(PyExc_TypeError, "%s: the ranks' tensors differ in shape, so a list of them is needed", what_);
      char* base = static_cast<char*>(call_.address(*whole_, dtype, at::IntArrayRef(shape, flat ? 2 : 3), what_));
      const int64_t step = shape[1] * (flat ? 1 : shape[2]) * static_cast<int64_t>(whole_->element_size());
      for (int r = 0; r < call_.P; ++r) to[r] = base + r * step;
      return;
    }
    for (int r = 0; r < call_.P; ++r) {
      const int64_t shape[2] = {rows(r), columns(r)};
      to[r] = call_.address(tensor(items_[r], what_), dtype, at::IntArrayRef(shape, flat ? 1 : 2), what_, r);
    }
  }

 private:
  const Call& call_;
  const char* what_;
  const at::Tensor* whole_ = nullptr;
  PyObject** items_ = nullptr;
  at::IntArrayRef sizes_;
  at::ScalarType dtype_;
};

// Rows or columns of n that rank r owns (the ceiling split).
struct Split {
  int64_t n;
  int P;
  int64_t operator()(int r) const {
    const int64_t each = (n + P - 1) / P, left = n - r * each;
    return left <= 0 ? 0 : (left < each ? left : each);
  }
};

struct Always {
  int64_t n;
  int64_t operator()(int) const { return n; }
};

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

void* pointer(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised();
  return p;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}

// Workspace of `bytes` from the caller's allocator (alloc(bytes) -> tensor).
class Scratch {
 public:
  Scratch(PyObject* alloc, size_t bytes) {
    if (bytes == 0) return;
    PyObject* n = PyLong_FromSize_t(bytes);
    held_ = n ? PyObject_CallOneArg(alloc, n) : nullptr;
    Py_XDECREF(n);
    if (!held_) throw Raised();
    if (!THPVariable_Check(held_)) {
      Py_DECREF(held_);
      raise(PyExc_TypeError, "the workspace is a tensor");
    }
  }
  ~Scratch() { Py_XDECREF(held_); }
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
  void* data() const { return held_ ? THPVariable_Unpack(held_).data_ptr() : nullptr; }

 private:
  PyObject* held_ = nullptr;
};

// Arguments common to all functions: (comm handle, P, device, stream, ...).
struct Head {
  hbmc_comm_t comm;
  Call call;
  void* stream;
  Head(PyObject* const* a)
      : comm(static_cast<hbmc_comm_t>(pointer(a[0]))), call{static_cast<int>(integer(a[1])), static_cast<int>(integer(a[2]))},
        stream(pointer(a[3])) {
    if (call.P < 1 || call.P > kMaxRanks) raise(PyExc_ValueError, "%d ranks", call.P);
  }
};

// The descriptor of the norms from the ranks' first argument and the weights.
hbmc_norm_t norm_of(const Call& c, const Ranks& first, const char* what, PyObject* pre, PyObject* post, PyObject* gate,
                    PyObject* scale, PyObject* eps, PyObject* post_eps, int64_t* groups) {
  hbmc_norm_t n = {};
  const int64_t rows = first.size(0, 0, 2), width = first.size(0, 1, 2);
  n.dtype = static_cast<hbmc_dtype_t>(dtype_code(first.first(), what));
  n.rows = static_cast<size_t>(rows);
  n.width = static_cast<size_t>(width);
  n.gate_rows = 1;
  n.scale = real(scale);
  n.pre_eps = real(eps);
  n.post_eps = post_eps == Py_None ? n.pre_eps : real(post_eps);
  n.pre_weight = c.address(pre, first.dtype(), {width}, "pre_weight");
  n.post_weight = c.optional(post, first.dtype(), {width}, "post_weight");
  *groups = 0;
  if (gate != Py_None) {
    const at::Tensor& g = tensor(gate, "gate");
    *groups = g.dim() == 2 ? g.size(0) : -1;
    if (*groups < 0 || (*groups == 0 ? rows != 0 : rows % *groups != 0))
      raise(PyExc_ValueError, "gate: [groups, width] is needed with groups dividing %lld rows evenly, got %s",
            static_cast<long long>(rows), text(g.sizes()).c_str());
    n.gate = c.address(g, first.dtype(), {*groups, width}, "gate");
    if (*groups > 0 && rows > 0) n.gate_rows = static_cast<size_t>(rows / *groups);
  }
  return n;
}

hbmc_status_t reduce_norm(PyObject* const* a) {
  // parts, residual, residual_out, out, sums, pre, post, gate, scale, eps, post_eps
  const Head h(a);
  const Call& c = h.call;
  const Ranks parts(a[4], c, "parts");
  int64_t groups;
  const hbmc_norm_t n = norm_of(c, parts, "parts", a[9], a[10], a[11], a[12], a[13], a[14], &groups);
  const at::ScalarType dt = parts.dtype();
  const Always rows{static_cast<int64_t>(n.rows)}, width{static_cast<int64_t>(n.width)};
  const Split mine{rows.n, c.P};
  void *p[kMaxRanks], *res[kMaxRanks], *res_out[kMaxRanks], *out[kMaxRanks], *sums[kMaxRanks];
  parts.addresses(dt, rows, width, false, p);
  Ranks(a[5], c, "residual").addresses(dt, mine, width, false, res);
  if (a[6] != Py_None) Ranks(a[6], c, "residual_out").addresses(dt, mine, width, false, res_out);
  Ranks(a[7], c, "out").addresses(dt, rows, width, false, out);
  if (a[8] != Py_None) Ranks(a[8], c, "sums").addresses(dt, mine, width, false, sums);
  return hbmc_reduce_norm(h.comm, &n, p, res, a[6] == Py_None ? res : res_out, out, a[8] == Py_None ? nullptr : sums, h.stream);
}

hbmc_status_t reduce_norm_grad(PyObject* const* a) {
  // out_grads, hidden, part_grads, residual_grad, pre, pre_grad, sums, residual_grad_in, post, post_grad, gate, gate_grad,
  // scale, eps, post_eps, alloc
  const Head h(a);
  const Call& c = h.call;
  const Ranks grads(a[4], c, "out_grads");
  int64_t groups;
  const hbmc_norm_t n = norm_of(c, grads, "out_grads", a[8], a[12], a[14], a[16], a[17], a[18], &groups);
  const bool has_post = a[12] != Py_None, has_gate = a[14] != Py_None, has_sums = a[10] != Py_None, has_in = a[11] != Py_None;
  if (has_post != (a[13] != Py_None) || has_gate != (a[15] != Py_None))
    raise(PyExc_ValueError, "post_weight_grad and gate_grad go with post_weight and gate");
  if ((has_post || has_gate) && !has_sums) raise(PyExc_ValueError, "the forward call's sums are needed with post_weight or gate");
  const at::ScalarType dt = grads.dtype();
  const Always rows{static_cast<int64_t>(n.rows)}, width{static_cast<int64_t>(n.width)};
  const Split mine{rows.n, c.P};
  void *g[kMaxRanks], *hid[kMaxRanks], *sums[kMaxRanks], *in[kMaxRanks], *part[kMaxRanks], *res[kMaxRanks];
  grads.addresses(dt, rows, width, false, g);
  Ranks(a[5], c, "hidden").addresses(dt, mine, width, false, hid);
  Ranks(a[6], c, "part_grads").addresses(dt, rows, width, false, part);
  Ranks(a[7], c, "residual_grad").addresses(dt, mine, width, false, res);
  if (has_sums) Ranks(a[10], c, "sums").addresses(dt, mine, width, false, sums);
  if (has_in) Ranks(a[11], c, "residual_grad_in").addresses(dt, mine, width, false, in);
  float* pre = static_cast<float*>(c.address(a[9], at::kFloat, {width.n}, "pre_weight_grad"));
  float* post = static_cast<float*>(c.optional(a[13], at::kFloat, {width.n}, "post_weight_grad"));
  float* gate = static_cast<float*>(c.optional(a[15], at::kFloat, {groups, width.n}, "gate_grad"));
  size_t bytes = 0;
  const hbmc_status_t st = hbmc_reduce_norm_grad_workspace(h.comm, &n, &bytes);
  if (st != HBMC_OK) return st;
  const Scratch ws(a[19], bytes);
  return hbmc_reduce_norm_grad(h.comm, &n, g, hid, has_sums ? sums : nullptr, has_in ? in : nullptr, part, res, pre, post, gate,
                              ws.data(), bytes, h.stream);
}

// The embedding's descriptor from its table (or the table's gradient) and ids.
hbmc_embedding_t embedding_of(const Call& c, const Ranks& table, const Ranks& ids, hbmc_dtype_t dtype, PyObject* scale,
                              void** rows, void** id, size_t* tokens) {
  hbmc_embedding_t m = {};
  int64_t vocab = 0;
  const int64_t width = table.size(0, 1, 2);
  for (int r = 0; r < c.P; ++r) vocab += table.size(r, 0, 2);
  table.addresses(table.dtype(), Split{vocab, c.P}, Always{width}, false, rows);
  m.id_bytes = id_bytes(ids.first(), "ids");
  for (int r = 0; r < c.P; ++r) tokens[r] = static_cast<size_t>(ids.size(r, 0, 1));
  ids.addresses(ids.dtype(), [&](int r) { return static_cast<int64_t>(tokens[r]); }, Always{1}, true, id);
  m.vocab = static_cast<size_t>(vocab);
  m.width = static_cast<size_t>(width);
  m.dtype = dtype;
  m.scale = real(scale);
  return m;
}

hbmc_status_t embedding(PyObject* const* a) {
  // tables, ids, out, scale
  const Head h(a);
  const Call& c = h.call;
  const Ranks tables(a[4], c, "tables"), ids(a[5], c, "ids");
  void *rows[kMaxRanks], *id[kMaxRanks], *out[kMaxRanks];
  size_t tokens[kMaxRanks];
  const hbmc_dtype_t code = static_cast<hbmc_dtype_t>(dtype_code(tables.first(), "tables"));
  const hbmc_embedding_t m = embedding_of(c, tables, ids, code, a[7], rows, id, tokens);
  Ranks(a[6], c, "out").addresses(tables.dtype(), [&](int r) { return static_cast<int64_t>(tokens[r]); },
                                  Always{static_cast<int64_t>(m.width)}, false, out);
  return hbmc_embedding(h.comm, &m, rows, id, tokens, out, h.stream);
}

hbmc_status_t embedding_grad(PyObject* const* a) {
  // out_grads, ids, table_grads, scale, accumulate, alloc
  const Head h(a);
  const Call& c = h.call;
  const Ranks grads(a[4], c, "out_grads"), ids(a[5], c, "ids"), table(a[6], c, "table_grads");
  void *rows[kMaxRanks], *id[kMaxRanks], *out[kMaxRanks];
  size_t tokens[kMaxRanks];
  const hbmc_dtype_t code = static_cast<hbmc_dtype_t>(dtype_code(grads.first(), "out_grads"));
  const hbmc_dtype_t grad = static_cast<hbmc_dtype_t>(dtype_code(table.first(), "table_grads"));
  if (grad != code && grad != HBMC_FP32) raise(PyExc_TypeError, "table_grads are fp32 or of out_grads' type");
  const hbmc_embedding_t m = embedding_of(c, table, ids, code, a[7], out, id, tokens);
  grads.addresses(grads.dtype(), [&](int r) { return static_cast<int64_t>(tokens[r]); }, Always{static_cast<int64_t>(m.width)},
                  false, rows);
  const int accumulate = PyObject_IsTrue(a[8]);
  if (accumulate < 0) throw Raised();
  size_t bytes = 0;
  const hbmc_status_t st = hbmc_embedding_grad_workspace(h.comm, &m, tokens, &bytes);
  if (st != HBMC_OK) return st;
  const Scratch ws(a[9], bytes);
  return hbmc_embedding_grad(h.comm, &m, rows, id, tokens, out, grad, accumulate, ws.data(), bytes, h.stream);
}

hbmc_distill_t distill_of(const Call& c, const Ranks& logits, PyObject* teacher, PyObject* ids, PyObject* temperature) {
  hbmc_distill_t d = {};
  const at::Tensor &t = tensor(teacher, "teacher_logits"), &k = tensor(ids, "teacher_ids");
  if (t.dim() != 2) raise(PyExc_ValueError, "teacher_logits: [rows, top] is needed, got %s", text(t.sizes()).c_str());
  int64_t vocab = 0;
  for (int r = 0; r < c.P; ++r) vocab += logits.size(r, 1, 2);
  d.rows = static_cast<size_t>(t.size(0));
  d.vocab = static_cast<size_t>(vocab);
  d.top = static_cast<size_t>(t.size(1));
  d.dtype = static_cast<hbmc_dtype_t>(dtype_code(logits.first(), "logits"));
  d.teacher_dtype = static_cast<hbmc_dtype_t>(dtype_code(t, "teacher_logits"));
  d.id_bytes = id_bytes(k, "teacher_ids");
  d.temperature = real(temperature);
  d.teacher_logits = c.address(t, t.scalar_type(), t.sizes(), "teacher_logits");
  d.teacher_ids = c.address(k, k.scalar_type(), t.sizes(), "teacher_ids");
  return d;
}

hbmc_status_t distill_loss(PyObject* const* a) {
  // logits, teacher_logits, teacher_ids, loss, lse, temperature, alloc
  const Head h(a);
  const Call& c = h.call;
  const Ranks logits(a[4], c, "logits");
  const hbmc_distill_t d = distill_of(c, logits, a[5], a[6], a[9]);
  const int64_t rows = static_cast<int64_t>(d.rows);
  void* z[kMaxRanks];
  logits.addresses(logits.dtype(), Always{rows}, Split{static_cast<int64_t>(d.vocab), c.P}, false, z);
  float* loss = static_cast<float*>(c.address(a[7], at::kFloat, {rows}, "loss"));
  float* lse = static_cast<float*>(c.address(a[8], at::kFloat, {rows}, "lse"));
  size_t bytes = 0;
  const hbmc_status_t st = hbmc_distill_loss_workspace(h.comm, &d, &bytes);
  if (st != HBMC_OK) return st;
  const Scratch ws(a[10], bytes);
  return hbmc_distill_loss(h.comm, &d, z, loss, lse, ws.data(), bytes, h.stream);
}

hbmc_status_t distill_loss_grad(PyObject* const* a) {
  // logits, teacher_logits, teacher_ids, lse, loss_grad, logit_grads, temperature
  const Head h(a);
  const Call& c = h.call;
  const Ranks logits(a[4], c, "logits");
  const hbmc_distill_t d = distill_of(c, logits, a[5], a[6], a[10]);
  const Always rows{static_cast<int64_t>(d.rows)};
  const Split columns{static_cast<int64_t>(d.vocab), c.P};
  void *z[kMaxRanks], *g[kMaxRanks];
  logits.addresses(logits.dtype(), rows, columns, false, z);
  const float* lse = static_cast<float*>(c.address(a[7], at::kFloat, {rows.n}, "lse"));
  const float* dl = static_cast<float*>(c.address(a[8], at::kFloat, {rows.n}, "loss_grad"));
  Ranks(a[9], c, "logit_grads").addresses(logits.dtype(), rows, columns, false, g);
  return hbmc_distill_loss_grad(h.comm, &d, z, lse, dl, g, h.stream);
}

// Entry of one function: its number of arguments, the status it returns, and no
// C++ exception past it.
template <hbmc_status_t (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(args));
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <hbmc_status_t (*F)(PyObject* const*), Py_ssize_t N>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<reduce_norm, 15>("reduce_norm"),
                         method<reduce_norm_grad, 20>("reduce_norm_grad"),
                         method<embedding, 8>("embedding"),
                         method<embedding_grad, 10>("embedding_grad"),
                         method<distill_loss, 11>("distill_loss"),
                         method<distill_loss_grad, 11>("distill_loss_grad"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
