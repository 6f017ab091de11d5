// Native front of the hard selections' Python binding: the calls of hard.py
// for arguments that need no conversion (right types, contiguous, on the current
// device), without the interpreter's share of the checks and allocations (about 4 us a
// call).  Every function returns None for anything else, refusals included, and hard.py then
// takes its own way, which converts or raises.  It holds no kernel and no formula: it calls
// the C ABI through addresses that hard.py hands over.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/lapsum.h"

namespace {

struct Entries {
  decltype(&lapsum_route_forward) route_forward;
  decltype(&lapsum_route_backward) route_backward;
  decltype(&lapsum_dispatch_plan_workspace_bytes) plan_bytes;
  decltype(&lapsum_dispatch_plan) plan;
  decltype(&lapsum_dispatch_forward) dispatch_forward;
  decltype(&lapsum_dispatch_backward) dispatch_backward;
  decltype(&lapsum_combine_forward) combine_forward;
  decltype(&lapsum_combine_backward) combine_backward;
  decltype(&lapsum_cache_attend_workspace_bytes) attend_bytes;
  decltype(&lapsum_cache_attend) attend;
  decltype(&lapsum_cache_evict_workspace_bytes) evict_bytes;
  decltype(&lapsum_cache_evict) evict;
  decltype(&lapsum_expert_product_forward) product_forward;
  decltype(&lapsum_expert_product_backward_rows) product_backward_rows;
  decltype(&lapsum_expert_product_backward_weights) product_backward_weights;
  decltype(&lapsum_beam_select_workspace_bytes) beam_bytes;
  decltype(&lapsum_beam_select) beam_select;
  decltype(&lapsum_cache_reorder) reorder;
};
Entries entry{};

PyObject *none() {
  if (PyErr_Occurred()) PyErr_Clear();
  Py_RETURN_NONE;
}

PyObject *failed = nullptr;  // raises for (status, name)

// After a C call that did not succeed.  Arguments that it refuses are hard.py's to explain; a
// launch that failed is raised here and not sent again, since an earlier one of the same call may
// have changed what it works on.
PyObject *refused(lapsum_status st, const char *name) {
  if (st != LAPSUM_ERR_HIP || failed == nullptr) return none();
  PyObject *done = PyObject_CallFunction(failed, "is", (int)st, name);
  if (done == nullptr) return nullptr;
  Py_DECREF(done);
  return none();
}

// A GPU tensor on the current device, or null.
const at::Tensor *gpu(int dev, PyObject *o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor &t = THPVariable_Unpack(o);
  return t.is_cuda() && t.device().index() == dev && t.numel() > 0 ? &t : nullptr;
}
int dtype_of(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return LAPSUM_F32;
    case at::kBFloat16: return LAPSUM_BF16;
    case at::kHalf: return LAPSUM_F16;
    default: return -1;
  }
}
// contiguous, of this type and of as many elements
bool plain(const at::Tensor *t, at::ScalarType type, int64_t numel) {
  return t != nullptr && t->scalar_type() == type && t->numel() == numel && t->is_contiguous();
}
bool rows(const at::Tensor *t) {  // [tokens, n], rows in order
  return t != nullptr && t->dim() == 2 && t->stride(1) == 1 && t->stride(0) >= t->size(1) && dtype_of(*t) >= 0;
}
void *stream_of(const at::Tensor &t) { return c10::hip::getCurrentHIPStream(t.device().index()).stream(); }
// A new tensor on the current device, from torch's pool for its current stream (without
// the dispatcher, which takes as long again).
at::Tensor make(int dev, at::IntArrayRef shape, at::ScalarType type) {
  return at::Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)dev),
                                           std::nullopt));
}
struct Workspace {
  at::Tensor buffer;
  void *at = nullptr;
  size_t bytes = 0;
  Workspace(int dev, size_t n) {
    if (n == 0) return;
    buffer = make(dev, {(int64_t)n + 256}, at::kByte);
    const uintptr_t p = reinterpret_cast<uintptr_t>(buffer.data_ptr()), up = (p + 255) / 256 * 256;
    at = reinterpret_cast<void *>(up);
    bytes = n;
  }
};
// A 32-bit integer; anything else leaves an error set.
int32_t int32_of(PyObject *o) {
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &over);
  if (over != 0 || x < INT32_MIN || x > INT32_MAX) PyErr_SetNone(PyExc_OverflowError);
  return (int32_t)x;
}
// A tensor of the caller has been changed in place, for autograd.
void written(const at::Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
PyObject *wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject *pair(at::Tensor a, at::Tensor b) { return Py_BuildValue("(NN)", wrap(std::move(a)), wrap(std::move(b))); }

#define BODY(count)                \
  if (n != (count)) return none(); \
  try {                            \
    const int dev = c10::hip::current_device();
#define END                        \
  }                                \
  catch (const std::exception &) { \
    return none();                 \
  }

PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != (Py_ssize_t)(sizeof(Entries) / sizeof(void *))) return none();
  void **to = reinterpret_cast<void **>(&entry);
  for (Py_ssize_t i = 0; i < n; ++i) to[i] = PyLong_AsVoidPtr(args[i]);
  Py_RETURN_NONE;
}

// (callable): what raises for a status and a name
PyObject *on_failure(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 1) return none();
  Py_INCREF(args[0]);
  Py_XDECREF(failed);
  failed = args[0];
  Py_RETURN_NONE;
}

// (logits, bias, k, score, groups, top_groups, renormalise, scale)
PyObject *route_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(8)
  const at::Tensor *x = gpu(dev, args[0]), *bias = args[1] == Py_None ? nullptr : gpu(dev, args[1]);
  if (!rows(x) || (args[1] != Py_None && !(plain(bias, at::kFloat, x->size(1)) && bias->dim() == 1))) return none();
  lapsum_route_options o;
  o.k = int32_of(args[2]);
  o.score = int32_of(args[3]);
  o.groups = int32_of(args[4]);
  o.top_groups = args[5] == Py_None ? o.groups : int32_of(args[5]);
  o.renormalise = PyObject_IsTrue(args[6]);
  o.scale = (float)PyFloat_AsDouble(args[7]);
  if (PyErr_Occurred() || o.k < 1 || o.k > LAPSUM_MAX_CHOICES) return none();
  at::Tensor w = make(dev, {x->size(0), o.k}, at::kFloat), c = make(dev, {x->size(0), o.k}, at::kInt);
  const lapsum_status st =
      entry.route_forward(x->data_ptr(), dtype_of(*x), x->size(0), x->size(1), x->stride(0),
                          bias ? static_cast<const float *>(bias->data_ptr()) : nullptr, &o,
                          static_cast<float *>(w.data_ptr()), static_cast<int32_t *>(c.data_ptr()), stream_of(*x));
  if (st != LAPSUM_OK) return refused(st, "lapsum_route_forward");
  return pair(std::move(w), std::move(c));
  END
}

// (dweights, logits, chosen, score, renormalise, scale)
PyObject *route_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(6)
  const at::Tensor *dw = gpu(dev, args[0]), *x = gpu(dev, args[1]), *c = gpu(dev, args[2]);
  if (!rows(x) || c == nullptr || c->dim() != 2 || c->size(0) != x->size(0) || !plain(c, at::kInt, c->numel()) ||
      !plain(dw, at::kFloat, c->numel()) || dw->sizes() != c->sizes())
    return none();
  lapsum_route_options o{};
  o.k = (int32_t)c->size(1);
  o.score = int32_of(args[3]);
  o.groups = o.top_groups = 1;
  o.renormalise = PyObject_IsTrue(args[4]);
  o.scale = (float)PyFloat_AsDouble(args[5]);
  if (PyErr_Occurred()) return none();
  at::Tensor dx = make(dev, {x->size(0), x->size(1)}, x->scalar_type());
  const lapsum_status st =
      entry.route_backward(static_cast<const float *>(dw->data_ptr()), x->data_ptr(), dtype_of(*x), x->size(0),
                           x->size(1), x->stride(0), static_cast<const int32_t *>(c->data_ptr()), &o, dx.data_ptr(),
                           stream_of(*x));
  if (st != LAPSUM_OK) return refused(st, "lapsum_route_backward");
  return wrap(std::move(dx));
  END
}

// (chosen, experts)
PyObject *dispatch_plan(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(2)
  const at::Tensor *c = gpu(dev, args[0]);
  const int64_t experts = PyLong_AsLongLong(args[1]);
  if (PyErr_Occurred() || c == nullptr || c->dim() != 2 || !plain(c, at::kInt, c->numel()) || experts < 1 ||
      experts > LAPSUM_MAX_EXPERTS)
    return none();
  const int64_t tokens = c->size(0), k = c->size(1);
  at::Tensor offsets = make(dev, {experts + 1}, at::kInt), slot = make(dev, {tokens, k}, at::kInt);
  at::Tensor order = make(dev, {tokens * k}, at::kInt);
  const Workspace ws(dev, entry.plan_bytes(tokens, k, experts));
  const lapsum_status st =
      entry.plan(static_cast<const int32_t *>(c->data_ptr()), tokens, k, experts,
                 static_cast<int32_t *>(offsets.data_ptr()), static_cast<int32_t *>(slot.data_ptr()),
                 static_cast<int32_t *>(order.data_ptr()), ws.at, ws.bytes, stream_of(*c));
  if (st != LAPSUM_OK) return refused(st, "lapsum_dispatch_plan");
  return Py_BuildValue("(NNN)", wrap(std::move(offsets)), wrap(std::move(slot)), wrap(std::move(order)));
  END
}

bool slots(const at::Tensor *s) { return s != nullptr && s->dim() == 2 && plain(s, at::kInt, s->numel()); }
bool offsets_of(const at::Tensor *o) { return o != nullptr && o->dim() == 1 && plain(o, at::kInt, o->numel()); }

// (x, slot, offsets)
PyObject *dispatch_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(3)
  const at::Tensor *x = gpu(dev, args[0]), *s = gpu(dev, args[1]), *o = gpu(dev, args[2]);
  if (!rows(x) || !slots(s) || s->size(0) != x->size(0) || !offsets_of(o)) return none();
  at::Tensor xs = make(dev, {s->numel(), x->size(1)}, x->scalar_type());
  const lapsum_status st =
      entry.dispatch_forward(x->data_ptr(), dtype_of(*x), x->size(0), s->size(1), x->size(1), x->stride(0),
                             static_cast<const int32_t *>(s->data_ptr()),
                             static_cast<const int32_t *>(o->data_ptr()), o->numel() - 1, xs.data_ptr(),
                             stream_of(*x));
  if (st != LAPSUM_OK) return refused(st, "lapsum_dispatch_forward");
  return wrap(std::move(xs));
  END
}

// rows in expert order for these slots: [slot.numel(), width], contiguous
bool expert_rows(const at::Tensor *t, const at::Tensor *s) {
  return t != nullptr && t->dim() == 2 && dtype_of(*t) >= 0 && t->size(0) == s->numel() && t->is_contiguous();
}

// (dxs, slot)
PyObject *dispatch_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(2)
  const at::Tensor *t = gpu(dev, args[0]), *s = gpu(dev, args[1]);
  if (!slots(s) || !expert_rows(t, s)) return none();
  at::Tensor dx = make(dev, {s->size(0), t->size(1)}, t->scalar_type());
  const lapsum_status st =
      entry.dispatch_backward(t->data_ptr(), dtype_of(*t), s->size(0), s->size(1), t->size(1),
                              static_cast<const int32_t *>(s->data_ptr()), dx.data_ptr(), stream_of(*t));
  if (st != LAPSUM_OK) return refused(st, "lapsum_dispatch_backward");
  return wrap(std::move(dx));
  END
}

// (ys, slot, weights)
PyObject *combine_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(3)
  const at::Tensor *t = gpu(dev, args[0]), *s = gpu(dev, args[1]), *w = gpu(dev, args[2]);
  if (!slots(s) || !expert_rows(t, s) || !plain(w, at::kFloat, s->numel()) || w->sizes() != s->sizes()) return none();
  at::Tensor y = make(dev, {s->size(0), t->size(1)}, t->scalar_type());
  const lapsum_status st =
      entry.combine_forward(t->data_ptr(), dtype_of(*t), s->size(0), s->size(1), t->size(1),
                            static_cast<const int32_t *>(s->data_ptr()), static_cast<const float *>(w->data_ptr()),
                            y.data_ptr(), stream_of(*t));
  if (st != LAPSUM_OK) return refused(st, "lapsum_combine_forward");
  return wrap(std::move(y));
  END
}

// (dy, ys, slot, weights, offsets)
PyObject *combine_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(5)
  const at::Tensor *dy = gpu(dev, args[0]), *t = gpu(dev, args[1]), *s = gpu(dev, args[2]), *w = gpu(dev, args[3]), *o = gpu(dev, args[4]);
  if (!rows(dy) || !slots(s) || s->size(0) != dy->size(0) || !expert_rows(t, s) || t->size(1) != dy->size(1) ||
      t->scalar_type() != dy->scalar_type() || !plain(w, at::kFloat, s->numel()) || w->sizes() != s->sizes() ||
      !offsets_of(o))
    return none();
  at::Tensor dys = make(dev, {t->size(0), t->size(1)}, t->scalar_type());
  at::Tensor dw = make(dev, {s->size(0), s->size(1)}, at::kFloat);
  const lapsum_status st =
      entry.combine_backward(dy->data_ptr(), dy->stride(0), t->data_ptr(), dtype_of(*t), s->size(0), s->size(1),
                             t->size(1), static_cast<const int32_t *>(s->data_ptr()),
                             static_cast<const float *>(w->data_ptr()), static_cast<const int32_t *>(o->data_ptr()),
                             o->numel() - 1, dys.data_ptr(), static_cast<float *>(dw.data_ptr()), stream_of(*t));
  if (st != LAPSUM_OK) return refused(st, "lapsum_combine_backward");
  return pair(std::move(dys), std::move(dw));
  END
}

bool cache_of(const at::Tensor *k, const at::Tensor *v, lapsum_cache &c) {
  if (k == nullptr || v == nullptr || k->dim() != 4 || v->dim() != 4 || k->sizes() != v->sizes() ||
      k->scalar_type() != v->scalar_type() || dtype_of(*k) < LAPSUM_BF16 || k->stride(3) != 1 || v->stride(3) != 1)
    return false;
  c.k = k->data_ptr();
  c.v = v->data_ptr();
  c.dtype = dtype_of(*k);
  c.width = (int32_t)k->size(3);
  c.batch = k->size(0);
  c.heads = k->size(1);
  c.capacity = k->size(2);
  c.k_stride_batch = k->stride(0);
  c.k_stride_head = k->stride(1);
  c.k_stride_entry = k->stride(2);
  c.v_stride_batch = v->stride(0);
  c.v_stride_head = v->stride(1);
  c.v_stride_entry = v->stride(2);
  return true;
}
bool per_entry(const at::Tensor *t, const at::Tensor &k, at::ScalarType type) {
  return t != nullptr && t->dim() == 3 && plain(t, type, t->numel()) && t->size(0) == k.size(0) &&
         t->size(1) == k.size(1) && t->size(2) == k.size(2);
}
bool per_sequence(const at::Tensor *t, const at::Tensor &k) {
  return t != nullptr && t->dim() == 1 && plain(t, at::kInt, k.size(0));
}

// (q, k, v, lengths, account, scale, account_out); scale None: 1/sqrt(width)
PyObject *cache_attend(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(7)
  const at::Tensor *q = gpu(dev, args[0]), *k = gpu(dev, args[1]), *v = gpu(dev, args[2]), *lengths = gpu(dev, args[3]);
  lapsum_cache c{};
  if (!cache_of(k, v, c) || q == nullptr || q->dim() != 4 || q->scalar_type() != k->scalar_type() ||
      !q->is_contiguous() || q->size(0) != c.batch || q->size(3) != c.width || !per_sequence(lengths, *k))
    return none();
  const bool accounts = args[4] != Py_None;
  const at::Tensor *in = accounts ? gpu(dev, args[4]) : nullptr;
  const at::Tensor *to = args[6] != Py_None ? gpu(dev, args[6]) : in;
  if (accounts ? !per_entry(in, *k, at::kFloat) || !per_entry(to, *k, at::kFloat) : args[6] != Py_None) return none();
  const double scale = args[5] == Py_None ? 1.0 / std::sqrt((double)c.width) : PyFloat_AsDouble(args[5]);
  if (PyErr_Occurred()) return none();
  at::Tensor out = make(dev, q->sizes(), q->scalar_type());
  const Workspace ws(dev, entry.attend_bytes(&c, q->size(1), q->size(2), accounts ? 1 : 0));
  const lapsum_status st =
      entry.attend(q->data_ptr(), &c, static_cast<const int32_t *>(lengths->data_ptr()), q->size(1), q->size(2),
                   (float)scale, accounts ? static_cast<const float *>(in->data_ptr()) : nullptr,
                   accounts ? static_cast<float *>(to->data_ptr()) : nullptr, out.data_ptr(), ws.at, ws.bytes,
                   stream_of(*q));
  if (st != LAPSUM_OK) return refused(st, "lapsum_cache_attend");
  if (accounts) written(*to);
  return wrap(std::move(out));
  END
}

// (k, v, account, positions, lengths, keep, next_position, sinks, recent, account_out, positions_out)
PyObject *cache_evict(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(11)
  const at::Tensor *k = gpu(dev, args[0]), *v = gpu(dev, args[1]), *account = gpu(dev, args[2]), *positions = gpu(dev, args[3]);
  const at::Tensor *lengths = gpu(dev, args[4]), *next = args[6] == Py_None ? nullptr : gpu(dev, args[6]);
  const at::Tensor *account_out = args[9] == Py_None ? account : gpu(dev, args[9]);
  const at::Tensor *positions_out = args[10] == Py_None ? positions : gpu(dev, args[10]);
  lapsum_cache c{};
  if (!cache_of(k, v, c) || !per_entry(account, *k, at::kFloat) || !per_entry(positions, *k, at::kInt) ||
      !per_sequence(lengths, *k) || (args[6] != Py_None && !per_sequence(next, *k)) ||
      !per_entry(account_out, *k, at::kFloat) || !per_entry(positions_out, *k, at::kInt))
    return none();
  const int64_t keep = PyLong_AsLongLong(args[5]);
  const int32_t sinks = int32_of(args[7]), recent = int32_of(args[8]);
  if (PyErr_Occurred() || keep < 1 || keep > c.capacity) return none();
  at::Tensor kept = make(dev, {c.batch, c.heads, keep}, at::kInt), after = make(dev, {c.batch}, at::kInt);
  const Workspace ws(dev, entry.evict_bytes(&c, keep));
  const lapsum_status st =
      entry.evict(&c, static_cast<const float *>(account->data_ptr()),
                  static_cast<const int32_t *>(positions->data_ptr()),
                  static_cast<const int32_t *>(lengths->data_ptr()), keep,
                  next ? static_cast<const int32_t *>(next->data_ptr()) : nullptr, sinks, recent,
                  static_cast<float *>(account_out->data_ptr()), static_cast<int32_t *>(positions_out->data_ptr()),
                  static_cast<int32_t *>(kept.data_ptr()), static_cast<int32_t *>(after.data_ptr()), ws.at, ws.bytes,
                  stream_of(*k));
  if (st != LAPSUM_OK) return refused(st, "lapsum_cache_evict");
  for (const at::Tensor *t : {k, v, account_out, positions_out}) written(*t);
  return pair(std::move(kept), std::move(after));
  END
}

// [experts, inputs, outputs], stored so or with inputs and outputs changed over
bool matrices(const at::Tensor *w, lapsum_experts &e) {
  if (w == nullptr || w->dim() != 3 || dtype_of(*w) < 0) return false;
  e = lapsum_experts{w->data_ptr(), dtype_of(*w),   0,           w->size(0),  w->size(1),
                     w->size(2),    w->stride(0), w->stride(1), w->stride(2)};
  return (e.stride_output == 1 && e.stride_input >= e.outputs) || (e.stride_input == 1 && e.stride_output >= e.inputs);
}
bool expert_offsets(const at::Tensor *o, const lapsum_experts &e) { return offsets_of(o) && o->numel() == e.experts + 1; }
bool expert_side(const at::Tensor *x, const at::Tensor &w, int64_t width) {
  return rows(x) && x->scalar_type() == w.scalar_type() && x->size(1) == width && x->stride(0) <= LAPSUM_MAX_EXPERT_STRIDE;
}

// (xs, w, offsets)
PyObject *expert_product_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(3)
  const at::Tensor *x = gpu(dev, args[0]), *w = gpu(dev, args[1]), *o = gpu(dev, args[2]);
  lapsum_experts e;
  if (!matrices(w, e) || !expert_side(x, *w, e.inputs) || !expert_offsets(o, e)) return none();
  at::Tensor ys = make(dev, {x->size(0), e.outputs}, w->scalar_type());
  const lapsum_status st =
      entry.product_forward(x->data_ptr(), x->stride(0), x->size(0), &e,
                            static_cast<const int32_t *>(o->data_ptr()), ys.data_ptr(), stream_of(*x));
  if (st != LAPSUM_OK) return refused(st, "lapsum_expert_product_forward");
  return wrap(std::move(ys));
  END
}

// (dys, w, offsets)
PyObject *expert_product_backward_rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(3)
  const at::Tensor *dy = gpu(dev, args[0]), *w = gpu(dev, args[1]), *o = gpu(dev, args[2]);
  lapsum_experts e;
  if (!matrices(w, e) || !expert_side(dy, *w, e.outputs) || !expert_offsets(o, e)) return none();
  at::Tensor dxs = make(dev, {dy->size(0), e.inputs}, w->scalar_type());
  const lapsum_status st =
      entry.product_backward_rows(dy->data_ptr(), dy->stride(0), dy->size(0), &e,
                                  static_cast<const int32_t *>(o->data_ptr()), dxs.data_ptr(), stream_of(*dy));
  if (st != LAPSUM_OK) return refused(st, "lapsum_expert_product_backward_rows");
  return wrap(std::move(dxs));
  END
}

// (dys, xs, w, offsets)
PyObject *expert_product_backward_weights(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(4)
  const at::Tensor *dy = gpu(dev, args[0]), *x = gpu(dev, args[1]), *w = gpu(dev, args[2]), *o = gpu(dev, args[3]);
  lapsum_experts e;
  if (!matrices(w, e) || !expert_side(x, *w, e.inputs) || !expert_side(dy, *w, e.outputs) ||
      x->size(0) != dy->size(0) || !expert_offsets(o, e))
    return none();
  // stored as w is
  const bool swapped = e.stride_output != 1;
  at::Tensor dw = swapped ? make(dev, {e.experts, e.outputs, e.inputs}, w->scalar_type())
                          : make(dev, {e.experts, e.inputs, e.outputs}, w->scalar_type());
  e.w = dw.data_ptr();
  e.stride_expert = e.inputs * e.outputs;
  e.stride_input = swapped ? 1 : e.outputs;
  e.stride_output = swapped ? e.inputs : 1;
  const lapsum_status st =
      entry.product_backward_weights(x->data_ptr(), x->stride(0), dy->data_ptr(), dy->stride(0), x->size(0),
                                     static_cast<const int32_t *>(o->data_ptr()), &e, stream_of(*x));
  if (st != LAPSUM_OK) return refused(st, "lapsum_expert_product_backward_weights");
  return wrap(swapped ? dw.transpose(1, 2) : std::move(dw));
  END
}

// (logits, scores, k, ended, end_token); k None: the beams
PyObject *beam_select(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(5)
  const at::Tensor *x = gpu(dev, args[0]), *scores = gpu(dev, args[1]);
  const at::Tensor *ended = args[3] == Py_None ? nullptr : gpu(dev, args[3]);
  if (x == nullptr || x->dim() != 3 || dtype_of(*x) < 0 || x->stride(2) != 1 || x->stride(1) < x->size(2) ||
      x->stride(0) != x->stride(1) * x->size(1))
    return none();
  const int64_t batch = x->size(0), beams = x->size(1), vocab = x->size(2);
  if (!plain(scores, at::kFloat, batch * beams) || scores->dim() != 2 || scores->size(0) != batch) return none();
  int32_t end = 0;
  if (args[3] != Py_None) {
    if (!plain(ended, at::kBool, batch * beams) || ended->dim() != 2 || ended->size(0) != batch || args[4] == Py_None)
      return none();
    end = int32_of(args[4]);
  }
  const int32_t k = args[2] == Py_None ? (int32_t)std::min<int64_t>(beams, INT32_MAX) : int32_of(args[2]);
  if (PyErr_Occurred() || k < 1 || k > LAPSUM_MAX_BEAMS) return none();
  at::Tensor out = make(dev, {batch, k}, at::kFloat), parents = make(dev, {batch, k}, at::kInt);
  at::Tensor tokens = make(dev, {batch, k}, at::kInt);
  const Workspace ws(dev, entry.beam_bytes(batch, beams, vocab, k));
  const lapsum_status st =
      entry.beam_select(x->data_ptr(), dtype_of(*x), batch, beams, vocab, x->stride(1),
                        static_cast<const float *>(scores->data_ptr()),
                        ended ? static_cast<const uint8_t *>(ended->data_ptr()) : nullptr, end, k,
                        static_cast<float *>(out.data_ptr()), static_cast<int32_t *>(parents.data_ptr()),
                        static_cast<int32_t *>(tokens.data_ptr()), ws.at, ws.bytes, stream_of(*x));
  if (st != LAPSUM_OK) return refused(st, "lapsum_beam_select");
  return Py_BuildValue("(NNN)", wrap(std::move(out)), wrap(std::move(parents)), wrap(std::move(tokens)));
  END
}

// (k, v, parents, lengths, account, positions)
PyObject *cache_reorder(PyObject *, PyObject *const *args, Py_ssize_t n) {
  BODY(6)
  const at::Tensor *k = gpu(dev, args[0]), *v = gpu(dev, args[1]), *parents = gpu(dev, args[2]);
  const at::Tensor *lengths = gpu(dev, args[3]);
  const at::Tensor *account = args[4] == Py_None ? nullptr : gpu(dev, args[4]);
  const at::Tensor *positions = args[5] == Py_None ? nullptr : gpu(dev, args[5]);
  lapsum_cache c{};
  if (!cache_of(k, v, c) || parents == nullptr || parents->dim() != 2 || !plain(parents, at::kInt, c.batch) ||
      !per_sequence(lengths, *k) || (args[4] != Py_None && !per_entry(account, *k, at::kFloat)) ||
      (args[5] != Py_None && !per_entry(positions, *k, at::kInt)))
    return none();
  at::Tensor after = make(dev, {c.batch}, at::kInt);
  const lapsum_status st =
      entry.reorder(&c, parents->size(1), static_cast<const int32_t *>(parents->data_ptr()),
                    static_cast<const int32_t *>(lengths->data_ptr()),
                    account ? static_cast<float *>(account->data_ptr()) : nullptr,
                    positions ? static_cast<int32_t *>(positions->data_ptr()) : nullptr,
                    static_cast<int32_t *>(after.data_ptr()), stream_of(*k));
  if (st != LAPSUM_OK) return refused(st, "lapsum_cache_reorder");
  for (const at::Tensor *t : {k, v, account, positions})
    if (t != nullptr) written(*t);
  return wrap(std::move(after));
  END
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),
                         METHOD(on_failure),
                         METHOD(route_forward),
                         METHOD(route_backward),
                         METHOD(dispatch_plan),
                         METHOD(dispatch_forward),
                         METHOD(dispatch_backward),
                         METHOD(combine_forward),
                         METHOD(combine_backward),
                         METHOD(cache_attend),
                         METHOD(cache_evict),
                         METHOD(expert_product_forward),
                         METHOD(expert_product_backward_rows),
                         METHOD(expert_product_backward_weights),
                         METHOD(beam_select),
                         METHOD(cache_reorder),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
