// The serving calls of the Python package on torch tensors: argument checks,
// output allocation, device and stream, then the C entry point (declared in
// bitnest.h; its address comes from the package, which has the library open).
// A decode step makes these calls for every layer, and its kernels take a few
// microseconds: the same checks in Python took 12 to 40 us a call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "bitnest.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr int64_t kD = 128;

// The library's entry points, in the order of kNames.
struct Entries {
  decltype(&bitnest_rope) rope;
  decltype(&bitnest_kv_append) kv_append;
  decltype(&bitnest_kv_read) kv_read;
  decltype(&bitnest_prefix_attention_ws_bytes) ws_bytes;
  decltype(&bitnest_prefix_attention) prefix_attention;
  decltype(&bitnest_kv_weights) kv_weights;
  decltype(&bitnest_kv_evict) kv_evict;
} lib;
const char *const kNames[] = {"bitnest_rope",
                              "bitnest_kv_append",
                              "bitnest_kv_read",
                              "bitnest_prefix_attention_ws_bytes",
                              "bitnest_prefix_attention",
                              "bitnest_kv_weights",
                              "bitnest_kv_evict"};
PyObject *error_type = nullptr;  // the package's BitnestError(status, what)

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char *what) {
  PyErr_SetString(PyExc_ValueError, what);
  throw Refused();
}
void need(bool ok, const char *what) {
  if (!ok) refuse(what);
}

PyObject *done(int status, const char *what, PyObject *result) {
  if (status == 0) return result;
  Py_XDECREF(result);
  PyObject *e = PyObject_CallFunction(error_type, "is", status, what);
  if (e) {
    PyErr_SetObject(error_type, e);
    Py_DECREF(e);
  }
  return nullptr;
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int small(PyObject *o) {
  const int64_t v = integer(o);
  need(v >= INT_MIN && v <= INT_MAX, "an integer is out of range");
  return (int)v;
}
double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}

const Tensor &tensor(PyObject *o, const char *what) {
  need(THPVariable_Check(o), what);
  return THPVariable_Unpack(o);
}

// t's address, where it is a contiguous array of this type and shape on `dev`.
template <typename T = void>
T *array(const Tensor &t, ScalarType type, at::IntArrayRef shape, const at::Device &dev,
         const char *what) {
  if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous()) {
    std::string m = std::string(what) + ": a contiguous " + c10::toString(type) + " array [";
    for (size_t i = 0; i < shape.size(); ++i) m += (i ? ", " : "") + std::to_string(shape[i]);
    refuse((m + "] on " + dev.str()).c_str());
  }
  return static_cast<T *>(t.data_ptr());
}
template <typename T = void>
T *array(PyObject *o, ScalarType type, at::IntArrayRef shape, const at::Device &dev,
         const char *what) {
  return array<T>(tensor(o, what), type, shape, dev, what);
}

// The three tensors of (hi, lo, scale).
struct Planes {
  const Tensor *hi, *lo, *scale;
};
Planes planes(PyObject *o, const char *what) {
  need(PyTuple_Check(o) || PyList_Check(o), what);
  need(PySequence_Fast_GET_SIZE(o) == 3, what);
  PyObject **p = PySequence_Fast_ITEMS(o);
  return {&tensor(p[0], what), &tensor(p[1], what), &tensor(p[2], what)};
}
struct Addresses {
  uint8_t *hi, *lo;
  uint16_t *scale;
};
Addresses addresses(const Planes &p, at::IntArrayRef rows, bool lo, const at::Device &dev,
                    const char *what) {
  c10::SmallVector<int64_t, 4> half(rows.begin(), rows.end());
  half.push_back(kD / 2);
  return {array<uint8_t>(*p.hi, at::kByte, half, dev, what),
          lo ? array<uint8_t>(*p.lo, at::kByte, half, dev, what) : nullptr,
          array<uint16_t>(*p.scale, at::kHalf, rows, dev, what)};
}
bitnest_kv_cache cache(const Planes &k, const Planes &v, at::IntArrayRef rows, bool lo,
                       const at::Device &dev, const char *what) {
  const Addresses a = addresses(k, rows, lo, dev, what), b = addresses(v, rows, lo, dev, what);
  return {a.hi, a.lo, a.scale, b.hi, b.lo, b.scale};
}

// Float types of bitnest.h.
int float_type(const Tensor &t, const char *what) {
  if (t.scalar_type() == at::kHalf) return BITNEST_F16;
  if (t.scalar_type() == at::kFloat) return BITNEST_F32;
  refuse(what);
}

// The tensors' device and its current stream for the call.
struct On {
  c10::cuda::CUDAGuard guard;
  explicit On(const at::Device &d) : guard(d) {}
  void *stream() const { return c10::cuda::getCurrentCUDAStream().stream(); }
};

PyObject *rope(PyObject *const *a, Py_ssize_t) {
  // x, pos, phases, magnitude, layout, inverse, out, dtype
  const Tensor &x = tensor(a[0], "rope: x, a tensor [M, heads, D]");
  need(x.dim() == 3, "rope: x [M, heads, D]");
  const int64_t M = x.size(0), heads = x.size(1), D = x.size(2);
  const int xt = float_type(x, "rope: fp16 or fp32 arrays");
  need(x.is_cuda(), "rope: x on a GPU");
  const at::Device dev = x.device();
  On on(dev);
  Tensor y;
  if (a[6] != Py_None) {
    y = tensor(a[6], "rope: out, a tensor like x");
  } else {
    ScalarType t = at::kHalf;
    if (a[7] != Py_None) {
      need(THPDtype_Check(a[7]), "rope: dtype torch.float16 or torch.float32");
      t = reinterpret_cast<THPDtype *>(a[7])->scalar_type;
    }
    need(t == at::kHalf || t == at::kFloat, "rope: dtype torch.float16 or torch.float32");
    y = at::empty({M, heads, D}, x.options().dtype(t));
  }
  const int yt = float_type(y, "rope: fp16 or fp32 arrays");
  need(y.device() == dev && y.sizes() == x.sizes(), "rope: out like x, on its device");
  need(x.numel() == 0 || (x.stride(2) == 1 && y.stride(2) == 1), "rope: a head's values lie together");
  const Tensor &ph = tensor(a[2], "rope: phases, a tensor [rot / 2]");
  need(ph.dim() == 1, "rope: phases [rot / 2]");
  const int s = lib.rope(x.data_ptr(), xt, x.stride(0), x.stride(1),
                         array<int32_t>(a[1], at::kInt, {M}, dev, "rope: pos"),
                         array<uint64_t>(ph, at::kLong, ph.sizes(), dev, "rope: phases"),
                         (float)real(a[3]), M, heads, D, 2 * ph.numel(), small(a[4]), truth(a[5]),
                         y.data_ptr(), yt, y.stride(0), y.stride(1), on.stream());
  return done(s, "bitnest_rope", THPVariable_Wrap(y));
}

PyObject *kv_append(PyObject *const *a, Py_ssize_t) {
  // k, v, start, k_planes, v_planes, pos, phases, magnitude, layout, count
  const char *const what = "kv_append: k and v fp16 or fp32 [B, L, Hkv, 128] on a GPU";
  const Tensor &k = tensor(a[0], what), &v = tensor(a[1], what);
  need(k.dim() == 4 && k.is_cuda() && v.device() == k.device() && v.sizes() == k.sizes() &&
           k.size(3) == kD && v.scalar_type() == k.scalar_type(),
       what);
  const int type = float_type(k, what);
  const int64_t B = k.size(0), L = k.size(1), Hkv = k.size(2);
  const at::Device dev = k.device();
  int64_t step[2];
  for (int i = 0; i < 2; ++i) {
    const Tensor &t = i ? v : k;
    step[i] = L > 1 ? t.stride(1) : B > 1 ? t.stride(0) : Hkv * kD;
    need(t.numel() == 0 || (t.stride(3) == 1 && (t.stride(2) == kD || Hkv == 1) &&
                            (B == 1 || t.stride(0) == L * step[i])),
         "kv_append: a token's heads lie together, tokens at one stride");
  }
  const Planes kp = planes(a[3], "kv_append: k_planes, (hi, lo, scale)"),
               vp = planes(a[4], "kv_append: v_planes, (hi, lo, scale)");
  need(kp.hi->dim() == 4, "kv_append: planes [B, cap, Hkv, 64]");
  const int64_t cap = kp.hi->size(1);
  const bitnest_kv_cache c = cache(kp, vp, {B, cap, Hkv}, true, dev, "kv_append: planes");
  const int32_t *pos = nullptr, *count = nullptr;
  const uint64_t *phase = nullptr;
  int64_t rot = 0;
  if (a[6] != Py_None) {
    const Tensor &ph = tensor(a[6], "kv_append: phases, a tensor [rot / 2]");
    need(a[5] != Py_None && ph.dim() == 1, "kv_append: pos and phases [rot / 2]");
    rot = 2 * ph.numel();
    phase = array<uint64_t>(ph, at::kLong, ph.sizes(), dev, "kv_append: phases");
    pos = array<int32_t>(a[5], at::kInt, {B, L}, dev, "kv_append: pos");
  }
  if (a[9] != Py_None) count = array<int32_t>(a[9], at::kInt, {B}, dev, "kv_append: count");
  On on(dev);
  const int s = lib.kv_append(k.data_ptr(), step[0], v.data_ptr(), step[1], type, B, L, Hkv,
                              array<int32_t>(a[2], at::kInt, {B}, dev, "kv_append: start"), count,
                              pos, phase, (float)real(a[7]), rot, small(a[8]), &c, cap, on.stream());
  Py_INCREF(Py_None);
  return done(s, "bitnest_kv_append", Py_None);
}

PyObject *kv_read(PyObject *const *a, Py_ssize_t) {
  // mode, start, L, k_planes, v_planes
  const Planes kp = planes(a[3], "kv_read: k_planes, (hi, lo, scale)"),
               vp = planes(a[4], "kv_read: v_planes, (hi, lo, scale)");
  const int mode = small(a[0]);
  const int64_t L = integer(a[2]);
  need(kp.hi->dim() == 4 && kp.hi->is_cuda() && L >= 0, "kv_read: L rows of a cache [B, cap, Hkv, 64] on a GPU");
  const int64_t B = kp.hi->size(0), cap = kp.hi->size(1), Hkv = kp.hi->size(2);
  const at::Device dev = kp.hi->device();
  const bitnest_kv_cache c = cache(kp, vp, {B, cap, Hkv}, mode != BITNEST_DRAFT, dev, "kv_read: planes");
  const int32_t *start = a[1] == Py_None ? nullptr : array<int32_t>(a[1], at::kInt, {B}, dev, "kv_read: start");
  On on(dev);
  const at::TensorOptions f16 = kp.scale->options();
  Tensor k = at::empty({B, L, Hkv, kD}, f16), v = at::empty({B, L, Hkv, kD}, f16);
  const int s = lib.kv_read(mode, &c, B, cap, Hkv, start, L, static_cast<uint16_t *>(k.data_ptr()),
                            static_cast<uint16_t *>(v.data_ptr()), on.stream());
  return done(s, "bitnest_kv_read", Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v)));
}

PyObject *prefix_attention(PyObject *const *a, Py_ssize_t) {
  // mode, q, prefix, own, lens, out, lse, ws
  const char *const what = "prefix_attention: q fp16 [B, L, H, 128] on a GPU";
  const Tensor &q = tensor(a[1], what);
  need(q.dim() == 4 && q.is_cuda() && q.size(3) == kD, what);
  const int mode = small(a[0]);
  const int64_t B = q.size(0), L = q.size(1), H = q.size(2);
  const at::Device dev = q.device();
  const bool lo = mode != BITNEST_DRAFT;
  int64_t P = 0, cap = 0, Hkv = 0;
  bitnest_kv_cache pc, oc;
  need(a[2] != Py_None || a[3] != Py_None, "prefix_attention: a prefix or own tokens");
  Planes c[2][2];
  for (int i = 1; i >= 0; --i) {  // the prefix's heads count where both are given
    if (a[2 + i] == Py_None) continue;
    const char *const w = i ? "prefix_attention: own, (k_planes, v_planes) [B, cap, Hkv, 64]"
                            : "prefix_attention: prefix, (k_planes, v_planes) [P, Hkv, 64]";
    need((PyTuple_Check(a[2 + i]) || PyList_Check(a[2 + i])) && PySequence_Fast_GET_SIZE(a[2 + i]) == 2, w);
    PyObject **p = PySequence_Fast_ITEMS(a[2 + i]);
    c[i][0] = planes(p[0], w);
    c[i][1] = planes(p[1], w);
    need(c[i][0].hi->dim() == 3 + i, w);
    (i ? cap : P) = c[i][0].hi->size(i);
    Hkv = c[i][0].hi->size(1 + i);
  }
  if (P > 0) pc = cache(c[0][0], c[0][1], {P, Hkv}, lo, dev, "prefix_attention: prefix");
  if (cap > 0) oc = cache(c[1][0], c[1][1], {B, cap, Hkv}, lo, dev, "prefix_attention: own");
  On on(dev);
  Tensor out, lse, ws;
  out = a[5] != Py_None ? tensor(a[5], "prefix_attention: out") : at::empty({B, L, H, kD}, q.options().dtype(at::kHalf));
  lse = a[6] != Py_None ? tensor(a[6], "prefix_attention: lse") : at::empty({B, L, H}, q.options().dtype(at::kFloat));
  if (a[7] != Py_None) {
    ws = tensor(a[7], "prefix_attention: ws");
    need(ws.scalar_type() == at::kByte && ws.device() == dev && ws.is_contiguous(),
         "prefix_attention: ws, bytes on q's device");
  } else {
    const int64_t n = lib.ws_bytes(B, L, H, Hkv, P, cap);
    if (n < 0) return done((int)-n, "bitnest_prefix_attention_ws_bytes", nullptr);
    ws = at::empty({n < 16 ? 16 : n}, q.options().dtype(at::kByte));
  }
  const int s = lib.prefix_attention(
      mode, array<uint16_t>(q, at::kHalf, q.sizes(), dev, "prefix_attention: q"), B, L, H, Hkv, kD,
      P > 0 ? &pc : nullptr, P, cap > 0 ? &oc : nullptr, cap,
      array<int32_t>(a[4], at::kInt, {B}, dev, "prefix_attention: lens"),
      array<uint16_t>(out, at::kHalf, {B, L, H, kD}, dev, "prefix_attention: out"),
      array<float>(lse, at::kFloat, {B, L, H}, dev, "prefix_attention: lse"), ws.data_ptr(),
      ws.numel(), on.stream());
  return done(s, "bitnest_prefix_attention", Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse)));
}

PyObject *kv_weights(PyObject *const *a, Py_ssize_t) {
  // mode, q, lse, k_planes, acc, lens
  const char *const what = "kv_weights: q fp16 [B, L, H, 128] on a GPU";
  const Tensor &q = tensor(a[1], what);
  need(q.dim() == 4 && q.is_cuda() && q.size(3) == kD, what);
  const int mode = small(a[0]);
  const int64_t B = q.size(0), L = q.size(1), H = q.size(2);
  const at::Device dev = q.device();
  const bool own = a[5] != Py_None;
  const Planes kp = planes(a[3], "kv_weights: k_planes, (hi, lo, scale)");
  need(kp.hi->dim() == (own ? 4 : 3), "kv_weights: planes [B, cap, Hkv, 64] with lens, [P, Hkv, 64] without");
  const int64_t cap = kp.hi->size(own), Hkv = kp.hi->size(own + 1);
  const int64_t rows[3] = {B, cap, Hkv}, sums[3] = {B, Hkv, cap};
  const int first = own ? 0 : 1;
  const Addresses k = addresses(kp, at::IntArrayRef(rows + first, 3 - first), mode != BITNEST_DRAFT,
                                dev, "kv_weights: k");
  On on(dev);
  const int s = lib.kv_weights(
      mode, array<uint16_t>(q, at::kHalf, q.sizes(), dev, "kv_weights: q"),
      array<float>(a[2], at::kFloat, {B, L, H}, dev, "kv_weights: lse"), B, L, H, Hkv, kD, k.hi,
      k.lo, k.scale, cap, own ? array<int32_t>(a[5], at::kInt, {B}, dev, "kv_weights: lens") : nullptr,
      array<float>(a[4], at::kFloat, at::IntArrayRef(sums + first, 3 - first), dev, "kv_weights: acc"),
      on.stream());
  Py_INCREF(a[4]);
  return done(s, "bitnest_kv_weights", a[4]);
}

PyObject *kv_evict(PyObject *const *a, Py_ssize_t) {
  // acc, lens, keep, sinks, recent, k_planes, v_planes, k_out, v_out, acc_out
  const Planes kp = planes(a[5], "kv_evict: k_planes, (hi, lo, scale)"),
               vp = planes(a[6], "kv_evict: v_planes, (hi, lo, scale)"),
               ko = planes(a[7], "kv_evict: k_out, (hi, lo, scale)"),
               vo = planes(a[8], "kv_evict: v_out, (hi, lo, scale)");
  need(kp.hi->dim() == 4 && ko.hi->dim() == 4 && kp.hi->is_cuda(), "kv_evict: caches [B, cap, Hkv, 64] on a GPU");
  const int64_t B = kp.hi->size(0), cap = kp.hi->size(1), Hkv = kp.hi->size(2), cap_out = ko.hi->size(1);
  const int64_t keep = integer(a[2]);
  const at::Device dev = kp.hi->device();
  const bitnest_kv_cache src = cache(kp, vp, {B, cap, Hkv}, true, dev, "kv_evict: planes"),
                         dst = cache(ko, vo, {B, cap_out, Hkv}, true, dev, "kv_evict: out");
  On on(dev);
  // a `keep` that the entry point refuses takes no memory here
  const bool held = keep >= 1 && keep <= cap_out;
  const at::TensorOptions ints = kp.hi->options().dtype(at::kInt);
  Tensor kept = at::empty({B, Hkv, held ? keep : 0}, ints), n = at::empty({B}, ints);
  const int s = lib.kv_evict(
      array<float>(a[0], at::kFloat, {B, Hkv, cap}, dev, "kv_evict: acc"),
      array<int32_t>(a[1], at::kInt, {B}, dev, "kv_evict: lens"), B, Hkv, cap, keep, integer(a[3]),
      integer(a[4]), &src, &dst, cap_out,
      array<float>(a[9], at::kFloat, {B, Hkv, cap_out}, dev, "kv_evict: acc_out"),
      static_cast<int32_t *>(kept.data_ptr()), static_cast<int32_t *>(n.data_ptr()), on.stream());
  return done(s, "bitnest_kv_evict", Py_BuildValue("(NN)", THPVariable_Wrap(kept), THPVariable_Wrap(n)));
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args, n);
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// open(addresses of kNames, BitnestError)
PyObject *open(PyObject *, PyObject *const *args, Py_ssize_t n) {
  constexpr Py_ssize_t count = sizeof(kNames) / sizeof(kNames[0]);
  static_assert(sizeof(lib) == count * sizeof(void *), "one entry a name");
  if (n != 2 || !PyTuple_Check(args[0]) || PyTuple_GET_SIZE(args[0]) != count) {
    PyErr_SetString(PyExc_TypeError, "open(addresses, error)");
    return nullptr;
  }
  void *p[count];
  for (Py_ssize_t i = 0; i < count; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[0], i));
    if (!p[i]) return nullptr;
  }
  memcpy(&lib, p, sizeof(lib));
  Py_INCREF(args[1]);
  Py_XSETREF(error_type, args[1]);
  Py_RETURN_NONE;
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("open", open),
                         FAST("rope", (call<rope, 8>)),
                         FAST("kv_append", (call<kv_append, 10>)),
                         FAST("kv_read", (call<kv_read, 5>)),
                         FAST("prefix_attention", (call<prefix_attention, 8>)),
                         FAST("kv_weights", (call<kv_weights, 6>)),
                         FAST("kv_evict", (call<kv_evict, 10>)),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject *m = PyModule_Create(&module);
  if (!m) return nullptr;
  PyObject *names = PyTuple_New(sizeof(kNames) / sizeof(kNames[0]));
  for (size_t i = 0; names && i < sizeof(kNames) / sizeof(kNames[0]); ++i)
    PyTuple_SET_ITEM(names, i, PyUnicode_FromString(kNames[i]));
  if (!names || PyModule_AddObject(m, "names", names) < 0) {
    Py_XDECREF(names);
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
