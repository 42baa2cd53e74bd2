// Python side of the batch operators' calls: torch tensors to the C ABI's pointers, strides and
// sizes, and nothing else (every computation runs in libvv's kernels).
//
// One decode step makes two of these calls per layer; written in Python, the argument checks and the
// foreign-function call cost about 20 us of host time each, more than the kernels they start.  The
// functions take their arguments by position; the documented, keyword-taking functions are in _vv.py.
// A call refuses a tensor of the wrong type, shape, layout or device with VVError
// (VV_ERR_INVALID_ARG) before anything is launched, and runs with the tensors' device current, on
// its current torch stream.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/api/include/torch/version.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <optional>

#include "../../include/vv.h"

namespace {

PyObject* g_error = nullptr;  // _vv.VVError

struct Refused {};  // a Python error has been set

[[noreturn]] void refuse(const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  PyObject* args = Py_BuildValue("(is)", VV_ERR_INVALID_ARG, text);
  if (args) {
    PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, args);
    Py_DECREF(args);
  }
  throw Refused();
}

void check(vv_status st) {
  if (st == VV_OK) return;
  char text[512];
  vv_last_error(text, sizeof(text));
  PyObject* args = Py_BuildValue("(is)", (int)st, text);
  if (args) {
    PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, args);
    Py_DECREF(args);
  }
  throw Refused();
}

// The arguments of one call, read in order.
struct Args {
  const char* who;
  PyObject* const* v;
  Py_ssize_t n, i = 0;
  PyObject* next() {
    if (i >= n) refuse("%s: too few arguments", who);
    return v[i++];
  }
  const at::Tensor* tensor_or_none(const char* name) {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse("%s: %s must be a tensor", who, name);
    return &THPVariable_Unpack(o);
  }
  const at::Tensor& tensor(const char* name) {
    const at::Tensor* t = tensor_or_none(name);
    if (!t) refuse("%s: %s must be a tensor", who, name);
    return *t;
  }
  int64_t integer(const char* name) {
    const int64_t x = PyLong_AsLongLong(next());
    if (x == -1 && PyErr_Occurred()) throw Refused();
    if (x != (int32_t)x) refuse("%s: %s = %lld does not fit 32 bits", who, name, (long long)x);
    return x;
  }
  bool truth() {
    const int x = PyObject_IsTrue(next());
    if (x < 0) throw Refused();
    return x == 1;
  }
  double number() {
    const double x = PyFloat_AsDouble(next());
    if (x == -1.0 && PyErr_Occurred()) throw Refused();
    return x;
  }
  void* address() {
    void* p = PyLong_AsVoidPtr(next());
    if (!p && PyErr_Occurred()) throw Refused();
    return p;
  }
};

// Where a call runs: the device of its first tensor; every other one has to be there too.
struct Place {
  const char* who;
  c10::Device device;
  std::optional<c10::cuda::CUDAGuard> guard;
  Place(const char* who_, const at::Tensor& t) : who(who_), device(t.device()) {
    if (!device.is_cuda()) refuse("%s: tensors must be on a CUDA device, got %s", who, device.str().c_str());
    if (c10::cuda::current_device() != device.index()) guard.emplace(device);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
  at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::detail::empty_cuda(sizes, type, device, std::nullopt);
  }
  void here(const char* name, const at::Tensor& t) const {
    if (t.device() != device)
      refuse("%s: %s is on %s, expected %s", who, name, t.device().str().c_str(), device.str().c_str());
  }
  // contiguous, of `type` and (when given) `sizes`; its data
  template <typename T>
  T* dense(const char* name, const at::Tensor* t, at::ScalarType type, at::IntArrayRef sizes) const {
    if (!t) return nullptr;
    here(name, *t);
    if (t->scalar_type() != type || !t->is_contiguous())
      refuse("%s: %s must be contiguous %s, got %s", who, name, c10::toString(type), c10::toString(t->scalar_type()));
    if (t->sizes() != sizes) refuse("%s: %s has the wrong shape (%lld elements)", who, name, (long long)t->numel());
    return static_cast<T*>(t->data_ptr());
  }
  template <typename T>
  T* dense(const char* name, const at::Tensor& t, at::ScalarType type, at::IntArrayRef sizes) const {
    return dense<T>(name, &t, type, sizes);
  }
  // [rows, a(, b)] of `type` whose rows are contiguous; the row stride in elements
  int64_t rows(const char* name, const at::Tensor& t, at::ScalarType type, int64_t n, int64_t a, int64_t b = -1) const {
    here(name, t);
    if (t.scalar_type() != type)
      refuse("%s: %s must be %s, got %s", who, name, c10::toString(type), c10::toString(t.scalar_type()));
    const bool flat = b < 0;
    if (t.dim() != (flat ? 2 : 3) || t.size(0) != n || t.size(1) != a || (!flat && t.size(2) != b))
      refuse("%s: %s has the wrong shape (expected %lld rows of %lld)", who, name, (long long)n, (long long)(flat ? a : a * b));
    const int64_t inner = flat ? t.stride(1) : t.stride(2);
    if (((flat ? a : b) > 1 && inner != 1) || (!flat && a > 1 && t.stride(1) != b))
      refuse("%s: the rows of %s must be contiguous", who, name);
    return n > 1 ? t.stride(0) : (flat ? a : a * b);
  }
};

int32_t i32(const char* who, const char* name, int64_t x) {
  if (x != (int32_t)x) refuse("%s: %s = %lld does not fit 32 bits", who, name, (long long)x);
  return (int32_t)x;
}

const auto kI32 = at::kInt;
const auto kI64 = at::kLong;
const auto kF32 = at::kFloat;

PyObject* tuple_of(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Refused();
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o = t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw Refused();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// A function of the module: C++ exceptions end here.
template <PyObject* (*F)(Args&)>
PyObject* entry(const char* who, PyObject* const* v, Py_ssize_t n) {
  try {
    Args a{who, v, n};
    return F(a);
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// lens, new_lens, block_tables, free_pages, page_size, pages, max_tokens, prefix_len, cursor,
// out_lens, out_offsets, out_slots, out_positions, out_cursor (all None: made here)
PyObject* paged_plan(Args& a) {
  const at::Tensor& lens = a.tensor("lens");
  const Place p(a.who, lens);
  const int64_t B = lens.numel();
  const auto* l = p.dense<int32_t>("lens", lens, kI32, {B});
  const auto* nl = p.dense<int32_t>("new_lens", a.tensor("new_lens"), kI32, {B});
  const at::Tensor& table = a.tensor("block_tables");
  if (table.dim() != 2) refuse("%s: block_tables must be [B, max_blocks]", a.who);
  auto* tb = p.dense<int32_t>("block_tables", table, kI32, {B, table.size(1)});
  const at::Tensor& pages_free = a.tensor("free_pages");
  const auto* fp = p.dense<int32_t>("free_pages", pages_free, kI32, {pages_free.numel()});
  const int64_t ps = a.integer("page_size"), pages = a.integer("pages"), mt = a.integer("max_tokens"),
                prefix = a.integer("prefix_len");
  const auto* cur = p.dense<int32_t>("cursor", a.tensor_or_none("cursor"), kI32, {1});
  const at::Tensor* given[5];
  for (auto& g : given) g = a.tensor_or_none("out");
  if (mt < 1) refuse("%s: max_tokens=%lld", a.who, (long long)mt);
  const int64_t sizes[5] = {B, B + 1, mt, mt, 1};
  void* out[5];
  at::Tensor made[5];
  if (!given[0] && !given[1] && !given[2] && !given[3] && !given[4]) {
    // one allocation, slots first: five took 8.3 us of host time a call
    int64_t at[5], words = 0;
    for (int i : {2, 0, 1, 3, 4}) {
      at[i] = words;
      words += ((i == 2 ? 2 : 1) * sizes[i] + 3) / 4 * 4;
    }
    made[0] = p.empty({words}, kI32);
    int32_t* base = made[0].data_ptr<int32_t>();
    for (int i = 4; i >= 0; --i) {
      const auto type = at::scalarTypeToTypeMeta(i == 2 ? kI64 : kI32);
      at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(made[0].storage()), made[0].key_set(), type);
      t.unsafeGetTensorImpl()->set_storage_offset(i == 2 ? at[i] / 2 : at[i]);
      t.unsafeGetTensorImpl()->set_sizes_contiguous({sizes[i]});
      out[i] = base + at[i];
      made[i] = std::move(t);
      given[i] = &made[i];
    }
  } else {
    for (int i = 0; i < 5; ++i) {
      const auto type = i == 2 ? kI64 : kI32;
      if (!given[i]) {
        made[i] = p.empty({sizes[i]}, type);
        given[i] = &made[i];
      }
      out[i] = p.dense<void>("out", given[i], type, {sizes[i]});
    }
  }
  check(vv_paged_plan(l, nl, i32(a.who, "B", B), prefix, ps, pages, fp, i32(a.who, "free_pages", pages_free.numel()), cur,
                      tb, i32(a.who, "max_blocks", table.size(1)), (int32_t*)out[0], (int32_t*)out[1], (int64_t*)out[2],
                      (int32_t*)out[3], mt, (int32_t*)out[4], p.stream()));
  return tuple_of({given[0], given[1], given[2], given[3], given[4]});
}

struct Pool {
  const vv_paged_kv* kv;
  int64_t heads, dim;
  at::ScalarType type;
};
// address of the vv_paged_kv, heads, head_dim, device index
Pool pool_of(Args& a, const Place& p) {
  Pool r;
  r.kv = static_cast<const vv_paged_kv*>(a.address());
  r.heads = a.integer("heads");
  r.dim = a.integer("head_dim");
  const int64_t dev = a.integer("device");
  if (!r.kv) refuse("%s: no page pool", a.who);
  if (dev != p.device.index()) refuse("%s: the pages are on cuda:%lld, expected %s", a.who, (long long)dev, p.device.str().c_str());
  r.type = r.kv->dtype == VV_F16 ? at::kHalf : at::kBFloat16;
  return r;
}

// q, k, v, positions, slots, pool (4), theta, q_gain, k_gain, eps, out
PyObject* qk_rope_append(Args& a) {
  const at::Tensor &q = a.tensor("q"), &k = a.tensor("k"), &v = a.tensor("v");
  const at::Tensor &pos = a.tensor("positions"), &slots = a.tensor("slots");
  const Place p(a.who, q);
  const Pool kv = pool_of(a, p);
  const double theta = a.number();
  const at::Tensor *qg = a.tensor_or_none("q_gain"), *kg = a.tensor_or_none("k_gain");
  const double eps = a.number();
  const at::Tensor* given = a.tensor_or_none("out");
  if (q.dim() != 3) refuse("%s: q must be [T, Hq, D]", a.who);
  const int64_t T = q.size(0), Hq = q.size(1), D = kv.dim;
  const int64_t qs = p.rows("q", q, kv.type, T, Hq, D), ks = p.rows("k", k, kv.type, T, kv.heads, D),
                vs = p.rows("v", v, kv.type, T, kv.heads, D);
  const auto* ps = p.dense<int32_t>("positions", pos, kI32, {T});
  const auto* sl = p.dense<int64_t>("slots", slots, kI64, {T});
  const void *g0 = p.dense<void>("q_gain", qg, kv.type, {D}), *g1 = p.dense<void>("k_gain", kg, kv.type, {D});
  at::Tensor made;
  if (!given) {
    made = p.empty({T, Hq, D}, kv.type);
    given = &made;
  }
  const int64_t os = p.rows("out", *given, kv.type, T, Hq, D);
  check(vv_qk_rope_append(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, i32(a.who, "Hq", Hq), kv.heads, D, g0,
                          g1, (float)eps, ps, (float)theta, sl, kv.kv, given->data_ptr(), os, p.stream()));
  return THPVariable_Wrap(*given);
}

// q, k_prefix, v_prefix, pool (4), block_tables, lens, scale, ws, out, lse
PyObject* gqa_prefix_attn(Args& a) {
  const at::Tensor& q = a.tensor("q");
  const at::Tensor *kp = a.tensor_or_none("k_prefix"), *vp = a.tensor_or_none("v_prefix");
  const Place p(a.who, q);
  const Pool kv = pool_of(a, p);
  const at::Tensor &table = a.tensor("block_tables"), &lens = a.tensor("lens");
  const double scale = a.number();
  const at::Tensor& ws = a.tensor("ws");
  const at::Tensor *given = a.tensor_or_none("out"), *lse = a.tensor_or_none("lse");
  if (q.dim() != 3) refuse("%s: q must be [B, Hq, D]", a.who);
  const int64_t B = q.size(0), Hq = q.size(1), D = kv.dim;
  const int64_t qs = p.rows("q", q, kv.type, B, Hq, D);
  int64_t P = 0, ph = 0, pt = 0;
  if (!kp != !vp) refuse("%s: k_prefix and v_prefix go together", a.who);
  if (kp) {
    p.here("k_prefix", *kp);
    p.here("v_prefix", *vp);
    if (kp->dim() != 3 || kp->size(0) != kv.heads || kp->size(2) != D || vp->sizes() != kp->sizes() ||
        vp->strides() != kp->strides() || kp->scalar_type() != kv.type || vp->scalar_type() != kv.type || kp->stride(2) != 1)
      refuse("%s: k_prefix and v_prefix must be %s [%lld, P, %lld] of one layout, the last dimension contiguous", a.who,
             c10::toString(kv.type), (long long)kv.heads, (long long)D);
    P = kp->size(1);
    ph = kv.heads > 1 ? kp->stride(0) : std::max(P, int64_t(1)) * D;
    pt = P > 1 ? kp->stride(1) : D;
  }
  if (table.dim() != 2) refuse("%s: block_tables must be [B, max_blocks]", a.who);
  const auto* tb = p.dense<int32_t>("block_tables", table, kI32, {B, table.size(1)});
  const auto* ln = p.dense<int32_t>("lens", lens, kI32, {B});
  float* ls = p.dense<float>("lse", lse, kF32, {B, Hq});
  p.here("ws", ws);
  if (!ws.is_contiguous()) refuse("%s: ws must be contiguous", a.who);
  at::Tensor made;
  if (!given) {
    made = p.empty({B, Hq, D}, kv.type);
    given = &made;
  }
  const int64_t os = p.rows("out", *given, kv.type, B, Hq, D);
  check(vv_gqa_prefix_attn(q.data_ptr(), qs, i32(a.who, "B", B), i32(a.who, "Hq", Hq), kv.heads, D, kp ? kp->data_ptr() : nullptr,
                           vp ? vp->data_ptr() : nullptr, ph, pt, i32(a.who, "P", P), kv.kv, tb,
                           i32(a.who, "max_blocks", table.size(1)), ln, (float)scale, given->data_ptr(), os, ls,
                           ws.data_ptr(), ws.nbytes(), p.stream()));
  return THPVariable_Wrap(*given);
}

// logits, ws, tokens, token_lens, prompt_lens, repetition, frequency, presence, bias_ids, bias_vals,
// bias_offsets, mask, argmax (bool), out
PyObject* logits_process(Args& a) {
  const at::Tensor& x = a.tensor("logits");
  const Place p(a.who, x);
  const at::Tensor* ws = a.tensor_or_none("ws");
  const at::Tensor* tokens = a.tensor_or_none("tokens");
  const at::Tensor *token_lens = a.tensor_or_none("token_lens"), *prompt_lens = a.tensor_or_none("prompt_lens");
  const at::Tensor *rep = a.tensor_or_none("repetition"), *freq = a.tensor_or_none("frequency"),
                   *pres = a.tensor_or_none("presence");
  const at::Tensor *ids = a.tensor_or_none("bias_ids"), *vals = a.tensor_or_none("bias_vals"),
                   *offs = a.tensor_or_none("bias_offsets");
  const at::Tensor* mask = a.tensor_or_none("mask");
  const bool argmax = a.truth();
  const at::Tensor* given = a.tensor_or_none("out");
  const auto type = x.scalar_type();
  if (x.dim() != 2 || (type != kF32 && type != at::kHalf && type != at::kBFloat16))
    refuse("%s: logits must be fp32, fp16 or bf16 [B, V]", a.who);
  const int64_t B = x.size(0), V = x.size(1);
  const int64_t xs = p.rows("logits", x, type, B, V);
  vv_logits_rules r = {};
  r.token_lens = p.dense<int32_t>("token_lens", token_lens, kI32, {B});
  r.prompt_lens = p.dense<int32_t>("prompt_lens", prompt_lens, kI32, {B});
  r.repetition = p.dense<float>("repetition", rep, kF32, {B});
  r.frequency = p.dense<float>("frequency", freq, kF32, {B});
  r.presence = p.dense<float>("presence", pres, kF32, {B});
  if (tokens) {
    if (!token_lens || tokens->dim() != 2) refuse("%s: tokens must be [B, width] and come with token_lens", a.who);
    r.tokens_stride = p.rows("tokens", *tokens, kI32, B, tokens->size(1));
    r.tokens = static_cast<const int32_t*>(tokens->data_ptr());
    r.max_tokens = i32(a.who, "width of tokens", tokens->size(1));
  } else if (rep || freq || pres) {
    refuse("%s: penalties need tokens", a.who);
  }
  if (ids) {
    if (!vals || !offs) refuse("%s: bias_ids, bias_vals and bias_offsets go together", a.who);
    const int64_t n = ids->numel();
    r.bias_ids = p.dense<int32_t>("bias_ids", ids, kI32, {n});
    r.bias_vals = p.dense<float>("bias_vals", vals, kF32, {n});
    r.bias_offsets = p.dense<int32_t>("bias_offsets", offs, kI32, {B + 1});
    r.n_bias = i32(a.who, "biases", n);
  }
  if (mask) {
    r.mask_stride = p.rows("mask", *mask, kI32, B, (V + 31) / 32);
    r.mask = static_cast<const uint32_t*>(mask->data_ptr());
  }
  if (argmax && (!ws || !ws->is_contiguous())) refuse("%s: argmax needs a contiguous workspace", a.who);
  if (argmax) p.here("ws", *ws);
  at::Tensor made, best;
  if (!given) {
    made = p.empty({B, V}, type);
    given = &made;
  }
  const int64_t os = p.rows("out", *given, type, B, V);
  if (argmax) best = p.empty({B}, kI32);
  check(vv_logits_process(x.data_ptr(), xs, type == kF32 ? VV_F32 : type == at::kHalf ? VV_F16 : VV_BF16,
                          i32(a.who, "B", B), V, &r, given->data_ptr(), os, argmax ? (int32_t*)best.data_ptr() : nullptr,
                          argmax ? ws->data_ptr() : nullptr, argmax ? ws->nbytes() : 0, p.stream()));
  return tuple_of({given, argmax ? &best : nullptr});
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  Py_RETURN_NONE;
}

#define VV_ENTRY(name) \
  PyObject* py_##name(PyObject*, PyObject* const* v, Py_ssize_t n) { return entry<name>("vv_" #name, v, n); }
VV_ENTRY(paged_plan)
VV_ENTRY(qk_rope_append)
VV_ENTRY(gqa_prefix_attn)
VV_ENTRY(logits_process)

#define VV_METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {VV_METHOD(paged_plan), VV_METHOD(qk_rope_append), VV_METHOD(gqa_prefix_attn),
                           VV_METHOD(logits_process), {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&g_module);
  // what torch it may be used with: its classes' layout is compiled in
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
