// Python side of the token mixers' calls (qmm_mix.h): checks the tensors, fills in pointers,
// sizes and the current stream, and calls the C ABI.  A decode step makes several of these
// calls, each a few microseconds of GPU work, so the marshalling is done here rather than in
// the interpreter (16 -> 5 us a call).  Every function returns the C status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qmm_mix.h"

namespace {

using at::ScalarType;
using at::Tensor;

// The entry points of the loaded library (bind).
decltype(&qmm_kv4_append) f_append = nullptr;
decltype(&qmm_kv4_attn) f_attn = nullptr;
decltype(&qmm_gdn) f_gdn = nullptr;

struct Bad {
  std::string what;
};
[[noreturn]] void bad(const std::string& s) { throw Bad{s}; }

// A call's tensors must live on the current device: the stream and the launch are its.
struct Call {
  int device = -1;
  hipStream_t stream = nullptr;
  explicit Call(PyObject* s) {
    c10::hip::HIPStream cur = c10::hip::getCurrentHIPStream();
    device = cur.device_index();
    stream = s == Py_None ? cur.stream() : static_cast<hipStream_t>(PyLong_AsVoidPtr(s));
    if (PyErr_Occurred()) bad("stream must be a stream or its handle");
  }
  Call() {}
  const Tensor* opt(PyObject* o, const char* name) const {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) bad(std::string(name) + " must be a device tensor");
    if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
    if (device >= 0 && t.get_device() != device)
      bad(std::string(name) + " is on device " + std::to_string(t.get_device()) + ", the current device is " +
          std::to_string(device));
    return &t;
  }
  const Tensor& get(PyObject* o, const char* name) const {
    const Tensor* t = opt(o, name);
    if (!t) bad(std::string(name) + " is missing");
    return *t;
  }
};

void need(bool ok, const char* what) {
  if (!ok) bad(what);
}
bool half_type(const Tensor& t) {
  const ScalarType s = t.scalar_type();
  return s == ScalarType::BFloat16 || s == ScalarType::Short || s == ScalarType::UInt16;
}
int out_type(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::Float) return QMM_OUT_F32;
  if (!half_type(t)) bad(std::string(name) + " must be bf16 or fp32");
  return QMM_OUT_BF16;
}
bool shaped(const Tensor& t, std::initializer_list<int64_t> s) {
  return t.sizes() == c10::IntArrayRef(s.begin(), s.size());
}
bool words(const Tensor& t) { return t.element_size() == 4 && !t.is_floating_point(); }
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Bad& b) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, b.what.c_str());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// cache(k_codes, k_meta, v_codes, v_meta) -> (struct bytes, device)
PyObject* cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 4, "cache takes 4 tensors");
    auto shape_of = [&](PyObject* o, const char* name) -> const Tensor& {
      if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
      return THPVariable_Unpack(o);
    };
    const Tensor &kc = shape_of(a[0], "k_codes"), &km = shape_of(a[1], "k_meta"), &vc = shape_of(a[2], "v_codes"),
                 &vm = shape_of(a[3], "v_meta");
    need(kc.dim() == 4 && words(kc), "k_codes must be [pages, heads, page_size, head_dim/8] 32-bit words");
    const int64_t p = kc.size(0), h = kc.size(1), s = kc.size(2), hd = kc.size(3) * 8;
    need(shaped(km, {p, h, s, hd / 64}) && words(km), "k_meta must be [pages, heads, page_size, head_dim/64] 32-bit words");
    need(shaped(vc, {p, h, s / 8, hd / 4, 8}) && vc.element_size() == 2 && !vc.is_floating_point(),
         "v_codes must be [pages, heads, page_size/8, head_dim/4, 8] 16-bit units");
    need(shaped(vm, {p, h, s, hd / 64}) && words(vm), "v_meta must be [pages, heads, page_size, head_dim/64] 32-bit words");
    Call c;
    c.get(a[0], "k_codes");
    c.device = kc.get_device();
    c.get(a[1], "k_meta"), c.get(a[2], "v_codes"), c.get(a[3], "v_meta");
    const qmm_kv4_cache v = {static_cast<uint32_t*>(kc.data_ptr()), static_cast<uint32_t*>(km.data_ptr()),
                             static_cast<uint16_t*>(vc.data_ptr()), static_cast<uint32_t*>(vm.data_ptr()), p, s, h, hd};
    return Py_BuildValue("y#i", reinterpret_cast<const char*>(&v), Py_ssize_t(sizeof v), c.device);
  });
}

qmm_kv4_cache cache_of(PyObject* o, const Call& c) {
  const char* p;
  Py_ssize_t n;
  int dev;
  if (!PyArg_ParseTuple(o, "y#i", &p, &n, &dev) || n != sizeof(qmm_kv4_cache)) bad("cache must be a KV4Cache");
  if (dev != c.device)
    bad("the cache is on device " + std::to_string(dev) + ", the current device is " + std::to_string(c.device));
  qmm_kv4_cache v;
  memcpy(&v, p, sizeof v);
  return v;
}

// append(cache, k, v, slots, positions, cos_sin, q, q_out, k_held, v_held, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 11, "append takes 11 arguments");
    const Call c(a[10]);
    const qmm_kv4_cache kv = cache_of(a[0], c);
    const Tensor &k = c.get(a[1], "k"), &v = c.get(a[2], "v"), &slots = c.get(a[3], "slots");
    const Tensor *pos = c.opt(a[4], "positions"), *cs = c.opt(a[5], "cos_sin"), *q = c.opt(a[6], "q"),
                 *qo = c.opt(a[7], "q_out"), *kh = c.opt(a[8], "k_held"), *vh = c.opt(a[9], "v_held");
    need(k.dim() == 3, "k, v must be [T, n_kv, head_dim]");
    const int64_t T = k.size(0), h = kv.n_kv_heads, hd = kv.head_dim;
    need(shaped(k, {T, h, hd}) && shaped(v, {T, h, hd}), "k, v must be [T, n_kv, head_dim]");
    const int dt = out_type(k, "k");
    need(out_type(v, "v") == dt && (!q || out_type(*q, "q") == dt), "q, k, v must share a dtype");
    need(slots.numel() == T && words(slots), "slots must be int32 [T]");
    need(!pos == !cs, "positions and cos_sin go together");
    if (pos) {
      need(pos->numel() == T && words(*pos), "positions must be int32 [T]");
      need(cs->dim() == 2 && cs->scalar_type() == ScalarType::Float, "cos_sin must be fp32 [max_pos, rot_dim]");
    }
    need(!q == !qo, "q and q_out go together");
    if (q) {
      need(q->dim() == 3 && q->size(0) == T && q->size(2) == hd, "q must be [T, n_q, head_dim]");
      need(qo->sizes() == q->sizes() && half_type(*qo), "q_out must be bf16, as q");
    }
    need(!kh || (shaped(*kh, {T, h, hd}) && half_type(*kh)), "k_held must be bf16 [T, n_kv, head_dim]");
    need(!vh || (shaped(*vh, {T, h, hd}) && half_type(*vh)), "v_held must be bf16 [T, n_kv, head_dim]");
    if (T == 0) return PyLong_FromLong(QMM_OK);
    return PyLong_FromLong(f_append(
        &kv, k.data_ptr(), v.data_ptr(), T, dt, static_cast<int32_t*>(slots.data_ptr()), static_cast<int32_t*>(ptr(pos)),
        static_cast<float*>(ptr(cs)), cs ? cs->size(0) : 0, cs ? cs->size(1) : 0, ptr(q), q ? q->size(1) : 0,
        static_cast<uint16_t*>(ptr(qo)), static_cast<uint16_t*>(ptr(kh)), static_cast<uint16_t*>(ptr(vh)), c.stream));
  });
}

// attn(q, cache, page_table, kv_lens, out, workspace, q_start, max_q, scale, causal, window, gate, stream)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 13, "attn takes 13 arguments");
    const Call c(a[12]);
    const Tensor& q = c.get(a[0], "q");
    const qmm_kv4_cache kv = cache_of(a[1], c);
    const Tensor &table = c.get(a[2], "page_table"), &lens = c.get(a[3], "kv_lens"), &out = c.get(a[4], "out"),
                 &ws = c.get(a[5], "workspace");
    const Tensor *start = c.opt(a[6], "q_start"), *gate = c.opt(a[11], "gate");
    const long long max_q = PyLong_AsLongLong(a[7]), window = PyLong_AsLongLong(a[10]);
    const long causal = PyLong_AsLong(a[9]);
    need(q.dim() == 3 && q.size(2) == kv.head_dim, "q must be [T, n_q, head_dim]");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt(double(kv.head_dim)) : PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) bad("max_q, scale, causal and window must be numbers");
    need(table.dim() == 2 && words(table), "page_table must be int32 [B, max_pages]");
    const int64_t B = table.size(0);
    need(lens.numel() == B && words(lens), "kv_lens must be int32 [B]");
    need(!start || (start->numel() == B + 1 && words(*start)), "q_start must be int32 [B + 1]");
    need(half_type(q) && half_type(out) && out.sizes() == q.sizes(), "q and out must be bf16 [T, n_q, head_dim]");
    need(!gate || (gate->sizes() == q.sizes() && half_type(*gate)), "gate must be bf16, as q");
    if (q.size(0) == 0) return PyLong_FromLong(QMM_OK);
    return PyLong_FromLong(f_attn(
        static_cast<uint16_t*>(q.data_ptr()), q.size(0), static_cast<int32_t*>(ptr(start)),
        static_cast<int32_t*>(lens.data_ptr()), static_cast<int32_t*>(table.data_ptr()), B, table.size(1), max_q, &kv,
        q.size(1), float(scale), int(causal), window, static_cast<uint16_t*>(ptr(gate)), ws.data_ptr(),
        ws.numel() * ws.element_size(), static_cast<uint16_t*>(out.data_ptr()), c.stream));
  });
}

// gdn(q, k, v, g, beta, state, y, workspace, state_out, seq_start, state_slots, max_len, scale, l2norm, stream)
PyObject* gdn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 15, "gdn takes 15 arguments");
    const Call c(a[14]);
    const Tensor &q = c.get(a[0], "q"), &k = c.get(a[1], "k"), &v = c.get(a[2], "v"), &g = c.get(a[3], "g"),
                 &beta = c.get(a[4], "beta"), &s = c.get(a[5], "state"), &y = c.get(a[6], "y"),
                 &ws = c.get(a[7], "workspace");
    const Tensor *so = c.opt(a[8], "state_out"), *start = c.opt(a[9], "seq_start"), *slots = c.opt(a[10], "state_slots");
    need(q.dim() == 3 && v.dim() == 3, "q, k must be [T, Hk, Dk], v [T, Hv, Dv]");
    const int64_t T = q.size(0), Hk = q.size(1), Dk = q.size(2), Hv = v.size(1), Dv = v.size(2);
    need(k.sizes() == q.sizes() && v.size(0) == T && y.sizes() == v.sizes(),
         "q, k must be [T, Hk, Dk], v and y [T, Hv, Dv]");
    need(half_type(q) && half_type(k) && half_type(v), "q, k, v must be bf16");
    need(shaped(g, {T, Hv}) && g.scalar_type() == ScalarType::Float, "g must be fp32 [T, Hv]");
    need(shaped(beta, {T, Hv}) && beta.scalar_type() == ScalarType::Float, "beta must be fp32 [T, Hv]");
    need(s.dim() == 4 && shaped(s, {s.size(0), Hv, Dv, Dk}) && s.scalar_type() == ScalarType::Float,
         "state must be fp32 [slots, Hv, Dv, Dk]");
    need(!so || (so->sizes() == s.sizes() && so->scalar_type() == ScalarType::Float), "state_out must be as state");
    need(!start || (start->numel() >= 1 && words(*start)), "seq_start must be int32 [B + 1]");
    const int64_t B = start ? start->numel() - 1 : T;
    need(!slots || (slots->numel() == B && words(*slots)), "state_slots must be int32 [B]");
    const long long max_len = PyLong_AsLongLong(a[11]);
    const double scale = a[12] == Py_None ? 1.0 / std::sqrt(double(Dk)) : PyFloat_AsDouble(a[12]);
    const long l2 = PyLong_AsLong(a[13]);
    if (PyErr_Occurred()) bad("max_len, scale and l2norm must be numbers");
    if (B == 0 || (T == 0 && (!so || so->data_ptr() == s.data_ptr()))) return PyLong_FromLong(QMM_OK);
    const int od = out_type(y, "y");
    return PyLong_FromLong(f_gdn(
        static_cast<uint16_t*>(q.data_ptr()), static_cast<uint16_t*>(k.data_ptr()), static_cast<uint16_t*>(v.data_ptr()),
        static_cast<float*>(g.data_ptr()), static_cast<float*>(beta.data_ptr()), T, static_cast<int32_t*>(ptr(start)), B,
        max_len, Hk, Hv, Dk, Dv, float(scale), int(l2), static_cast<float*>(s.data_ptr()),
        static_cast<float*>(so ? so->data_ptr() : s.data_ptr()), static_cast<int32_t*>(ptr(slots)), s.size(0),
        ws.data_ptr(), ws.numel() * ws.element_size(), y.data_ptr(), od, c.stream));
  });
}

// bind(append, attn, gdn): addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 3, "bind takes 3 addresses");
    f_append = reinterpret_cast<decltype(f_append)>(PyLong_AsVoidPtr(a[0]));
    f_attn = reinterpret_cast<decltype(f_attn)>(PyLong_AsVoidPtr(a[1]));
    f_gdn = reinterpret_cast<decltype(f_gdn)>(PyLong_AsVoidPtr(a[2]));
    need(f_append && f_attn && f_gdn && !PyErr_Occurred(), "bind takes 3 addresses");
    Py_RETURN_NONE;
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(bind), FAST(cache), FAST(append), FAST(attn), FAST(gdn), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_qmm_mix", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_mix(void) { return PyModule_Create(&kModule); }
