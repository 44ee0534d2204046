// Python side of a serving step's calls (qmm_serve.h): checks the tensors, fills in pointers,
// sizes and the current stream, and calls the C ABI (as mix_binding.cpp).  Every function
// returns the C status.
#include "binding.h"
#include "qmm_serve.h"

namespace {

// The entry points of the loaded library (bind).
decltype(&qmm_kv8_append) f_append = nullptr;
decltype(&qmm_kv8_attn) f_attn = nullptr;
decltype(&qmm_spec_verify) f_verify = nullptr;
decltype(&qmm_lora) f_lora = nullptr;

bool f32(const Tensor& t) { return t.scalar_type() == ScalarType::Float; }

// cache(k_codes, k_scale, v_codes, v_scale) -> (struct bytes, device)
PyObject* cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 4, "cache takes 4 tensors");
    auto shape_of = [&](PyObject* o, const char* name) -> const Tensor& {
      if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
      return THPVariable_Unpack(o);
    };
    const Tensor &kc = shape_of(a[0], "k_codes"), &ks = shape_of(a[1], "k_scale"), &vc = shape_of(a[2], "v_codes"),
                 &vs = shape_of(a[3], "v_scale");
    need(kc.dim() == 4 && kc.scalar_type() == ScalarType::Char, "k_codes must be int8 [pages, heads, page_size, head_dim]");
    const int64_t p = kc.size(0), h = kc.size(1), s = kc.size(2), hd = kc.size(3);
    need(shaped(ks, {p, h, s / 16}) && f32(ks), "k_scale must be fp32 [pages, heads, page_size/16]");
    need(shaped(vc, {p, h, s / 8, hd, 8}) && vc.scalar_type() == ScalarType::Char,
         "v_codes must be int8 [pages, heads, page_size/8, head_dim, 8]");
    need(shaped(vs, {p, h, s / 16}) && f32(vs), "v_scale must be fp32 [pages, heads, page_size/16]");
    Call c;
    c.get(a[0], "k_codes");
    c.device = kc.get_device();
    c.get(a[1], "k_scale"), c.get(a[2], "v_codes"), c.get(a[3], "v_scale");
    const qmm_kv8_cache v = {static_cast<int8_t*>(kc.data_ptr()), static_cast<float*>(ks.data_ptr()),
                             static_cast<int8_t*>(vc.data_ptr()), static_cast<float*>(vs.data_ptr()), p, s, h, hd};
    return Py_BuildValue("y#i", reinterpret_cast<const char*>(&v), Py_ssize_t(sizeof v), c.device);
  });
}

qmm_kv8_cache cache_of(PyObject* o, const Call& c) {
  const char* p;
  Py_ssize_t n;
  int dev;
  if (!PyArg_ParseTuple(o, "y#i", &p, &n, &dev) || n != sizeof(qmm_kv8_cache)) bad("cache must be a KV8Cache");
  if (dev != c.device)
    bad("the cache is on device " + std::to_string(dev) + ", the current device is " + std::to_string(c.device));
  qmm_kv8_cache v;
  memcpy(&v, p, sizeof v);
  return v;
}

// The sequences of a call: page_table int32 [B, max_pages], kv_lens int32 [B], q_start int32 [B + 1].
struct Seqs {
  const Tensor &table, &lens, *start;
  Seqs(const Call& c, PyObject* t, PyObject* l, PyObject* s)
      : table(c.get(t, "page_table")), lens(c.get(l, "kv_lens")), start(c.opt(s, "q_start")) {
    need(table.dim() == 2 && words(table), "page_table must be int32 [B, max_pages]");
    need(lens.numel() == B() && words(lens), "kv_lens must be int32 [B]");
    need(!start || (start->numel() == B() + 1 && words(*start)), "q_start must be int32 [B + 1]");
  }
  int64_t B() const { return table.size(0); }
  const int32_t* q_start() const { return static_cast<int32_t*>(ptr(start)); }
  const int32_t* kv_lens() const { return static_cast<int32_t*>(lens.data_ptr()); }
  const int32_t* pages() const { return static_cast<int32_t*>(table.data_ptr()); }
};

// append(cache, k, v, page_table, kv_lens, q_start, max_q, positions, cos_sin, q, q_out, k_held, v_held, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 14, "append takes 14 arguments");
    const Call c(a[13]);
    const qmm_kv8_cache kv = cache_of(a[0], c);
    const Tensor &k = c.get(a[1], "k"), &v = c.get(a[2], "v");
    const Seqs s(c, a[3], a[4], a[5]);
    const Tensor *pos = c.opt(a[7], "positions"), *cs = c.opt(a[8], "cos_sin"), *q = c.opt(a[9], "q"),
                 *qo = c.opt(a[10], "q_out"), *kh = c.opt(a[11], "k_held"), *vh = c.opt(a[12], "v_held");
    const long long max_q = PyLong_AsLongLong(a[6]);
    if (PyErr_Occurred()) bad("max_q must be a number");
    need(k.dim() == 3, "k, v must be [T, n_kv, head_dim]");
    const int64_t T = k.size(0), h = kv.n_kv_heads, hd = kv.head_dim;
    need(shaped(k, {T, h, hd}) && shaped(v, {T, h, hd}), "k, v must be [T, n_kv, head_dim]");
    const int dt = out_type(k, "k");
    need(out_type(v, "v") == dt && (!q || out_type(*q, "q") == dt), "q, k, v must share a dtype");
    need(!pos || (pos->numel() == T && words(*pos)), "positions must be int32 [T]");
    need(!cs || (cs->dim() == 2 && f32(*cs)), "cos_sin must be fp32 [max_pos, rot_dim]");
    need(cs || (!pos && !q), "positions and q need cos_sin");
    need(!q == !qo, "q and q_out go together");
    if (q) {
      need(q->dim() == 3 && q->size(0) == T && q->size(2) == hd, "q must be [T, n_q, head_dim]");
      need(qo->sizes() == q->sizes() && half_type(*qo), "q_out must be bf16, as q");
    }
    need(!kh || (shaped(*kh, {T, h, hd}) && half_type(*kh)), "k_held must be bf16 [T, n_kv, head_dim]");
    need(!vh || (shaped(*vh, {T, h, hd}) && half_type(*vh)), "v_held must be bf16 [T, n_kv, head_dim]");
    if (T == 0 || s.B() == 0) return PyLong_FromLong(QMM_OK);
    return PyLong_FromLong(f_append(
        &kv, k.data_ptr(), v.data_ptr(), T, dt, s.q_start(), s.kv_lens(), s.pages(), s.B(), s.table.size(1), max_q,
        static_cast<int32_t*>(ptr(pos)), static_cast<float*>(ptr(cs)), cs ? cs->size(0) : 0, cs ? cs->size(1) : 0,
        ptr(q), q ? q->size(1) : 0, static_cast<uint16_t*>(ptr(qo)), static_cast<uint16_t*>(ptr(kh)),
        static_cast<uint16_t*>(ptr(vh)), c.stream));
  });
}

// attn(q, cache, page_table, kv_lens, out, workspace, q_start, max_q, scale, causal, window, sinks, gate, stream)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 14, "attn takes 14 arguments");
    const Call c(a[13]);
    const Tensor& q = c.get(a[0], "q");
    const qmm_kv8_cache kv = cache_of(a[1], c);
    const Seqs s(c, a[2], a[3], a[6]);
    const Tensor &out = c.get(a[4], "out"), &ws = c.get(a[5], "workspace");
    const Tensor* gate = c.opt(a[12], "gate");
    const long long max_q = PyLong_AsLongLong(a[7]), window = PyLong_AsLongLong(a[10]), sinks = PyLong_AsLongLong(a[11]);
    const long causal = PyLong_AsLong(a[9]);
    need(q.dim() == 3 && q.size(2) == kv.head_dim, "q must be [T, n_q, head_dim]");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt(double(kv.head_dim)) : PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) bad("max_q, scale, causal, window and sinks must be numbers");
    need(half_type(q) && half_type(out) && out.sizes() == q.sizes(), "q and out must be bf16 [T, n_q, head_dim]");
    need(!gate || (gate->sizes() == q.sizes() && half_type(*gate)), "gate must be bf16, as q");
    if (q.size(0) == 0 || s.B() == 0) return PyLong_FromLong(QMM_OK);
    return PyLong_FromLong(f_attn(
        static_cast<uint16_t*>(q.data_ptr()), q.size(0), s.q_start(), s.kv_lens(), s.pages(), s.B(), s.table.size(1),
        max_q, &kv, q.size(1), float(scale), int(causal), window, sinks, static_cast<uint16_t*>(ptr(gate)),
        ws.data_ptr(), ws.numel() * ws.element_size(), static_cast<uint16_t*>(out.data_ptr()), c.stream));
  });
}

// verify(draft, target, u, tokens, accepted, workspace, draft_start, draft_probs, stream)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 9, "verify takes 9 arguments");
    const Call c(a[8]);
    const Tensor &draft = c.get(a[0], "draft"), &p = c.get(a[1], "target"), &u = c.get(a[2], "u"),
                 &tokens = c.get(a[3], "tokens"), &accepted = c.get(a[4], "accepted"), &ws = c.get(a[5], "workspace"),
                 &start = c.get(a[6], "draft_start");
    const Tensor* q = c.opt(a[7], "draft_probs");
    need(tokens.dim() == 2 && tokens.size(1) >= 1 && words(tokens), "tokens must be int32 [B, max_draft + 1]");
    const int64_t B = tokens.size(0), D = draft.numel();
    need(words(draft), "draft must be int32 [D]");
    need(start.numel() == B + 1 && words(start), "draft_start must be int32 [B + 1]");
    need(accepted.numel() == B && words(accepted), "accepted must be int32 [B]");
    need(p.dim() == 2 && p.size(0) == D + B, "target must be [D + B, V]");
    const int64_t V = p.size(1);
    const auto prob = [](const Tensor& t) { return t.scalar_type() == ScalarType::BFloat16 || f32(t); };
    need(prob(p), "target must be bf16 or fp32");
    need(!q || (shaped(*q, {D, V}) && q->scalar_type() == p.scalar_type()), "draft_probs must be [D, V], as target");
    need(u.numel() == D + B && f32(u), "u must be fp32 [D + B]");
    if (B == 0) return PyLong_FromLong(QMM_OK);
    // of no drafts there are no probabilities: an empty tensor has no address
    return PyLong_FromLong(f_verify(
        static_cast<int32_t*>(draft.data_ptr()), D, static_cast<int32_t*>(start.data_ptr()), B, tokens.size(1) - 1,
        p.data_ptr(), ptr(q), V, f32(p) ? QMM_OUT_F32 : QMM_OUT_BF16, static_cast<float*>(u.data_ptr()),
        static_cast<int32_t*>(tokens.data_ptr()), static_cast<int32_t*>(accepted.data_ptr()), ws.data_ptr(),
        ws.numel() * ws.element_size(), c.stream));
  });
}

// lora(x, a, b, ids, y, workspace, base, scales, stream); y and base: tuples of 1 .. 3 tensors, base may be None
PyObject* lora(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 9, "lora takes 9 arguments");
    const Call c(a[8]);
    const Tensor &x = c.get(a[0], "x"), &A = c.get(a[1], "a"), &Bw = c.get(a[2], "b"), &ids = c.get(a[3], "ids"),
                 &ws = c.get(a[5], "workspace");
    const Tensor* scales = c.opt(a[7], "scales");
    need(PyTuple_Check(a[4]) && (a[6] == Py_None || PyTuple_Check(a[6])), "y and base must be tuples of tensors");
    const Py_ssize_t parts = PyTuple_GET_SIZE(a[4]);
    need(parts >= 1 && parts <= 3, "y must be 1 to 3 tensors");
    need(a[6] == Py_None || PyTuple_GET_SIZE(a[6]) == parts, "base must be as many tensors as y");
    need(x.dim() == 2 && half_type(x), "x must be bf16 [T, K]");
    const int64_t T = x.size(0), K = x.size(1);
    need(Bw.dim() == 3 && half_type(Bw), "b must be bf16 [adapters, rows, rank]");
    const int64_t ad = Bw.size(0), rank = Bw.size(2);
    need(shaped(A, {ad, parts * rank, K}) && half_type(A), "a must be bf16 [adapters, parts * rank, K]");
    need(ids.numel() == T && words(ids), "ids must be int32 [T]");
    need(!scales || (scales->numel() == ad && f32(*scales)), "scales must be fp32 [adapters]");
    int64_t rows[3] = {}, total = 0;
    const void* from[3] = {};
    void* to[3] = {};
    int base_type = 0, type = 0;
    for (Py_ssize_t p = 0; p < parts; ++p) {
      const Tensor& y = c.get(PyTuple_GET_ITEM(a[4], p), "y");
      need(y.dim() == 2 && y.size(0) == T, "y must be [T, rows]");
      const int t = out_type(y, "y");
      need(p == 0 || t == type, "the parts of y must share a dtype");
      type = t, rows[p] = y.size(1), total += rows[p], to[p] = y.data_ptr();
      if (a[6] != Py_None) {
        const Tensor& base = c.get(PyTuple_GET_ITEM(a[6], p), "base");
        need(base.sizes() == y.sizes(), "base must be shaped as y");
        const int bt = out_type(base, "base");
        need(p == 0 || bt == base_type, "the parts of base must share a dtype");
        base_type = bt, from[p] = base.data_ptr();
      }
    }
    need(Bw.size(1) == total, "b must have the parts' rows");
    if (T == 0) return PyLong_FromLong(QMM_OK);
    return PyLong_FromLong(f_lora(
        static_cast<uint16_t*>(x.data_ptr()), T, K, static_cast<uint16_t*>(A.data_ptr()),
        static_cast<uint16_t*>(Bw.data_ptr()), ad, rank, static_cast<int32_t*>(ids.data_ptr()),
        static_cast<float*>(ptr(scales)), parts, rows, a[6] == Py_None ? nullptr : from, base_type, to, type,
        ws.data_ptr(), ws.numel() * ws.element_size(), c.stream));
  });
}

// bind(append, attn, verify, lora): addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need(n == 4, "bind takes 4 addresses");
    f_append = reinterpret_cast<decltype(f_append)>(PyLong_AsVoidPtr(a[0]));
    f_attn = reinterpret_cast<decltype(f_attn)>(PyLong_AsVoidPtr(a[1]));
    f_verify = reinterpret_cast<decltype(f_verify)>(PyLong_AsVoidPtr(a[2]));
    f_lora = reinterpret_cast<decltype(f_lora)>(PyLong_AsVoidPtr(a[3]));
    need(f_append && f_attn && f_verify && f_lora && !PyErr_Occurred(), "bind takes 4 addresses");
    Py_RETURN_NONE;
  });
}

PyMethodDef kMethods[] = {FAST(bind),   FAST(cache), FAST(append), FAST(attn),
                          FAST(verify), FAST(lora),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_qmm_serve", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_serve(void) { return PyModule_Create(&kModule); }
