// Argument marshalling of the paged-cache calls and of the head norm with
// rotation, as a CPython module: checks tensors, allocates outputs and calls
// the C ABI of include/ffpa.h.  paged.py wraps it (keyword arguments,
// documentation, statuses to exceptions) and gives it the library's functions.
//
// Why not ctypes, as for the attention calls: these calls take 3 to 12 us on
// the device when they serve single tokens, and the marshalling in Python took
// 14 to 27 us of the 26 to 44 us that a call took (now 7 to 13 us a call).
#include <ATen/ATen.h>
#include <ATen/FunctionalTensorWrapper.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ffpa.h"

namespace {

using at::Tensor;

// The C ABI's functions, from the library that the package has loaded.
struct Abi {
  decltype(&ffpa_decode_paged) decode = nullptr;
  decltype(&ffpa_decode_paged_workspace_bytes) decode_bytes = nullptr;
  decltype(&ffpa_qk_norm_rope) rope = nullptr;
  decltype(&ffpa_qk_norm_rope_bwd) rope_bwd = nullptr;
  decltype(&ffpa_qk_norm_rope_bwd_workspace_bytes) rope_bwd_bytes = nullptr;
  decltype(&ffpa_kv_append) append = nullptr;
  decltype(&ffpa_page_plan) plan = nullptr;
} abi;

// ---- arguments
const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch.Tensor");
  const Tensor& t = THPVariable_Unpack(o);
  // (Tracers' and transforms' tensors have no memory that a kernel could use: a pointer
  // of theirs is null or anything.  They go through the torch operators.)
  TORCH_CHECK_TYPE(!t.unsafeGetTensorImpl()->is_python_dispatch() && !at::functionalization::impl::isFunctionalTensor(t) &&
                       t.layout() == at::kStrided && t.has_storage() && !t.is_meta(),
                   name, " must be a tensor with memory of its own, not one that is traced or transformed");
  return t;
}
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
bool truth(PyObject* o) {
  const int b = PyObject_IsTrue(o);
  if (b < 0) throw python_error();
  return b != 0;
}
float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}
int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}
int small(int64_t x, const char* name) {
  TORCH_CHECK_VALUE(x >= INT_MIN && x <= INT_MAX, name, " = ", x, " is beyond 32 bits");
  return static_cast<int>(x);
}
const ffpa_options* options(PyObject* o) {
  return o == Py_None ? nullptr : reinterpret_cast<const ffpa_options*>(integer(o));
}
// A stream handle that the caller named, or torch's current stream of t's device.
ffpa_stream_t stream_of(PyObject* o, const Tensor& t) {
  if (o != Py_None) return reinterpret_cast<ffpa_stream_t>(integer(o));
  if (!t.is_cuda()) return nullptr;   // host tensors never reach a launch (the ABI rejects them)
  return reinterpret_cast<ffpa_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}
ffpa_dtype dtype_of(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? FFPA_BF16
         : t.scalar_type() == at::kHalf   ? FFPA_FP16
                                          : static_cast<ffpa_dtype>(-1);
}
const void* ptr(const Tensor* t) { return t ? t->const_data_ptr() : nullptr; }

// A new tensor beside `like`; on the GPU without the dispatcher's way round (a
// call makes up to five: the plan 13.8 -> 9.5 us of host time, a decode 13.3 -> 10.2).
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  if (like.is_cuda()) return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
  return at::empty(shape, like.options().dtype(type));
}

// A caller's output: what the library writes (it sizes every write from the
// inputs), or a new one.
Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const Tensor& like,
              bool contiguous = false) {
  if (o == Py_None) return fresh(shape, type, like);
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
  TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.device() == like.device(), name, " must be on ", like.device(), ", got ", t.device());
  TORCH_CHECK_VALUE(!contiguous || t.is_contiguous(), name, " must be contiguous");
  return t;
}
Tensor workspace(PyObject* o, size_t need, const Tensor& like) {
  if (o == Py_None) return fresh({static_cast<int64_t>(need < 256 ? 256 : need)}, at::kByte, like);
  const Tensor& t = tensor(o, "workspace");
  TORCH_CHECK_VALUE(t.scalar_type() == at::kByte && t.dim() == 1 && t.is_contiguous(),
                    "workspace must be a contiguous 1-D uint8 tensor");
  return t;
}
// A contiguous 1-D integer tensor with n entries (any number for n < 0).
const Tensor& integers(PyObject* o, const char* name, int64_t n, at::ScalarType type) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 1 && (n < 0 || t.size(0) == n), name, " must have ", n, " entries in one dimension, got ",
                    t.sizes());
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  return t;
}
const Tensor& table_of(PyObject* o) {
  const Tensor& t = tensor(o, "block_table");
  TORCH_CHECK_TYPE(t.scalar_type() == at::kInt, "block_table must be int32, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1),
                    "block_table must be 2-D [B, max_pages] with adjacent entries");
  return t;
}
void check_cache(const Tensor& kc, const Tensor& vc, at::ScalarType type, int64_t D) {
  TORCH_CHECK_VALUE(kc.dim() == 4 && vc.sizes() == kc.sizes(),
                    "k_cache and v_cache must be 4-D [num_pages, page_size, Hkv, D] of one shape");
  TORCH_CHECK_TYPE(kc.scalar_type() == type && vc.scalar_type() == type, "the cache must be ", type, ", got ",
                   kc.scalar_type(), " and ", vc.scalar_type());
  TORCH_CHECK_VALUE(kc.size(3) == D, "the cache has head dim ", kc.size(3), ", the call ", D);
}

// Queries and keys [B, H, N, D] or packed [T, H, D].  (That every tensor of a
// call is memory of one device is the C ABI's check.)
struct Shape {
  int B, Hq, Hkv, N, D;
};
Shape qk_shape(const Tensor& q, const Tensor& k) {
  TORCH_CHECK_VALUE(q.dim() == k.dim() && (q.dim() == 3 || q.dim() == 4),
                    "q and k must both be 4-D [B, H, N, D] or 3-D [T, H, D]");
  TORCH_CHECK_TYPE(q.scalar_type() == k.scalar_type(), "q and k must share one dtype");
  const bool dense = q.dim() == 4;
  const int h = 1, n = dense ? 2 : 0, d = dense ? 3 : 2;
  TORCH_CHECK_VALUE(q.size(n) == k.size(n) && q.size(d) == k.size(d) && (!dense || q.size(0) == k.size(0)),
                    "shape mismatch: q ", q.sizes(), ", k ", k.sizes());
  return {dense ? small(q.size(0), "B") : 1, small(q.size(h), "Hq"), small(k.size(h), "Hkv"), small(q.size(n), "N"),
          small(q.size(d), "D")};
}
// Strides of such rows as (b, h, n, d).
struct Rows {
  int64_t s[4];
  explicit Rows(const Tensor& t) {
    const auto x = t.strides();
    if (x.size() == 4)
      for (int i = 0; i < 4; ++i) s[i] = x[i];
    else
      s[0] = 0, s[1] = x[1], s[2] = x[0], s[3] = x[2];
  }
};

const void* weight(const Tensor* w, const char* name, const Tensor& k, int64_t D, ffpa_rope* r) {
  if (!w) return nullptr;
  TORCH_CHECK_TYPE(w->scalar_type() == at::kFloat || w->scalar_type() == k.scalar_type(), name, " must be float32 or ",
                   k.scalar_type(), ", got ", w->scalar_type());
  TORCH_CHECK_VALUE(w->dim() == 1 && w->size(0) == D && w->is_contiguous(), name, " must be contiguous [", D, "], got ",
                    w->sizes());
  r->weight_f32 = w->scalar_type() == at::kFloat;
  return w->const_data_ptr();
}
// positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale: seven arguments from a[0] on.
ffpa_rope rope_of(PyObject* const* a, const Tensor& k, const Shape& s) {
  ffpa_rope r{};
  const Tensor *positions = maybe(a[0], "positions"), *freq = maybe(a[1], "inv_freq");
  const Tensor *qw = maybe(a[2], "q_weight"), *kw = maybe(a[3], "k_weight");
  if (freq) {
    TORCH_CHECK_TYPE(freq->scalar_type() == at::kDouble, "inv_freq must be float64, got ", freq->scalar_type());
    TORCH_CHECK_VALUE(freq->dim() == 1 && freq->is_contiguous() && freq->size(0) > 0 && 2 * freq->size(0) <= s.D,
                      "inv_freq must be contiguous [rot_dim / 2] with rot_dim in 8..", s.D);
    TORCH_CHECK_VALUE(positions, "a rotation needs positions");
    const bool wide = positions->scalar_type() == at::kLong;
    TORCH_CHECK_TYPE(wide || positions->scalar_type() == at::kInt, "positions must be int32 or int64, got ",
                     positions->scalar_type());
    const auto n = positions->sizes();
    if (n.size() == 1 && n[0] == s.N) {
      r.position_str[1] = positions->stride(0);
    } else {
      TORCH_CHECK_VALUE(n.size() == 2 && n[1] == s.N && (n[0] == s.B || n[0] == 1), "positions must have shape [", s.N,
                        "] or [", s.B, ", ", s.N, "], got ", n);
      r.position_str[0] = n[0] == s.B ? positions->stride(0) : 0;
      r.position_str[1] = positions->stride(1);
    }
    r.positions = positions->const_data_ptr();
    r.position_bits = wide ? 64 : 32;
    r.inv_freq = static_cast<const double*>(freq->const_data_ptr());
    r.rot_dim = static_cast<int>(2 * freq->size(0));
  }
  TORCH_CHECK_TYPE(!qw || !kw || qw->scalar_type() == kw->scalar_type(), "q_weight and k_weight must share one dtype");
  r.q_weight = weight(qw, "q_weight", k, s.D, &r);
  r.k_weight = weight(kw, "k_weight", k, s.D, &r);
  r.eps = number(a[4]);
  r.interleaved = truth(a[5]);
  r.rope_scale = number(a[6]);
  return r;
}

// ---- results: the outputs, or the status of a call that was refused
template <class F>
ffpa_status call(F f) {
  ffpa_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}
PyObject* status(ffpa_status st) { return PyLong_FromLong(st); }
PyObject* none() { Py_RETURN_NONE; }
PyObject* wrap(const Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : none(); }
template <size_t N>
PyObject* tuple(const Tensor (&ts)[N]) {
  PyObject* r = PyTuple_New(N);
  if (!r) throw python_error();
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(r, i, wrap(ts[i]));
  return r;
}
void count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "takes ", want, " arguments, got ", n); }

// (q, k, <rope: 7>, q_out, k_out, stream)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 12);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  const Shape s = qk_shape(q, k);
  const ffpa_rope r = rope_of(a + 2, k, s);
  const Tensor qo = output(a[9], "q_out", q.sizes(), q.scalar_type(), q);
  const Tensor ko = output(a[10], "k_out", k.sizes(), k.scalar_type(), k);
  const Rows qs(q), ks(k), qos(qo), kos(ko);
  const ffpa_stream_t stream = stream_of(a[11], q);
  const ffpa_status st = call([&] {
    return abi.rope(q.const_data_ptr(), k.const_data_ptr(), qo.data_ptr(), ko.data_ptr(), dtype_of(q), s.B, s.Hq, s.Hkv,
                    s.N, s.D, qs.s, ks.s, qos.s, kos.s, &r, stream);
  });
  return st == FFPA_OK ? tuple({qo, ko}) : status(st);
  END_HANDLE_TH_ERRORS
}

// (dq_out, dk_out, q, k, <rope: 7>, dq, dk, workspace, stream)
PyObject* py_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 15);
  const Tensor &gq = tensor(a[0], "dq_out"), &gk = tensor(a[1], "dk_out"), &q = tensor(a[2], "q"), &k = tensor(a[3], "k");
  const Shape s = qk_shape(q, k);
  TORCH_CHECK_TYPE(gq.scalar_type() == q.scalar_type() && gk.scalar_type() == q.scalar_type(),
                   "dq_out and dk_out must be ", q.scalar_type(), ", got ", gq.scalar_type(), " and ", gk.scalar_type());
  TORCH_CHECK_VALUE(gq.sizes() == q.sizes() && gk.sizes() == k.sizes(), "dq_out and dk_out must have the shapes ",
                    q.sizes(), " and ", k.sizes(), ", got ", gq.sizes(), " and ", gk.sizes());
  const ffpa_rope r = rope_of(a + 4, k, s);
  const Tensor dq = output(a[11], "dq", q.sizes(), q.scalar_type(), q);
  const Tensor dk = output(a[12], "dk", k.sizes(), k.scalar_type(), k);
  const at::ScalarType wt = r.weight_f32 ? at::kFloat : k.scalar_type();
  Tensor dqw, dkw, ws;
  if (r.q_weight) dqw = fresh({s.D}, wt, q);
  if (r.k_weight) dkw = fresh({s.D}, wt, q);
  if (r.q_weight || r.k_weight) ws = workspace(a[13], abi.rope_bwd_bytes(s.D), q);
  const Rows gqs(gq), gks(gk), qs(q), ks(k), dqs(dq), dks(dk);
  const ffpa_stream_t stream = stream_of(a[14], q);
  const ffpa_status st = call([&] {
    return abi.rope_bwd(gq.const_data_ptr(), gk.const_data_ptr(), q.const_data_ptr(), k.const_data_ptr(), dq.data_ptr(),
                        dk.data_ptr(), dqw.defined() ? dqw.data_ptr() : nullptr,
                        dkw.defined() ? dkw.data_ptr() : nullptr, dtype_of(q), s.B, s.Hq, s.Hkv, s.N, s.D, gqs.s, gks.s,
                        qs.s, ks.s, dqs.s, dks.s, &r, ws.defined() ? ws.data_ptr() : nullptr,
                        ws.defined() ? static_cast<size_t>(ws.numel()) : 0, stream);
  });
  return st == FFPA_OK ? tuple({dq, dk, dqw, dkw}) : status(st);
  END_HANDLE_TH_ERRORS
}

// (q, k, v, k_cache, v_cache, slots, <rope: 7>, q_out, stream, options)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 16);
  const Tensor* q = maybe(a[0], "q");
  const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache");
  TORCH_CHECK_VALUE(k.dim() == 3 && v.sizes() == k.sizes(), "k and v must be 3-D [T, Hkv, D] of one shape");
  TORCH_CHECK_TYPE(v.scalar_type() == k.scalar_type(), "k and v must share one dtype");
  const Shape s = qk_shape(q ? *q : k, k);
  TORCH_CHECK_VALUE(q || (a[13] == Py_None && a[8] == Py_None), "q_out and q_weight need q");
  check_cache(kc, vc, k.scalar_type(), s.D);
  TORCH_CHECK_VALUE(kc.size(2) == s.Hkv, "the cache has ", kc.size(2), " key heads, the keys have ", s.Hkv);
  const Tensor& slots = integers(a[5], "slots", s.N, at::kLong);
  const ffpa_rope r = rope_of(a + 6, k, s);
  Tensor qo;
  if (q) qo = output(a[13], "q_out", q->sizes(), q->scalar_type(), *q);
  const int pages = small(kc.size(0), "num_pages"), page = small(kc.size(1), "page_size");
  const ffpa_stream_t stream = stream_of(a[14], k);
  const ffpa_options* opt = options(a[15]);
  const ffpa_status st = call([&] {
    return abi.append(ptr(q), k.const_data_ptr(), v.const_data_ptr(), q ? qo.data_ptr() : nullptr, kc.data_ptr(),
                      vc.data_ptr(), dtype_of(k), s.N, s.Hq, s.Hkv, s.D, pages, page, q ? q->strides().data() : nullptr,
                      k.strides().data(), v.strides().data(), q ? qo.strides().data() : nullptr, kc.strides().data(),
                      vc.strides().data(), static_cast<const int64_t*>(slots.const_data_ptr()), &r, stream, opt);
  });
  return st == FFPA_OK ? wrap(qo) : status(st);
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, block_table, seq_lens, scale, enable_gqa, return_lse, out, lse, workspace, stream, options)
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
  TORCH_CHECK_VALUE(q.dim() == 3, "q must be 3-D [B, Hq, D]");
  const int B = small(q.size(0), "B"), Hq = small(q.size(1), "Hq"), D = small(q.size(2), "D");
  check_cache(kc, vc, q.scalar_type(), D);
  const Tensor& table = table_of(a[3]);
  TORCH_CHECK_VALUE(table.size(0) == B, "block_table has ", table.size(0), " rows for ", B, " requests");
  const Tensor& lens = integers(a[4], "seq_lens", B, at::kInt);
  const int pages = small(kc.size(0), "num_pages"), page = small(kc.size(1), "page_size"), Hkv = small(kc.size(2), "Hkv");
  const bool scaled = a[5] != Py_None, gqa = truth(a[6]), want = truth(a[7]);
  const float scale = scaled ? number(a[5]) : 0.0f;
  const Tensor out = output(a[8], "out", q.sizes(), q.scalar_type(), q);
  Tensor lse;
  if (want || a[9] != Py_None) lse = output(a[9], "lse", {B, Hq}, at::kFloat, q, true);
  const Tensor ws = workspace(a[10], abi.decode_bytes(Hq, Hkv, D), q);
  const ffpa_stream_t stream = stream_of(a[11], q);
  const ffpa_options* opt = options(a[12]);
  const ffpa_status st = call([&] {
    return abi.decode(q.const_data_ptr(), kc.const_data_ptr(), vc.const_data_ptr(), out.data_ptr(),
                      lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, dtype_of(q), B, Hq, Hkv, D, pages,
                      page, static_cast<int>(table.size(1)), q.strides().data(), kc.strides().data(),
                      vc.strides().data(), out.strides().data(), static_cast<const int32_t*>(table.const_data_ptr()),
                      table.stride(0), static_cast<const int32_t*>(lens.const_data_ptr()), scaled ? &scale : nullptr, gqa,
                      ws.data_ptr(), static_cast<size_t>(ws.numel()), stream, opt);
  });
  return st != FFPA_OK ? status(st) : want ? tuple({out, lse}) : wrap(out);
  END_HANDLE_TH_ERRORS
}

// (block_table, seq_lens, new_lens, free_pages, free_count, page_size, num_tokens, stream, options)
PyObject* py_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Tensor& table = table_of(a[0]);
  const int64_t B = table.size(0);
  const Tensor &old = integers(a[1], "seq_lens", B, at::kInt), &add = integers(a[2], "new_lens", B, at::kInt);
  const Tensor &free = integers(a[3], "free_pages", -1, at::kInt), &left = integers(a[4], "free_count", 1, at::kInt);
  const int page = small(integer(a[5]), "page_size"), tokens = small(integer(a[6]), "num_tokens");
  TORCH_CHECK_VALUE(tokens >= 0 && page >= 1, "num_tokens must not be negative and page_size must be positive");
  const Tensor slots = fresh({tokens}, at::kLong, table), positions = fresh({tokens}, at::kInt, table);
  const Tensor cu = fresh({B + 1}, at::kInt, table), lens = fresh({B}, at::kInt, table), rest = fresh({1}, at::kInt, table);
  const int rows = small(B, "B"), width = small(table.size(1), "max_pages"), n_free = small(free.size(0), "free_pages");
  const ffpa_stream_t stream = stream_of(a[7], table);
  const ffpa_options* opt = options(a[8]);
  auto in = [](const Tensor& t) { return static_cast<const int32_t*>(t.const_data_ptr()); };
  auto to = [](const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
  const ffpa_status st = call([&] {
    return abi.plan(to(table), table.stride(0), rows, width, in(old), in(add), in(free), n_free, in(left), page, tokens,
                    static_cast<int64_t*>(slots.data_ptr()), to(positions), to(cu), to(lens), to(rest), stream, opt);
  });
  return st == FFPA_OK ? tuple({slots, positions, cu, lens, rest}) : status(st);
  END_HANDLE_TH_ERRORS
}

// The addresses of the library's functions, in the order of Abi.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  void* p[7];
  for (int i = 0; i < 7; ++i) p[i] = reinterpret_cast<void*>(integer(a[i]));
  abi.decode = reinterpret_cast<decltype(abi.decode)>(p[0]);
  abi.decode_bytes = reinterpret_cast<decltype(abi.decode_bytes)>(p[1]);
  abi.rope = reinterpret_cast<decltype(abi.rope)>(p[2]);
  abi.rope_bwd = reinterpret_cast<decltype(abi.rope_bwd)>(p[3]);
  abi.rope_bwd_bytes = reinterpret_cast<decltype(abi.rope_bwd_bytes)>(p[4]);
  abi.append = reinterpret_cast<decltype(abi.append)>(p[5]);
  abi.plan = reinterpret_cast<decltype(abi.plan)>(p[6]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FFPA_PY(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FFPA_PY("bind", py_bind),         FFPA_PY("qk_norm_rope", py_rope),
                         FFPA_PY("qk_norm_rope_bwd", py_rope_bwd), FFPA_PY("kv_append", py_append),
                         FFPA_PY("decode_paged", py_decode), FFPA_PY("page_plan", py_plan),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "ffpa_paged_binding", nullptr, -1, methods,
                          nullptr,               nullptr,              nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ffpa_paged_binding() { return PyModule_Create(&module_def); }
