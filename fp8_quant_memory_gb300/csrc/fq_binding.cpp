// fq_binding.cpp -- CPython module over the FP8 serving entry points of include/fq.h. It checks devices, dtypes
// and shapes of torch tensors, allocates outputs and workspaces with torch, and calls libfq on the current stream
// of the tensors' device. It is compiled, where the other entry points go through ctypes, because a decoding step
// makes these calls with a few microseconds of GPU work in each: checking a dozen tensors attribute by attribute
// from Python took 14 to 24 us a call.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>

#include "fq.h"

namespace {

PyObject* g_fq_error = nullptr;  // the package's FqError

// Raises ValueError (the package's answer to arguments that do not fit).
struct Refused {};

[[noreturn]] void refuse(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(PyExc_ValueError, fmt, ap);
  va_end(ap);
  throw Refused{};
}

using Tensor = const at::Tensor&;

const at::Tensor& tensor(const char* fn, const char* name, PyObject* o, bool optional = false) {
  static const at::Tensor none;
  if (optional && o == Py_None) return none;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: %s must be a tensor", fn, name);
    throw Refused{};
  }
  return THPVariable_Unpack(o);
}

void same_device(const char* fn, std::initializer_list<const at::Tensor*> ts) {
  const at::Device dev = (*ts.begin())->device();
  for (const at::Tensor* t : ts) {
    if (!t->defined()) continue;
    if (!t->is_cuda()) refuse("%s: every tensor must be on a CUDA device", fn);
    if (t->device() != dev) refuse("%s: tensors are on different devices", fn);
  }
}

bool codes(Tensor t) { return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn; }

int out_code(at::ScalarType t) { return t == at::kBFloat16 ? FQ_BF16 : t == at::kHalf ? FQ_FP16 : -1; }

at::ScalarType dtype_arg(const char* fn, PyObject* o) {
  if (!THPDtype_Check(o)) refuse("%s: out_dtype must be bfloat16 or float16", fn);
  const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  if (out_code(t) < 0) refuse("%s: out_dtype must be bfloat16 or float16", fn);
  return t;
}

bool shape(Tensor t, std::initializer_list<int64_t> want) { return t.sizes() == at::IntArrayRef(want); }

int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

cudaStream_t stream_of(Tensor t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

// Runs an entry point without the interpreter lock (strict mode waits in it) and raises FqError on failure.
template <typename F>
void launch(const char* fn, F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS
  if (rc == FQ_OK) return;
  PyObject* e = PyObject_CallFunction(g_fq_error, "sis", fn, rc, fq_last_error());
  if (e != nullptr) {
    PyErr_SetObject(g_fq_error, e);
    Py_DECREF(e);
  }
  throw Refused{};
}

void want_args(const char* fn, Py_ssize_t got, Py_ssize_t want) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments expected, got %zd", fn, want, got);
    throw Refused{};
  }
}

template <typename T>
T* ptr(Tensor t) {
  return static_cast<T*>(t.data_ptr());
}

// --------------------------------------------------------------------------- matrix product
// (a, a_scale, b, b_scale, out_dtype, out or None) -> out
PyObject* matmul(PyObject* const* args, Py_ssize_t n) {
  const char* fn = "fp8_matmul";
  want_args(fn, n, 6);
  Tensor a = tensor(fn, "a", args[0]), sa = tensor(fn, "a_scale", args[1]), b = tensor(fn, "b", args[2]),
         sb = tensor(fn, "b_scale", args[3]), given = tensor(fn, "out", args[5], true);
  same_device(fn, {&a, &sa, &b, &sb, &given});
  if (a.dim() != 2 || b.dim() != 2) refuse("%s: a and b must be [M, K] and [N, K]", fn);
  const int64_t M = a.size(0), K = a.size(1), N = b.size(0), g = (K + 127) / 128, blocks = (N + 127) / 128;
  if (b.size(1) != K || K < 1) refuse("%s: a and b must share K >= 1, got %lld and %lld", fn, (long long)K, (long long)b.size(1));
  if (!codes(a) || !codes(b)) refuse("%s: a and b must hold e4m3 codes (uint8 or float8_e4m3fn)", fn);
  if (sa.scalar_type() != at::kFloat || sb.scalar_type() != at::kFloat) refuse("%s: scales must be float32", fn);
  if (!shape(sa, {M, g}) || !shape(sb, {blocks, g}))
    refuse("%s: a_scale must be [%lld, %lld] and b_scale [%lld, %lld]", fn, (long long)M, (long long)g, (long long)blocks, (long long)g);
  if ((K > 1 && (a.stride(1) != 1 || b.stride(1) != 1)) || (g > 1 && (sa.stride(1) != 1 || sb.stride(1) != 1)))
    refuse("%s: rows of the operands and of their scales must be contiguous", fn);
  const c10::DeviceGuard guard(a.device());
  at::Tensor out = given;
  if (!out.defined()) {
    out = at::empty({M, N}, a.options().dtype(dtype_arg(fn, args[4])));
  } else if (out_code(out.scalar_type()) < 0 || !shape(out, {M, N}) || (N > 1 && out.stride(1) != 1)) {
    refuse("%s: out must be [%lld, %lld] bfloat16 or float16 with contiguous rows", fn, (long long)M, (long long)N);
  }
  launch("fq_fp8_matmul", [&] {
    return fq_fp8_matmul(ptr<uint8_t>(a), a.stride(0), ptr<float>(sa), sa.stride(0), ptr<uint8_t>(b), b.stride(0), ptr<float>(sb),
                         sb.stride(0), out.data_ptr(), out.stride(0), M, N, K, out_code(out.scalar_type()), stream_of(a));
  });
  return THPVariable_Wrap(out);
}

// ------------------------------------------------------------------------------------ cache
fq_paged_cache cache_of(const char* fn, Tensor k, Tensor v, Tensor ks, Tensor vs) {
  if (k.dim() != 4 || v.sizes() != k.sizes()) refuse("%s: k_cache and v_cache must be [pages, Hk, page_size, D] of the same shape", fn);
  if (ks.sizes() != k.sizes().slice(0, 3) || vs.sizes() != ks.sizes()) refuse("%s: k_scale and v_scale must be [pages, Hk, page_size]", fn);
  if (!codes(k) || !codes(v)) refuse("%s: the cache must hold e4m3 codes (uint8 or float8_e4m3fn)", fn);
  if (ks.scalar_type() != at::kFloat || vs.scalar_type() != at::kFloat) refuse("%s: scales must be float32", fn);
  if (v.strides() != k.strides() || vs.strides() != ks.strides()) refuse("%s: k and v must share their strides", fn);
  if (k.stride(3) != 1 && k.size(3) != 1) refuse("%s: rows of the cache must be contiguous", fn);
  fq_paged_cache c;
  c.k = ptr<uint8_t>(k);
  c.v = ptr<uint8_t>(v);
  c.k_scale = ptr<float>(ks);
  c.v_scale = ptr<float>(vs);
  c.pages = k.size(0);
  c.page_size = k.size(2);
  c.page_stride = k.stride(0);
  c.head_stride = k.stride(1);
  c.token_stride = k.stride(2);
  c.scale_page_stride = ks.stride(0);
  c.scale_head_stride = ks.stride(1);
  c.scale_token_stride = ks.stride(2);
  return c;
}

// (qkv, wq, wk, cos, sin, slots, k_cache, v_cache, k_scale, v_scale, Hq, Hk, eps, fp8_max, rope_dim or None,
//  q_out or None, q_scale or None) -> (q_out, q_scale)
PyObject* append(PyObject* const* args, Py_ssize_t n) {
  const char* fn = "qkv_norm_rope_append";
  want_args(fn, n, 17);
  Tensor qkv = tensor(fn, "qkv", args[0]), wq = tensor(fn, "wq", args[1]), wk = tensor(fn, "wk", args[2]),
         cos = tensor(fn, "cos", args[3]), sin = tensor(fn, "sin", args[4]), slots = tensor(fn, "slots", args[5]),
         k = tensor(fn, "k_cache", args[6]), v = tensor(fn, "v_cache", args[7]), ks = tensor(fn, "k_scale", args[8]),
         vs = tensor(fn, "v_scale", args[9]), given_q = tensor(fn, "q_out", args[15], true),
         given_s = tensor(fn, "q_scale", args[16], true);
  same_device(fn, {&qkv, &wq, &wk, &cos, &sin, &slots, &k, &v, &ks, &vs, &given_q, &given_s});
  const fq_paged_cache c = cache_of(fn, k, v, ks, vs);
  const int64_t Hq = whole(args[10]), Hk = whole(args[11]), D = k.size(3);
  const double eps = real(args[12]), fp8_max = real(args[13]);
  if (Hq < 0 || Hk < 1 || Hq > (1 << 24) || k.size(1) != Hk) refuse("%s: need Hq >= 0 and a cache of Hk >= 1 heads", fn);
  if (qkv.dim() != 2 || qkv.size(1) < (Hq + 2 * Hk) * D || (qkv.stride(1) != 1 && qkv.size(1) > 1))
    refuse("%s: qkv must be [T, S] with contiguous rows of S >= (Hq + 2*Hk)*D", fn);
  const int64_t T = qkv.size(0), R = args[14] == Py_None ? D : whole(args[14]);
  const int dt = out_code(qkv.scalar_type());
  if (dt < 0 || wq.scalar_type() != qkv.scalar_type() || wk.scalar_type() != qkv.scalar_type())
    refuse("%s: qkv, wq and wk must share bfloat16 or float16", fn);
  if (!shape(wq, {D}) || !shape(wk, {D}) || !wq.is_contiguous() || !wk.is_contiguous())
    refuse("%s: wq and wk must be contiguous [%lld]", fn, (long long)D);
  if (R < 0 || R > D || R % 2 != 0) refuse("%s: rope_dim must be even and in [0, %lld]", fn, (long long)D);
  const int td = cos.scalar_type() == at::kFloat ? FQ_FP32 : out_code(cos.scalar_type());
  if (td < 0 || sin.scalar_type() != cos.scalar_type()) refuse("%s: cos and sin must share one of bfloat16/float16/float32", fn);
  if (!shape(cos, {T, R / 2}) || !shape(sin, {T, R / 2}) || !cos.is_contiguous() || !sin.is_contiguous())
    refuse("%s: cos and sin must be contiguous [%lld, %lld]", fn, (long long)T, (long long)(R / 2));
  if (slots.scalar_type() != at::kLong || !shape(slots, {T}) || !slots.is_contiguous())
    refuse("%s: slots must be contiguous int64 [%lld]", fn, (long long)T);
  const c10::DeviceGuard guard(qkv.device());
  at::Tensor q = given_q, qs = given_s;
  if (!q.defined()) q = at::empty({T, Hq, D}, qkv.options().dtype(at::kByte));
  else if (!codes(q) || !shape(q, {T, Hq, D}) || !q.is_contiguous())
    refuse("%s: q_out must be contiguous codes [%lld, %lld, %lld]", fn, (long long)T, (long long)Hq, (long long)D);
  if (!qs.defined()) qs = at::empty({T, Hq}, qkv.options().dtype(at::kFloat));
  else if (qs.scalar_type() != at::kFloat || !shape(qs, {T, Hq}) || !qs.is_contiguous())
    refuse("%s: q_scale must be contiguous float32 [%lld, %lld]", fn, (long long)T, (long long)Hq);
  launch("fq_qkv_norm_rope_append", [&] {
    return fq_qkv_norm_rope_append(qkv.data_ptr(), qkv.stride(0), wq.data_ptr(), wk.data_ptr(), cos.data_ptr(), sin.data_ptr(),
                                   ptr<int64_t>(slots), ptr<uint8_t>(q), ptr<float>(qs), &c, T, Hq, Hk, D, R, dt, td,
                                   static_cast<float>(eps), static_cast<float>(fp8_max), stream_of(qkv));
  });
  PyObject* pair = PyTuple_New(2);
  if (pair == nullptr) throw Refused{};
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(q));
  PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(qs));
  return pair;
}

// -------------------------------------------------------------------------------- attention
// (q, q_scale, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, softmax_scale or None, out_dtype,
//  max_seq_len or None, want_lse, out or None, lse or None, workspace or None) -> (out, lse or None)
PyObject* attention(PyObject* const* args, Py_ssize_t n) {
  const char* fn = "paged_attention";
  want_args(fn, n, 15);
  Tensor q = tensor(fn, "q", args[0]), qs = tensor(fn, "q_scale", args[1]), k = tensor(fn, "k_cache", args[2]),
         v = tensor(fn, "v_cache", args[3]), ks = tensor(fn, "k_scale", args[4]), vs = tensor(fn, "v_scale", args[5]),
         table = tensor(fn, "page_table", args[6]), lens = tensor(fn, "seq_lens", args[7]),
         given_out = tensor(fn, "out", args[12], true), given_lse = tensor(fn, "lse", args[13], true),
         given_ws = tensor(fn, "workspace", args[14], true);
  same_device(fn, {&q, &qs, &k, &v, &ks, &vs, &table, &lens, &given_out, &given_lse, &given_ws});
  const fq_paged_cache c = cache_of(fn, k, v, ks, vs);
  if (q.dim() != 3 || !codes(q)) refuse("%s: q must hold e4m3 codes [B, Hq, D]", fn);
  const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hk = k.size(1);
  if (k.size(3) != D || Hk < 1 || Hq < 1 || Hq % Hk != 0)
    refuse("%s: q and the cache must share D, and Hq must be a multiple of the cache's heads", fn);
  if ((q.stride(2) != 1 && D != 1) || (q.stride(1) != D && Hq != 1)) refuse("%s: the heads of a sequence must be contiguous in q", fn);
  if (qs.scalar_type() != at::kFloat || !shape(qs, {B, Hq}) || (qs.stride(1) != 1 && Hq != 1))
    refuse("%s: q_scale must be float32 [%lld, %lld] with contiguous rows", fn, (long long)B, (long long)Hq);
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B || (table.size(1) > 1 && table.stride(1) != 1))
    refuse("%s: page_table must be int32 [%lld, max_pages] with contiguous rows", fn, (long long)B);
  if (lens.scalar_type() != at::kInt || !shape(lens, {B}) || (B > 1 && lens.stride(0) != 1))
    refuse("%s: seq_lens must be contiguous int32 [%lld]", fn, (long long)B);
  const int64_t max_pages = table.size(1);
  int64_t max_len = max_pages > INT64_MAX / std::max<int64_t>(c.page_size, 1) ? INT64_MAX : max_pages * c.page_size;
  if (args[10] != Py_None) max_len = std::min(max_len, whole(args[10]));
  if (max_len < 0) refuse("%s: max_seq_len must be >= 0", fn);
  const double scale = args[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : real(args[8]);
  const int want_lse = PyObject_IsTrue(args[11]);
  if (want_lse < 0) throw Refused{};
  const c10::DeviceGuard guard(q.device());
  at::Tensor out = given_out, lse = given_lse, ws = given_ws;
  if (!out.defined()) out = at::empty({B, Hq, D}, q.options().dtype(dtype_arg(fn, args[9])));
  else if (out_code(out.scalar_type()) < 0 || !shape(out, {B, Hq, D}) || !out.is_contiguous())
    refuse("%s: out must be contiguous bfloat16 or float16 [%lld, %lld, %lld]", fn, (long long)B, (long long)Hq, (long long)D);
  if (lse.defined()) {
    if (lse.scalar_type() != at::kFloat || !shape(lse, {B, Hq}) || !lse.is_contiguous())
      refuse("%s: lse must be contiguous float32 [%lld, %lld]", fn, (long long)B, (long long)Hq);
  } else if (want_lse) {
    lse = at::empty({B, Hq}, q.options().dtype(at::kFloat));
  }
  size_t bytes = 0;
  if (ws.defined()) {
    if (!ws.is_contiguous()) refuse("%s: workspace must be contiguous", fn);
    bytes = ws.nbytes();
  } else {
    bytes = fq_paged_attention_workspace_bytes(B, Hq, Hk, D, max_len);
    if (bytes > 0) ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
  }
  launch("fq_paged_attention", [&] {
    return fq_paged_attention(ptr<uint8_t>(q), q.stride(0), ptr<float>(qs), qs.stride(0), &c, ptr<int32_t>(table), table.stride(0),
                              ptr<int32_t>(lens), out.data_ptr(), lse.defined() ? ptr<float>(lse) : nullptr,
                              ws.defined() ? ws.data_ptr() : nullptr, bytes, B, Hq, Hk, D, max_pages, max_len,
                              static_cast<float>(scale), out_code(out.scalar_type()), stream_of(q));
  });
  PyObject* pair = PyTuple_New(2);
  if (pair == nullptr) throw Refused{};
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
  if (lse.defined()) {
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(pair, 1, Py_None);
  }
  return pair;
}

// No C++ exception leaves the module: a refusal has set its Python error, torch's own become theirs.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error_class(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_fq_error);
  g_fq_error = cls;
  Py_RETURN_NONE;
}

#define FQ_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FQ_METHOD("fp8_matmul", matmul), FQ_METHOD("qkv_norm_rope_append", append),
                           FQ_METHOD("paged_attention", attention), {"set_error_class", set_error_class, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fq_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fq_binding() { return PyModule_Create(&g_module); }
