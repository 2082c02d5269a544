// The way in from Python of the FP8 layer's and the prompt's operators: checks torch
// tensors and calls the C ABI.  A small call's kernel takes two microseconds; the same
// checks made in Python (shapes, types, strides and pointers of up to seven tensors,
// then ctypes) took seven, this module about one.  No arithmetic happens here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <string>

#include "../../include/mla_decode.h"

namespace {

PyObject* g_error_type = nullptr;  // binding.MlaError

// A refusal on its way to Python.
struct Refused {
  int code;
  std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused{MLA_ERR_ARG, what}; }

enum Kind { kBf16 = MLA_OUT_BF16, kE4m3 = MLA_OUT_E4M3, kFp32 = MLA_OUT_FP32, kInt32, kInt64 };

// Element types that hold a kind (stored bits included).
bool holds(at::ScalarType t, int kind) {
  switch (kind) {
    case kBf16: return t == at::kBFloat16 || t == at::kShort || t == at::kUInt16;
    case kE4m3: return t == at::kFloat8_e4m3fn || t == at::kByte || t == at::kChar;
    case kFp32: return t == at::kFloat;
    case kInt32: return t == at::kInt;
    case kInt64: return t == at::kLong;
  }
  return false;
}

const at::Tensor& tensor(PyObject* o, const char* name, int dims, int kind) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a torch tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != dims) refuse(std::string(name) + " must be " + std::to_string(dims) + "-dimensional");
  if (!holds(t.scalar_type(), kind)) refuse(std::string(name) + " has the wrong element type");
  return t;
}

void on_this_gpu(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != c10::cuda::current_device()) refuse(std::string(name) + " is on another device than the current one");
}

void shaped(const at::Tensor& t, const char* name, int64_t rows, int64_t cols) {
  if (t.size(0) != rows || t.size(1) != cols)
    refuse(std::string(name) + " has shape (" + std::to_string(t.size(0)) + ", " + std::to_string(t.size(1)) +
           "), expected (" + std::to_string(rows) + ", " + std::to_string(cols) + ")");
}

// Row stride of a 2-D CUDA tensor with contiguous columns (one row: any serves).
int64_t row_stride(const at::Tensor& t, const char* name) {
  if (t.size(0) > 0 && t.size(1) > 1 && t.stride(1) != 1) refuse(std::string(name) + " must have contiguous columns");
  on_this_gpu(t, name);
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

void packed(const at::Tensor& t, const char* name) {
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  on_this_gpu(t, name);
}

int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::exception();
  if (v < INT32_MIN || v > INT32_MAX) refuse("an integer argument does not fit 32 bits");
  return (int)v;
}

int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + " must be < 2^31");
  return (int)v;
}

void* as_stream(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  void* s = PyLong_AsVoidPtr(o);
  if (!s && PyErr_Occurred()) throw std::exception();
  return s;
}

void check(int rc) {
  if (rc != MLA_OK) throw Refused{rc, mla_decode_last_error_string()};
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// Run `f`, turning what it throws into a Python exception.
template <class F>
PyObject* call(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    f();
    Py_RETURN_NONE;
  } catch (const Refused& r) {
    PyObject* e = g_error_type ? PyObject_CallFunction(g_error_type, "is", r.code, r.what.c_str()) : nullptr;
    if (e) {
      PyErr_SetObject(g_error_type, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_SetString(PyExc_RuntimeError, r.what.c_str());
    }
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

struct Scales {
  float* p = nullptr;
  int64_t stride = 0;
};

// fp32 [blocks, rows], or None
Scales block_scales(PyObject* o, const char* name, int64_t cols, int64_t rows, bool optional) {
  Scales s;
  if (optional && o == Py_None) return s;
  const at::Tensor& t = tensor(o, name, 2, kFp32);
  shaped(t, name, blocks(cols), rows);
  s.stride = row_stride(t, name);
  s.p = static_cast<float*>(t.data_ptr());
  return s;
}

// (x, residual, residual_out, residual_dtype, weight, eps, y, y_dtype, y_scales, stream)
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&] {
    const at::Tensor& x = tensor(a[0], "x", 2, kBf16);
    const int64_t t = x.size(0), d = x.size(1), xs = row_stride(x, "x");
    const int residual_dtype = as_int(a[3]), y_dtype = as_int(a[7]);
    void *rin = nullptr, *rout = nullptr;
    int64_t rs = 0;
    if (a[1] != Py_None || a[2] != Py_None) {
      if (a[1] == Py_None || a[2] == Py_None) refuse("residual and residual_out go together");
      const at::Tensor& r = tensor(a[1], "residual", 2, residual_dtype);
      const at::Tensor& ro = tensor(a[2], "residual_out", 2, residual_dtype);
      shaped(r, "residual", t, d);
      shaped(ro, "residual_out", t, d);
      rs = row_stride(r, "residual");
      if (row_stride(ro, "residual_out") != rs) refuse("residual and residual_out differ in their row stride");
      rin = r.data_ptr();
      rout = ro.data_ptr();
    }
    const at::Tensor& w = tensor(a[4], "weight", 1, kBf16);
    if (w.size(0) != d) refuse("weight must have as many elements as x has columns");
    packed(w, "weight");
    const double eps = PyFloat_AsDouble(a[5]);
    if (eps == -1.0 && PyErr_Occurred()) throw std::exception();
    const at::Tensor& y = tensor(a[6], "y", 2, y_dtype);
    shaped(y, "y", t, d);
    const int64_t ys = row_stride(y, "y");
    const Scales s = block_scales(a[8], "y_scales", d, t, true);
    check(mla_add_rmsnorm(x.data_ptr(), xs, rin, rout, residual_dtype, rs, w.data_ptr(), size32(t, "tokens"),
                          size32(d, "dim"), (float)eps, y.data_ptr(), y_dtype, ys, s.p, s.stride, as_stream(a[9])));
  });
}

// (x, act, y, y_dtype, y_scales, stream)
PyObject* act_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 6, [&] {
    const int act = as_int(a[1]), y_dtype = as_int(a[3]);
    const at::Tensor& y = tensor(a[2], "y", 2, y_dtype);
    const int64_t t = y.size(0), d = y.size(1);
    const at::Tensor& x = tensor(a[0], "x", 2, kBf16);
    shaped(x, "x", t, act == MLA_ACT_SILU_MUL ? 2 * d : d);
    const int64_t xs = row_stride(x, "x"), ys = row_stride(y, "y");
    const Scales s = block_scales(a[4], "y_scales", d, t, true);
    check(mla_act_quantize(x.data_ptr(), xs, act, size32(t, "tokens"), size32(d, "dim"), y.data_ptr(), y_dtype, ys, s.p,
                           s.stride, as_stream(a[5])));
  });
}

// (a, a_scales, w, w_scales, out, out_dtype, stream)
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 7, [&] {
    const at::Tensor& x = tensor(a[0], "a", 2, kE4m3);
    const at::Tensor& w = tensor(a[2], "w", 2, kE4m3);
    const int64_t t = x.size(0), k = x.size(1), rows = w.size(0);
    shaped(w, "w", rows, k);
    const int64_t lda = row_stride(x, "a"), ldw = row_stride(w, "w");
    const Scales s = block_scales(a[1], "a_scales", k, t, false);
    const at::Tensor& ws = tensor(a[3], "w_scales", 2, kFp32);
    shaped(ws, "w_scales", blocks(rows), blocks(k));
    packed(ws, "w_scales");
    const int out_dtype = as_int(a[5]);
    const at::Tensor& out = tensor(a[4], "out", 2, out_dtype);
    shaped(out, "out", t, rows);
    const int64_t ldo = row_stride(out, "out");
    check(mla_gemm_fp8(x.data_ptr(), lda, s.p, s.stride, w.data_ptr(), ldw, static_cast<float*>(ws.data_ptr()),
                       size32(t, "tokens"), size32(rows, "n"), size32(k, "k"), out.data_ptr(), out_dtype, ldo,
                       as_stream(a[6])));
  });
}

// (a, a_scales, w, w_scales, expert_offsets, out, out_dtype, stream)
PyObject* grouped_gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&] {
    const at::Tensor& x = tensor(a[0], "a", 2, kE4m3);
    const at::Tensor& w = tensor(a[2], "w", 3, kE4m3);
    const int64_t t = x.size(0), k = x.size(1), experts = w.size(0), rows = w.size(1);
    // every row of every expert `ldw` apart, the experts `rows` rows
    const int64_t ldw = rows > 1 ? w.stride(1) : experts > 1 ? w.stride(0) : k;
    if (w.size(2) != k || w.stride(2) != 1 || (experts > 1 && w.stride(0) != rows * ldw))
      refuse("w must be [experts, n, k] with contiguous columns and one row stride");
    on_this_gpu(w, "w");
    const int64_t lda = row_stride(x, "a");
    const Scales s = block_scales(a[1], "a_scales", k, t, false);
    const at::Tensor& ws = tensor(a[3], "w_scales", 3, kFp32);
    if (ws.size(0) != experts || ws.size(1) != blocks(rows) || ws.size(2) != blocks(k))
      refuse("w_scales must be [experts, ceil(n / 128), ceil(k / 128)]");
    packed(ws, "w_scales");
    const at::Tensor& off = tensor(a[4], "expert_offsets", 1, kInt32);
    if (off.size(0) != experts + 1) refuse("expert_offsets must have experts + 1 elements");
    packed(off, "expert_offsets");
    const int out_dtype = as_int(a[6]);
    const at::Tensor& out = tensor(a[5], "out", 2, out_dtype);
    shaped(out, "out", t, rows);
    const int64_t ldo = row_stride(out, "out");
    check(mla_grouped_gemm_fp8(x.data_ptr(), lda, s.p, s.stride, w.data_ptr(), ldw, static_cast<float*>(ws.data_ptr()),
                               static_cast<int32_t*>(off.data_ptr()), size32(experts, "experts"),
                               size32(t, "tokens"), size32(rows, "n"), size32(k, "k"), out.data_ptr(), out_dtype, ldo,
                               as_stream(a[7])));
  });
}

// ---- the prompt's operators

struct Heads {
  void* p = nullptr;
  int64_t token_stride = 0, head_stride = 0;
};

// bf16 [tokens, heads, cols] with contiguous columns; a dimension of one has any stride.
Heads heads(PyObject* o, const char* name, int64_t t, int64_t h, int64_t cols) {
  const at::Tensor& x = tensor(o, name, 3, kBf16);
  if (x.size(0) != t || x.size(1) != h || x.size(2) != cols)
    refuse(std::string(name) + " has shape (" + std::to_string(x.size(0)) + ", " + std::to_string(x.size(1)) + ", " +
           std::to_string(x.size(2)) + "), expected (" + std::to_string(t) + ", " + std::to_string(h) + ", " +
           std::to_string(cols) + ")");
  if (x.numel() > 0 && x.stride(2) != 1) refuse(std::string(name) + " must have contiguous columns");
  on_this_gpu(x, name);
  Heads r;
  r.p = x.data_ptr();
  r.head_stride = h > 1 ? x.stride(1) : cols;
  r.token_stride = t > 1 ? x.stride(0) : h * r.head_stride;
  return r;
}

// bf16 [tokens, cols], or None
Heads rows(PyObject* o, const char* name, int64_t t, int64_t cols) {
  const at::Tensor& x = tensor(o, name, 2, kBf16);
  shaped(x, name, t, cols);
  Heads r;
  r.token_stride = row_stride(x, name);
  r.p = x.data_ptr();
  return r;
}

float* packed_lse(PyObject* o, const char* name, int64_t t, int64_t h) {
  const at::Tensor& x = tensor(o, name, 2, kFp32);
  shaped(x, name, t, h);
  packed(x, name);
  return static_cast<float*>(x.data_ptr());
}

double as_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::exception();
  return v;
}

int64_t as_int64(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::exception();
  return v;
}

bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw std::exception();
  return v != 0;
}

// (table, first_position, base, scaling, factor, original_max_position, beta_fast, beta_slow, magnitude, stream)
PyObject* rope_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&] {
    const at::Tensor& t = tensor(a[0], "table", 2, kFp32);
    packed(t, "table");
    check(mla_rope_table(static_cast<float*>(t.data_ptr()), as_int64(a[1]), t.size(0), size32(t.size(1), "rotary_dim"),
                         as_double(a[2]), as_int(a[3]), as_double(a[4]), as_int64(a[5]), as_double(a[6]), as_double(a[7]),
                         as_double(a[8]), as_stream(a[9])));
  });
}

// (q, k, positions, cos_sin_cache, is_neox, q_out, k_out, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&] {
    const at::Tensor& pos = tensor(a[2], "positions", 1, kInt64);
    packed(pos, "positions");
    const at::Tensor& table = tensor(a[3], "cos_sin_cache", 2, kFp32);
    packed(table, "cos_sin_cache");
    const int64_t t = pos.size(0), r = table.size(1);
    int64_t h = 0;
    Heads q, qo, k, ko;
    if (a[0] != Py_None || a[5] != Py_None) {
      if (a[0] == Py_None || a[5] == Py_None) refuse("q and q_out go together");
      h = tensor(a[0], "q", 3, kBf16).size(1);
      if (h < 1) refuse("q has no head");
      q = heads(a[0], "q", t, h, r);
      qo = heads(a[5], "q_out", t, h, r);
    }
    if (a[1] != Py_None || a[6] != Py_None) {
      if (a[1] == Py_None || a[6] == Py_None) refuse("k and k_out go together");
      k = rows(a[1], "k", t, r);
      ko = rows(a[6], "k_out", t, r);
    }
    check(mla_rope(q.p, q.token_stride, q.head_stride, k.p, k.token_stride, size32(t, "tokens"), size32(h, "heads"),
                   size32(r, "rotary_dim"), static_cast<int64_t*>(pos.data_ptr()), static_cast<float*>(table.data_ptr()),
                   table.size(0), as_bool(a[4]), qo.p, qo.token_stride, qo.head_stride, ko.p, ko.token_stride,
                   as_stream(a[7])));
  });
}

// (kv_pages, kv_dtype, block_table, starts, cu_seqlens, k_scale, latent, latent_dtype, latent_scales, k_pe, stream)
PyObject* cache_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&] {
    const int kv_dtype = as_int(a[1]), latent_dtype = as_int(a[7]);
    const at::Tensor& kv = tensor(a[0], "kv_pages", 3, kv_dtype == MLA_KV_E4M3 ? kE4m3 : kBf16);
    if (kv.size(2) != MLA_KV_DIM) refuse("kv_pages must be [pages, page_size, 576]");
    packed(kv, "kv_pages");
    const at::Tensor& table = tensor(a[2], "block_table", 2, kInt32);
    const int64_t batch = table.size(0);
    packed(table, "block_table");
    int32_t* starts = nullptr;
    if (a[3] != Py_None) {
      const at::Tensor& s = tensor(a[3], "starts", 1, kInt32);
      if (s.size(0) != batch) refuse("starts must have one element a request");
      packed(s, "starts");
      starts = static_cast<int32_t*>(s.data_ptr());
    }
    const at::Tensor& cu = tensor(a[4], "cu_seqlens", 1, kInt32);
    if (cu.size(0) != batch + 1) refuse("cu_seqlens must have batch + 1 elements");
    packed(cu, "cu_seqlens");
    const at::Tensor& latent = tensor(a[6], "latent", 2, latent_dtype);
    const int64_t t = latent.size(0);
    shaped(latent, "latent", t, MLA_KV_LORA_RANK);
    const int64_t ls = row_stride(latent, "latent");
    const Scales s = block_scales(a[8], "latent_scales", MLA_KV_LORA_RANK, t, latent_dtype != MLA_OUT_E4M3);
    const Heads pe = rows(a[9], "k_pe", t, MLA_ROPE_DIM);
    check(mla_cache_gather(kv.data_ptr(), kv_dtype, kv.size(0), size32(kv.size(1), "page_size"),
                           static_cast<int32_t*>(table.data_ptr()), table.size(1), starts,
                           static_cast<int32_t*>(cu.data_ptr()), size32(batch, "batch"), size32(t, "tokens"),
                           (float)as_double(a[5]), latent.data_ptr(), latent_dtype, ls, s.p, s.stride, pe.p,
                           pe.token_stride, as_stream(a[10])));
  });
}

// (q_nope, q_pe, k_nope, k_pe, v, cu_seqlens_q, cu_seqlens_k, causal, scale, out, lse, workspace, stream)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 13, [&] {
    const at::Tensor& q0 = tensor(a[0], "q_nope", 3, kBf16);
    const at::Tensor& k0 = tensor(a[2], "k_nope", 3, kBf16);
    const int64_t tq = q0.size(0), tk = k0.size(0), h = q0.size(1);
    const Heads q = heads(a[0], "q_nope", tq, h, MLA_NOPE_DIM), qp = heads(a[1], "q_pe", tq, h, MLA_ROPE_DIM),
                k = heads(a[2], "k_nope", tk, h, MLA_NOPE_DIM), kp = rows(a[3], "k_pe", tk, MLA_ROPE_DIM),
                v = heads(a[4], "v", tk, h, MLA_V_DIM), out = heads(a[9], "out", tq, h, MLA_V_DIM);
    const at::Tensor& cu_q = tensor(a[5], "cu_seqlens_q", 1, kInt32);
    const at::Tensor& cu_k = tensor(a[6], "cu_seqlens_k", 1, kInt32);
    packed(cu_q, "cu_seqlens_q");
    packed(cu_k, "cu_seqlens_k");
    if (cu_q.size(0) < 2 || cu_k.size(0) != cu_q.size(0)) refuse("cu_seqlens_q and cu_seqlens_k must have batch + 1 elements");
    float* lse = packed_lse(a[10], "lse", tq, h);
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[11] != Py_None) {
      if (!THPVariable_Check(a[11])) refuse("workspace must be a torch tensor");
      const at::Tensor& w = THPVariable_Unpack(a[11]);
      packed(w, "workspace");
      ws = w.data_ptr();
      ws_bytes = w.nbytes();
    }
    check(mla_prefill(q.p, q.token_stride, q.head_stride, qp.p, qp.token_stride, qp.head_stride, k.p, k.token_stride,
                      k.head_stride, kp.p, kp.token_stride, v.p, v.token_stride, v.head_stride,
                      static_cast<int32_t*>(cu_q.data_ptr()), static_cast<int32_t*>(cu_k.data_ptr()),
                      size32(cu_q.size(0) - 1, "batch"), size32(tq, "query tokens"), size32(tk, "key tokens"),
                      size32(h, "heads"), as_bool(a[7]), (float)as_double(a[8]), out.p, out.token_stride, out.head_stride,
                      lse, ws, ws_bytes, as_stream(a[12])));
  });
}

// (out_a, lse_a, out_b, lse_b, out, lse, stream)
PyObject* merge_states(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 7, [&] {
    const at::Tensor& x = tensor(a[0], "out_a", 3, kBf16);
    const int64_t t = x.size(0), h = x.size(1), d = x.size(2);
    const Heads xa = heads(a[0], "out_a", t, h, d), xb = heads(a[2], "out_b", t, h, d), o = heads(a[4], "out", t, h, d);
    const float *la = packed_lse(a[1], "lse_a", t, h), *lb = packed_lse(a[3], "lse_b", t, h);
    float* l = packed_lse(a[5], "lse", t, h);
    check(mla_merge_states(xa.p, xa.token_stride, xa.head_stride, la, xb.p, xb.token_stride, xb.head_stride, lb,
                           size32(t, "tokens"), size32(h, "heads"), size32(d, "dim"), o.p, o.token_stride, o.head_stride,
                           l, as_stream(a[6])));
  });
}

PyObject* set_error_type(PyObject*, PyObject* type) {
  Py_XINCREF(type);
  Py_XSETREF(g_error_type, type);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef fast(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {fast<add_rmsnorm>("add_rmsnorm"),
                         fast<act_quantize>("act_quantize"),
                         fast<gemm_fp8>("gemm_fp8"),
                         fast<grouped_gemm_fp8>("grouped_gemm_fp8"),
                         fast<rope_table>("rope_table"),
                         fast<rope>("rope"),
                         fast<cache_gather>("cache_gather"),
                         fast<prefill>("prefill"),
                         fast<merge_states>("merge_states"),
                         {"set_error_type", set_error_type, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mla_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_calls() { return PyModule_Create(&module); }
