// Argument marshalling of the per-layer entry points for Python callers:
// quantize, gemm, gemm_grouped, qk_norm_rope, gemm_gated, layer_norm and the two
// backward passes on torch tensors.
//
// A decode step makes one such call per layer, and there the time of the call
// on the host is what counts: quantize, gemm, gemm_grouped and qk_norm_rope of
// one token take 6.3, 5.0, 4.9 and 5.5 us of it, through ctypes 9.1, 7.4, 7.3
// and 11.1 (of either the launch is 2.6).  This module reads the tensors and
// allocates the output in C++ and calls the C ABI (through the addresses that
// the ctypes binding resolved; it links nothing of libmxq).  It holds no
// arithmetic.  It refuses (ValueError) what the C ABI cannot see: tensors in
// host memory, of another type, or smaller than the call reads or writes; the
// rest is refused by the library.  A failing call returns the status as an int.
#include <Python.h>

#include <algorithm>
#include <initializer_list>

#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>

#include "mxq.h"

namespace {

decltype(&mxq_quantize) g_quantize;
decltype(&mxq_gemm) g_gemm;
decltype(&mxq_gemm_grouped) g_grouped;
decltype(&mxq_qk_norm_rope) g_qk;
decltype(&mxq_gemm_gated) g_gated;
decltype(&mxq_gemm_gated_backward) g_gated_bwd;
decltype(&mxq_layer_norm) g_norm;
decltype(&mxq_layer_norm_backward) g_norm_bwd;
decltype(&mxq_workspace_size) g_ws_size;

PyObject *s_fmt, *s_rows, *s_cols, *s_codes, *s_scales, *s_tensor_scale;

bool fail(const char* what) {
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, what);
  return false;
}

bool to_i64(PyObject* o, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  return !(*v == -1 && PyErr_Occurred());
}

// None leaves *t null.  The argument keeps the tensor alive.
bool to_tensor(PyObject* o, const at::Tensor** t, const char* what) {
  *t = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return fail(what);
  *t = &THPVariable_Unpack(o);
  return (*t)->is_cuda() || fail("tensors are in device memory");
}

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// Rows of a 2-D tensor are ld elements apart; with a single row any stride is that row's.
int64_t ld(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1)); }

bool row_major(const at::Tensor& t) { return t.dim() == 2 && (t.stride(1) == 1 || t.size(1) <= 1); }

// bf16 values, or their bits under an integer type
bool bf16_bits(const at::Tensor& t) {
  const auto ty = t.scalar_type();
  return ty == at::kBFloat16 || ty == at::kShort || ty == at::kUInt16;
}

bool one_float(const at::Tensor* t, const char* what) {
  return !t || (t->scalar_type() == at::kFloat && t->numel() >= 1) || fail(what);
}

// Attribute `name` of a quantized operand, undefined for None.
bool part(PyObject* q, PyObject* name, at::Tensor* t) {
  PyObject* o = PyObject_GetAttr(q, name);
  if (!o) return false;
  const at::Tensor* p;
  const bool ok = to_tensor(o, &p, "an operand's codes and scales are tensors");
  if (ok && p) *t = *p;
  Py_DECREF(o);
  return ok;
}

bool number(PyObject* q, PyObject* name, int64_t* v) {
  PyObject* o = PyObject_GetAttr(q, name);
  if (!o) return false;
  const bool ok = to_i64(o, v);
  Py_DECREF(o);
  return ok;
}

constexpr int64_t kMaxCols = int64_t(1) << 40;   // more than any tensor has: no overflow in what follows

// A quantized operand, with the tensors it reads held for the call.
struct Operand : mxq_qtensor {
  at::Tensor t_codes, t_scales, t_tensor_scale;

  bool read(PyObject* q) {
    int64_t f;
    if (!number(q, s_fmt, &f) || !number(q, s_rows, &rows) || !number(q, s_cols, &cols) ||
        !part(q, s_codes, &t_codes) || !part(q, s_scales, &t_scales) || !part(q, s_tensor_scale, &t_tensor_scale))
      return false;
    fmt = (int32_t)f;
    reserved = 0;
    if (t_tensor_scale.defined() && !one_float(&t_tensor_scale, "an operand's tensor_scale is a float32 tensor")) return false;
    tensor_scale = static_cast<float*>(t_tensor_scale.defined() ? t_tensor_scale.data_ptr() : nullptr);
    return side(t_codes, rows, code_bytes(), code_type(), &codes, &ld_codes) &&
           side(t_scales, scale_rows(), scale_bytes(), scale_type(), &scales, &ld_scales);
  }

 private:
  // Bytes of a row's codes and scales; formats that the library does not know
  // have none, and are refused there.
  int64_t code_bytes() const {
    const int64_t k = std::min(cols, kMaxCols);
    switch (fmt) {
      case MXQ_FMT_BF16: return 2 * k;
      case MXQ_FMT_MXFP8: case MXQ_FMT_INT8: case MXQ_FMT_FP8: case MXQ_FMT_FP8_TILE: return k;
      case MXQ_FMT_MXFP4: case MXQ_FMT_NVFP4: case MXQ_FMT_INT4: return k / 2;
      default: return 0;
    }
  }
  int64_t scale_bytes() const {
    const int64_t k = std::min(cols, kMaxCols);
    switch (fmt) {
      case MXQ_FMT_INT8: return 4;
      case MXQ_FMT_FP8: return 4 * std::min(rows, kMaxCols);
      case MXQ_FMT_FP8_TILE: return (k + 127) / 128 * 4;
      case MXQ_FMT_INT4: return k / 32 * 4;
      case MXQ_FMT_NVFP4: return k / 16;
      case MXQ_FMT_MXFP4: case MXQ_FMT_MXFP8: return k / 32;
      default: return 0;
    }
  }

  // Rows of the scales: one per row, K-block (FP8) or 128 rows (FP8_TILE).
  int64_t scale_rows() const {
    return fmt == MXQ_FMT_FP8 ? (std::min(cols, kMaxCols) + 127) / 128 : fmt == MXQ_FMT_FP8_TILE ? rows / 128 + (rows % 128 > 0) : rows;
  }

  // Codes and the scale codes of the block formats are bytes under any type but
  // the wider floating ones, whose values would be taken for them; bf16
  // operands, integers and fp32 scales are what they say.
  enum Type { kBytes, kBits16, kInt8, kFloat32 };
  Type code_type() const { return fmt == MXQ_FMT_BF16 ? kBits16 : fmt == MXQ_FMT_INT8 ? kInt8 : kBytes; }
  Type scale_type() const {
    return fmt == MXQ_FMT_INT8 || fmt == MXQ_FMT_INT4 || fmt == MXQ_FMT_FP8 || fmt == MXQ_FMT_FP8_TILE ? kFloat32 : kBytes;
  }
  static bool is(const at::Tensor& t, Type ty) {
    const auto s = t.scalar_type();
    switch (ty) {
      case kBits16: return bf16_bits(t);
      case kInt8: return s == at::kChar || s == at::kByte;
      case kFloat32: return s == at::kFloat;
      default: return !(at::isFloatingType(s) && t.element_size() > 1) && !at::isComplexType(s);
    }
  }

  bool side(const at::Tensor& t, int64_t n, int64_t need, Type type, void** p, int64_t* bytes) {
    *p = nullptr;
    *bytes = 0;
    if (!t.defined()) return true;
    if (t.dim() < 1 || t.size(0) < n) return fail("an operand's codes and scales have its rows");
    *p = t.data_ptr();
    *bytes = t.stride(0) * (int64_t)t.element_size();
    if (rows <= 0 || cols <= 0) return true;
    if (!is(t, type)) return fail("an operand's codes and scales have its format's types");
    int64_t row = (int64_t)t.element_size();   // bytes of a row, which lie together
    for (int64_t d = t.dim() - 1; d > 0; --d) {
      if (t.size(d) != 1 && t.stride(d) * (int64_t)t.element_size() != row)
        return fail("the rows of an operand's codes and scales are contiguous");
      row *= t.size(d);
    }
    // a single row may have any stride: it is given one that the library takes
    if (n == 1) *bytes = (row + 15) / 16 * 16;
    return row >= need || fail("an operand's codes and scales are as wide as its columns");
  }
};

at::Tensor bf16_like(const at::Tensor& t, at::IntArrayRef sizes) {
  return at::empty(sizes, t.options().dtype(at::kBFloat16).requires_grad(false));
}

// [rows, cols], rows any stride apart; bf16, or a 16-bit type that its bits are put into
bool output(const at::Tensor& t, int64_t rows, int64_t cols) {
  return (t.element_size() == 2 && row_major(t) && t.size(0) >= rows && t.size(1) >= cols) ||
         fail("out is a row-major tensor of the product's size, bfloat16 or its bits");
}

bool bias_of(const at::Tensor* t, int64_t n) {
  return !t || (bf16_bits(*t) && t->is_contiguous() && t->numel() >= n) ||
         fail("bias is a contiguous bfloat16 tensor, one element per output column");
}

// u of the low-rank branch: fp32 [rows, rank], rows any stride apart
bool lowrank_u(const at::Tensor* u, int64_t rows, int64_t rank) {
  return !u || (u->scalar_type() == at::kFloat && row_major(*u) && u->size(0) >= rows && u->size(1) >= rank) ||
         fail("u is a row-major float32 tensor [rows, rank]");
}

template <class F>
PyObject* guarded(F f) {   // no C++ exception crosses into Python
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  return n == want || fail("wrong number of arguments");
}

// quantize(x, dtype, hadamard, static_tensor_scale, l1t, u, out, ws, ws_bytes, stream)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x, *g, *l1t, *u, *ws;
    Operand q;
    int64_t dt, had, wsn, stream;
    if (!count(n, 10) || !to_tensor(a[0], &x, "x is a tensor") || !to_i64(a[1], &dt) || !to_i64(a[2], &had) ||
        !to_tensor(a[3], &g, "static_tensor_scale is a tensor") || !to_tensor(a[4], &l1t, "l1t is a tensor") ||
        !to_tensor(a[5], &u, "u is a tensor") || !q.read(a[6]) ||
        !to_tensor(a[7], &ws, "workspace is a tensor") || !to_i64(a[8], &wsn) || !to_i64(a[9], &stream))
      return nullptr;
    if (!x || !row_major(*x) || x->scalar_type() != (dt == MXQ_DT_BF16 ? at::kBFloat16 : at::kFloat)) {
      fail("quantize needs a row-major 2-D float32 or bfloat16 tensor");
      return nullptr;
    }
    if (l1t && (!bf16_bits(*l1t) || l1t->dim() != 2 || l1t->size(1) != x->size(1) || !l1t->is_contiguous())) {
      fail("l1t is a contiguous bfloat16 tensor [rank, cols]");
      return nullptr;
    }
    if ((l1t && !lowrank_u(u, x->size(0), l1t->size(0))) || !one_float(g, "static_tensor_scale is a float32 tensor"))
      return nullptr;
    mxq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_quantize(x->data_ptr(), (int32_t)dt, x->size(0), x->size(1), ld(*x), (int32_t)had,
                    static_cast<const float*>(ptr(g)), ptr(l1t), l1t ? (int32_t)l1t->size(0) : 0,
                    static_cast<float*>(ptr(u)), u && l1t ? ld(*u) : 0, &q, ptr(ws), (size_t)wsn,
                    reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
  });
}

// empty_rows(x, fmt) -> (codes uint8 [rows, cols], scales float32) for a quantized x:
// int8 [rows, 1], FP8 [cols / 128, rows], FP8_TILE [rows / 128, cols / 128]
PyObject* empty_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* x;
    int64_t fmt;
    if (!count(n, 2) || !to_tensor(a[0], &x, "x is a tensor") || !to_i64(a[1], &fmt)) return nullptr;
    if (!x || x->dim() != 2) {
      fail("quantize needs a 2-D tensor");
      return nullptr;
    }
    const auto opt = x->options().requires_grad(false);
    const int64_t rows = x->size(0), blocks = (x->size(1) + 127) / 128;
    const int64_t shape[2] = {fmt == MXQ_FMT_FP8 ? blocks : fmt == MXQ_FMT_FP8_TILE ? (rows + 127) / 128 : rows,
                              fmt == MXQ_FMT_FP8 ? rows : fmt == MXQ_FMT_FP8_TILE ? blocks : 1};
    PyObject* c = THPVariable_Wrap(at::empty(x->sizes(), opt.dtype(at::kByte).memory_format(at::MemoryFormat::Contiguous)));
    PyObject* s = THPVariable_Wrap(at::empty(at::IntArrayRef(shape, 2), opt.dtype(at::kFloat)));
    PyObject* r = c && s ? PyTuple_Pack(2, c, s) : nullptr;
    Py_XDECREF(c);
    Py_XDECREF(s);
    return r;
  });
}

// gemm(a, w, n_out, w_out_col, u, l2t, bias, out, ws, ws_bytes, stream) -> out or status
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Operand qa, qw;
    const at::Tensor *map, *u, *l2t, *bias, *out, *ws;
    int64_t n_out, wsn, stream;
    if (!count(n, 11) || !qa.read(a[0]) || !qw.read(a[1]) || !to_i64(a[2], &n_out) ||
        !to_tensor(a[3], &map, "w_out_col is a tensor") || !to_tensor(a[4], &u, "u is a tensor") ||
        !to_tensor(a[5], &l2t, "l2t is a tensor") || !to_tensor(a[6], &bias, "bias is a tensor") ||
        !to_tensor(a[7], &out, "out is a tensor") || !to_tensor(a[8], &ws, "workspace is a tensor") ||
        !to_i64(a[9], &wsn) || !to_i64(a[10], &stream))
      return nullptr;
    if (!qa.t_codes.defined() || n_out < 0) {
      fail("gemm needs the operand's codes");
      return nullptr;
    }
    if (map && (map->scalar_type() != at::kInt || !map->is_contiguous() || map->numel() < qw.rows)) {
      fail("w_out_col is a contiguous int32 tensor, one element per weight row");
      return nullptr;
    }
    if (l2t && (!bf16_bits(*l2t) || l2t->dim() != 2 || l2t->size(0) < n_out || !l2t->is_contiguous())) {
      fail("l2t is a contiguous bfloat16 tensor [n_out, rank]");
      return nullptr;
    }
    if (l2t && !lowrank_u(u, qa.rows, l2t->size(1))) return nullptr;
    if (!bias_of(bias, n_out) || (out && !output(*out, qa.rows, n_out))) return nullptr;
    at::Tensor made;
    if (!out) {
      made = bf16_like(qa.t_codes, {qa.rows, n_out});
      out = &made;
    }
    mxq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_gemm(&qa, &qw, static_cast<const int32_t*>(ptr(map)), static_cast<const float*>(ptr(u)),
                u && l2t ? ld(*u) : 0, ptr(l2t), l2t ? (int32_t)l2t->size(1) : 0, ptr(bias), out->data_ptr(),
                ld(*out), n_out, ptr(ws), (size_t)wsn, reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (st != MXQ_OK) return PyLong_FromLong(st);
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[7]);
    return a[7];
  });
}

// gemm_grouped(a, w, offsets, bias, out, stream) -> out or status
PyObject* gemm_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Operand qa, qw;
    const at::Tensor *off, *bias, *out;
    int64_t stream;
    if (!count(n, 6) || !qa.read(a[0]) || !qw.read(a[1]) ||
        !to_tensor(a[2], &off, "offsets is a tensor") || !to_tensor(a[3], &bias, "bias is a tensor") ||
        !to_tensor(a[4], &out, "out is a tensor") || !to_i64(a[5], &stream))
      return nullptr;
    if (!qa.t_codes.defined() || !off || off->scalar_type() != at::kInt || off->dim() != 1 || !off->is_contiguous()) {
      fail("gemm_grouped needs the operand's codes and contiguous 1-D int32 offsets");
      return nullptr;
    }
    const int64_t groups = off->size(0) - 1;
    const int64_t n_out = groups > 0 ? qw.rows / groups : 0;
    if (!bias_of(bias, groups * n_out) || (out && !output(*out, qa.rows, n_out))) return nullptr;
    at::Tensor made;
    if (!out) {
      made = bf16_like(qa.t_codes, {qa.rows, n_out});
      out = &made;
    }
    mxq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_grouped(&qa, &qw, (int32_t)std::min<int64_t>(groups, INT32_MAX), static_cast<const int32_t*>(ptr(off)),
                   ptr(bias), out->data_ptr(), ld(*out), reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (st != MXQ_OK) return PyLong_FromLong(st);
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[4]);
    return a[4];
  });
}

// qk_norm_rope(x, n_q, n_k, head_dim, q_weight, k_weight, cos, sin, positions, eps, interleaved, q_out,
// k_out, stream) -> (q, k) or status
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x, *wq, *wk, *cos, *sin, *pos, *q, *k;
    int64_t nq, nk, d, inter, stream;
    if (!count(n, 14) || !to_tensor(a[0], &x, "x is a tensor") || !to_i64(a[1], &nq) || !to_i64(a[2], &nk) ||
        !to_i64(a[3], &d) || !to_tensor(a[4], &wq, "q_weight is a tensor") ||
        !to_tensor(a[5], &wk, "k_weight is a tensor") || !to_tensor(a[6], &cos, "cos is a tensor") ||
        !to_tensor(a[7], &sin, "sin is a tensor") || !to_tensor(a[8], &pos, "positions is a tensor") ||
        !to_i64(a[10], &inter) || !to_tensor(a[11], &q, "q_out is a tensor") ||
        !to_tensor(a[12], &k, "k_out is a tensor") || !to_i64(a[13], &stream))
      return nullptr;
    const double eps = PyFloat_AsDouble(a[9]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    auto refuse = [](const char* what) -> PyObject* {
      fail(what);
      return nullptr;
    };
    const auto dt = x ? x->scalar_type() : at::kHalf;
    if ((dt != at::kBFloat16 && dt != at::kFloat) || !row_major(*x))
      return refuse("qk_norm_rope needs a row-major 2-D float32 or bfloat16 tensor");
    const int64_t tokens = x->size(0);
    if (nq < 0 || nk < 0 || d < 1 || d > 512 || nq > (1 << 20) || nk > (1 << 20) || x->size(1) < (nq + nk) * d)
      return refuse("qk_norm_rope: x is narrower than its heads");
    for (const at::Tensor* g : {wq, wk})
      if (g && (g->scalar_type() != dt || g->dim() != 1 || g->size(0) != d || g->stride(0) != 1))
        return refuse("qk_norm_rope: weights are contiguous [head_dim] tensors of x's dtype");
    int64_t n_pos = 0, rot = 0;
    if (cos) {
      if (!sin || cos->scalar_type() != at::kFloat || sin->scalar_type() != at::kFloat || cos->dim() != 2 ||
          sin->sizes() != cos->sizes() || !cos->is_contiguous() || !sin->is_contiguous())
        return refuse("qk_norm_rope: cos and sin are contiguous float32 [n_pos, rot / 2]");
      n_pos = cos->size(0);
      rot = 2 * cos->size(1);
      if (pos && (pos->scalar_type() != at::kInt || pos->dim() != 1 || pos->size(0) != tokens || !pos->is_contiguous()))
        return refuse("qk_norm_rope: positions are contiguous int32 [tokens]");
    }
    at::Tensor mq, mk;
    const auto opt = x->options().requires_grad(false);
    if (!q) {
      mq = at::empty({tokens, nq, d}, opt);
      q = &mq;
    }
    if (!k) {
      mk = at::empty({tokens, nk, d}, opt);
      k = &mk;
    }
    for (const auto& [t, heads] : {std::pair{q, nq}, std::pair{k, nk}})
      if (t->scalar_type() != dt || t->dim() != 3 || t->size(0) != tokens || t->size(1) != heads || t->size(2) != d ||
          t->stride(2) != 1)
        return refuse("qk_norm_rope: outputs are [tokens, heads, head_dim] of x's dtype");
    mxq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_qk(x->data_ptr(), dt == at::kBFloat16 ? MXQ_DT_BF16 : MXQ_DT_F32, tokens, ld(*x), (int32_t)nq,
              (int32_t)nk, (int32_t)d, ptr(wq), ptr(wk), (float)eps, static_cast<const float*>(ptr(cos)),
              static_cast<const float*>(cos ? ptr(sin) : nullptr), n_pos, (int32_t)rot, inter != 0,
              static_cast<const int32_t*>(cos ? ptr(pos) : nullptr), q->data_ptr(), q->stride(0), q->stride(1),
              k->data_ptr(), k->stride(0), k->stride(1), reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (st != MXQ_OK) return PyLong_FromLong(st);
    PyObject* oq = mq.defined() ? THPVariable_Wrap(std::move(mq)) : (Py_INCREF(a[11]), a[11]);
    PyObject* ok = mk.defined() ? THPVariable_Wrap(std::move(mk)) : (Py_INCREF(a[12]), a[12]);
    PyObject* r = oq && ok ? PyTuple_Pack(2, oq, ok) : nullptr;
    Py_XDECREF(oq);
    Py_XDECREF(ok);
    return r;
  });
}

// Whether all of them (null and undefined ones aside) are on device `dev`, whose stream the call uses.
bool on_device(int64_t dev, std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts)
    if (t && t->defined() && t->get_device() != dev) return fail("tensors are on the device of the call's stream");
  return true;
}

PyObject* give(at::Tensor& made, PyObject* given) {
  if (made.defined()) return THPVariable_Wrap(std::move(made));
  Py_INCREF(given);
  return given;
}

PyObject* pack3(PyObject* a, PyObject* b, PyObject* c) {
  PyObject* r = a && b && c ? PyTuple_Pack(3, a, b, c) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  Py_XDECREF(c);
  return r;
}

// gemm_gated(x, w_gate, w_up, act, saved, out, device, stream) -> out or status
PyObject* gemm_gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Operand x, g, u;
    const at::Tensor *saved, *out;
    int64_t act, dev, stream;
    if (!count(n, 8) || !x.read(a[0]) || !g.read(a[1]) || !u.read(a[2]) || !to_i64(a[3], &act) ||
        !to_tensor(a[4], &saved, "saved is a tensor") || !to_tensor(a[5], &out, "out is a tensor") ||
        !to_i64(a[6], &dev) || !to_i64(a[7], &stream))
      return nullptr;
    if (!x.t_codes.defined()) {
      fail("gemm_gated needs the operand's codes");
      return nullptr;
    }
    if (saved && (saved->scalar_type() != at::kFloat || !saved->is_contiguous() || saved->dim() != 3 ||
                  saved->size(0) != 2 || saved->size(1) != x.rows || saved->size(2) != g.rows)) {
      fail("saved is a contiguous float32 tensor [2, rows, outputs]");
      return nullptr;
    }
    if ((out && !output(*out, x.rows, g.rows)) ||
        !on_device(dev, {&x.t_codes, &x.t_scales, &g.t_codes, &g.t_scales, &u.t_codes, &u.t_scales, saved, out}))
      return nullptr;
    at::Tensor made;
    if (!out) {
      made = bf16_like(x.t_codes, {x.rows, g.rows});
      out = &made;
    }
    mxq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_gated(&x, &g, &u, (int32_t)act, static_cast<float*>(ptr(saved)), out->data_ptr(), ld(*out),
                 reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (st != MXQ_OK) return PyLong_FromLong(st);
    return give(made, a[5]);
  });
}

// gemm_gated_backward(dy, x, w_gate, w_up, act, saved, want_dx, want_dw, dx, dw_gate, dw_up, ws, device, stream)
// -> (dx, dw_gate, dw_up), None for those not wanted, or status
PyObject* gemm_gated_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Operand x, g, u;
    const at::Tensor *dy, *saved, *dx, *dg, *du, *ws;
    int64_t act, want_dx, want_dw, dev, stream;
    if (!count(n, 14) || !to_tensor(a[0], &dy, "dy is a tensor") || !x.read(a[1]) || !g.read(a[2]) || !u.read(a[3]) ||
        !to_i64(a[4], &act) || !to_tensor(a[5], &saved, "saved is a tensor") || !to_i64(a[6], &want_dx) ||
        !to_i64(a[7], &want_dw) || !to_tensor(a[8], &dx, "dx is a tensor") || !to_tensor(a[9], &dg, "dw_gate is a tensor") ||
        !to_tensor(a[10], &du, "dw_up is a tensor") || !to_tensor(a[11], &ws, "workspace is a tensor") ||
        !to_i64(a[12], &dev) || !to_i64(a[13], &stream))
      return nullptr;
    auto refuse = [](const char* what) -> PyObject* {
      fail(what);
      return nullptr;
    };
    const int64_t rows = x.rows, outs = g.rows, k = x.cols;
    if (!x.t_codes.defined() || !dy || dy->scalar_type() != at::kBFloat16 || !row_major(*dy) || dy->size(0) != rows ||
        dy->size(1) != outs)
      return refuse("gemm_gated_backward: dy is a row-major bfloat16 tensor [rows, outputs]");
    if (!saved || saved->scalar_type() != at::kFloat || !saved->is_contiguous() || saved->dim() != 3 ||
        saved->size(0) != 2 || saved->size(1) != rows || saved->size(2) != outs)
      return refuse("saved is a contiguous float32 tensor [2, rows, outputs]");
    at::Tensor mx, mg, mu, mw;
    auto gradient = [&](const at::Tensor*& t, at::Tensor& made, int64_t want, int64_t r) {
      if (!want) {
        t = nullptr;
      } else if (!t) {
        made = bf16_like(x.t_codes, {r, k});
        t = &made;
      } else if (!output(*t, r, k)) {
        return false;
      }
      return true;
    };
    if (!gradient(dx, mx, want_dx, rows) || !gradient(dg, mg, want_dw, outs) || !gradient(du, mu, want_dw, outs)) return nullptr;
    if (dg && outs > 1 && ld(*dg) != ld(*du)) return refuse("dw_gate and dw_up have one row stride");
    const int64_t need = g_ws_size(MXQ_OP_GATED_BACKWARD, rows, outs, (int32_t)std::min<int64_t>(k, INT32_MAX));
    if (!ws && need > 0) {
      mw = at::empty({need}, x.t_codes.options().dtype(at::kByte).requires_grad(false));
      ws = &mw;
    }
    if (ws && !ws->is_contiguous()) return refuse("the workspace is a contiguous tensor");
    if (!on_device(dev, {dy, &x.t_codes, &g.t_codes, &u.t_codes, saved, dx, dg, du, ws})) return nullptr;
    mxq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_gated_bwd(dy->data_ptr(), ld(*dy), &x, &g, &u, (int32_t)act, static_cast<const float*>(ptr(saved)), ptr(dx),
                     dx ? ld(*dx) : 0, ptr(dg), ptr(du), dg ? ld(*dg) : 0, ptr(ws), ws ? ws->nbytes() : 0,
                     reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (st != MXQ_OK) return PyLong_FromLong(st);
    return pack3(give(mx, want_dx ? a[8] : Py_None), give(mg, want_dw ? a[9] : Py_None), give(mu, want_dw ? a[10] : Py_None));
  });
}

bool norm_param(const at::Tensor* t, const at::Tensor& x, const char* what) {
  return !t || (t->scalar_type() == x.scalar_type() && t->dim() == 1 && t->size(0) == x.size(1) && t->is_contiguous()) ||
         fail(what);
}

bool norm_rows(const at::Tensor* t, const at::Tensor& x, const char* what) {
  return !t || (t->scalar_type() == x.scalar_type() && row_major(*t) && t->sizes() == x.sizes()) || fail(what);
}

bool norm_input(const at::Tensor* x) {
  return (x && (x->scalar_type() == at::kBFloat16 || x->scalar_type() == at::kFloat) && row_major(*x)) ||
         fail("layer_norm needs a row-major 2-D float32 or bfloat16 tensor");
}

bool norm_stats(const at::Tensor* t, const at::Tensor& x) {
  return !t || (t->scalar_type() == at::kFloat && t->is_contiguous() && t->dim() == 2 && t->size(0) == x.size(0) &&
                t->size(1) == 2) || fail("stats is a contiguous float32 tensor [rows, 2]");
}

// layer_norm(x, weight, bias, eps, stats, out, device, stream) -> out or status
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x, *w, *b, *stats, *out;
    int64_t dev, stream;
    if (!count(n, 8) || !to_tensor(a[0], &x, "x is a tensor") || !to_tensor(a[1], &w, "weight is a tensor") ||
        !to_tensor(a[2], &b, "bias is a tensor") || !to_tensor(a[4], &stats, "stats is a tensor") ||
        !to_tensor(a[5], &out, "out is a tensor") || !to_i64(a[6], &dev) || !to_i64(a[7], &stream))
      return nullptr;
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    if (!norm_input(x) || !norm_param(w, *x, "weight is a contiguous [cols] tensor of x's dtype") ||
        !norm_param(b, *x, "bias is a contiguous [cols] tensor of x's dtype") || !norm_stats(stats, *x) ||
        !norm_rows(out, *x, "out is a row-major tensor of x's dtype and size") || !on_device(dev, {x, w, b, stats, out}))
      return nullptr;
    at::Tensor made;
    if (!out) {
      made = at::empty(x->sizes(), x->options().requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
      out = &made;
    }
    mxq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_norm(x->data_ptr(), x->scalar_type() == at::kFloat ? MXQ_DT_F32 : MXQ_DT_BF16, x->size(0), x->size(1), ld(*x),
                ptr(w), ptr(b), (float)eps, out->data_ptr(), ld(*out), static_cast<float*>(ptr(stats)),
                reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (st != MXQ_OK) return PyLong_FromLong(st);
    return give(made, a[5]);
  });
}

// layer_norm_backward(dy, x, stats, weight, want_dx, want_params, dx, dweight, dbias, ws, device, stream)
// -> (dx, dweight, dbias), None for those not wanted, or status
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *dy, *x, *stats, *w, *dx, *dw, *db, *ws;
    int64_t want_dx, want_p, dev, stream;
    if (!count(n, 12) || !to_tensor(a[0], &dy, "dy is a tensor") || !to_tensor(a[1], &x, "x is a tensor") ||
        !to_tensor(a[2], &stats, "stats is a tensor") || !to_tensor(a[3], &w, "weight is a tensor") ||
        !to_i64(a[4], &want_dx) || !to_i64(a[5], &want_p) || !to_tensor(a[6], &dx, "dx is a tensor") ||
        !to_tensor(a[7], &dw, "dweight is a tensor") || !to_tensor(a[8], &db, "dbias is a tensor") ||
        !to_tensor(a[9], &ws, "workspace is a tensor") || !to_i64(a[10], &dev) || !to_i64(a[11], &stream))
      return nullptr;
    if (!norm_input(x)) return nullptr;
    if (!dy || !stats) {
      fail("layer_norm_backward needs dy and stats");
      return nullptr;
    }
    if (!norm_rows(dy, *x, "dy is a row-major tensor of x's dtype and size") || !norm_stats(stats, *x) ||
        !norm_param(w, *x, "weight is a contiguous [cols] tensor of x's dtype"))
      return nullptr;
    const auto opt = x->options().requires_grad(false);
    at::Tensor mx, mw, mb, ms;
    if (!want_dx) dx = nullptr;
    if (!want_p) dw = db = nullptr;
    if (want_dx && !dx) {
      mx = at::empty(x->sizes(), opt.memory_format(at::MemoryFormat::Contiguous));
      dx = &mx;
    }
    if (want_p && !dw) {
      mw = at::empty({x->size(1)}, opt);
      dw = &mw;
    }
    if (want_p && !db) {
      mb = at::empty({x->size(1)}, opt);
      db = &mb;
    }
    if (!norm_rows(dx, *x, "dx is a row-major tensor of x's dtype and size") ||
        !norm_param(dw, *x, "dweight is a contiguous [cols] tensor of x's dtype") ||
        !norm_param(db, *x, "dbias is a contiguous [cols] tensor of x's dtype"))
      return nullptr;
    if (want_p && !ws) {
      const int64_t need = g_ws_size(MXQ_OP_LAYER_NORM_BACKWARD, x->size(0), x->size(1), 0);
      if (need > 0) {
        ms = at::empty({need}, opt.dtype(at::kByte));
        ws = &ms;
      }
    }
    if (ws && !ws->is_contiguous()) {
      fail("the workspace is a contiguous tensor");
      return nullptr;
    }
    if (!on_device(dev, {dy, x, stats, w, dx, dw, db, ws})) return nullptr;
    mxq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_norm_bwd(dy->data_ptr(), ld(*dy), x->data_ptr(), x->scalar_type() == at::kFloat ? MXQ_DT_F32 : MXQ_DT_BF16,
                    x->size(0), x->size(1), ld(*x), static_cast<const float*>(ptr(stats)), ptr(w), ptr(dx),
                    dx ? ld(*dx) : 0, ptr(dw), ptr(db), ptr(ws), ws ? ws->nbytes() : 0, reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
    if (st != MXQ_OK) return PyLong_FromLong(st);
    return pack3(give(mx, want_dx ? a[6] : Py_None), give(mw, want_p ? a[7] : Py_None), give(mb, want_p ? a[8] : Py_None));
  });
}

// bind(quantize, gemm, gemm_grouped, qk_norm_rope, gemm_gated, gemm_gated_backward, layer_norm,
// layer_norm_backward, workspace_size): the addresses of the C ABI
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int64_t p[9];
  if (!count(n, 9)) return nullptr;
  for (int i = 0; i < 9; ++i)
    if (!to_i64(a[i], &p[i])) return nullptr;
  g_quantize = reinterpret_cast<decltype(g_quantize)>(p[0]);
  g_gemm = reinterpret_cast<decltype(g_gemm)>(p[1]);
  g_grouped = reinterpret_cast<decltype(g_grouped)>(p[2]);
  g_qk = reinterpret_cast<decltype(g_qk)>(p[3]);
  g_gated = reinterpret_cast<decltype(g_gated)>(p[4]);
  g_gated_bwd = reinterpret_cast<decltype(g_gated_bwd)>(p[5]);
  g_norm = reinterpret_cast<decltype(g_norm)>(p[6]);
  g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[7]);
  g_ws_size = reinterpret_cast<decltype(g_ws_size)>(p[8]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<bind>("bind"), method<quantize>("quantize"), method<empty_rows>("empty_rows"), method<gemm>("gemm"),
    method<gemm_grouped>("gemm_grouped"), method<qk_norm_rope>("qk_norm_rope"), method<gemm_gated>("gemm_gated"),
    method<gemm_gated_backward>("gemm_gated_backward"), method<layer_norm>("layer_norm"),
    method<layer_norm_backward>("layer_norm_backward"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() {
  s_fmt = PyUnicode_InternFromString("fmt");
  s_rows = PyUnicode_InternFromString("rows");
  s_cols = PyUnicode_InternFromString("cols");
  s_codes = PyUnicode_InternFromString("codes");
  s_scales = PyUnicode_InternFromString("scales");
  s_tensor_scale = PyUnicode_InternFromString("tensor_scale");
  return PyModule_Create(&g_module);
}
