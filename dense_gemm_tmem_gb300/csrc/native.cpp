// native.cpp: the Python calls that a decode step makes many times, from tensors
// straight to the C-ABI: argument checks, output allocation and the call, without
// an interpreter step in between (a product through ctypes costs 9 us of host
// time, its kernel 7).  The entry points' addresses come from the loaded library
// (init); nothing is computed here.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_fp4.h"
#include "../../include/gemm_fp8.h"
#include "../../include/gemm_ortho.h"

namespace {

using QuantizeFn = int (*)(gemm_handle_t, int64_t, int64_t, const void*, int64_t, int,
                           const gemm_fp8_matrix_t*, const gemm_fp8_matrix_t*, void*);
using RunFn = int (*)(gemm_handle_t, int64_t, int64_t, int64_t, const gemm_fp8_matrix_t*,
                      const gemm_fp8_matrix_t*, const float*, void*, int64_t, int, int, int,
                      void*);
using MoeSpaceFn = int (*)(gemm_handle_t, const gemm_moe_fp8_t*, int64_t*);
using MoeFn = int (*)(gemm_handle_t, const gemm_moe_fp8_t*, void*, int64_t, void*);
using Quantize4Fn = int (*)(gemm_handle_t, int64_t, int64_t, const void*, int64_t, int,
                            const gemm_fp4_matrix_t*, void*);
using Dequantize4Fn = int (*)(gemm_handle_t, int64_t, int64_t, const gemm_fp4_matrix_t*, void*,
                              int64_t, int, void*);
using Run4Fn = int (*)(gemm_handle_t, int64_t, int64_t, int64_t, const gemm_fp4_matrix_t*,
                       const gemm_fp4_matrix_t*, const float*, void*, int64_t, int, void*);
using LinearRow4Fn = int (*)(gemm_handle_t, int64_t, int64_t, const void*, int,
                             const gemm_fp4_matrix_t*, const float*, void*, int, void*);
using OneRow4Fn = int (*)(gemm_handle_t, int64_t, int64_t);
using OrthoSpaceFn = int (*)(gemm_handle_t, const gemm_orthogonalize_t*, int64_t*);
using OrthoFn = int (*)(gemm_handle_t, const gemm_orthogonalize_t*, void*, int64_t, void*);
QuantizeFn quantize_fn = nullptr;
RunFn run_fn = nullptr;
MoeSpaceFn moe_space_fn = nullptr;
MoeFn moe_fn = nullptr;
Quantize4Fn quantize4_fn = nullptr;
Dequantize4Fn dequantize4_fn = nullptr;
Run4Fn run4_fn = nullptr;
OrthoSpaceFn ortho_space_fn = nullptr;
OrthoFn ortho_fn = nullptr;
LinearRow4Fn linear_row4_fn = nullptr;
OneRow4Fn one_row4_fn = nullptr;

constexpr int64_t kBlock = 128;
int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// A Python error has been set.
struct Raised {};
[[noreturn]] void fail(PyObject* type, const char* what) {
  PyErr_SetString(type, what);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, what);
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
template <class T>
T* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised{};
  return static_cast<T*>(p);
}

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return GEMM_F16;
    case at::kFloat: return GEMM_F32;
    case at::kBFloat16: return GEMM_BF16;
    default: return -1;
  }
}

void on_device(const at::Tensor& t, int64_t index) {
  if (!t.is_cuda() || t.get_device() != index)
    fail(PyExc_ValueError, "tensor is not on the handle's device");
}

// Unit stride along the rows of a 2-D tensor, and the row pitch.
int64_t pitch_of(const at::Tensor& t, const char* what) {
  const int64_t rows = t.size(0), cols = t.size(1);
  if ((cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols))
    fail(PyExc_ValueError, what);
  return rows > 1 ? t.stride(0) : std::max(t.stride(0), cols);
}

// A view of `buf`'s bytes from `at` on, as another type.
at::Tensor carve(const at::Tensor& buf, at::ScalarType type, int64_t at, int64_t rows,
                 int64_t cols, int64_t stride_r, int64_t stride_c) {
  const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::TensorImpl::VIEW, c10::Storage(buf.storage()), buf.key_set(), meta);
  const int64_t sizes[2] = {rows, cols}, strides[2] = {stride_r, stride_c};
  t.unsafeGetTensorImpl()->set_storage_offset(at / int64_t(meta.itemsize()));
  t.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, strides);
  return t;
}

// The same, flat.
at::Tensor carve_flat(const at::Tensor& buf, at::ScalarType type, int64_t at, int64_t count) {
  const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::TensorImpl::VIEW, c10::Storage(buf.storage()), buf.key_set(), meta);
  t.unsafeGetTensorImpl()->set_storage_offset(at / int64_t(meta.itemsize()));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(count);
  return t;
}

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11) fail(PyExc_TypeError, "init takes 11 addresses");
    quantize_fn = reinterpret_cast<QuantizeFn>(address<void>(args[0]));
    run_fn = reinterpret_cast<RunFn>(address<void>(args[1]));
    moe_space_fn = reinterpret_cast<MoeSpaceFn>(address<void>(args[2]));
    moe_fn = reinterpret_cast<MoeFn>(address<void>(args[3]));
    quantize4_fn = reinterpret_cast<Quantize4Fn>(address<void>(args[4]));
    dequantize4_fn = reinterpret_cast<Dequantize4Fn>(address<void>(args[5]));
    run4_fn = reinterpret_cast<Run4Fn>(address<void>(args[6]));
    ortho_space_fn = reinterpret_cast<OrthoSpaceFn>(address<void>(args[7]));
    ortho_fn = reinterpret_cast<OrthoFn>(address<void>(args[8]));
    linear_row4_fn = reinterpret_cast<LinearRow4Fn>(address<void>(args[9]));
    one_row4_fn = reinterpret_cast<OneRow4Fn>(address<void>(args[10]));
    Py_RETURN_NONE;
  });
}

// quantize(handle, device, x, first kind, second kind or -1, stream)
//   -> (data, scale) or (data, scale, data2, scale2), or a gemm_status_t
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) fail(PyExc_TypeError, "quantize takes 6 arguments");
    const int64_t device = integer(args[1]);
    const at::Tensor& x = tensor(args[2], "x must be a tensor");
    const int64_t kinds[2] = {integer(args[3]), integer(args[4])};
    const int code = code_of(x.scalar_type());
    if (code < 0) fail(PyExc_TypeError, "x must be float16, bfloat16 or float32");
    if (x.dim() != 2) fail(PyExc_ValueError, "x must be 2-D");
    on_device(x, device);
    const int64_t ld_x = pitch_of(x, "rows of x must be contiguous and not overlap");
    const int64_t rows = x.size(0), cols = x.size(1), ld = (cols + 15) & ~int64_t(15);
    const int64_t values = (rows * ld + 255) & ~int64_t(255);
    const int count = kinds[1] >= 0 ? 2 : 1;
    const auto opt = x.options().dtype(at::kByte).requires_grad(false);
    gemm_fp8_matrix_t m[2];
    at::Tensor out[4];
    for (int i = 0; i < count; ++i) {
      // values and scales in one allocation, each matrix in its own: a program that
      // keeps one of the two does not hold the other's bytes
      const bool row = kinds[i] == GEMM_FP8_ROW;
      const int64_t sr = row ? rows : blocks_of(rows);
      const int64_t sc = kinds[i] == GEMM_FP8_COL ? cols : blocks_of(cols);
      const at::Tensor buf = at::empty({values + sr * sc * 4}, opt);
      uint8_t* base = static_cast<uint8_t*>(buf.data_ptr());
      // row blocks: the scales of one k-block next to each other
      const int64_t s_r = row ? 1 : sc, s_c = row ? sr : 1;
      m[i] = gemm_fp8_matrix_t{base, ld, reinterpret_cast<float*>(base + values),
                               s_r,  s_c, int32_t(kinds[i]), 0};
      out[2 * i] = carve(buf, at::kFloat8_e4m3fn, 0, rows, cols, ld, 1);
      out[2 * i + 1] = carve(buf, at::kFloat, values, sr, sc, s_r, s_c);
    }
    const int rc = quantize_fn(address<gemm_ctx>(args[0]), rows, cols, x.data_ptr(), ld_x, code,
                               &m[0], count == 2 ? &m[1] : nullptr, address<void>(args[5]));
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    PyObject* r = PyTuple_New(2 * count);
    if (!r) throw Raised{};
    for (int i = 0; i < 2 * count; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
    return r;
  });
}

// Types of a block-scaled matrix's tensors, and the shape of its scales.  They are
// looked at on every call: a program may replace the tensors of an Fp8Matrix.
void check_types(const at::Tensor& q, const at::Tensor& s) {
  if (q.scalar_type() != at::kFloat8_e4m3fn && q.scalar_type() != at::kByte)
    fail(PyExc_TypeError, "data must be float8_e4m3fn (or its bytes as uint8)");
  if (s.scalar_type() != at::kFloat) fail(PyExc_TypeError, "scale must be float32");
}
void check_scales(const at::Tensor& s, int64_t rows, int64_t cols) {
  const int64_t d = s.dim();
  if (s.size(d - 2) != rows || s.size(d - 1) != cols) {
    PyErr_Format(PyExc_ValueError, "scale has shape (%lld, %lld), expected (%lld, %lld)",
                 (long long)s.size(d - 2), (long long)s.size(d - 1), (long long)rows,
                 (long long)cols);
    throw Raised{};
  }
}

gemm_fp8_matrix_t matrix(PyObject* data, PyObject* scale, PyObject* blocks) {
  const at::Tensor& q = tensor(data, "data must be a tensor");
  const at::Tensor& s = tensor(scale, "scale must be a tensor");
  if (q.dim() != 2 || s.dim() != 2) fail(PyExc_ValueError, "A and B must be 2-D");
  check_types(q, s);
  const int64_t kind = integer(blocks);
  if (kind < GEMM_FP8_ROW || kind > GEMM_FP8_TILE) fail(PyExc_ValueError, "unknown blocks");
  check_scales(s, kind == GEMM_FP8_ROW ? q.size(0) : blocks_of(q.size(0)),
               kind == GEMM_FP8_COL ? q.size(1) : blocks_of(q.size(1)));
  return gemm_fp8_matrix_t{q.data_ptr(), pitch_of(q, "rows of data must be contiguous"),
                           static_cast<float*>(s.data_ptr()), s.stride(0), s.stride(1),
                           int32_t(kind), 0};
}

// The arguments that both product calls take: handle, device, A data, A scale, A kind,
// B data, B scale, B kind, bias or None, a_major, b_major.
struct Product {
  gemm_ctx* h;
  int64_t device;
  gemm_fp8_matrix_t a, b;
  int64_t a_major, b_major, M, N, K;
  const float* bias = nullptr;
  explicit Product(PyObject* const* args)
      : h(address<gemm_ctx>(args[0])),
        device(integer(args[1])),
        a(matrix(args[2], args[3], args[4])),
        b(matrix(args[5], args[6], args[7])),
        a_major(integer(args[9])),
        b_major(integer(args[10])) {
    for (int i : {2, 3, 5, 6}) on_device(THPVariable_Unpack(args[i]), device);
    const at::Tensor& qa = THPVariable_Unpack(args[2]);
    const at::Tensor& qb = THPVariable_Unpack(args[5]);
    const bool ar = a_major == GEMM_ROW_MAJOR, br = b_major == GEMM_ROW_MAJOR;
    M = qa.size(ar ? 0 : 1);
    K = qa.size(ar ? 1 : 0);
    N = qb.size(br ? 1 : 0);
    if (qb.size(br ? 0 : 1) != K) {
      PyErr_Format(PyExc_ValueError, "inner dimensions differ: %lld vs %lld", (long long)K,
                   (long long)qb.size(br ? 0 : 1));
      throw Raised{};
    }
    if (args[8] != Py_None) {
      const at::Tensor& t = tensor(args[8], "bias must be a tensor");
      if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != N || !t.is_contiguous())
        fail(PyExc_ValueError, "bias must be contiguous float32 of shape (N,)");
      on_device(t, device);
      bias = static_cast<const float*>(t.data_ptr());
    }
  }
  int run(void* C, int64_t ldc, int code, PyObject* stream) const {
    return run_fn(h, M, N, K, &a, &b, bias, C, ldc, int(a_major), int(b_major), code,
                  address<void>(stream));
  }
};

// matmul(the product's arguments, output type's code, stream) -> C or a gemm_status_t
PyObject* matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13) fail(PyExc_TypeError, "matmul takes 13 arguments");
    const Product p(args);
    const int64_t code = integer(args[11]);
    const at::ScalarType type = code == GEMM_F16    ? at::kHalf
                                : code == GEMM_BF16 ? at::kBFloat16
                                                    : at::kFloat;
    const auto opt = THPVariable_Unpack(args[2]).options().dtype(type).requires_grad(false);
    at::Tensor C = at::empty({p.M, p.N}, opt);
    const int rc = p.run(C.data_ptr(), p.N, int(code), args[12]);
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    return THPVariable_Wrap(std::move(C));
  });
}

// run(the product's arguments, C, stream) -> a gemm_status_t
PyObject* run(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13) fail(PyExc_TypeError, "run takes 13 arguments");
    const Product p(args);
    const at::Tensor& C = tensor(args[11], "C must be a tensor");
    const int code = code_of(C.scalar_type());
    if (code < 0) fail(PyExc_TypeError, "C must be float16, bfloat16 or float32");
    if (C.dim() != 2 || C.size(0) != p.M || C.size(1) != p.N) {
      PyErr_Format(PyExc_ValueError, "C must have shape (%lld, %lld)", (long long)p.M,
                   (long long)p.N);
      throw Raised{};
    }
    on_device(C, p.device);
    const int64_t ldc = pitch_of(C, "rows of C must be contiguous and not overlap");
    return PyLong_FromLong(p.run(C.data_ptr(), ldc, code, args[12]));
  });
}

gemm_fp8_experts_t experts(PyObject* data, PyObject* scale, int64_t E, int64_t rows,
                           int64_t cols) {
  const at::Tensor& q = tensor(data, "data must be a tensor");
  const at::Tensor& s = tensor(scale, "scale must be a tensor");
  if (q.dim() != 3 || s.dim() != 3)
    fail(PyExc_ValueError, "gate, up and down must be (experts, rows, cols)");
  if (q.size(0) != E || q.size(1) != rows || q.size(2) != cols) {
    PyErr_Format(PyExc_ValueError,
                 "weights have shape (%lld, %lld, %lld), expected (%lld, %lld, %lld)",
                 (long long)q.size(0), (long long)q.size(1), (long long)q.size(2), (long long)E,
                 (long long)rows, (long long)cols);
    throw Raised{};
  }
  check_types(q, s);
  if (s.size(0) != E) fail(PyExc_ValueError, "scale must have one matrix per expert");
  check_scales(s, blocks_of(rows), blocks_of(cols));
  if (cols > 1 && q.stride(2) != 1) fail(PyExc_ValueError, "rows of data must be contiguous");
  return gemm_fp8_experts_t{q.data_ptr(),
                            rows > 1 ? q.stride(1) : std::max(q.stride(1), cols),
                            q.stride(0),
                            static_cast<const float*>(s.data_ptr()),
                            s.stride(0),
                            s.stride(1),
                            s.stride(2)};
}

// moe(handle, device, x, router, gate data, scale, up data, scale, down data,
// scale, top_k, renormalize, stream) -> (out, ids, gates) or a gemm_status_t.
// `stream` is the current stream: the scratch is freed on return, in that stream's
// order.
PyObject* moe(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13) fail(PyExc_TypeError, "moe takes 13 arguments");
    const int64_t device = integer(args[1]);
    const at::Tensor& x = tensor(args[2], "x must be a tensor");
    const at::Tensor& router = tensor(args[3], "router must be a tensor");
    if (x.dim() != 2 || router.dim() != 2 || router.size(1) != x.size(1))
      fail(PyExc_ValueError, "x must be (tokens, hidden), router (experts, hidden)");
    if (x.scalar_type() != router.scalar_type() ||
        (x.scalar_type() != at::kHalf && x.scalar_type() != at::kBFloat16))
      fail(PyExc_TypeError, "x and router: both float16 or both bfloat16");
    gemm_moe_fp8_t L = {};
    L.tokens = x.size(0);
    L.hidden = x.size(1);
    L.experts = router.size(0);
    const at::Tensor& g = tensor(args[4], "gate must be a tensor");
    L.inner = g.dim() == 3 ? g.size(1) : 0;
    const int64_t top_k = integer(args[10]);
    if (top_k < 1 || top_k > L.experts)
      fail(PyExc_ValueError, "top_k must be between 1 and the number of experts");
    L.top_k = int32_t(std::min<int64_t>(top_k, INT32_MAX));
    L.renormalize = int32_t(integer(args[11]));
    L.dtype = code_of(x.scalar_type());
    L.gate = experts(args[4], args[5], L.experts, L.inner, L.hidden);
    L.up = experts(args[6], args[7], L.experts, L.inner, L.hidden);
    L.down = experts(args[8], args[9], L.experts, L.hidden, L.inner);
    for (int i = 2; i < 10; ++i) on_device(THPVariable_Unpack(args[i]), device);
    L.x = x.data_ptr();
    L.ld_x = pitch_of(x, "rows of x must be contiguous and not overlap");
    L.router = router.data_ptr();
    L.ld_router = pitch_of(router, "rows of router must be contiguous and not overlap");
    gemm_ctx* h = address<gemm_ctx>(args[0]);
    int64_t bytes = 0;
    int rc = moe_space_fn(h, &L, &bytes);
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    const auto opt = x.options().requires_grad(false);
    at::Tensor out = at::empty({L.tokens, L.hidden}, opt);
    at::Tensor ids = at::empty({L.tokens, L.top_k}, opt.dtype(at::kInt));
    at::Tensor gates = at::empty({L.tokens, L.top_k}, opt.dtype(at::kFloat));
    at::Tensor space = at::empty({bytes}, opt.dtype(at::kByte));
    L.out = out.data_ptr();
    L.ld_out = L.hidden;
    L.ids = static_cast<int32_t*>(ids.data_ptr());
    L.gates = static_cast<float*>(gates.data_ptr());
    rc = moe_fn(h, &L, space.data_ptr(), bytes, address<void>(args[12]));
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    PyObject* r = PyTuple_New(3);
    if (!r) throw Raised{};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(out)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(ids)));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(gates)));
    return r;
  });
}

// ------------------------------------------------------------------ 4 bits --
int64_t scale_bytes4(int64_t rows, int64_t cols, int64_t kind) {
  const int64_t per = kind == GEMM_MXFP4 ? 128 : 64;
  return blocks_of(rows) * ((cols + per - 1) / per) * 512;
}

at::ScalarType type_of(int64_t code) {
  return code == GEMM_F16 ? at::kHalf : code == GEMM_BF16 ? at::kBFloat16 : at::kFloat;
}

// A 4-bit matrix and what it is stored in.
struct Made4 {
  gemm_fp4_matrix_t m;
  at::Tensor buf;
  int64_t rows, cols, scales_at, rows_at;
  // values, block scales and row scales in one allocation
  Made4(const at::TensorOptions& opt, int64_t r, int64_t c, int64_t kind) : rows(r), cols(c) {
    const int64_t ld = ((c + 1) / 2 + 15) & ~int64_t(15);
    scales_at = (r * ld + 255) & ~int64_t(255);
    rows_at = scales_at + scale_bytes4(r, c, kind);  // a multiple of 256
    buf = at::empty({rows_at + (kind == GEMM_NVFP4 ? 4 * r : 0)}, opt);
    uint8_t* base = static_cast<uint8_t*>(buf.data_ptr());
    m = gemm_fp4_matrix_t{base, ld, base + scales_at,
                          kind == GEMM_NVFP4 ? reinterpret_cast<float*>(base + rows_at) : nullptr,
                          kind == GEMM_NVFP4, int32_t(kind), 0};
  }
};

// The tensors of an Fp4Matrix of `cols` columns, looked at on every call (and when one is
// made, wherever they are: device < 0).
struct Given4 {
  gemm_fp4_matrix_t m;
  int64_t rows;
  Given4(PyObject* data, PyObject* scale, PyObject* row_scale, int64_t cols, int64_t kind,
         int64_t device) {
    const at::Tensor& q = tensor(data, "data must be a tensor");
    const at::Tensor& s = tensor(scale, "scale must be a tensor");
    if (kind != GEMM_MXFP4 && kind != GEMM_NVFP4) fail(PyExc_ValueError, "unknown format");
    if (q.scalar_type() != at::kByte && q.scalar_type() != at::ScalarType::Float4_e2m1fn_x2)
      fail(PyExc_TypeError, "data must be uint8 (or float4_e2m1fn_x2)");
    if (s.scalar_type() != at::kByte &&
        s.scalar_type() != (kind == GEMM_MXFP4 ? at::ScalarType::Float8_e8m0fnu
                                               : at::ScalarType::Float8_e4m3fn))
      fail(PyExc_TypeError, "scale must be uint8 or the format's scale type");
    if (q.dim() != 2 || cols < 0 || q.size(1) != (cols + 1) / 2)
      fail(PyExc_ValueError, "data must be (rows, ceil(cols / 2))");
    rows = q.size(0);
    if (s.dim() != 1 || s.size(0) != scale_bytes4(rows, cols, kind) || !s.is_contiguous())
      fail(PyExc_ValueError, "scale must be flat and contiguous, of the format's size");
    on(q, device);
    on(s, device < 0 ? place(q) : device);
    // a lone row needs no pitch
    const int64_t pitch = pitch_of(q, "rows of data must be contiguous and not overlap");
    m = gemm_fp4_matrix_t{q.data_ptr(), rows > 1 ? pitch : (q.size(1) + 15) & ~int64_t(15),
                          s.data_ptr(), nullptr, 0, int32_t(kind), 0};
    if (row_scale != Py_None) {
      const at::Tensor& r = tensor(row_scale, "row_scale must be a tensor or None");
      if (r.scalar_type() != at::kFloat) fail(PyExc_TypeError, "row_scale must be float32");
      if (r.dim() != 1 || r.size(0) != rows)
        fail(PyExc_ValueError, "row_scale must have shape (rows,)");
      on(r, device < 0 ? place(q) : device);
      m.row_scale = static_cast<float*>(r.data_ptr());
      m.row_scale_stride = r.stride(0);
    }
  }

 private:
  static constexpr int64_t kHost = -2;
  static int64_t place(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : kHost; }
  static void on(const at::Tensor& t, int64_t device) {
    if (device == kHost) {
      if (t.is_cuda()) fail(PyExc_ValueError, "the scales are on another device than data");
    } else if (device >= 0) {
      on_device(t, device);
    }
  }
};

// check4(data, scale, row_scale or None, rows, cols, kind): refuses what is no 4-bit matrix.
PyObject* check4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) fail(PyExc_TypeError, "check4 takes 6 arguments");
    const Given4 q(args[0], args[1], args[2], integer(args[4]), integer(args[5]), -1);
    if (q.rows != integer(args[3])) fail(PyExc_ValueError, "data must be (rows, ceil(cols / 2))");
    Py_RETURN_NONE;
  });
}

const float* bias_of(PyObject* o, int64_t N, int64_t device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "bias must be a tensor");
  if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != N || !t.is_contiguous())
    fail(PyExc_ValueError, "bias must be contiguous float32 of shape (N,)");
  on_device(t, device);
  return static_cast<const float*>(t.data_ptr());
}

// A matrix of the caller's: checked, with its type's code and row pitch.
const at::Tensor& rows_of(PyObject* o, int64_t device, int* code, int64_t* ld) {
  const at::Tensor& x = tensor(o, "x must be a tensor");
  *code = code_of(x.scalar_type());
  if (*code < 0) fail(PyExc_TypeError, "x must be float16, bfloat16 or float32");
  if (x.dim() != 2) fail(PyExc_ValueError, "x must be 2-D");
  on_device(x, device);
  *ld = pitch_of(x, "rows of x must be contiguous and not overlap");
  return x;
}

// quantize4(handle, device, x, kind, stream) -> (data, scale, row_scale or None)
// or a gemm_status_t
PyObject* quantize4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) fail(PyExc_TypeError, "quantize4 takes 5 arguments");
    int code;
    int64_t ld;
    const at::Tensor& x = rows_of(args[2], integer(args[1]), &code, &ld);
    const int64_t kind = integer(args[3]);
    const Made4 q(x.options().dtype(at::kByte).requires_grad(false), x.size(0), x.size(1), kind);
    const int rc = quantize4_fn(address<gemm_ctx>(args[0]), q.rows, q.cols, x.data_ptr(), ld,
                                code, &q.m, address<void>(args[4]));
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    PyObject* r = PyTuple_New(3);
    if (!r) throw Raised{};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(carve(q.buf, at::kByte, 0, q.rows, (q.cols + 1) / 2,
                                                  q.m.ld, 1)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(carve_flat(q.buf, at::kByte, q.scales_at,
                                                       q.rows_at - q.scales_at)));
    if (kind == GEMM_NVFP4) {
      PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(carve_flat(q.buf, at::kFloat, q.rows_at, q.rows)));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, 2, Py_None);
    }
    return r;
  });
}

// dequantize4(handle, device, data, scale, row_scale, cols, kind, output type's code,
// stream) -> a tensor or a gemm_status_t
PyObject* dequantize4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) fail(PyExc_TypeError, "dequantize4 takes 9 arguments");
    const int64_t cols = integer(args[5]), code = integer(args[7]);
    const Given4 q(args[2], args[3], args[4], cols, integer(args[6]), integer(args[1]));
    at::Tensor out = at::empty({q.rows, cols}, THPVariable_Unpack(args[2]).options()
                                                   .dtype(type_of(code)).requires_grad(false));
    const int rc = dequantize4_fn(address<gemm_ctx>(args[0]), q.rows, cols, &q.m, out.data_ptr(),
                                  cols, int(code), address<void>(args[8]));
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    return THPVariable_Wrap(std::move(out));
  });
}

// What both product calls take: handle, device, A data, scale, row_scale, B data, scale,
// row_scale, K, kind, bias or None.
struct Product4 {
  gemm_ctx* h;
  int64_t device, K;
  Given4 a, b;
  const float* bias;
  explicit Product4(PyObject* const* args)
      : h(address<gemm_ctx>(args[0])),
        device(integer(args[1])),
        K(integer(args[8])),
        a(args[2], args[3], args[4], K, integer(args[9]), device),
        b(args[5], args[6], args[7], K, integer(args[9]), device),
        bias(bias_of(args[10], b.rows, device)) {}
};

// matmul4(the product's arguments, output type's code, stream) -> C or a gemm_status_t
PyObject* matmul4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13) fail(PyExc_TypeError, "matmul4 takes 13 arguments");
    const Product4 p(args);
    const int64_t code = integer(args[11]);
    at::Tensor C = at::empty({p.a.rows, p.b.rows}, THPVariable_Unpack(args[2]).options()
                                                       .dtype(type_of(code)).requires_grad(false));
    const int rc = run4_fn(p.h, p.a.rows, p.b.rows, p.K, &p.a.m, &p.b.m, p.bias, C.data_ptr(),
                           p.b.rows, int(code), address<void>(args[12]));
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    return THPVariable_Wrap(std::move(C));
  });
}

// run4(the product's arguments, C, stream) -> a gemm_status_t
PyObject* run4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 13) fail(PyExc_TypeError, "run4 takes 13 arguments");
    const Product4 p(args);
    const at::Tensor& C = tensor(args[11], "C must be a tensor");
    const int code = code_of(C.scalar_type());
    if (code < 0) fail(PyExc_TypeError, "C must be float16, bfloat16 or float32");
    if (C.dim() != 2 || C.size(0) != p.a.rows || C.size(1) != p.b.rows) {
      PyErr_Format(PyExc_ValueError, "C must have shape (%lld, %lld)", (long long)p.a.rows,
                   (long long)p.b.rows);
      throw Raised{};
    }
    on_device(C, p.device);
    const int64_t ldc = pitch_of(C, "rows of C must be contiguous and not overlap");
    return PyLong_FromLong(run4_fn(p.h, p.a.rows, p.b.rows, p.K, &p.a.m, &p.b.m, p.bias,
                                   C.data_ptr(), ldc, code, address<void>(args[12])));
  });
}

// linear4(handle, device, x, W data, scale, row_scale, K, kind, bias or None, stream)
// -> y or a gemm_status_t.  `stream` is the current stream: the quantised x is freed
// on return, in that stream's order.
PyObject* linear4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10) fail(PyExc_TypeError, "linear4 takes 10 arguments");
    gemm_ctx* h = address<gemm_ctx>(args[0]);
    const int64_t device = integer(args[1]), K = integer(args[6]), kind = integer(args[7]);
    int code;
    int64_t ld;
    const at::Tensor& x = rows_of(args[2], device, &code, &ld);
    const Given4 w(args[3], args[4], args[5], K, kind, device);
    if (x.size(1) != K) {
      PyErr_Format(PyExc_ValueError, "inner dimensions differ: %lld vs %lld",
                   (long long)x.size(1), (long long)K);
      throw Raised{};
    }
    const float* bias = bias_of(args[8], w.rows, device);
    void* stream = address<void>(args[9]);
    const auto opt = x.options().requires_grad(false);
    at::Tensor y = at::empty({x.size(0), w.rows}, opt);
    int rc;
    if (x.size(0) == 1 && K <= GEMM_FP4_ROW_MOST && one_row4_fn(h, w.rows, K)) {  // one launch
      rc = linear_row4_fn(h, w.rows, K, x.data_ptr(), code, &w.m, bias, y.data_ptr(), code, stream);
    } else {
      const Made4 q(opt.dtype(at::kByte), x.size(0), K, kind);
      rc = quantize4_fn(h, q.rows, K, x.data_ptr(), ld, code, &q.m, stream);
      if (rc == GEMM_OK)
        rc = run4_fn(h, q.rows, w.rows, K, &q.m, &w.m, bias, y.data_ptr(), w.rows, code, stream);
    }
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    return THPVariable_Wrap(std::move(y));
  });
}

// orthogonalize(handle, device, G, coefficients as fp32 bytes, eps, stream) -> a tensor or
// a gemm_status_t.  `stream` is the current stream: the scratch is freed on return, in
// that stream's order.
PyObject* orthogonalize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) fail(PyExc_TypeError, "orthogonalize takes 6 arguments");
    gemm_ctx* h = address<gemm_ctx>(args[0]);
    const at::Tensor& g = tensor(args[2], "G must be a tensor");
    const int code = code_of(g.scalar_type());
    if (code < 0) fail(PyExc_TypeError, "G must be float16, bfloat16 or float32");
    const int64_t d = g.dim();
    if (d != 2 && d != 3) fail(PyExc_ValueError, "G must be 2-D, or 3-D with a batch");
    on_device(g, integer(args[1]));
    if (!PyBytes_Check(args[3]) || PyBytes_GET_SIZE(args[3]) % 12 != 0)
      fail(PyExc_TypeError, "coefficients must be bytes of three floats a step");
    gemm_orthogonalize_t p = {};
    p.batch = d == 3 ? g.size(0) : 1;
    p.rows = g.size(d - 2);
    p.cols = g.size(d - 1);
    p.steps = int32_t(PyBytes_GET_SIZE(args[3]) / 12);
    p.dtype = code;
    p.coefficients = reinterpret_cast<const float*>(PyBytes_AS_STRING(args[3]));
    p.eps = PyFloat_AsDouble(args[4]);
    if (p.eps == -1 && PyErr_Occurred()) throw Raised{};
    if ((p.cols > 1 && g.stride(d - 1) != 1) || (p.rows > 1 && g.stride(d - 2) < p.cols))
      fail(PyExc_ValueError, "rows of G must be contiguous and not overlap");
    p.g = g.data_ptr();
    p.ld_g = p.rows > 1 ? g.stride(d - 2) : p.cols;
    p.stride_g = d == 3 && p.batch > 1 ? g.stride(0) : 0;
    int64_t bytes = 0;
    int rc = ortho_space_fn(h, &p, &bytes);
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    const auto opt = g.options().requires_grad(false);
    at::Tensor out = at::empty(g.sizes(), opt.dtype(at::kBFloat16));
    at::Tensor space = at::empty({bytes}, opt.dtype(at::kByte));
    p.out = out.data_ptr();
    p.ld_out = p.cols;
    p.stride_out = p.rows * p.cols;
    rc = ortho_fn(h, &p, space.data_ptr(), bytes, address<void>(args[5]));
    if (rc != GEMM_OK) return PyLong_FromLong(rc);
    return THPVariable_Wrap(std::move(out));
  });
}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(init), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(quantize), METH_FASTCALL, nullptr},
    {"matmul", reinterpret_cast<PyCFunction>(matmul), METH_FASTCALL, nullptr},
    {"run", reinterpret_cast<PyCFunction>(run), METH_FASTCALL, nullptr},
    {"moe", reinterpret_cast<PyCFunction>(moe), METH_FASTCALL, nullptr},
    {"check4", reinterpret_cast<PyCFunction>(check4), METH_FASTCALL, nullptr},
    {"quantize4", reinterpret_cast<PyCFunction>(quantize4), METH_FASTCALL, nullptr},
    {"dequantize4", reinterpret_cast<PyCFunction>(dequantize4), METH_FASTCALL, nullptr},
    {"matmul4", reinterpret_cast<PyCFunction>(matmul4), METH_FASTCALL, nullptr},
    {"run4", reinterpret_cast<PyCFunction>(run4), METH_FASTCALL, nullptr},
    {"linear4", reinterpret_cast<PyCFunction>(linear4), METH_FASTCALL, nullptr},
    {"orthogonalize", reinterpret_cast<PyCFunction>(orthogonalize), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dgemm_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dgemm_native() { return PyModule_Create(&module); }
