// Argument marshalling of the binding's short calls, as a Python extension.
//
// At decode a call's kernels run for a few microseconds, and checking the
// arguments, allocating the results and calling through ctypes takes longer
// than that in Python. Each function here does it for the ordinary call (plain
// CUDA tensors on the current device and its current stream, shapes that fit)
// and returns None for any other, and where the library refuses: the caller
// (_lib.py) then goes its own way, which raises what is to be raised. No step
// of any operator is here.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "mm.h"

namespace {

using at::Tensor;

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

// Other threads of Python run while this lives: a launch waits where the device's
// queue is full, and an allocation may wait for the device.
struct Released {
  PyThreadState* state = PyEval_SaveThread();
  ~Released() { PyEval_RestoreThread(state); }
};

// One call: the device of its first tensor, and whether all fit so far. Python is
// released from its first allocation to the end of the library's call.
struct Call {
  bool ok = true;
  int device = -1;
  std::optional<Released> released;

  // A contiguous tensor of `type` on the one device; NULL (ok stays) for None
  // if `optional`.
  const Tensor* take(PyObject* o, at::ScalarType type, bool optional = false) {
    const Tensor* t = any(o, optional);
    if (t != nullptr && t->scalar_type() != type) ok = false;
    return t;
  }

  const Tensor* any(PyObject* o, bool optional = false) {
    if (o == Py_None) {
      ok = ok && optional;
      return nullptr;
    }
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || !t.is_contiguous()) {
      ok = false;
      return &t;
    }
    if (device < 0) {
      device = t.get_device();
      if (device != c10::cuda::current_device()) ok = false;
    } else if (device != t.get_device()) {
      ok = false;
    }
    return &t;
  }

  Tensor make(at::IntArrayRef shape, at::ScalarType type) {
    if (!released) released.emplace();
    return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)device),
                                  std::nullopt);
  }

  // Tensors of `type` and the next shapes out of one allocation, 256-byte aligned
  // each: an allocation takes longer than the rest of a tensor.
  Tensor part(const Tensor& bytes, int64_t& at, at::IntArrayRef shape, at::ScalarType type) const {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(bytes.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
        c10::scalarTypeToTypeMeta(type));
    c10::TensorImpl* i = t.unsafeGetTensorImpl();
    i->set_sizes_contiguous(shape);
    i->set_storage_offset(at / (int64_t)c10::elementSize(type));
    at += round256(t.numel() * (int64_t)c10::elementSize(type));
    return t;
  }

  template <typename... P, typename... A>
  int run(int (*fn)(P...), A... a) {
    if (!released) released.emplace();
    const int rc = fn(a...);
    released.reset();
    return rc;
  }

  void* stream() const {
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  }
};

int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? MM_DTYPE_FP32 : t == at::kBFloat16 ? MM_DTYPE_BF16
       : t == at::kHalf ? MM_DTYPE_FP16 : -1;
}

at::ScalarType dtype_of(long code) {
  return code == MM_DTYPE_FP32 ? at::kFloat : code == MM_DTYPE_BF16 ? at::kBFloat16 : at::kHalf;
}

bool fits_int(int64_t v) { return v >= 0 && v < (int64_t(1) << 31); }

// An int argument that is a Python int; sets ok to false otherwise.
long integer(PyObject* o, bool& ok) {
  if (!PyLong_CheckExact(o)) {
    ok = false;
    return 0;
  }
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    ok = false;
  }
  if (v < 0 || v >= (1L << 31)) ok = false;
  return v;
}

int64_t tiles(int64_t n) { return (n + 127) / 128; }

bool shape_is(const Tensor& t, at::IntArrayRef s) { return t.sizes() == s; }

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

#define MARSHAL_BEGIN try {
#define MARSHAL_END        \
  }                        \
  catch (...) {            \
  }                        \
  Py_RETURN_NONE;

// (logits, top_k, renorm, token_mask) -> (ids, w, counts, prob_sums, loss)
PyObject* route_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 4) Py_RETURN_NONE;
  Call c;
  const Tensor* x = c.any(a[0]);
  const Tensor* mask = c.any(a[3], true);
  const long k = integer(a[1], c.ok);
  const int renorm = PyObject_IsTrue(a[2]);
  if (!c.ok || renorm < 0 || x->dim() != 2) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const int64_t T = x->size(0), E = x->size(1);
  const int dt = dtype_code(x->scalar_type());
  if (dt < 0 || !fits_int(T) || !fits_int(E) || k < 1 || k > E || !fits_int(T * k))
    Py_RETURN_NONE;
  if (mask != nullptr && (!shape_is(*mask, {T}) || (mask->scalar_type() != at::kBool &&
                                                    mask->scalar_type() != at::kByte)))
    Py_RETURN_NONE;
  const int64_t need = mm_route_logits_workspace_size((int)T, (int)E);
  if (need < 0) Py_RETURN_NONE;
  // Two allocations for five results: what is the tokens', what is the batch's
  // (64 tokens: 6.6 -> 5.2 us a call). Codes and scales keep one each: weights are
  // stored, and formats that store tensors refuse shared memory.
  const Tensor tokens = c.make({2 * round256(4 * T * k)}, at::kByte),
               batch = c.make({2 * round256(4 * E) + 4}, at::kByte);
  int64_t in_tokens = 0, in_batch = 0;
  Tensor ids = c.part(tokens, in_tokens, {T, k}, at::kInt),
         w = c.part(tokens, in_tokens, {T, k}, at::kFloat),
         counts = c.part(batch, in_batch, {E}, at::kInt),
         sums = c.part(batch, in_batch, {E}, at::kFloat),
         loss = c.part(batch, in_batch, {1}, at::kFloat), ws;
  if (need > 0) ws = c.make({need}, at::kByte);
  const int rc = c.run(
      mm_route_logits, x->data_ptr(), dt,
      mask ? static_cast<const uint8_t*>(mask->data_ptr()) : nullptr, (int)T,
      (int)E, (int)k, renorm, static_cast<int32_t*>(ids.data_ptr()),
      static_cast<float*>(w.data_ptr()), static_cast<int32_t*>(counts.data_ptr()),
      static_cast<float*>(sums.data_ptr()), static_cast<float*>(loss.data_ptr()),
      need > 0 ? ws.data_ptr() : nullptr, (size_t)need, c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  PyObject* r = PyTuple_New(5);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrap(std::move(ids)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(w)));
  PyTuple_SET_ITEM(r, 2, wrap(std::move(counts)));
  PyTuple_SET_ITEM(r, 3, wrap(std::move(sums)));
  PyTuple_SET_ITEM(r, 4, wrap(std::move(loss)));
  return r;
  MARSHAL_END
}

// (logits, ids, counts, renorm, d_topk_w, d_loss, token_mask) -> d_logits
PyObject* route_logits_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 7) Py_RETURN_NONE;
  Call c;
  const Tensor* x = c.any(a[0]);
  const Tensor* ids = c.take(a[1], at::kInt);
  const Tensor* counts = c.take(a[2], at::kInt);
  const int renorm = PyObject_IsTrue(a[3]);
  const Tensor* dw = c.take(a[4], at::kFloat, true);
  const Tensor* dl = c.take(a[5], at::kFloat, true);
  const Tensor* mask = c.any(a[6], true);
  if (!c.ok || renorm < 0 || x->dim() != 2 || ids->dim() != 2) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const int64_t T = x->size(0), E = x->size(1), k = ids->size(1);
  const int dt = dtype_code(x->scalar_type());
  if (dt < 0 || !fits_int(T) || !fits_int(E) || !fits_int(k) || ids->size(0) != T ||
      !shape_is(*counts, {E}) || (dw && !shape_is(*dw, {T, k})) || (dl && dl->numel() != 1))
    Py_RETURN_NONE;
  if (mask != nullptr && (!shape_is(*mask, {T}) || (mask->scalar_type() != at::kBool &&
                                                    mask->scalar_type() != at::kByte)))
    Py_RETURN_NONE;
  Tensor grad = c.make({T, E}, x->scalar_type());
  const int rc = c.run(
      mm_route_logits_backward, x->data_ptr(), dt,
      mask ? static_cast<const uint8_t*>(mask->data_ptr()) : nullptr,
      static_cast<const int32_t*>(ids->data_ptr()), static_cast<const int32_t*>(counts->data_ptr()),
      dw ? static_cast<const float*>(dw->data_ptr()) : nullptr,
      dl ? static_cast<const float*>(dl->data_ptr()) : nullptr, (int)T, (int)E, (int)k, renorm,
      grad.data_ptr(), c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  return wrap(std::move(grad));
  MARSHAL_END
}

// (x) -> (codes, scales)
PyObject* mxfp4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 1) Py_RETURN_NONE;
  Call c;
  const Tensor* x = c.any(a[0]);
  if (!c.ok || (x->dim() != 2 && x->dim() != 3)) Py_RETURN_NONE;
  const bool lead = x->dim() == 3;
  const int64_t batch = lead ? x->size(0) : 1, rows = x->size(-2), K = x->size(-1);
  const int dt = dtype_code(x->scalar_type());
  if (dt < 0 || !fits_int(batch) || !fits_int(rows) || !fits_int(K) || K == 0 || K % 32 != 0)
    Py_RETURN_NONE;
  Tensor codes = lead ? c.make({batch, rows, K / 2}, at::kByte) : c.make({rows, K / 2}, at::kByte);
  Tensor scales = lead ? c.make({batch, tiles(rows), tiles(K), 512}, at::kByte)
                       : c.make({tiles(rows), tiles(K), 512}, at::kByte);
  const int rc = c.run(
      mm_mxfp4_quantize, x->data_ptr(), dt, (int)batch, (int)rows, (int)K,
      static_cast<uint8_t*>(codes.data_ptr()), static_cast<uint8_t*>(scales.data_ptr()),
      c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  PyObject* r = PyTuple_New(2);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrap(std::move(codes)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(scales)));
  return r;
  MARSHAL_END
}

// (codes, scales, dtype code) -> values
PyObject* mxfp4_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 3) Py_RETURN_NONE;
  Call c;
  const Tensor* codes = c.take(a[0], at::kByte);
  const Tensor* scales = c.take(a[1], at::kByte);
  const long dt = integer(a[2], c.ok);
  if (!c.ok || dt > 2 || (codes->dim() != 2 && codes->dim() != 3)) Py_RETURN_NONE;
  const bool lead = codes->dim() == 3;
  const int64_t batch = lead ? codes->size(0) : 1, rows = codes->size(-2), K = 2 * codes->size(-1);
  if (!fits_int(batch) || !fits_int(rows) || !fits_int(K) ||
      !(lead ? shape_is(*scales, {batch, tiles(rows), tiles(K), 512})
             : shape_is(*scales, {tiles(rows), tiles(K), 512})))
    Py_RETURN_NONE;
  Tensor out = lead ? c.make({batch, rows, K}, dtype_of(dt)) : c.make({rows, K}, dtype_of(dt));
  const int rc = c.run(
      mm_mxfp4_dequantize, static_cast<const uint8_t*>(codes->data_ptr()),
      static_cast<const uint8_t*>(scales->data_ptr()), (int)batch, (int)rows, (int)K,
      out.data_ptr(), (int)dt, c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  return wrap(std::move(out));
  MARSHAL_END
}

// One 4-bit matrix (a leading dimension of 1 allowed) whose scales fit.
bool matrix(const Tensor& codes, const Tensor& scales, int64_t& rows, int64_t& K) {
  const int64_t d = codes.dim();
  if (d != 2 && !(d == 3 && codes.size(0) == 1)) return false;
  rows = codes.size(-2);
  K = 2 * codes.size(-1);
  return fits_int(rows) && fits_int(K) &&
         (shape_is(scales, {tiles(rows), tiles(K), 512}) ||
          shape_is(scales, {1, tiles(rows), tiles(K), 512}));
}

// (a, a_scales, b, b_scales, out dtype code) -> c
PyObject* mxfp4_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 5) Py_RETURN_NONE;
  Call c;
  const Tensor *x = c.take(a[0], at::kByte), *sx = c.take(a[1], at::kByte),
               *w = c.take(a[2], at::kByte), *sw = c.take(a[3], at::kByte);
  const long dt = integer(a[4], c.ok);
  int64_t M = 0, N = 0, K = 0, Kw = 0;
  if (!c.ok || dt > 1 || !matrix(*x, *sx, M, K) || !matrix(*w, *sw, N, Kw) || K != Kw)
    Py_RETURN_NONE;
  Tensor out = c.make({M, N}, dtype_of(dt));
  const int rc = c.run(
      mm_mxfp4_gemm, static_cast<const uint8_t*>(x->data_ptr()),
      static_cast<const uint8_t*>(sx->data_ptr()),
      static_cast<const uint8_t*>(w->data_ptr()), static_cast<const uint8_t*>(sw->data_ptr()),
      (int)M, (int)N, (int)K, out.data_ptr(), (int)dt, c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  return wrap(std::move(out));
  MARSHAL_END
}

// (hidden, ids, w, w_gate_up, scales, w_down, scales, out, workspace) -> out
PyObject* experts_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 9) Py_RETURN_NONE;
  Call c;
  const Tensor *x = c.take(a[0], at::kBFloat16), *ids = c.take(a[1], at::kInt),
               *w = c.take(a[2], at::kFloat), *gu = c.take(a[3], at::kByte),
               *sgu = c.take(a[4], at::kByte), *dn = c.take(a[5], at::kByte),
               *sdn = c.take(a[6], at::kByte), *given = c.take(a[7], at::kBFloat16, true),
               *space = c.take(a[8], at::kByte, true);
  if (!c.ok || x->dim() != 2 || ids->dim() != 2 || dn->dim() != 3) Py_RETURN_NONE;
  const int64_t T = x->size(0), H = x->size(1), k = ids->size(1), E = dn->size(0),
                I = 2 * dn->size(2);
  if (!fits_int(T) || !fits_int(H) || !fits_int(2 * E) || !fits_int(2 * I) || !fits_int(k) ||
      ids->size(0) != T || !shape_is(*w, {T, k}) || dn->size(1) != H ||
      !(shape_is(*gu, {2 * E, I, H / 2}) || shape_is(*gu, {E, 2 * I, H / 2})) ||
      !shape_is(*sgu, {2 * E, tiles(I), tiles(H), 512}) ||
      !shape_is(*sdn, {E, tiles(H), tiles(I), 512}) || (given && !shape_is(*given, {T, H})))
    Py_RETURN_NONE;
  const int64_t need =
      mm_moe_experts_mxfp4_workspace_size((int)T, (int)H, (int)E, (int)I, (int)k);
  if (need < 0) Py_RETURN_NONE;
  Tensor made, scratch;
  if (given == nullptr) made = c.make({T, H}, at::kBFloat16);
  if (space == nullptr) scratch = c.make({need}, at::kByte);
  const Tensor &out = given != nullptr ? *given : made, &ws = space != nullptr ? *space : scratch;
  const int rc = c.run(
      mm_moe_experts_mxfp4, static_cast<const uint16_t*>(x->data_ptr()),
      static_cast<const int32_t*>(ids->data_ptr()),
      static_cast<const float*>(w->data_ptr()), static_cast<const uint8_t*>(gu->data_ptr()),
      static_cast<const uint8_t*>(sgu->data_ptr()), static_cast<const uint8_t*>(dn->data_ptr()),
      static_cast<const uint8_t*>(sdn->data_ptr()), (int)T, (int)H, (int)E, (int)I, (int)k,
      static_cast<uint16_t*>(out.data_ptr()), ws.data_ptr(), (size_t)ws.numel(), c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  if (given != nullptr) {
    Py_INCREF(a[7]);
    return a[7];
  }
  return wrap(std::move(made));
  MARSHAL_END
}

// bf16 and fp16, the types of rows.
bool is_row_type(at::ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }

template <typename T>
T* ptr(const Tensor* t) {
  return t != nullptr ? static_cast<T*>(t->data_ptr()) : nullptr;
}
template <typename T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// A result: the given tensor (a reference to it for the caller) or a new one.
PyObject* result(PyObject* given, const Tensor* g, Tensor& made) {
  if (g == nullptr) return wrap(std::move(made));
  Py_INCREF(given);
  return given;
}

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* r = PyTuple_New(2);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, a);
  PyTuple_SET_ITEM(r, 1, b);
  return r;
}

PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// Results of one call: small ones (under 1 MB together, where an allocation takes
// longer than the kernel needs) out of one allocation, as in _lib.py.
struct Together {
  Call& c;
  Tensor bytes;
  int64_t at = 0;
  bool one;

  Together(Call& call, int64_t total) : c(call), one(total < (int64_t(1) << 20)) {
    if (one) bytes = c.make({total}, at::kByte);
  }
  Tensor make(at::IntArrayRef shape, at::ScalarType type) {
    return one ? c.part(bytes, at, shape, type) : c.make(shape, type);
  }
};

// (topk_ids, E, token_mask) -> (places, offsets)
PyObject* group_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 3) Py_RETURN_NONE;
  Call c;
  const Tensor* ids = c.take(a[0], at::kInt);
  const long E = integer(a[1], c.ok);
  const Tensor* mask = c.any(a[2], true);
  if (!c.ok || ids->dim() != 2) Py_RETURN_NONE;
  const int64_t T = ids->size(0), k = ids->size(1);
  if (!fits_int(T) || !fits_int(k) || !fits_int(E) ||
      (mask && (!shape_is(*mask, {T}) ||
                (mask->scalar_type() != at::kBool && mask->scalar_type() != at::kByte))))
    Py_RETURN_NONE;
  const int64_t need = mm_group_slots_workspace_size((int)T, (int)k, (int)E);
  if (need < 0) Py_RETURN_NONE;
  Together both(c, round256(4 * T * k) + round256(4 * (E + 1)));
  Tensor places = both.make({T, k}, at::kInt), offsets = both.make({E + 1}, at::kInt), ws;
  if (need > 0) ws = c.make({need}, at::kByte);
  const int rc = c.run(mm_group_slots, ptr<const int32_t>(ids), ptr<const uint8_t>(mask), (int)T,
                       (int)k, (int)E, ptr<int32_t>(places), ptr<int32_t>(offsets),
                       need > 0 ? ws.data_ptr() : nullptr, (size_t)need, c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  return pair(wrap(std::move(places)), wrap(std::move(offsets)));
  MARSHAL_END
}

// (x, places, w, rows, row_w) -> (rows, row_w)
PyObject* dispatch_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 5) Py_RETURN_NONE;
  Call c;
  const Tensor *x = c.any(a[0]), *places = c.take(a[1], at::kInt),
               *w = c.take(a[2], at::kFloat, true), *rows = c.any(a[3], true),
               *row_w = c.take(a[4], at::kFloat, true);
  if (!c.ok || x->dim() != 2 || places->dim() != 2 || !is_row_type(x->scalar_type()))
    Py_RETURN_NONE;
  const int64_t T = x->size(0), H = x->size(1), k = places->size(1);
  if (places->size(0) != T || (w && !shape_is(*w, {T, k})) || (row_w && !w) ||
      (rows && (rows->dim() != 2 || rows->size(1) != H ||
                rows->scalar_type() != x->scalar_type())))
    Py_RETURN_NONE;
  const int64_t R = rows ? rows->size(0) : T * k;
  if (!fits_int(T) || !fits_int(H) || !fits_int(k) || !fits_int(R) ||
      (row_w && !shape_is(*row_w, {R})))
    Py_RETURN_NONE;
  Tensor new_rows, new_w;
  if (rows == nullptr) new_rows = c.make({R, H}, x->scalar_type());
  if (w != nullptr && row_w == nullptr) new_w = c.make({R}, at::kFloat);
  const int rc = c.run(mm_dispatch_rows, ptr<const void>(x), dtype_code(x->scalar_type()),
                       ptr<const int32_t>(places), ptr<const float>(w), (int)T, (int)k, (int)H,
                       (int)R, rows ? ptr<void>(rows) : ptr<void>(new_rows),
                       w == nullptr ? nullptr : row_w ? ptr<float>(row_w) : ptr<float>(new_w),
                       c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  return pair(result(a[3], rows, new_rows), w == nullptr ? none() : result(a[4], row_w, new_w));
  MARSHAL_END
}

// (rows, places, w, row_values, out) -> out, or (out, values) with row_values
PyObject* combine_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 5) Py_RETURN_NONE;
  Call c;
  const Tensor *rows = c.any(a[0]), *places = c.take(a[1], at::kInt),
               *w = c.take(a[2], at::kFloat, true), *vals = c.take(a[3], at::kFloat, true),
               *out = c.any(a[4], true);
  if (!c.ok || rows->dim() != 2 || places->dim() != 2 || !is_row_type(rows->scalar_type()))
    Py_RETURN_NONE;
  const int64_t R = rows->size(0), H = rows->size(1), T = places->size(0), k = places->size(1);
  if (!fits_int(T) || !fits_int(H) || !fits_int(k) || !fits_int(R) ||
      (w && !shape_is(*w, {T, k})) || (vals && !shape_is(*vals, {R})) ||
      (out && (!shape_is(*out, {T, H}) || out->scalar_type() != rows->scalar_type())))
    Py_RETURN_NONE;
  Tensor new_out, values;
  if (out == nullptr) new_out = c.make({T, H}, rows->scalar_type());
  if (vals != nullptr) values = c.make({T, k}, at::kFloat);
  const int rc = c.run(mm_combine_rows, ptr<const void>(rows), dtype_code(rows->scalar_type()),
                       ptr<const int32_t>(places), ptr<const float>(w), ptr<const float>(vals),
                       (int)T, (int)k, (int)H, (int)R, out ? ptr<void>(out) : ptr<void>(new_out),
                       vals ? ptr<float>(values) : nullptr, c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  PyObject* r = result(a[4], out, new_out);
  return vals ? pair(r, wrap(std::move(values))) : r;
  MARSHAL_END
}

// (x, w, offsets, out, transposed) -> out
PyObject* grouped_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 5) Py_RETURN_NONE;
  Call c;
  const Tensor *x = c.any(a[0]), *w = c.any(a[1]), *off = c.take(a[2], at::kInt),
               *out = c.any(a[3], true);
  const bool tr = a[4] == Py_True;
  if (!c.ok || x->dim() != 2 || w->dim() != 3 || !is_row_type(x->scalar_type()) ||
      w->scalar_type() != x->scalar_type())
    Py_RETURN_NONE;
  const int64_t R = x->size(0), E = w->size(0), N = w->size(1), K = w->size(2), M = tr ? K : N;
  if (!fits_int(R) || !fits_int(E) || !fits_int(N) || !fits_int(K) ||
      x->size(1) != (tr ? N : K) || !shape_is(*off, {E + 1}) ||
      (out && (!shape_is(*out, {R, M}) || out->scalar_type() != x->scalar_type())))
    Py_RETURN_NONE;
  Tensor made;
  if (out == nullptr) made = c.make({R, M}, x->scalar_type());
  const int rc = c.run(tr ? mm_grouped_product_dx : mm_grouped_product, ptr<const void>(x),
                       ptr<const void>(w), dtype_code(x->scalar_type()), ptr<const int32_t>(off),
                       (int)R, (int)E, (int)N, (int)K, out ? ptr<void>(out) : ptr<void>(made),
                       c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  return result(a[3], out, made);
  MARSHAL_END
}

// (dy, x, offsets, out, dtype code of the result, accumulate) -> out
PyObject* grouped_product_dw(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 6) Py_RETURN_NONE;
  Call c;
  const Tensor *dy = c.any(a[0]), *x = c.any(a[1]), *off = c.take(a[2], at::kInt),
               *out = c.any(a[3], true);
  const long dt = integer(a[4], c.ok);
  const int add = PyObject_IsTrue(a[5]);
  if (add < 0) PyErr_Clear();
  if (!c.ok || dt > 2 || dy->dim() != 2 || x->dim() != 2 || off->dim() != 1 ||
      !is_row_type(dy->scalar_type()) || x->scalar_type() != dy->scalar_type() || add < 0 ||
      (add && !out))
    Py_RETURN_NONE;
  const int64_t R = dy->size(0), N = dy->size(1), K = x->size(1), E = off->size(0) - 1;
  const at::ScalarType type = dtype_of(dt);
  if (!fits_int(R) || !fits_int(E) || !fits_int(N) || !fits_int(K) || x->size(0) != R || E < 1 ||
      (type != at::kFloat && type != dy->scalar_type()) ||
      (out && (!shape_is(*out, {E, N, K}) || out->scalar_type() != type)))
    Py_RETURN_NONE;
  const int64_t need =
      mm_grouped_product_dw_workspace_size((int)R, (int)E, (int)N, (int)K, (int)dt);
  if (need < 0) Py_RETURN_NONE;
  Tensor made, ws;
  if (out == nullptr) made = c.make({E, N, K}, type);
  if (need > 0) ws = c.make({need}, at::kByte);
  const int rc = c.run(mm_grouped_product_dw, ptr<const void>(dy), ptr<const void>(x),
                       dtype_code(dy->scalar_type()), ptr<const int32_t>(off), (int)R, (int)E,
                       (int)N, (int)K, out ? ptr<void>(out) : ptr<void>(made), (int)dt, add,
                       need > 0 ? ws.data_ptr() : nullptr, (size_t)need, c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  return result(a[3], out, made);
  MARSHAL_END
}

// The address of the number of rows in use, the last of `offsets`.
const int32_t* rows_end(const Tensor* offsets, bool& ok) {
  if (offsets == nullptr) return nullptr;
  if (offsets->dim() != 1 || offsets->size(0) == 0) {
    ok = false;
    return nullptr;
  }
  return ptr<const int32_t>(offsets) + offsets->size(0) - 1;
}

// (z, offsets) -> (act, codes, scales)
PyObject* swiglu_pack(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 2) Py_RETURN_NONE;
  Call c;
  const Tensor *z = c.any(a[0]), *off = c.take(a[1], at::kInt, true);
  if (!c.ok || z->dim() != 2 || !is_row_type(z->scalar_type())) Py_RETURN_NONE;
  const int64_t R = z->size(0), C = z->size(1);
  const int32_t* end = rows_end(off, c.ok);
  if (!c.ok || !fits_int(R) || !fits_int(C) || C == 0 || C % 64 != 0) Py_RETURN_NONE;
  Together all(c, 2 * round256(R * C) + round256(R * (C / 32)));
  Tensor act = all.make({R, C / 2}, z->scalar_type()), codes = all.make({R, C}, at::kChar),
         scales = all.make({R, C / 32}, at::kByte);
  const int rc = c.run(mm_swiglu_pack, ptr<const void>(z), dtype_code(z->scalar_type()), end,
                       (int)R, (int)(C / 2), ptr<void>(act), ptr<int8_t>(codes),
                       ptr<uint8_t>(scales), c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  PyObject* r = PyTuple_New(3);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrap(std::move(act)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(codes)));
  PyTuple_SET_ITEM(r, 2, wrap(std::move(scales)));
  return r;
  MARSHAL_END
}

// (codes, scales, d_act, row_w, offsets) -> (dz, act, d_row_w or None)
PyObject* swiglu_pack_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 5) Py_RETURN_NONE;
  Call c;
  const Tensor *codes = c.take(a[0], at::kChar), *scales = c.take(a[1], at::kByte),
               *da = c.any(a[2]), *w = c.take(a[3], at::kFloat, true),
               *off = c.take(a[4], at::kInt, true);
  if (!c.ok || da->dim() != 2 || !is_row_type(da->scalar_type())) Py_RETURN_NONE;
  const int64_t R = da->size(0), I = da->size(1);
  const int32_t* end = rows_end(off, c.ok);
  if (!c.ok || !fits_int(R) || !fits_int(2 * I) || I == 0 || I % 32 != 0 ||
      !shape_is(*codes, {R, 2 * I}) || !shape_is(*scales, {R, I / 16}) || (w && !shape_is(*w, {R})))
    Py_RETURN_NONE;
  Together all(c, round256(4 * R * I) + round256(2 * R * I) + (w ? round256(4 * R) : 0));
  Tensor dz = all.make({R, 2 * I}, da->scalar_type()), act = all.make({R, I}, da->scalar_type()),
         dw;
  if (w != nullptr) dw = all.make({R}, at::kFloat);
  const int rc = c.run(mm_swiglu_pack_backward, ptr<const int8_t>(codes),
                       ptr<const uint8_t>(scales), ptr<const void>(da),
                       dtype_code(da->scalar_type()), ptr<const float>(w), end, (int)R, (int)I,
                       ptr<void>(dz), ptr<void>(act), w ? ptr<float>(dw) : nullptr, c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  PyObject* r = PyTuple_New(3);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrap(std::move(dz)));
  PyTuple_SET_ITEM(r, 1, wrap(std::move(act)));
  PyTuple_SET_ITEM(r, 2, w ? wrap(std::move(dw)) : none());
  return r;
  MARSHAL_END
}

// (codes, scales, dtype code) -> values
PyObject* mxint8_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MARSHAL_BEGIN
  if (n != 3) Py_RETURN_NONE;
  Call c;
  const Tensor *codes = c.take(a[0], at::kChar), *scales = c.take(a[1], at::kByte);
  const long dt = integer(a[2], c.ok);
  if (!c.ok || dt > 2 || codes->dim() != 2) Py_RETURN_NONE;
  const int64_t rows = codes->size(0), K = codes->size(1);
  if (!fits_int(rows) || !fits_int(K) || K == 0 || K % 32 != 0 ||
      !shape_is(*scales, {rows, K / 32}))
    Py_RETURN_NONE;
  Tensor out = c.make({rows, K}, dtype_of(dt));
  const int rc = c.run(mm_mxint8_dequantize, ptr<const int8_t>(codes), ptr<const uint8_t>(scales),
                       (int)rows, (int)K, ptr<void>(out), (int)dt, c.stream());
  if (rc != MM_OK) Py_RETURN_NONE;
  return wrap(std::move(out));
  MARSHAL_END
}

#define MARSHAL_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {MARSHAL_METHOD(route_logits),
                         MARSHAL_METHOD(route_logits_backward),
                         MARSHAL_METHOD(mxfp4_quantize),
                         MARSHAL_METHOD(mxfp4_dequantize),
                         MARSHAL_METHOD(mxfp4_gemm),
                         MARSHAL_METHOD(experts_mxfp4),
                         MARSHAL_METHOD(group_slots),
                         MARSHAL_METHOD(dispatch_rows),
                         MARSHAL_METHOD(combine_rows),
                         MARSHAL_METHOD(grouped_product),
                         MARSHAL_METHOD(grouped_product_dw),
                         MARSHAL_METHOD(swiglu_pack),
                         MARSHAL_METHOD(swiglu_pack_backward),
                         MARSHAL_METHOD(mxint8_dequantize),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// MARSHAL_TAG: a digest of this file, the C ABI and the torch and Python it was
// compiled for. The binding uses the module where it would be built from the same.
PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "tag", MARSHAL_TAG) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
