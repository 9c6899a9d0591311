// The Python calls of the 4-bit operators and of the norm: checks of the tensors,
// results, device, stream, and the library's entry point.  Compiled, because a small
// call is bound by this: a product of one row takes 4.4 us a call in place of 7.6 through
// ctypes, 3.2 of them the launch and 0.65 the result.  The entry points come from
// binding.py (bind), so that there is one library in a process, and so do the parts of a
// call that are not the ordinary ones: results on a stream that is not the current one,
// and the exception for a status.
#include <Python.h>

#include <algorithm>
#include <cstring>
#include <initializer_list>
#include <utility>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty_strided.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

struct {
  decltype(&moe_quant_mxfp4) quant_mxfp4, silu_mul_quant_mxfp4;
  decltype(&moe_dequant_mxfp4) dequant_mxfp4;
  decltype(&moe_gemm_mxfp4) gemm_mxfp4;
  decltype(&moe_add_rms_norm) add_rms_norm;
  decltype(&moe_add_rms_norm_quant_fp8) add_rms_norm_quant_fp8;
} entry;
PyObject *raw_stream_of, *empty_on, *check_status;

// A check that failed, or a call of Python: its exception is set.
struct Refused {};
template <typename... A>
[[noreturn]] void refuse(const char* format, A... args) {
  PyErr_Format(PyExc_ValueError, format, args...);
  throw Refused();
}
// A reference of our own; null: Python's exception is set.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {
    if (p == nullptr) throw Refused();
  }
  Ref(const Ref&) = delete;
  ~Ref() { Py_DECREF(p); }
};

enum class Types { kBytes, kMxScales, kCodes, kF32, kBf16, kFloats };

bool among(at::ScalarType t, Types types) {
  switch (types) {
    case Types::kBytes: return t == at::kByte;
    case Types::kMxScales: return t == at::kByte || t == at::kFloat8_e8m0fnu;
    case Types::kCodes: return t == at::kByte || t == at::kFloat8_e4m3fn;
    case Types::kF32: return t == at::kFloat;
    case Types::kBf16: return t == at::kBFloat16;
    default: return t == at::kFloat || t == at::kBFloat16;
  }
}
const char* names_of(Types types) {
  switch (types) {
    case Types::kBytes: return "torch.uint8";
    case Types::kMxScales: return "torch.uint8 or torch.float8_e8m0fnu";
    case Types::kCodes: return "torch.uint8 or torch.float8_e4m3fn";
    case Types::kF32: return "torch.float32";
    case Types::kBf16: return "torch.bfloat16";
    default: return "torch.float32 or torch.bfloat16";
  }
}
int32_t dtype_code(at::ScalarType t) { return t == at::kBFloat16 ? MOE_BF16 : MOE_F32; }

const at::Tensor& tensor(PyObject* t, const char* name) {
  if (!THPVariable_Check(t)) {
    PyErr_Format(PyExc_TypeError, "%s: a tensor expected, not %S", name, (PyObject*)Py_TYPE(t));
    throw Refused();
  }
  return THPVariable_Unpack(t);
}
// "torch.uint8 (3, 5)"
PyObject* type_and_shape(PyObject* t) {
  const Ref shape(PyObject_GetAttrString(t, "shape"));
  const Ref sizes(PySequence_Tuple(shape.p)), dtype(PyObject_GetAttrString(t, "dtype"));
  return PyUnicode_FromFormat("%S %S", dtype.p, sizes.p);
}

// The rows and columns of a matrix of `multiple` n columns.
std::pair<int64_t, int64_t> matrix_sizes(PyObject* obj, const char* name, int64_t multiple) {
  const at::Tensor& t = tensor(obj, name);
  if (t.dim() != 2 || t.size(1) % multiple != 0)
    refuse("%s: a matrix of %lld n columns expected, not %S", name, (long long)multiple,
           Ref(type_and_shape(obj)).p);
  // (the descriptors hold 32 bits)
  if (std::max(t.size(0), t.size(1)) > INT32_MAX)
    refuse("%s: sizes (%lld, %lld), less than 2^31 expected", name, (long long)t.size(0), (long long)t.size(1));
  return {t.size(0), t.size(1)};
}

at::ScalarType float_type(PyObject* dtype) {
  if (THPDtype_Check(dtype))
    if (const auto t = reinterpret_cast<THPDtype*>(dtype)->scalar_type; among(t, Types::kFloats)) return t;
  refuse("out_dtype %S: float32 or bfloat16 expected", dtype);
}

// The storage of one result among several in one allocation, the room: it begins where the
// room does and ends with the result, so that a result that grows gets memory of its own, as
// any tensor does, and leaves the ones behind it.  The room lives as long as one of its
// storages.  The pointer frees nothing and carries the allocator's deleter, by which
// record_stream knows the allocator's own blocks.
struct Share final : c10::StorageImpl {
  Share(const c10::Storage& room, int64_t end)
      : StorageImpl(use_byte_size_t(), (size_t)end,
                    at::DataPtr(room.mutable_data(), nullptr, room.data_ptr().get_deleter(), room.device()),
                    room.allocator(), /*resizable=*/true),
        room_(room) {}
  ~Share() override { let_go(); }
  void release_resources() override {
    let_go();
    StorageImpl::release_resources();
  }

 private:
  void let_go() {
    // Handed to another process (torch has put its own count of readers in the pointer's
    // place, which does not know of the room): the other side may read it still, so it stays.
    if (room_ && data_ptr().get() == room_.data() && data_ptr().get_deleter() != room_.data_ptr().get_deleter())
      (void)c10::Storage(room_).unsafeReleaseStorageImpl();
    room_ = c10::Storage();
  }
  c10::Storage room_;
};

// What all tensors of a call share.
struct Call {
  explicit Call(PyObject* stream) : stream_(stream) {}

  // rows x cols with contiguous rows; ld: their stride (0: dense, or one row, whose
  // stride says nothing)
  const at::Tensor& matrix(PyObject* obj, const char* name, Types types, int64_t rows, int64_t cols, int64_t* ld) {
    const at::Tensor& t = tensor(obj, name);
    if (!among(t.scalar_type(), types) || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
      refuse("%s: %S, expected %s (%lld, %lld)", name, Ref(type_and_shape(obj)).p, names_of(types),
             (long long)rows, (long long)cols);
    *ld = 0;
    if (!t.is_contiguous()) {
      if (t.stride(1) != 1 && cols > 1) refuse("%s must have contiguous rows", name);
      if (rows != 1) {
        *ld = t.stride(0);
        if (*ld < cols) refuse("%s has rows that overlap (stride %lld)", name, (long long)*ld);
      }
    }
    on_device(t);
    return t;
  }
  void on_device(const at::Tensor& t) {
    if (!t.is_cuda()) {
      off_gpu_ = true;   // (said behind what is wrong with the tensors themselves)
      return;
    }
    const int d = t.get_device();
    if (device_ >= 0 && d != device_) refuse("tensors on cuda:%d and cuda:%d: one GPU expected", device_, d);
    device_ = d;
  }

  // Results of these bytes (0: given) in one allocation, up to 1 MB in all: an allocation
  // costs 0.65 us of a call, a tensor in one that is there 0.25.  Larger ones apart, so that
  // a result that is kept keeps no other one's memory.
  void together(std::initializer_list<int64_t> bytes) {
    int count = 0;
    int64_t all = 0;
    for (const int64_t n : bytes) count += n > 0, all += whole(n);
    if (count > 1 && all <= (1 << 20) && stream_ == Py_None && !off_gpu_)
      room_ = at::empty_strided({all}, {1}, on_gpu(at::kByte));
  }
  // A result that is written on the call's stream (its memory is reused in that
  // stream's order).
  at::Tensor empty(int64_t rows, int64_t cols, at::ScalarType dtype) {
    all_on_gpu();
    const int64_t size[2] = {rows, cols}, stride[2] = {cols, 1};
    if (room_.defined()) {
      const auto type = c10::scalarTypeToTypeMeta(dtype);
      const int64_t bytes = rows * cols * (int64_t)type.itemsize();
      at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
          c10::Storage(c10::make_intrusive<Share>(room_.storage(), taken_ + bytes)), room_.key_set(), type);
      t.unsafeGetTensorImpl()->set_storage_offset(taken_ / (int64_t)type.itemsize());
      t.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(size, 2), at::IntArrayRef(stride, 2));
      taken_ += whole(bytes);
      return t;
    }
    if (stream_ == Py_None)
      return at::empty_strided(at::IntArrayRef(size, 2), at::IntArrayRef(stride, 2), on_gpu(dtype));
    const Ref t(PyObject_CallFunction(empty_on, "(LL)OiO", (long long)rows, (long long)cols,
                                      reinterpret_cast<PyObject*>(torch::getTHPDtype(dtype)), device_, stream_));
    return tensor(t.p, "result");
  }
  // `given`, or a new one
  at::Tensor result(PyObject* given, const char* name, Types types, int64_t rows, int64_t cols, at::ScalarType dtype,
                    int64_t* ld) {
    *ld = 0;
    return given == Py_None ? empty(rows, cols, dtype) : matrix(given, name, types, rows, cols, ld);
  }

  // The entry point with that GPU current, on the given stream or its current one.
  template <typename F>
  void enqueue(F&& launch) const {
    all_on_gpu();
    void* stream;
    if (stream_ == Py_None) {
      const Ref index(PyLong_FromLong(device_));
      stream = PyLong_AsVoidPtr(Ref(PyObject_CallOneArg(raw_stream_of, index.p)).p);
    } else {
      const long at = PyLong_AsLong(Ref(PyObject_GetAttrString(stream_, "device_index")).p);
      if (at != device_ && !PyErr_Occurred()) refuse("stream on cuda:%ld, tensors on cuda:%d", at, device_);
      stream = PyLong_AsVoidPtr(Ref(PyObject_GetAttrString(stream_, "cuda_stream")).p);
    }
    if (PyErr_Occurred()) throw Refused();
    int status;
    {
      const c10::DeviceGuard guard(at::Device(at::kCUDA, (at::DeviceIndex)device_));
      Py_BEGIN_ALLOW_THREADS
      status = launch(stream);
      Py_END_ALLOW_THREADS
    }
    if (status != MOE_OK) {
      const Ref raised(PyObject_CallFunction(check_status, "i", status));
      refuse("status %d", status);
    }
  }

 private:
  void all_on_gpu() const {
    if (off_gpu_) refuse("tensors must be on the GPU");
  }
  at::TensorOptions on_gpu(at::ScalarType dtype) const {
    return at::TensorOptions().dtype(dtype).device(at::kCUDA, (at::DeviceIndex)device_);
  }
  static int64_t whole(int64_t bytes) { return (bytes + 255) / 256 * 256; }
  PyObject* stream_;
  bool off_gpu_ = false;
  int device_ = -1;
  at::Tensor room_;     // of `together`, of which the first bytes are taken
  int64_t taken_ = 0;
};
// The bytes of a result that is not given.
int64_t wanted(PyObject* given, int64_t rows, int64_t cols, int64_t size) {
  return given == Py_None ? rows * cols * size : 0;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  const Ref x(THPVariable_Wrap(a)), y(THPVariable_Wrap(b));
  return PyTuple_Pack(2, x.p, y.p);
}

// Every call: no exception leaves it, and its number of arguments is what its function
// in binding.py hands on.
template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != N) refuse("%zd arguments expected", N);
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (x, codes, scales, stream)
template <bool SILU>
PyObject* quant_mxfp4(PyObject* const* a) {
  const auto [M, n] = matrix_sizes(a[0], "input", SILU ? 64 : 32);
  const int64_t K = SILU ? n / 2 : n;
  Call c(a[3]);
  moe_quant_desc d{(int32_t)M, (int32_t)K};
  const at::Tensor& x = c.matrix(a[0], "input", Types::kFloats, M, n, &d.ld_in);
  c.together({wanted(a[1], M, K / 2, 1), wanted(a[2], M, K / 32, 1)});
  const at::Tensor codes = c.result(a[1], "codes", Types::kBytes, M, K / 2, at::kByte, &d.ld_codes);
  const at::Tensor scales = c.result(a[2], "scales", Types::kMxScales, M, K / 32, at::kByte, &d.ld_scales);
  d.in_dtype = dtype_code(x.scalar_type());
  c.enqueue([&](void* stream) {
    return (SILU ? entry.silu_mul_quant_mxfp4 : entry.quant_mxfp4)(
        &d, x.const_data_ptr(), codes.mutable_data_ptr(), scales.mutable_data_ptr(), stream);
  });
  return pair(codes, scales);
}

// (codes, scales, out, out_dtype, stream)
PyObject* dequant_mxfp4(PyObject* const* a) {
  const auto [M, half] = matrix_sizes(a[0], "codes", 16);
  const int64_t K = 2 * half;
  if (K > INT32_MAX) refuse("%lld columns, less than 2^31 expected", (long long)K);
  Call c(a[4]);
  moe_quant_desc d{(int32_t)M, (int32_t)K};
  const at::Tensor& codes = c.matrix(a[0], "codes", Types::kBytes, M, half, &d.ld_codes);
  const at::Tensor& scales = c.matrix(a[1], "scales", Types::kMxScales, M, K / 32, &d.ld_scales);
  const at::Tensor out = c.result(a[2], "out", Types::kFloats, M, K, a[2] == Py_None ? float_type(a[3]) : at::kFloat,
                                  &d.ld_in);
  d.in_dtype = dtype_code(out.scalar_type());
  c.enqueue([&](void* stream) {
    return entry.dequant_mxfp4(&d, codes.const_data_ptr(), scales.const_data_ptr(), out.mutable_data_ptr(), stream);
  });
  return THPVariable_Wrap(out);
}

// (a, a_scale, b, b_scale, out, out_dtype, stream)
PyObject* gemm_mxfp4(PyObject* const* a) {
  const auto [M, half] = matrix_sizes(a[0], "a", 1);
  const auto [N, width] = matrix_sizes(a[2], "b", 1);
  const int64_t K = 2 * half;
  if (K > INT32_MAX) refuse("%lld columns, less than 2^31 expected", (long long)K);
  Call c(a[6]);
  moe_mx_gemm_desc d{(int32_t)M, (int32_t)N, (int32_t)K};
  const at::Tensor& x = c.matrix(a[0], "a", Types::kBytes, M, half, &d.lda);
  const at::Tensor& w = c.matrix(a[2], "b", Types::kBytes, N, half, &d.ldb);
  const at::Tensor& xs = c.matrix(a[1], "a_scale", Types::kMxScales, M, K / 32, &d.ld_as);
  const at::Tensor& ws = c.matrix(a[3], "b_scale", Types::kMxScales, N, K / 32, &d.ld_bs);
  const at::Tensor out = c.result(a[4], "out", Types::kFloats, M, N, a[4] == Py_None ? float_type(a[5]) : at::kFloat,
                                  &d.ldo);
  d.out_dtype = dtype_code(out.scalar_type());
  c.enqueue([&](void* stream) {
    return entry.gemm_mxfp4(&d, x.const_data_ptr(), xs.const_data_ptr(), w.const_data_ptr(), ws.const_data_ptr(),
                            out.mutable_data_ptr(), stream);
  });
  return THPVariable_Wrap(out);
}

// What both norms take: x, residual (None: absent), weight, eps and residual_out.
struct Norm {
  Call c;
  moe_norm_desc d{};
  const at::Tensor *x, *res = nullptr, *w;
  at::Tensor kept;   // residual_out
  // others: the other results' bytes, of the rows and columns
  template <typename F>
  Norm(PyObject* x_obj, PyObject* residual, PyObject* weight, PyObject* eps, PyObject* residual_out, PyObject* stream,
       F&& others)
      : c(stream) {
    const auto [M, H] = matrix_sizes(x_obj, "x", 1);
    d.rows = (int32_t)M;
    d.cols = (int32_t)H;
    d.eps = (float)PyFloat_AsDouble(eps);
    if (PyErr_Occurred()) throw Refused();
    x = &c.matrix(x_obj, "x", Types::kFloats, M, H, &d.ld_x);
    d.x_dtype = dtype_code(x->scalar_type());
    w = &tensor(weight, "weight");
    if (!among(w->scalar_type(), Types::kFloats) || w->dim() != 1 || w->size(0) != H || !w->is_contiguous())
      refuse("weight: %S, expected contiguous torch.float32 or torch.bfloat16 (%lld,)",
             Ref(type_and_shape(weight)).p, (long long)H);
    c.on_device(*w);
    d.w_dtype = dtype_code(w->scalar_type());
    const std::pair<int64_t, int64_t> more = others(M, H);
    if (residual == Py_None) {
      if (residual_out != Py_None) refuse("residual_out without a residual");
      c.together({more.first, more.second});
      return;
    }
    res = &c.matrix(residual, "residual", Types::kFloats, M, H, &d.ld_res);
    const auto type = res->scalar_type();
    c.together({wanted(residual_out, M, H, type == at::kFloat ? 4 : 2), more.first, more.second});
    kept = c.result(residual_out, "residual_out", type == at::kFloat ? Types::kF32 : Types::kBf16, M, H, type,
                    &d.ld_res_out);
    d.res_dtype = dtype_code(type);
  }
  const void* residual() const { return res ? res->const_data_ptr() : nullptr; }
  void* residual_out() const { return res ? kept.mutable_data_ptr() : nullptr; }
  PyObject* wrapped_residual_out() const { return res ? THPVariable_Wrap(kept) : Py_NewRef(Py_None); }
};

// (x, residual, weight, eps, out, residual_out, out_dtype, stream)
PyObject* add_rms_norm(PyObject* const* a) {
  const at::ScalarType type = a[4] == Py_None ? float_type(a[6]) : at::kFloat;
  Norm n(a[0], a[1], a[2], a[3], a[5], a[7], [&](int64_t M, int64_t H) {
    return std::pair(wanted(a[4], M, H, type == at::kFloat ? 4 : 2), (int64_t)0);
  });
  const at::Tensor out = n.c.result(a[4], "out", Types::kFloats, n.d.rows, n.d.cols, type, &n.d.ld_out);
  n.d.out_dtype = dtype_code(out.scalar_type());
  n.c.enqueue([&](void* stream) {
    return entry.add_rms_norm(&n.d, n.x->const_data_ptr(), n.residual(), n.w->const_data_ptr(), n.residual_out(),
                              out.mutable_data_ptr(), stream);
  });
  const Ref first(THPVariable_Wrap(out)), second(n.wrapped_residual_out());
  return PyTuple_Pack(2, first.p, second.p);
}

// (x, residual, weight, eps, codes, scales, residual_out, out, stream)
PyObject* add_rms_norm_quant_fp8(PyObject* const* a) {
  Norm n(a[0], a[1], a[2], a[3], a[6], a[8], [&](int64_t M, int64_t H) {
    return std::pair(wanted(a[4], M, H, 1), wanted(a[5], M, (H + 127) / 128, 4));
  });
  const int64_t M = n.d.rows, H = n.d.cols;
  const at::Tensor codes = n.c.result(a[4], "codes", Types::kCodes, M, H, at::kByte, &n.d.ld_codes);
  const at::Tensor scales = n.c.result(a[5], "scales", Types::kF32, M, (H + 127) / 128, at::kFloat, &n.d.ld_scales);
  const at::Tensor* out = nullptr;
  if (a[7] != Py_None) {
    out = &n.c.matrix(a[7], "out", Types::kFloats, M, H, &n.d.ld_out);
    n.d.out_dtype = dtype_code(out->scalar_type());
  }
  n.c.enqueue([&](void* stream) {
    return entry.add_rms_norm_quant_fp8(&n.d, n.x->const_data_ptr(), n.residual(), n.w->const_data_ptr(),
                                        n.residual_out(), out ? out->mutable_data_ptr() : nullptr,
                                        codes.mutable_data_ptr(), static_cast<float*>(scales.mutable_data_ptr()),
                                        stream);
  });
  const Ref first(THPVariable_Wrap(codes)), second(THPVariable_Wrap(scales)), third(n.wrapped_residual_out());
  return PyTuple_Pack(3, first.p, second.p, third.p);
}

// (addresses of the six entry points in the order of `entry`, raw stream of a device,
// new tensor on a stream, exception for a status)
PyObject* bind(PyObject* const* a) {
  void* at[6];
  for (int i = 0; i < 6; ++i) at[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) throw Refused();
  static_assert(sizeof(entry) == sizeof(at));
  std::memcpy(&entry, at, sizeof(at));
  raw_stream_of = Py_NewRef(a[6]);
  empty_on = Py_NewRef(a[7]);
  check_status = Py_NewRef(a[8]);
  Py_RETURN_NONE;
}

template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<N, F>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {
    method<9, bind>("bind"),
    method<4, quant_mxfp4<false>>("quant_mxfp4"),
    method<4, quant_mxfp4<true>>("silu_mul_quant_mxfp4"),
    method<5, dequant_mxfp4>("dequant_mxfp4"),
    method<7, gemm_mxfp4>("gemm_mxfp4"),
    method<8, add_rms_norm>("add_rms_norm"),
    method<9, add_rms_norm_quant_fp8>("add_rms_norm_quant_fp8"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__moe_calls() { return PyModule_Create(&module); }
