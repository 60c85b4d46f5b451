// What the torch calls share: access to tensors and their checks, the stream of
// a call, its outputs.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <initializer_list>
#include <optional>

#include "fa_cache.h"

namespace {

[[noreturn]] void refuse(PyObject* type, const char* what) {
  PyErr_SetString(type, what);
  throw python_error();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %.100s", what, Py_TYPE(o)->tp_name);
    throw python_error();
  }
  return THPVariable_Unpack(o);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// An int argument of the C ABI.
int narrow(long long v, const char* what) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, what);
  return static_cast<int>(v);
}

int cuda_device(const at::Tensor& t) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "tensors must be on a CUDA device");
  return t.get_device();
}

bool on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// The address of a contiguous int32 tensor of shape [a] or [a, b] (b < 0: one axis) on `dev`.
int32_t* index(const at::Tensor& t, int dev, int64_t a, int64_t b, const char* what) {
  const bool shape = b < 0 ? t.dim() == 1 && t.size(0) == a
                           : t.dim() == 2 && t.size(0) == a && t.size(1) == b;
  if (!(t.scalar_type() == at::kInt && shape && on(t, dev) && t.is_contiguous())) {
    if (b < 0)
      PyErr_Format(PyExc_ValueError, "%s must be a contiguous int32 tensor [%lld] on CUDA device %d",
                   what, static_cast<long long>(a), dev);
    else
      PyErr_Format(PyExc_ValueError,
                   "%s must be a contiguous int32 tensor [%lld, %lld] on CUDA device %d", what,
                   static_cast<long long>(a), static_cast<long long>(b), dev);
    throw python_error();
  }
  return static_cast<int32_t*>(t.data_ptr());
}

fa_dtype dtype16(const at::Tensor& t) {
  if (t.scalar_type() == at::kHalf) return FA_DTYPE_FP16;
  if (t.scalar_type() == at::kBFloat16) return FA_DTYPE_BF16;
  refuse(PyExc_TypeError, "unsupported dtype (fp16 or bf16)");
}

// The stream of a call: the given torch.cuda.Stream, which tensors that the
// call creates are then allocated on, or the device's current one.
struct CallStream {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard given;
  cudaStream_t stream = nullptr;

  CallStream(PyObject* s, int dev) {
    if (s == Py_None) {
      device.set_index(static_cast<c10::DeviceIndex>(dev));
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
      return;
    }
    long long v[3];
    const char* names[3] = {"stream_id", "device_index", "device_type"};
    for (int i = 0; i < 3; ++i) {
      PyObject* o = PyObject_GetAttrString(s, names[i]);
      if (!o) throw python_error();
      v[i] = PyLong_AsLongLong(o);
      Py_DECREF(o);
      if (v[i] == -1 && PyErr_Occurred()) throw python_error();
    }
    if (v[1] != dev) refuse(PyExc_ValueError, "the stream is on another device than the tensors");
    const c10::cuda::CUDAStream cs = c10::cuda::CUDAStream::unpack3(
        v[0], static_cast<c10::DeviceIndex>(v[1]), static_cast<c10::DeviceType>(v[2]));
    given.reset_stream(cs);
    stream = cs.stream();
  }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::Tensor(at::detail::empty_cuda(
      shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
}

// A contiguous tensor of `shape` on the memory of `whole`, from element `from` on (of
// `type`, where that is another one than the whole's).
at::Tensor part(const at::Tensor& whole, int64_t from, at::IntArrayRef shape,
                at::ScalarType type) {
  auto t = c10::make_intrusive<at::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                               c10::scalarTypeToTypeMeta(type));
  t->set_storage_offset(from);
  t->set_sizes_contiguous(shape);
  return at::Tensor(std::move(t));
}
at::Tensor part(const at::Tensor& whole, int64_t from, int64_t n) {
  return part(whole, from, {n}, whole.scalar_type());
}

// A call has written to tensors of the caller's: autograd then refuses the backward pass of
// an operation that saved what they held before, as after torch's own in-place calls.
void wrote(std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts)
    if (t->defined() && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
void wrote_cache(PyObject* cache) {  // one that describe() has checked
  for (Py_ssize_t i = 0; i < 4; ++i) wrote({&THPVariable_Unpack(PyTuple_GET_ITEM(cache, i))});
}

PyObject* status(fa_status s) { return PyLong_FromLong(static_cast<long>(s)); }

// fa_cache of a (k, v, k_scales, v_scales) tuple on device `dev`.
fa_cache describe(PyObject* o, int dev) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4)
    refuse(PyExc_TypeError, "a cache is a tuple (k, v, k_scales, v_scales)");
  const at::Tensor& k = tensor(PyTuple_GET_ITEM(o, 0), "cache k");
  const at::Tensor& v = tensor(PyTuple_GET_ITEM(o, 1), "cache v");
  const at::Tensor& ks = tensor(PyTuple_GET_ITEM(o, 2), "cache k_scales");
  const at::Tensor& vs = tensor(PyTuple_GET_ITEM(o, 3), "cache v_scales");
  auto scales = [&](const at::Tensor& s) {
    return s.dim() == 2 && s.size(0) == k.size(0) && s.size(1) == k.size(1) &&
           s.scalar_type() == at::kFloat && s.is_contiguous();
  };
  auto codes = [](const at::Tensor& t) {
    return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte;
  };
  if (!(k.dim() == 4 && k.sizes() == v.sizes() && k.strides() == v.strides() && k.stride(3) == 1 &&
        codes(k) && codes(v) && scales(ks) && scales(vs)))
    refuse(PyExc_ValueError,
           "cache: k, v must be [blocks, heads, block, d] float8_e4m3fn or uint8 tensors of equal "
           "strides (1 along d) and k_scales, v_scales contiguous float32 [blocks, heads]");
  if (!(on(k, dev) && on(v, dev) && on(ks, dev) && on(vs, dev)))
    refuse(PyExc_ValueError, "cache: tensors must be on the same CUDA device as the other arguments");
  fa_cache c{};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.k_scales = static_cast<float*>(ks.data_ptr());
  c.v_scales = static_cast<float*>(vs.data_ptr());
  c.num_blocks = narrow(k.size(0), "cache: too many blocks");
  c.Hkv = narrow(k.size(1), "cache: too many heads");
  c.block = narrow(k.size(2), "cache: block too large");
  c.d = narrow(k.size(3), "cache: d too large");
  // an axis of length one has no stride of its own
  c.block_stride = c.num_blocks > 1 ? k.stride(0) : 16;
  c.head_stride = c.Hkv > 1 ? k.stride(1) : 16;
  c.token_stride = k.stride(2);
  return c;
}

void count_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "wrong number of arguments");
}

// The tensors as a tuple, None for one that is not there.
PyObject* tuple_of(std::initializer_list<const at::Tensor*> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o = Py_None;
    if (t != nullptr && t->defined()) o = THPVariable_Wrap(*t);
    else Py_INCREF(Py_None);
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

}  // namespace
