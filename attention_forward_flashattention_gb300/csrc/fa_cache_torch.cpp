// The block cache's calls on torch tensors: checks of shapes, types and
// devices, output allocation and the call into the C ABI (fa_cache.h). Host
// code only. A call of these costs a few microseconds of host time where the
// same marshalling in Python costs twenty, which a decoding step of short
// sequences would spend waiting.
//
// Functions return their tensors, or the fa_status of a failed call as an int.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
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

// Elements from .. from + n - 1 of `whole`, a tensor of one axis, on its memory.
at::Tensor part(const at::Tensor& whole, int64_t from, int64_t n) {
  auto t = c10::make_intrusive<at::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                               whole.dtype());
  t->set_storage_offset(from);
  t->set_sizes_contiguous({n});
  return at::Tensor(std::move(t));
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

// (lens, new_lens, block_table, free_blocks, free_pos, out, n_tokens, block, stream);
// out: None, or (slots, cu_new, kv_lens, free_next). Returns those.
PyObject* cache_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 9);
  const at::Tensor& lens = tensor(a[0], "lens");
  const int dev = cuda_device(lens);
  const at::Tensor& table = tensor(a[2], "block_table");
  const at::Tensor& free = tensor(a[3], "free_blocks");
  if (lens.dim() != 1 || table.dim() != 2 || free.dim() != 1)
    refuse(PyExc_ValueError, "lens and free_blocks have one axis, block_table has two");
  const int64_t B = lens.size(0), width = table.size(1);
  CallStream cs(a[8], dev);
  at::Tensor slots, cu, kv, next;
  if (a[5] == Py_None) {
    const long long T = integer(a[6]);
    if (T < 0 || T > INT32_MAX) refuse(PyExc_ValueError, "n_tokens out of range");
    // one allocation for all four, each from a multiple of 16 bytes on (a call
    // takes 4.5 us of host time so, 6.3 with four)
    auto up = [](int64_t x) { return (x + 3) & ~int64_t{3}; };
    const int64_t at_cu = up(T), at_kv = at_cu + up(B + 1), at_next = at_kv + up(B);
    const at::Tensor all = empty({at_next + 1}, at::kInt, dev);
    slots = part(all, 0, T);
    cu = part(all, at_cu, B + 1);
    kv = part(all, at_kv, B);
    next = part(all, at_next, 1);
  } else {
    if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 4)
      refuse(PyExc_TypeError, "out is (slots, cu_new, kv_lens, free_next)");
    slots = tensor(PyTuple_GET_ITEM(a[5], 0), "slots");
    cu = tensor(PyTuple_GET_ITEM(a[5], 1), "cu_new");
    kv = tensor(PyTuple_GET_ITEM(a[5], 2), "kv_lens");
    next = tensor(PyTuple_GET_ITEM(a[5], 3), "free_next");
    if (slots.dim() != 1) refuse(PyExc_ValueError, "slots has one axis");
  }
  const int T = narrow(slots.size(0), "too many tokens");
  const int32_t* p_lens = index(lens, dev, B, -1, "lens");
  const int32_t* p_new = index(tensor(a[1], "new_lens"), dev, B, -1, "new_lens");
  int32_t* p_table = index(table, dev, B, width, "block_table");
  const int32_t* p_free = index(free, dev, free.size(0), -1, "free_blocks");
  const int32_t* p_pos = index(tensor(a[4], "free_pos"), dev, 1, -1, "free_pos");
  int32_t* p_slots = index(slots, dev, T, -1, "slots");
  int32_t* p_cu = index(cu, dev, B + 1, -1, "cu_new");
  int32_t* p_kv = index(kv, dev, B, -1, "kv_lens");
  int32_t* p_next = index(next, dev, 1, -1, "free_next");
  const int w = narrow(width, "block_table too wide");
  const int nf = narrow(free.size(0), "too many free blocks");
  const int b = narrow(B, "too many requests"), block = narrow(integer(a[7]), "block out of range");
  fa_status rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fa_cache_plan(p_lens, p_new, p_table, w, p_free, nf, p_pos, p_slots, T, p_cu, p_kv, p_next, b,
                     block, cs.stream);
  Py_END_ALLOW_THREADS;
  if (rc != FA_OK) return status(rc);
  if (a[5] != Py_None) {
    Py_INCREF(a[5]);
    return a[5];
  }
  PyObject* out = PyTuple_New(4);
  if (!out) throw python_error();
  const at::Tensor* ts[4] = {&slots, &cu, &kv, &next};
  for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(out, i, THPVariable_Wrap(*ts[i]));
  return out;
  END_HANDLE_TH_ERRORS
}

// (k, v, slots, cache, stream). Returns None.
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 5);
  const at::Tensor& k = tensor(a[0], "k");
  const at::Tensor& v = tensor(a[1], "v");
  const int dev = cuda_device(k);
  const fa_cache c = describe(a[3], dev);
  if (!(k.dim() == 3 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() && on(v, dev) &&
        k.size(1) == c.Hkv && k.size(2) == c.d && k.stride(2) == 1 && v.stride(2) == 1))
    refuse(PyExc_ValueError,
           "k, v must be [T, heads, d] tensors of one dtype with the cache's heads and d, and unit "
           "d stride");
  const fa_dtype dt = dtype16(k);
  const int T = narrow(k.size(0), "too many tokens");
  const int32_t* slots = index(tensor(a[2], "slots"), dev, T, -1, "slots");
  if (T == 0) Py_RETURN_NONE;
  CallStream cs(a[4], dev);
  // an axis of length one has no stride of its own
  fa_strides st[2];
  const at::Tensor* ts[2] = {&k, &v};
  for (int i = 0; i < 2; ++i)
    st[i] = fa_strides{0, c.Hkv > 1 ? ts[i]->stride(1) : c.d, T > 1 ? ts[i]->stride(0) : c.d};
  fa_status rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fa_cache_append(k.data_ptr(), v.data_ptr(), st, slots, T, &c, dt, cs.stream);
  Py_END_ALLOW_THREADS;
  if (rc != FA_OK) return status(rc);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (q, cache, block_table, kv_lens, cu_q, out, causal, scale, stream); out:
// None, or (o, lse, workspace). Returns (o, lse).
PyObject* attention_forward_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 9);
  const at::Tensor& q = tensor(a[0], "q");
  const int dev = cuda_device(q);
  const fa_cache c = describe(a[1], dev);
  const at::Tensor& table = tensor(a[2], "block_table");
  if (table.dim() != 2) refuse(PyExc_ValueError, "block_table has two axes");
  const int B = narrow(table.size(0), "too many sequences");
  const int width = narrow(table.size(1), "block_table too wide");
  const bool ragged = a[4] != Py_None;
  const int64_t dims = q.dim();
  if (!(ragged ? dims == 3 : (dims == 3 || dims == 4) && q.size(0) == B))
    refuse(PyExc_ValueError, "q must be [T, H, d] with cu_q, or [B, H, d] or [B, H, n, d] without");
  if (q.size(dims - 1) != c.d || q.stride(dims - 1) != 1)
    refuse(PyExc_ValueError, "q must have the cache's d and unit d stride");
  const int H = narrow(q.size(1), "too many heads");
  if (H <= 0 || c.Hkv <= 0 || H % c.Hkv != 0)
    refuse(PyExc_ValueError, "the query heads do not share the K / V heads evenly");
  const fa_dtype dt = dtype16(q);
  const int64_t rows = ragged ? q.size(0) : B * (dims == 4 ? q.size(2) : 1);
  const int T = narrow(rows, "too many query rows");
  const int32_t* p_table = index(table, dev, B, width, "block_table");
  const int32_t* p_kv = index(tensor(a[3], "kv_lens"), dev, B, -1, "kv_lens");
  const int32_t* p_cu = ragged ? index(tensor(a[4], "cu_q"), dev, B + 1, -1, "cu_q") : nullptr;
  const int causal = PyObject_IsTrue(a[6]);
  if (causal < 0) throw python_error();
  double scale = 1.0 / std::sqrt(static_cast<double>(c.d));
  if (a[7] != Py_None) {
    scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  }
  CallStream cs(a[8], dev);
  at::Tensor o, lse, ws;
  const auto lse_shape = q.sizes().slice(0, static_cast<size_t>(dims - 1));
  if (a[5] == Py_None) {
    size_t bytes = 0;
    const fa_status s = fa_fwd_cache_workspace_size(B, T, H, c.Hkv, c.d, &bytes);
    if (s != FA_OK) return status(s);
    o = empty(q.sizes(), q.scalar_type(), dev);
    lse = empty(lse_shape, at::kFloat, dev);
    ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
  } else {
    if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 3)
      refuse(PyExc_TypeError, "out is (o, lse, workspace)");
    o = tensor(PyTuple_GET_ITEM(a[5], 0), "o");
    lse = tensor(PyTuple_GET_ITEM(a[5], 1), "lse");
    ws = tensor(PyTuple_GET_ITEM(a[5], 2), "workspace");
    if (!(o.sizes() == q.sizes() && o.scalar_type() == q.scalar_type() && o.stride(dims - 1) == 1 &&
          lse.sizes() == lse_shape && lse.scalar_type() == at::kFloat && lse.is_contiguous() &&
          ws.scalar_type() == at::kByte && ws.is_contiguous() && on(o, dev) && on(lse, dev) &&
          on(ws, dev)))
      refuse(PyExc_ValueError,
             "o must have q's shape and dtype and unit d stride, lse be contiguous float32 of its "
             "shape without d, workspace contiguous uint8, all on q's device");
  }
  if (T > 0) {
    // element strides of batch, head and row; an axis of length one has none of its own
    fa_strides st[2];
    const at::Tensor* ts[2] = {&q, &o};
    for (int i = 0; i < 2; ++i) {
      const at::Tensor& t = *ts[i];
      const long long head = H > 1 ? t.stride(1) : c.d;
      if (ragged) st[i] = fa_strides{8, head, T > 1 ? t.stride(0) : c.d};
      else
        st[i] = fa_strides{B > 1 ? t.stride(0) : 8, head,
                           dims == 4 && t.size(2) > 1 ? t.stride(2) : c.d};
    }
    const size_t ws_bytes = static_cast<size_t>(ws.numel());
    fa_status rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fa_fwd_cache(q.data_ptr(), &c, p_table, width, p_kv, p_cu, o.data_ptr(),
                      static_cast<float*>(lse.data_ptr()), B, T, H, st, causal,
                      static_cast<float>(scale), dt, ws.data_ptr(), ws_bytes, cs.stream);
    Py_END_ALLOW_THREADS;
    if (rc != FA_OK) return status(rc);
  }
  PyObject* out = PyTuple_New(2);
  if (!out) throw python_error();
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(o));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(lse));
  return out;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef kMethods[] = {
    {"cache_plan", fast<cache_plan>(), METH_FASTCALL, nullptr},
    {"cache_append", fast<cache_append>(), METH_FASTCALL, nullptr},
    {"attention_forward_cache", fast<attention_forward_cache>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fa_cache_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_cache_torch() { return PyModule_Create(&kModule); }
