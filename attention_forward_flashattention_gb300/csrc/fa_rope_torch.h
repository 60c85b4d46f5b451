// fa_qk_norm_rope and its gradients on torch tensors (see fa_cache_torch.cpp).
#pragma once

#include "fa_rope.h"
#include "fa_torch.h"

namespace {

// Shape of q or k: [B, H, N, d], or [T, H, d] as one batch of T tokens.
struct HeadsView {
  int64_t B, H, N, d;
};
HeadsView heads_view(const at::Tensor& t, const char* what) {
  if ((t.dim() != 3 && t.dim() != 4) || (t.numel() > 0 && t.stride(t.dim() - 1) != 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be [B, H, N, d] or [T, H, d] with unit d stride", what);
    throw python_error();
  }
  if (t.dim() == 3) return {1, t.size(1), t.size(0), t.size(2)};
  return {t.size(0), t.size(1), t.size(2), t.size(3)};
}
// Its strides; an axis of length one has none of its own, a tensor without elements no axis.
fa_strides heads_strides(const at::Tensor& t, const HeadsView& v) {
  if (t.numel() == 0) return {v.d, v.d, v.d};
  const bool rows = t.dim() == 3;
  return {v.B > 1 ? t.stride(0) : 8, v.H > 1 ? t.stride(1) : v.d,
          v.N > 1 ? t.stride(rows ? 0 : 2) : v.d};
}

// A tensor's address; one of its own for a tensor without elements, which has none.
void* address(const at::Tensor& t) {
  alignas(16) static char none[16];
  return t.numel() > 0 ? t.data_ptr() : static_cast<void*>(none);
}

// Tensors of one call: every one like the first of its pair.
void same_rows(const at::Tensor& t, const at::Tensor& like, const char* what) {
  if (!(t.sizes() == like.sizes() && t.scalar_type() == like.scalar_type() &&
        (t.numel() == 0 || t.stride(t.dim() - 1) == 1) && on(t, like.get_device()))) {
    PyErr_Format(PyExc_ValueError,
                 "%s must have the shape, dtype and device of its input and unit d stride", what);
    throw python_error();
  }
}

// fa_rope of (table, positions, q_weight, k_weight, eps, interleaved) at a[0].
fa_rope describe_rope(PyObject* const* a, const HeadsView& q, fa_dtype dt, int dev) {
  fa_rope r{};
  const at::Tensor& table = tensor(a[0], "rope");
  if (!(table.dim() == 2 && table.scalar_type() == at::kFloat && table.is_contiguous() &&
        on(table, dev)))
    refuse(PyExc_ValueError,
           "rope must be a contiguous float32 tensor [positions, rotary_dim] on q's device");
  r.table = static_cast<const float*>(table.data_ptr());
  r.n_positions = narrow(table.size(0), "rope: too many positions");
  r.rotary_dim = narrow(table.size(1), "rope: rotary_dim too large");
  const at::Tensor& pos = tensor(a[1], "positions");
  const bool shared = pos.dim() == 1;
  if (!(pos.scalar_type() == at::kInt && on(pos, dev) &&
        (shared ? pos.size(0) == q.N : pos.dim() == 2 && pos.size(0) == q.B && pos.size(1) == q.N) &&
        (q.N <= 1 || pos.stride(pos.dim() - 1) == 1)))
    refuse(PyExc_ValueError,
           "positions must be int32 [N] ([T]) or [B, N] on q's device, without gaps along N");
  r.positions = static_cast<const int32_t*>(address(pos));
  r.positions_b = shared || q.B == 1 ? 0 : pos.stride(0);
  r.weights_fp32 = -1;
  const void** to[2] = {&r.q_weight, &r.k_weight};
  for (int i = 0; i < 2; ++i) {
    if (a[2 + i] == Py_None) continue;
    const at::Tensor& w = tensor(a[2 + i], "weight");
    const bool fp32 = w.scalar_type() == at::kFloat;
    if (!(w.dim() == 1 && w.size(0) == q.d && w.is_contiguous() && on(w, dev) &&
          (fp32 || w.scalar_type() == (dt == FA_DTYPE_FP16 ? at::kHalf : at::kBFloat16)) &&
          (r.weights_fp32 < 0 || r.weights_fp32 == static_cast<int>(fp32))))
      refuse(PyExc_ValueError,
             "weights must be contiguous [d] tensors on q's device, both float32 or both of q's dtype");
    r.weights_fp32 = fp32;
    *to[i] = w.data_ptr();
  }
  r.weights_fp32 = r.weights_fp32 > 0;
  r.eps = static_cast<float>(PyFloat_AsDouble(a[4]));
  if (PyErr_Occurred()) throw python_error();
  r.interleaved = PyObject_IsTrue(a[5]);
  if (r.interleaved < 0) throw python_error();
  return r;
}

// q and k of a call: shapes that go together.
void check_qk(const at::Tensor& q, const at::Tensor& k, const HeadsView& vq, const HeadsView& vk) {
  if (!(q.dim() == k.dim() && vk.B == vq.B && vk.N == vq.N && vk.d == vq.d &&
        k.scalar_type() == q.scalar_type() && on(k, q.get_device())))
    refuse(PyExc_ValueError, "q and k must be of one dtype and device and differ in their heads only");
}

// (q, k, table, positions, q_weight, k_weight, eps, interleaved, out, stream);
// out: None, or (q_out, k_out). Returns those.
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 10);
  const at::Tensor& q = tensor(a[0], "q");
  const at::Tensor& k = tensor(a[1], "k");
  const int dev = cuda_device(q);
  const HeadsView vq = heads_view(q, "q"), vk = heads_view(k, "k");
  check_qk(q, k, vq, vk);
  const fa_dtype dt = dtype16(q);
  const fa_rope r = describe_rope(a + 2, vq, dt, dev);
  CallStream cs(a[9], dev);
  at::Tensor qo, ko;
  if (a[8] == Py_None) {
    qo = empty(q.sizes(), q.scalar_type(), dev);
    ko = empty(k.sizes(), k.scalar_type(), dev);
  } else {
    if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 2)
      refuse(PyExc_TypeError, "out is (q_out, k_out)");
    qo = tensor(PyTuple_GET_ITEM(a[8], 0), "q_out");
    ko = tensor(PyTuple_GET_ITEM(a[8], 1), "k_out");
    same_rows(qo, q, "q_out");
    same_rows(ko, k, "k_out");
    if (c10::GradMode::is_enabled() && (qo.requires_grad() || ko.requires_grad()))
      refuse(PyExc_ValueError,
             "q_out and k_out must not require gradients: what is written to them has none (use "
             "qk_norm_rope, or torch.no_grad)");
  }
  const int B = narrow(vq.B, "too many batches"), N = narrow(vq.N, "too many tokens");
  const int H = narrow(vq.H, "too many heads"), Hkv = narrow(vk.H, "too many heads");
  const int d = narrow(vq.d, "d too large");
  if (B > 0 && N > 0) {
    const fa_strides st[4] = {heads_strides(q, vq), heads_strides(k, vk), heads_strides(qo, vq),
                              heads_strides(ko, vk)};
    fa_status rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fa_qk_norm_rope(q.data_ptr(), k.data_ptr(), qo.data_ptr(), ko.data_ptr(), B, H, Hkv, N, d,
                         st, &r, dt, cs.stream);
    Py_END_ALLOW_THREADS;
    if (rc != FA_OK) return status(rc);
    if (a[8] != Py_None) wrote({&qo, &ko});
  }
  return tuple_of({&qo, &ko});
  END_HANDLE_TH_ERRORS
}

// (dq_out, dk_out, q, k, table, positions, q_weight, k_weight, eps, interleaved,
// stream, of_q_weight, of_k_weight). Returns (dq, dk, dq_weight, dk_weight), None for a
// weight that is None or whose gradient is not asked for.
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 13);
  bool wanted[2];
  for (int i = 0; i < 2; ++i) {
    const int truth = PyObject_IsTrue(a[11 + i]);
    if (truth < 0) throw python_error();
    wanted[i] = truth != 0;
  }
  const at::Tensor& dqo = tensor(a[0], "dq_out");
  const at::Tensor& dko = tensor(a[1], "dk_out");
  const at::Tensor& q = tensor(a[2], "q");
  const at::Tensor& k = tensor(a[3], "k");
  const int dev = cuda_device(q);
  const HeadsView vq = heads_view(q, "q"), vk = heads_view(k, "k");
  check_qk(q, k, vq, vk);
  same_rows(dqo, q, "dq_out");
  same_rows(dko, k, "dk_out");
  const fa_dtype dt = dtype16(q);
  const fa_rope r = describe_rope(a + 4, vq, dt, dev);
  CallStream cs(a[10], dev);
  const at::Tensor dq = empty(q.sizes(), q.scalar_type(), dev);
  const at::Tensor dk = empty(k.sizes(), k.scalar_type(), dev);
  at::Tensor dqw, dkw, ws;
  if (r.q_weight && wanted[0]) dqw = empty({vq.d}, at::kFloat, dev);
  if (r.k_weight && wanted[1]) dkw = empty({vq.d}, at::kFloat, dev);
  const int B = narrow(vq.B, "too many batches"), N = narrow(vq.N, "too many tokens");
  const int H = narrow(vq.H, "too many heads"), Hkv = narrow(vk.H, "too many heads");
  const int d = narrow(vq.d, "d too large");
  if (H == 0 || Hkv == 0) refuse(PyExc_ValueError, "no heads");
  size_t bytes = 0;
  if (dqw.defined() || dkw.defined()) {
    const fa_status s = fa_qk_norm_rope_bwd_workspace_size(d, &bytes);
    if (s != FA_OK) return status(s);
    ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
  }
  const fa_strides st[6] = {heads_strides(dqo, vq), heads_strides(dko, vk), heads_strides(q, vq),
                            heads_strides(k, vk),   heads_strides(dq, vq),  heads_strides(dk, vk)};
  float* const pqw = dqw.defined() ? static_cast<float*>(dqw.data_ptr()) : nullptr;
  float* const pkw = dkw.defined() ? static_cast<float*>(dkw.data_ptr()) : nullptr;
  void* const pws = ws.defined() ? ws.data_ptr() : nullptr;
  fa_status rc;
  Py_BEGIN_ALLOW_THREADS;
  // (no batches: as one without tokens)
  rc = fa_qk_norm_rope_bwd(address(dqo), address(dko), address(q), address(k), address(dq), address(dk),
                           pqw, pkw, B > 0 ? B : 1, H, Hkv, B > 0 ? N : 0, d, st, &r, dt, pws, bytes,
                           cs.stream);
  Py_END_ALLOW_THREADS;
  if (rc != FA_OK) return status(rc);
  return tuple_of({&dq, &dk, &dqw, &dkw});
  END_HANDLE_TH_ERRORS
}

}  // namespace
