// fa_pages.h on torch tensors (see fa_cache_torch.cpp).
#pragma once

#include "fa_pages.h"
#include "fa_torch.h"

namespace {

// The device of a cache.
int cache_device(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4)
    refuse(PyExc_TypeError, "a cache is a tuple (k, v, k_scales, v_scales)");
  return cuda_device(tensor(PyTuple_GET_ITEM(o, 0), "cache k"));
}

const at::Tensor& table_of(PyObject* o) {
  const at::Tensor& t = tensor(o, "block_table");
  if (t.dim() != 2) refuse(PyExc_ValueError, "block_table has two axes");
  return t;
}
const at::Tensor& one_axis(PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 1) {
    PyErr_Format(PyExc_ValueError, "%s has one axis", what);
    throw python_error();
  }
  return t;
}

// (cache, block_table, kv_lens, cu, keep, out, stream); out: None, or lens_out. Returns that.
PyObject* cache_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 7);
  const int dev = cache_device(a[0]);
  const fa_cache c = describe(a[0], dev);
  const at::Tensor& table = table_of(a[1]);
  const int B = narrow(table.size(0), "too many sequences");
  const int width = narrow(table.size(1), "block_table too wide");
  const int32_t* p_table = index(table, dev, B, width, "block_table");
  const int32_t* p_kv = index(tensor(a[2], "kv_lens"), dev, B, -1, "kv_lens");
  const int32_t* p_cu = index(tensor(a[3], "cu"), dev, int64_t{B} + 1, -1, "cu");
  const at::Tensor& keep = tensor(a[4], "keep");
  if (!(keep.scalar_type() == at::kLong && keep.dim() == 2 && keep.size(0) == B &&
        keep.is_contiguous() && on(keep, dev)))
    refuse(PyExc_ValueError, "keep must be a contiguous int64 tensor [B, words] on the cache's device");
  const int words = narrow(keep.size(1), "keep: too many words");
  CallStream cs(a[6], dev);
  const at::Tensor out = a[5] == Py_None ? empty({B}, at::kInt, dev) : tensor(a[5], "lens_out");
  int32_t* const p_out = index(out, dev, B, -1, "lens_out");
  fa_status rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fa_cache_keep(&c, p_table, width, p_kv, p_cu, static_cast<const uint64_t*>(keep.data_ptr()), words,
                     p_out, B, cs.stream);
  Py_END_ALLOW_THREADS;
  if (rc != FA_OK) return status(rc);
  wrote_cache(a[0]);
  if (a[5] != Py_None) wrote({&out});
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (block_table, lens, new_lens, free_blocks, free_pos, block, shares, out, stream);
// shares: or None; out: None, or free_next. Returns that.
PyObject* cache_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 9);
  const at::Tensor& table = table_of(a[0]);
  const int dev = cuda_device(table);
  const int B = narrow(table.size(0), "too many requests");
  const int width = narrow(table.size(1), "block_table too wide");
  const int32_t* p_table = index(table, dev, B, width, "block_table");
  const int32_t* p_lens = index(tensor(a[1], "lens"), dev, B, -1, "lens");
  const int32_t* p_new = index(tensor(a[2], "new_lens"), dev, B, -1, "new_lens");
  const at::Tensor& free = one_axis(a[3], "free_blocks");
  const int n_free = narrow(free.size(0), "too many free blocks");
  int32_t* const p_free = index(free, dev, n_free, -1, "free_blocks");
  const int32_t* p_pos = index(tensor(a[4], "free_pos"), dev, 1, -1, "free_pos");
  const int block = narrow(integer(a[5]), "block out of range");
  int32_t* p_shares = nullptr;
  int num_blocks = 0;
  if (a[6] != Py_None) {
    const at::Tensor& shares = one_axis(a[6], "shares");
    num_blocks = narrow(shares.size(0), "too many blocks");
    p_shares = index(shares, dev, num_blocks, -1, "shares");
    if (num_blocks == 0) refuse(PyExc_ValueError, "shares is empty");
  }
  CallStream cs(a[8], dev);
  const at::Tensor next = a[7] == Py_None ? empty({1}, at::kInt, dev) : tensor(a[7], "free_next");
  int32_t* const p_next = index(next, dev, 1, -1, "free_next");
  fa_status rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fa_cache_release(p_table, width, p_lens, p_new, p_shares, num_blocks, p_free, n_free, p_pos, p_next,
                        B, block, cs.stream);
  Py_END_ALLOW_THREADS;
  if (rc != FA_OK) return status(rc);
  wrote({&free});
  if (a[6] != Py_None) wrote({&THPVariable_Unpack(a[6])});
  if (a[7] != Py_None) wrote({&next});
  return THPVariable_Wrap(next);
  END_HANDLE_TH_ERRORS
}

// (block_table, lens, src, free_blocks, free_pos, shares, block, out, stream); out:
// None, or (new_table, new_lens, copies, free_next). Returns those.
PyObject* cache_fork(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count_args(n_args, 9);
  const at::Tensor& table = table_of(a[0]);
  const int dev = cuda_device(table);
  const int B = narrow(table.size(0), "too many requests");
  const int width = narrow(table.size(1), "block_table too wide");
  const int32_t* p_table = index(table, dev, B, width, "block_table");
  const int32_t* p_lens = index(tensor(a[1], "lens"), dev, B, -1, "lens");
  const at::Tensor& src = one_axis(a[2], "src");
  const int n = narrow(src.size(0), "too many new requests");
  const int32_t* p_src = index(src, dev, n, -1, "src");
  const at::Tensor& free = one_axis(a[3], "free_blocks");
  const int n_free = narrow(free.size(0), "too many free blocks");
  const int32_t* p_free = index(free, dev, n_free, -1, "free_blocks");
  const int32_t* p_pos = index(tensor(a[4], "free_pos"), dev, 1, -1, "free_pos");
  const at::Tensor& shares = one_axis(a[5], "shares");
  const int num_blocks = narrow(shares.size(0), "too many blocks");
  int32_t* const p_shares = index(shares, dev, num_blocks, -1, "shares");
  const int block = narrow(integer(a[6]), "block out of range");
  CallStream cs(a[8], dev);
  at::Tensor rows, lens, copies, next;
  if (a[7] == Py_None) {
    // one allocation for all four, each from a multiple of 16 bytes on
    auto up = [](int64_t x) { return (x + 3) & ~int64_t{3}; };
    const int64_t at_lens = up(int64_t{n} * width), at_copies = at_lens + up(n);
    const int64_t at_next = at_copies + up(int64_t{3} * n);
    const at::Tensor all = empty({at_next + 1}, at::kInt, dev);
    rows = part(all, 0, {n, width}, at::kInt);
    lens = part(all, at_lens, n);
    copies = part(all, at_copies, {n, 3}, at::kInt);
    next = part(all, at_next, 1);
  } else {
    if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 4)
      refuse(PyExc_TypeError, "out is (new_table, new_lens, copies, free_next)");
    rows = tensor(PyTuple_GET_ITEM(a[7], 0), "new_table");
    lens = tensor(PyTuple_GET_ITEM(a[7], 1), "new_lens");
    copies = tensor(PyTuple_GET_ITEM(a[7], 2), "copies");
    next = tensor(PyTuple_GET_ITEM(a[7], 3), "free_next");
  }
  int32_t* const p_rows = index(rows, dev, n, width, "new_table");
  int32_t* const p_new = index(lens, dev, n, -1, "new_lens");
  int32_t* const p_copies = index(copies, dev, n, 3, "copies");
  int32_t* const p_next = index(next, dev, 1, -1, "free_next");
  fa_status rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fa_cache_fork(p_table, width, p_lens, B, p_src, n, p_shares, num_blocks, p_free, n_free, p_pos,
                     p_rows, p_new, p_copies, p_next, block, cs.stream);
  Py_END_ALLOW_THREADS;
  if (rc != FA_OK) return status(rc);
  wrote({&shares});
  if (a[7] != Py_None) wrote({&rows, &lens, &copies, &next});
  return tuple_of({&rows, &lens, &copies, &next});
  END_HANDLE_TH_ERRORS
}

// (cache, copies, stream). Returns None.
PyObject* cache_copy(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count_args(n_args, 3);
  const int dev = cache_device(a[0]);
  const fa_cache c = describe(a[0], dev);
  const at::Tensor& copies = tensor(a[1], "copies");
  if (copies.dim() != 2) refuse(PyExc_ValueError, "copies has two axes");
  const int n = narrow(copies.size(0), "too many copies");
  const int32_t* p = index(copies, dev, n, 3, "copies");
  if (n == 0) Py_RETURN_NONE;
  CallStream cs(a[2], dev);
  fa_status rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = fa_cache_copy(&c, p, n, cs.stream);
  Py_END_ALLOW_THREADS;
  if (rc != FA_OK) return status(rc);
  wrote_cache(a[0]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

}  // namespace
