// fa_cache_tree on torch tensors (see fa_cache_torch.cpp).
#pragma once

#include <algorithm>

#include "fa_check.h"
#include "fa_draft.h"
#include "fa_torch.h"

namespace {

using fa::kMaxWords;

// (parents, cu, lens, words, out, stream); words: or None, as many as one request of all the
// tokens needs (up to the most there are); out: None, or (masks, positions). Returns those.
PyObject* cache_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 6);
  const at::Tensor& parents = tensor(a[0], "parents");
  const at::Tensor& lens = tensor(a[2], "lens");
  const int dev = cuda_device(parents);
  if (parents.dim() != 1 || lens.dim() != 1)
    refuse(PyExc_ValueError, "parents and lens have one axis");
  const int T = narrow(parents.size(0), "too many tokens");
  const int B = narrow(lens.size(0), "too many requests");
  const int words = a[3] == Py_None ? std::min(std::max((T - 1) / 64 + 1, 1), kMaxWords)
                                    : narrow(integer(a[3]), "words out of range");
  const int32_t* p_parents = index(parents, dev, T, -1, "parents");
  const int32_t* p_cu = index(tensor(a[1], "cu"), dev, int64_t{B} + 1, -1, "cu");
  const int32_t* p_lens = index(lens, dev, B, -1, "lens");
  CallStream cs(a[5], dev);
  at::Tensor masks, positions;
  if (a[4] == Py_None) {
    if (words < 1) return status(FA_ERR_INVALID_ARG);
    // one allocation for both, the positions behind the masks
    const int64_t n_masks = int64_t{T} * words;
    const at::Tensor all = empty({n_masks + (int64_t{T} + 1) / 2}, at::kLong, dev);
    masks = part(all, 0, {T, words}, at::kLong);
    positions = part(all, 2 * n_masks, {T}, at::kInt);
  } else {
    if (!PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 2)
      refuse(PyExc_TypeError, "out is (masks, positions)");
    masks = tensor(PyTuple_GET_ITEM(a[4], 0), "masks");
    positions = tensor(PyTuple_GET_ITEM(a[4], 1), "positions");
    if (!(masks.scalar_type() == at::kLong && masks.dim() == 2 && masks.size(0) == T &&
          masks.size(1) == words && masks.is_contiguous() && on(masks, dev)))
      refuse(PyExc_ValueError,
             "masks must be a contiguous int64 tensor [T, words] on the device of the parents");
  }
  int32_t* const p_pos = index(positions, dev, T, -1, "positions");
  if (T > 0) {
    fa_status rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fa_cache_tree(p_parents, p_cu, p_lens, static_cast<uint64_t*>(masks.data_ptr()), p_pos, B, T,
                       words, cs.stream);
    Py_END_ALLOW_THREADS;
    if (rc != FA_OK) return status(rc);
    if (a[4] != Py_None) wrote({&masks, &positions});
  }
  return tuple_of({&masks, &positions});
  END_HANDLE_TH_ERRORS
}

}  // namespace
