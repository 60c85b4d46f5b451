/*
 * fa_rope.h - C ABI of the pass before attention: an RMS norm of every head of
 * Q and K, and the rotation by the tokens' positions, together.
 *
 * For a row x of d elements (one head of one token at position p) and the
 * head's weights w:
 *
 *     n = x / sqrt(mean(x^2) + eps)       y = R(p) (n * w)
 *
 * R(p) turns the pairs (a, b) of the first rotary_dim elements by the angles
 * whose cosines and sines the table's row p holds: (a cos - b sin, b cos + a
 * sin). Elements behind rotary_dim are not turned. Pair i is (i, i +
 * rotary_dim / 2), or with `interleaved` (2 i, 2 i + 1).
 *
 * Conventions are fa.h's: plain C, device pointers unless said otherwise,
 * asynchronous on `stream`, arguments checked before anything is enqueued,
 * fa_status results, no device memory allocated.
 */
#ifndef FA_SM103_ROPE_H
#define FA_SM103_ROPE_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct fa_rope {
  const float* table;       /* [n_positions][rotary_dim], 16-byte aligned: a row's cosines, then its
                               sines */
  const int32_t* positions; /* [B][N], 4-byte aligned; taken as within 0 .. n_positions - 1 */
  long long positions_b;    /* elements from one batch's positions to the next one's; 0: shared */
  const void* q_weight;     /* [d], 16-byte aligned, read only; NULL: ones */
  const void* k_weight;
  int weights_fp32;         /* not 0: the weights are float32, else of `dtype` */
  int n_positions;          /* >= 1 */
  int rotary_dim;           /* a multiple of 8, 8 .. d */
  int interleaved;
  float eps;                /* > 0, finite */
} fa_rope;

/*
 * fa_qk_norm_rope - y of all heads of q and k.
 *
 * q, k         : [B][H][N][d] and [B][Hkv][N][d] views of `dtype`, read only.
 * q_out, k_out : the same shapes, written. Either may be its input itself, with
 *                the same strides (in place); no other overlap. (An output at the
 *                address of another operand, or of its input with other strides, is
 *                refused.)
 * strides      : host pointer to four fa_strides, of q, k, q_out, k_out, in
 *                elements: positive multiples of 8 below 2^38. A batch of one
 *                token each row is [1][H][T][d].
 * rope         : host pointer, read during the call.
 * Pointers 16-byte aligned; d 64 or 128; B, H, Hkv >= 1, N >= 0 (0: nothing is
 * enqueued), B * N * (H + Hkv) <= 2^31 - 1.
 * Squares and sums are formed in fp32 (elements beyond 2^60 overflow them), the
 * result is rounded once. An infinity or NaN in a row makes its results NaN or
 * 0, and reaches no other row. One launch.
 */
fa_status fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int H,
                          int Hkv, int N, int d, const fa_strides* strides, const fa_rope* rope,
                          fa_dtype dtype, void* stream);

/*
 * fa_qk_norm_rope_bwd - gradients of fa_qk_norm_rope, from its inputs.
 *
 *     t = R(p)^T dy    dw = sum over rows of t * n    dx = (t w - n mean(t w n)) / sqrt(mean(x^2) + eps)
 *
 * dq_out, dk_out       : gradients of q_out and k_out, read only.
 * q, k                 : the forward's inputs, read only.
 * dq, dk               : written; either may be its dq_out or dk_out itself, with
 *                        the same strides; no other overlap (refused as above).
 * dq_weight, dk_weight : float32 [d], written; NULL: not wanted.
 * strides              : of dq_out, dk_out, q, k, dq, dk, as above.
 * workspace            : device scratch of fa_qk_norm_rope_bwd_workspace_size bytes,
 *                        16-byte aligned, overwritten; not to be used by another call
 *                        at the same time. May be NULL if neither dq_weight nor
 *                        dk_weight is wanted.
 * N = 0: weight gradients that are wanted are set to 0.
 * dw is summed in fp32 in a fixed order: the same call gives the same bits. One
 * launch, and a second one if weight gradients are wanted.
 */
fa_status fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k,
                              void* dq, void* dk, float* dq_weight, float* dk_weight, int B, int H,
                              int Hkv, int N, int d, const fa_strides* strides, const fa_rope* rope,
                              fa_dtype dtype, void* workspace, size_t workspace_size, void* stream);

/* Bytes of the workspace on the current device. Host only. */
fa_status fa_qk_norm_rope_bwd_workspace_size(int d, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* FA_SM103_ROPE_H */
