/*
 * ge_block.h -- transformer-block operators around the fused products, for AMD Instinct MI355X
 * (gfx950): the gated feed-forward block with its backward pass, the per-head norm of queries
 * and keys with the position rotation (and its gradient), and the global gradient norm with
 * clipping.  Library: libge_block.so.  Status codes, element types, activations and weight
 * layouts are those of gemm_epilogue.h.
 *
 * Model of use, as in gemm_epilogue.h: a descriptor is checked and turned into a handle once
 * (*_create), then executed many times against a pack of borrowed device pointers on a stream.
 * A handle owns host memory only and belongs to the device that was current when it was created;
 * executing it while another device is current returns GE_ERR_DEVICE.  The library never
 * allocates or frees device memory and never synchronises: every call can be captured into a
 * graph.  Calls only read the handle, so several threads may use one handle at once, each with
 * its own outputs and workspace.
 *
 * Workspace: device scratch of the size *_workspace_size reports, 16-byte aligned, owned by the
 * caller, ZERO-FILLED before its first use; each call that completes leaves its counters at zero
 * again.  One workspace of the largest size may serve handles of all operators of this header in
 * turn; where anything else wrote to it, it is cleared again.  HAZARD: calls that share a workspace
 * must not overlap in time (two streams, or two graphs replayed at once); give concurrent calls
 * workspaces of their own, and clear a workspace again after a call that did not complete.
 *
 * Errors: every call returns a status, nothing is enqueued unless it is GE_OK (GE_ERR_HIP: a
 * launch failed, and earlier launches of the same call may have run), nothing aborts.
 */
#ifndef GE_BLOCK_H
#define GE_BLOCK_H

#include "gemm_epilogue.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------------------
 * Gated feed-forward block.  With X [M][d], Wg, Wu : d -> h, Wd : h -> d, all bf16:
 *
 *   forward   G = X Wg   U = X Wu   H = act(G) * U   Y = H Wd (+ R)
 *   backward  dH = dY Wd^T   dG = dH * U * act'(G)   dU = dH * act(G)
 *             dX = dG Wg^T + dU Wu^T   dWg = X^T dG   dWu = X^T dU   dWd = H^T dY
 *
 * Activations: GE_ACT_NONE, GE_ACT_RELU (its derivative is 1 above zero, else 0),
 * GE_ACT_GELU_TANH, GE_ACT_SILU, with the formulas of gemm_epilogue.h.  A NaN gate stays NaN with
 * each of them.
 *
 * Numerics: products are summed in fp32.  Rounded to bf16, to nearest even: H before its product
 * with Wd, dG and dU (and, in the backward pass, H rebuilt from the given G and U) before theirs,
 * because the matrix cores take bf16 operands; and every output.  Everything between is fp32.
 * Results do not depend on the order in which workgroups run: equal calls give equal bits.
 *
 * Layouts (row-major, leading dimensions in elements): X [M][ldx], Y [M][ldy], R [M][ldr],
 * G and U [M][ldg], dY [M][lddy], dX [M][lddx].  w_layout GE_LAYOUT_KN: Wg, Wu [d][ldw >= h],
 * Wd [h][ldwd >= d]; GE_LAYOUT_NK (linear layers' [out][in]): Wg, Wu [h][ldw >= d], Wd
 * [d][ldwd >= h].  dWg, dWu (lddw) and dWd (lddwd) have their weights' layout.
 *
 * Supported: M >= 0 (any value), d and h >= 0 and multiples of 8, every leading dimension a
 * multiple of 8 and below 2^22, M, d and h below 2^31 - 512; every pointer 16-byte aligned.
 * Outputs must not overlap inputs or each other, but Y may be the residual R itself (same
 * leading dimension).  Elements between a row's length and its leading dimension are neither
 * read nor written.
 * ------------------------------------------------------------------------------------------- */
typedef struct {
  int64_t M, d, h;
  int64_t ldx, ldy, ldr, ldg, lddy, lddx;   /* activations and their gradients */
  int64_t ldw, ldwd, lddw, lddwd;           /* weights and their gradients */
  int32_t act;                              /* ge_act_t */
  int32_t w_layout;                         /* ge_layout_t of all weights and their gradients */
  int32_t residual;                         /* 1: forward adds R */
  int32_t save;                             /* 1: forward also writes G and U */
  int32_t tile;                             /* 0 = chosen by size; 1 + ge_ffn_tile_t = that tile */
} ge_ffn_desc_t;

/* Output tiles of the block's products (rows x columns of one workgroup; the gate/up pair halves
 * the columns of the largest).  A requested tile sums every product in ascending order of its
 * contraction, so that all tiles give the same bits; the library's own choice may split a long
 * contraction over workgroups and add the parts (in a fixed order: equal calls give equal bits). */
typedef enum { GE_FFN_TILE_256 = 0, GE_FFN_TILE_128 = 1, GE_FFN_TILE_64 = 2, GE_FFN_TILE_COUNT = 3 } ge_ffn_tile_t;

typedef struct {
  const void *X, *Wg, *Wu, *Wd;
  const void* residual;      /* forward, with desc.residual */
  void* Y;                   /* forward */
  void *G, *U;               /* forward with desc.save: written; backward: read */
  const void* dY;            /* backward */
  void* dX;                  /* backward; NULL: not computed */
  void *dWg, *dWu, *dWd;     /* backward; all three NULL: not computed (X may then be NULL) */
  void* workspace;
  size_t workspace_bytes;
} ge_ffn_args_t;

typedef struct ge_ffn_plan* ge_ffn_handle_t;

/* Checks a descriptor without touching any device.  GE_OK, GE_ERR_INVALID_ARG (NULL, a negative
 * size, a leading dimension below its row, an unknown enum value or flag) or GE_ERR_UNSUPPORTED. */
ge_status_t ge_ffn_validate(const ge_ffn_desc_t* desc);
/* Validates, checks that the current device is gfx950 (GE_ERR_DEVICE) and builds the handle;
 * *out is NULL on failure. */
ge_status_t ge_ffn_create(const ge_ffn_desc_t* desc, ge_ffn_handle_t* out);
/* Workspace bytes of ge_ffn_forward (backward = 0: H) or ge_ffn_backward (backward = 1: dG, dU and
 * H), each with the tickets and partial sums of split contractions.  One workspace of the larger
 * size serves both calls in turn. */
ge_status_t ge_ffn_workspace_size(ge_ffn_handle_t handle, int32_t backward, size_t* bytes);
/* Y (and, with desc.save, G and U) from X, the weights and R.  Two launches. */
ge_status_t ge_ffn_forward(ge_ffn_handle_t handle, const ge_ffn_args_t* args, void* stream);
/* The gradients from dY, X, G, U and the weights; overwritten, not accumulated.  Three launches
 * (two or one where dX or the weight gradients are not asked for). */
ge_status_t ge_ffn_backward(ge_ffn_handle_t handle, const ge_ffn_args_t* args, void* stream);
void ge_ffn_destroy(ge_ffn_handle_t handle);
/* One line on the kernels the handle launches. */
ge_status_t ge_ffn_describe(ge_ffn_handle_t handle, char* buf, size_t len);

/* ---------------------------------------------------------------------------------------------
 * Per-head norm of queries and keys with the position rotation, in one pass.  For each token and
 * head with D = head_dim values x (fp32 arithmetic, one rounding at the end):
 *
 *   r = 1 / sqrt(mean(x^2) + eps)    y = x * r * gain         (desc.norm; otherwise y = x)
 *   angle_i = position * inv_freq[i], i < rot_dim / 2          (product and reduction in 64 bits)
 *   (y_a, y_b) -> amplitude * (y_a cos - y_b sin, y_b cos + y_a sin)    for each pair i
 *   GE_PAIRS_HALF:        a = i, b = i + rot_dim / 2
 *   GE_PAIRS_INTERLEAVED: a = 2i, b = 2i + 1
 *   values rot_dim .. D-1 are y, unturned
 *
 * Scaled positions for long contexts are a choice of inv_freq and amplitude, which the caller
 * gives.  Backward: from the gradients of the outputs, those of x (the inputs are read again and
 * the norm is rebuilt) and of the two gains (fp32 sums over tokens and heads in a fixed order).
 *
 * Element types: q, k, their outputs and gradients and the gains all bf16 or all fp32; inv_freq
 * fp32 [rot_dim / 2]; positions int32 or int64 [tokens], |position| < 2^31; gains' gradients
 * fp32 [D].  Any of tokens, heads_q, heads_k may be 0.  head_dim even, 2 .. 512; rot_dim even,
 * 0 .. head_dim (0: only the norm).  Value e of head j of token t is at t * *_token + j * *_head
 * + e; strides are non-negative, and those of outputs keep elements apart.  Outputs may be the
 * inputs themselves (same pointer and strides), otherwise they must not overlap inputs or each
 * other.  Pointers need their element's alignment; 16-byte aligned pointers and strides that are
 * multiples of 8 elements, with head_dim and rot_dim multiples of 8, take wide accesses.
 * ------------------------------------------------------------------------------------------- */
typedef enum { GE_PAIRS_INTERLEAVED = 0, GE_PAIRS_HALF = 1 } ge_pairs_t;

typedef struct {
  int64_t tokens, heads_q, heads_k;
  int64_t q_token, q_head, k_token, k_head;         /* inputs q, k */
  int64_t oq_token, oq_head, ok_token, ok_head;     /* outputs; backward: their gradients */
  int64_t dq_token, dq_head, dk_token, dk_head;     /* backward: gradients of the inputs */
  int32_t head_dim, rot_dim;
  int32_t pairs;                                    /* ge_pairs_t */
  int32_t norm;                                     /* 1: normalise, with gains */
  int32_t dtype;                                    /* GE_DT_BF16 or GE_DT_FP32 */
  int32_t pos64;                                    /* 1: positions are int64, 0: int32 */
  float eps;                                        /* finite, >= 0 */
} ge_qk_desc_t;

typedef struct {
  const void *q, *k;                  /* forward; backward with norm */
  void *q_out, *k_out;                /* forward */
  const void* positions;              /* with rot_dim > 0 */
  const float* inv_freq;              /* with rot_dim > 0 */
  const void *gain_q, *gain_k;        /* with norm */
  const void *dq_out, *dk_out;        /* backward */
  void *dq, *dk;                      /* backward */
  float *dgain_q, *dgain_k;           /* backward with norm: overwritten */
  void* workspace;                    /* backward with norm */
  size_t workspace_bytes;
  float amplitude;
} ge_qk_args_t;

typedef struct ge_qk_plan* ge_qk_handle_t;

ge_status_t ge_qk_validate(const ge_qk_desc_t* desc);
ge_status_t ge_qk_create(const ge_qk_desc_t* desc, ge_qk_handle_t* out);
/* Workspace bytes of ge_qk_backward (partial sums of the gains' gradients, every one written by
 * each call: one that no other operator uses needs no zero fill); 0 without norm.  ge_qk_forward
 * needs none. */
ge_status_t ge_qk_workspace_size(ge_qk_handle_t handle, size_t* bytes);
/* One launch. */
ge_status_t ge_qk_forward(ge_qk_handle_t handle, const ge_qk_args_t* args, void* stream);
/* One launch, and with norm a second one for the gains' gradients. */
ge_status_t ge_qk_backward(ge_qk_handle_t handle, const ge_qk_args_t* args, void* stream);
void ge_qk_destroy(ge_qk_handle_t handle);

/* ---------------------------------------------------------------------------------------------
 * Global gradient norm over many tensors, and clipping:
 *
 *   norm = sqrt(sum over all tensors of the sum of squares)      (64-bit sums in a fixed order)
 *   out_t = in_t * min(1, max_norm / (norm + eps))               (fp32 product, one rounding)
 *
 * A NaN or infinite gradient makes the norm NaN or infinite, and the products what the formula
 * gives (times NaN, or times 0).  Tensors are dense arrays of bf16 or fp32 values (mixed freely),
 * any length including 0, aligned to their elements.  out_t may be in_t (in place; nothing is
 * written when the factor is 1); otherwise outputs must not overlap inputs or each other.
 * ------------------------------------------------------------------------------------------- */
typedef struct {
  int64_t numel;
  int32_t dtype;                      /* GE_DT_BF16 or GE_DT_FP32 */
} ge_clip_tensor_t;

typedef struct {
  const void* const* in;              /* host array of n device pointers, read during the call */
  void* const* out;                   /* host array of n device pointers; NULL: only the norm */
  float* norm;                        /* device, one float; may be NULL with out */
  void* workspace;                    /* (one that no other operator uses needs no zero fill) */
  size_t workspace_bytes;
  float max_norm;                     /* >= 0 (may be infinite) */
  float eps;                          /* finite, >= 0 */
} ge_clip_args_t;

typedef struct ge_clip_plan* ge_clip_handle_t;

/* tensors: host array of n entries, copied into the handle.  GE_ERR_INVALID_ARG (n < 0, NULL with
 * n > 0, a negative length, an unknown type), GE_ERR_UNSUPPORTED (fp8 values, 2^45 values or more
 * in all, more than 32768 non-empty tensors). */
ge_status_t ge_clip_create(const ge_clip_tensor_t* tensors, int32_t n, ge_clip_handle_t* out);
ge_status_t ge_clip_workspace_size(ge_clip_handle_t handle, size_t* bytes);
/* Two launches for up to 128 non-empty tensors (one more pair for each further 128). */
ge_status_t ge_clip_run(ge_clip_handle_t handle, const ge_clip_args_t* args, void* stream);
void ge_clip_destroy(ge_clip_handle_t handle);

#ifdef __cplusplus
}
#endif

#endif /* GE_BLOCK_H */
