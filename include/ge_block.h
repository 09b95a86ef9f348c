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
 * Workspace: device scratch of the size *_workspace_size reports, 256-byte aligned, owned by the
 * caller, ZERO-FILLED before its first use; each call that completes leaves its counters at zero
 * again.  HAZARD: calls that share a workspace must not overlap in time (two streams, or two
 * graphs replayed at once); give concurrent calls workspaces of their own, and clear a workspace
 * again after a call that did not complete.
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
 * GE_ACT_GELU_TANH, GE_ACT_SILU, with the formulas of gemm_epilogue.h.
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
 * the columns of the largest).  Results do not depend on the tile, bit for bit. */
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
/* Workspace bytes of ge_ffn_forward (backward = 0: H, and the split sums of few-row calls) or
 * ge_ffn_backward (backward = 1: dG, dU and H). */
ge_status_t ge_ffn_workspace_size(ge_ffn_handle_t handle, int32_t backward, size_t* bytes);
/* Y (and, with desc.save, G and U) from X, the weights and R.  Two launches. */
ge_status_t ge_ffn_forward(ge_ffn_handle_t handle, const ge_ffn_args_t* args, void* stream);
/* The gradients from dY, X, G, U and the weights; overwritten, not accumulated.  Three launches
 * (two or one where dX or the weight gradients are not asked for). */
ge_status_t ge_ffn_backward(ge_ffn_handle_t handle, const ge_ffn_args_t* args, void* stream);
void ge_ffn_destroy(ge_ffn_handle_t handle);
/* One line on the kernels the handle launches. */
ge_status_t ge_ffn_describe(ge_ffn_handle_t handle, char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* GE_BLOCK_H */
