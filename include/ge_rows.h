/*
 * ge_rows.h -- operators on the rows between a transformer's products, for AMD Instinct MI355X
 * (gfx950): layer norm with dropout and residual add in front of it, forward and backward; dropout
 * from a counter-based generator; int8 codes with a scale per row; and the product of int8 codes
 * with scales per token and per channel.  Library: libge_rows.so.  Status codes, element types and
 * activations are those of gemm_epilogue.h.
 *
 * Model of use, as in ge_block.h: a descriptor is checked and turned into a handle once (*_create),
 * then executed many times against a pack of borrowed device pointers on a stream.  A handle owns
 * host memory only and belongs to the device that was current when it was created; executing it
 * while another device is current returns GE_ERR_DEVICE.  The library never allocates or frees
 * device memory and never synchronises: every call can be captured into a graph.  Calls only read
 * the handle, so several threads may use one handle at once, each with its own outputs and workspace.
 *
 * Workspace: device scratch of the size *_workspace_size reports, 16-byte aligned, owned by the
 * caller, ZERO-FILLED before its first use; each call that completes leaves its counters at zero
 * again.  One workspace of the largest size may serve handles of this header and of ge_block.h in
 * turn; where anything else wrote to it, it is cleared again.  HAZARD: calls that share a workspace
 * must not overlap in time (two streams, or two graphs replayed at once); give concurrent calls
 * workspaces of their own, and clear a workspace again after a call that did not complete.
 *
 * Rows: every matrix is row-major, its leading dimension in elements.  Elements between a row's
 * length and its leading dimension are not written, and nothing depends on them.  Outputs must not overlap inputs or
 * each other, except where an operator says that an output may be an input itself (same pointer and
 * leading dimension).
 *
 * Sizes: besides what each operator says, the row operators (ge_norm, ge_dropout, ge_quant) take up to 2^40 rows,
 * leading dimensions up to 2^40, and rows times each leading dimension up to 10^18; what is larger is
 * GE_ERR_UNSUPPORTED.
 *
 * Errors: every call returns a status, nothing is enqueued unless it is GE_OK (GE_ERR_HIP: a
 * launch failed, and earlier launches of the same call may have run), nothing aborts.
 */
#ifndef GE_ROWS_H
#define GE_ROWS_H

#include "gemm_epilogue.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------------------
 * Dropout's random numbers.  rng points to two 64-bit integers in device memory, a seed and an
 * offset, read by the kernels: a captured graph draws new numbers when the offset is changed between
 * its replays.  `site` tells the dropouts of one step apart.  A row of d columns has ceil(d / 8)
 * blocks of eight; block b of row i takes the four words of Philox4x32-10 (Salmon, Moraes, Dror and
 * Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with
 *
 *   key      seed, seed >> 32                                         (each word the low 32 bits)
 *   counter  i * ceil(d / 8) + b, site, offset, offset >> 32
 *
 * and value j of the block their half-word j (low half of word 0, high half of word 0, ...).  With
 * t = round(p 65536) a value is dropped (becomes 0, whatever it was) where its half-word is below t, and
 * multiplied by 65536 / (65536 - t) elsewhere: p counts in steps of 2^-16.  The mask depends on
 * nothing but these numbers and d, so the backward pass draws it again; it is never stored.
 * Supported: 0 <= p <= 65535 / 65536, rows * ceil(d / 8) <= 2^32.
 * ------------------------------------------------------------------------------------------- */

/* ---------------------------------------------------------------------------------------------
 * Layer norm of rows of d values, with dropout and residual add in front of it, in one pass
 * (fp32 arithmetic, one rounding of each output):
 *
 *   forward   s = R + drop(X)   (without residual s = drop(X); without dropout drop(X) = X)
 *             n = (s - mean) * rstd,  rstd = 1 / sqrt(mean((s - mean)^2) + eps)
 *             Y = n * gain + bias
 *   backward  e = dY * gain
 *             g = rstd * (e - mean(e) - n * mean(e * n)) + dS
 *             dR = g   dX = drop(g)   dgain = sum over rows of dY * n   dbias = sum over rows of dY
 *
 * The statistics are those of s as S holds it (rounded to the element type), so that the backward
 * pass, which reads S, differentiates what was computed.  dS is the gradient that reaches S from
 * elsewhere (the residual stream goes on past the norm).
 *
 * Element types: X, R, S, Y, gain, bias and their gradients all bf16 or all fp32; mean, rstd, dgain
 * and dbias fp32.  rows >= 0, 1 <= d <= 32768.  Pointers need their element's alignment only;
 * 16-byte aligned rows are fastest.  Forward: S and Y may be X or R; backward: dX and dR may be dY, S or
 * dS.  Sums over rows are taken in a fixed order: equal calls give equal bits.
 *
 * Range: the arithmetic is fp32's.  A row whose sum of values, or of squared deviations (each about 1.8e19 or more),
 * passes 3.4e38 does not get the formula's outputs, nor does one whose squared deviations are below 1e-38 (each about
 * 1e-19 or less) with an eps that is no larger, nor a row of equal values with eps = 0 (NaN).  Such rows, and
 * rows with infinities or NaN, change no other row's outputs; dgain and dbias are sums over all of them.
 * ------------------------------------------------------------------------------------------- */
typedef struct {
  int64_t rows, d;
  int64_t ldx, ldr, lds, ldy;             /* X, R, S, Y */
  int64_t lddy, ldds, lddx, lddr;         /* their gradients */
  int32_t dtype;                          /* GE_DT_BF16 or GE_DT_FP32 */
  int32_t residual;                       /* 1: forward adds R */
  uint32_t site;                          /* with dropout > 0 */
  float dropout;                          /* p; 0: none */
  float eps;                              /* finite, >= 0 */
} ge_norm_desc_t;

typedef struct {
  const void* X;                          /* forward */
  const void* residual;                   /* forward, with desc.residual */
  void* S;                                /* forward: written (NULL: not kept); backward: read (without
                                             residual and dropout it is X) */
  void* Y;                                /* forward */
  const void *gain, *bias;                /* NULL: ones, zeros (bias: forward only) */
  float *mean, *rstd;                     /* [rows]; forward: written (NULL: not kept); backward: read */
  const int64_t* rng;                     /* with dropout */
  const void *dY, *dS;                    /* backward; dS NULL: none */
  void *dX, *dR;                          /* backward; NULL: not computed */
  float *dgain, *dbias;                   /* backward, [d], overwritten; NULL: not computed */
  void* workspace;                        /* backward with dgain or dbias */
  size_t workspace_bytes;
} ge_norm_args_t;

typedef struct ge_norm_plan* ge_norm_handle_t;

/* Checks a descriptor without touching any device.  GE_OK, GE_ERR_INVALID_ARG (NULL, a negative
 * size, a leading dimension below d, an unknown type or flag, a p or eps outside its range) or
 * GE_ERR_UNSUPPORTED. */
ge_status_t ge_norm_validate(const ge_norm_desc_t* desc);
/* Validates, checks that the current device is gfx950 (GE_ERR_DEVICE) and builds the handle;
 * *out is NULL on failure. */
ge_status_t ge_norm_create(const ge_norm_desc_t* desc, ge_norm_handle_t* out);
/* Workspace bytes of ge_norm_backward (partial sums of dgain and dbias); ge_norm_forward needs none. */
ge_status_t ge_norm_workspace_size(ge_norm_handle_t handle, size_t* bytes);
/* One launch. */
ge_status_t ge_norm_forward(ge_norm_handle_t handle, const ge_norm_args_t* args, void* stream);
/* One launch, and a second one for dgain and dbias. */
ge_status_t ge_norm_backward(ge_norm_handle_t handle, const ge_norm_args_t* args, void* stream);
void ge_norm_destroy(ge_norm_handle_t handle);

/* ---------------------------------------------------------------------------------------------
 * Dropout of rows of d values:  forward Y = drop(X) (+ R),  backward dX = drop(dY)  with the same mask
 * (fp32 arithmetic, one rounding).  All of one type, bf16 or fp32.  rows >= 0, 0 <= d <= 2^31 - 16 (and
 * rows * ceil(d / 8) <= 2^32, as above).  Y may be X or R, dX may be dY.
 * ------------------------------------------------------------------------------------------- */
typedef struct {
  int64_t rows, d;
  int64_t ldx, ldr, ldy, lddy, lddx;
  int32_t dtype;                          /* GE_DT_BF16 or GE_DT_FP32 */
  int32_t residual;                       /* 1: forward adds R */
  uint32_t site;
  float p;
} ge_dropout_desc_t;

typedef struct {
  const void *X, *residual;               /* forward */
  void* Y;                                /* forward */
  const void* dY;                         /* backward */
  void* dX;                               /* backward */
  const int64_t* rng;
} ge_dropout_args_t;

typedef struct ge_dropout_plan* ge_dropout_handle_t;

ge_status_t ge_dropout_validate(const ge_dropout_desc_t* desc);
ge_status_t ge_dropout_create(const ge_dropout_desc_t* desc, ge_dropout_handle_t* out);
/* One launch. */
ge_status_t ge_dropout_forward(ge_dropout_handle_t handle, const ge_dropout_args_t* args, void* stream);
/* One launch. */
ge_status_t ge_dropout_backward(ge_dropout_handle_t handle, const ge_dropout_args_t* args, void* stream);
void ge_dropout_destroy(ge_dropout_handle_t handle);

/* ---------------------------------------------------------------------------------------------
 * int8 codes and a scale for every row (tokens, or the output channels of an [out][in] weight):
 *
 *   a = max |x| of the row     scale = a / 127     code = 127 x / a to the nearest integer
 *
 * The exact quotient decides, ties go to the even code.  A row of zeros (or of no values) has scale 0
 * and codes 0.  A row that holds a NaN or an infinity has scale NaN and codes 0: a product with it is NaN.
 * X bf16 or fp32 [rows][ldx], codes [rows][ldq], scale [rows].  rows >= 0, 0 <= d <= 32768.
 * ------------------------------------------------------------------------------------------- */
typedef struct {
  int64_t rows, d;
  int64_t ldx, ldq;
  int32_t dtype;                          /* of X: GE_DT_BF16 or GE_DT_FP32 */
} ge_quant_desc_t;

typedef struct {
  const void* X;
  int8_t* codes;
  float* scale;
} ge_quant_args_t;

typedef struct ge_quant_plan* ge_quant_handle_t;

ge_status_t ge_quant_validate(const ge_quant_desc_t* desc);
ge_status_t ge_quant_create(const ge_quant_desc_t* desc, ge_quant_handle_t* out);
/* One launch. */
ge_status_t ge_quant_run(ge_quant_handle_t handle, const ge_quant_args_t* args, void* stream);
void ge_quant_destroy(ge_quant_handle_t handle);

/* ---------------------------------------------------------------------------------------------
 * Product of int8 codes:  X [M][K] (tokens), W [N][K] (a linear layer's [out][in]),
 *
 *   Y[m][n] = act(x_scale[m] * w_scale[n] * sum over k of X[m][k] W[n][k] + bias[n]) + R[m][n]
 *
 * The sums are int32 and exact; everything after them is fp32, one rounding at the end.  Y, bias and R
 * all bf16 or all fp32; scales fp32 [M] and [N].  A sum is multiplied with its row's scale first: scales may be any numbers
 * as long as that product, of a sum up to 2^14 K, stays below 3.4e38 (magnitudes of x_scale up to 1e29 always do); a NaN
 * scale gives NaN.  Activations as in gemm_epilogue.h; a NaN stays NaN with each of them.  Equal calls give equal bits.
 *
 * Supported: M >= 0, N >= 0 and a multiple of 8, K >= 0 and a multiple of 16 below 2^17 (sums
 * of any codes, -128 among them, fit 32 bits); ldx and ldw multiples of 16, ldy and ldr of 8, all
 * below 2^22 (fp32: ldy and ldr below 2^21); M and N below 2^31 - 512, and ceil(M / 256) * ceil(N / 256) below 2^23
 * (with a tile named, its own rows and columns instead of 256: below 2^23, of 64 below 2^24); 16-byte aligned pointers (scales:
 * 4-byte).  Y may be R.
 * ------------------------------------------------------------------------------------------- */
typedef struct {
  int64_t M, N, K;
  int64_t ldx, ldw, ldy, ldr;
  int32_t act;                            /* ge_act_t */
  int32_t bias, residual;                 /* 1: added */
  int32_t dtype;                          /* of Y, bias and R: GE_DT_BF16 or GE_DT_FP32 */
  int32_t tile;                           /* 0 = chosen by size; 1 + ge_i8_tile_t = that tile */
} ge_i8_desc_t;

/* Output tiles (rows x columns of a workgroup), all with the same results. */
typedef enum { GE_I8_TILE_256 = 0, GE_I8_TILE_128 = 1, GE_I8_TILE_64 = 2, GE_I8_TILE_COUNT = 3 } ge_i8_tile_t;

typedef struct {
  const int8_t *X, *W;
  const float *x_scale, *w_scale;
  const void *bias, *residual;
  void* Y;
  void* workspace;
  size_t workspace_bytes;
} ge_i8_args_t;

typedef struct ge_i8_plan* ge_i8_handle_t;

ge_status_t ge_i8_validate(const ge_i8_desc_t* desc);
ge_status_t ge_i8_create(const ge_i8_desc_t* desc, ge_i8_handle_t* out);
/* Workspace bytes (tickets and partial sums of a contraction that is split over workgroups; 0: none
 * is needed). */
ge_status_t ge_i8_workspace_size(ge_i8_handle_t handle, size_t* bytes);
/* One launch. */
ge_status_t ge_i8_run(ge_i8_handle_t handle, const ge_i8_args_t* args, void* stream);
void ge_i8_destroy(ge_i8_handle_t handle);
/* One line on the kernel the handle launches. */
ge_status_t ge_i8_describe(ge_i8_handle_t handle, char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* GE_ROWS_H */
