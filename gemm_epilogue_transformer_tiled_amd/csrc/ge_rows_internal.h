// Internal interface between the C-ABI of the row operators (rows_api.cpp) and their HIP kernels.
#pragma once

#include "ge_block_internal.h"

namespace ge {

// ---- how a row lies on threads ----
// Eight values are a vector; thread t of a row's `threads` holds vectors t, t + threads, ... up to `vecs`
// of them.  So a wave reads 1 KB of bf16 at a time, and the whole row is in registers between its
// sums and its outputs.  More threads with fewer vectors each are slower (norm of 65536 x 1024 bf16 90
// us, with four times the threads 113; codes 39 against 52; 4096 x 16384 with 512 threads 91, with 1024 98),
// but for few rows (16 x 11008 with 512 threads 5.6 us, with 1024 5.0).
struct RowShape { int threads, vecs; };
constexpr int kRowShapes = 7;
constexpr RowShape kRowShape[kRowShapes] = {{64, 1}, {64, 2}, {256, 1}, {256, 2}, {512, 2}, {512, 4}, {1024, 4}};
// The backward pass holds the sums of its columns too: more threads for a row (16384 x 4096 bf16 with 512 threads
// 114 us, with 256 124).
constexpr RowShape kGradShape[kRowShapes] = {{64, 1}, {64, 2}, {256, 1}, {512, 1}, {1024, 1}, {1024, 2}, {1024, 4}};
constexpr int64_t kRowMax = 8 * 1024 * 4;
// The same widths in both tables: 512, 1024, 2048, ... 32768.
inline int row_shape(int64_t d) {
  for (int i = 0; i < kRowShapes - 1; ++i)
    if (d <= 8 * kRowShape[i].threads * kRowShape[i].vecs) return i;
  return kRowShapes - 1;
}
// Rows a workgroup takes at a time: workgroups have 256 threads at least.
inline int rows_at_once(const RowShape& s) { return s.threads < 256 ? 256 / s.threads : 1; }

// Cache policy of large calls (past kRowsLarge bytes of outputs): nothing of them would
// be left in the caches for the next call, so their loads and stores do not push other lines out, nor wait for
// room (16384 x 4096 bf16, 134 MB an array, residual and dropout: norm 90 us against 100, its gradient 124 against 131, before
// its grid was halved).  Ragged rows keep the default, though it goes both ways there (8192 x 11007 with
// residual and dropout: bf16 248 us against 226 past the caches, fp32 375 against 422; codes 67 against 66 and 88 against 95).
enum RowsPolicy : int { kRowsLoadsOnce = 1, kRowsStoresThrough = 2 };
constexpr int64_t kRowsLarge = int64_t(64) << 20;

struct DropParams {
  const int64_t* rng;         // seed, offset
  uint32_t site, below;       // dropped: half-words below `below` (0: no dropout)
  float factor;               // of kept values
};

struct NormParams {
  const void *x, *r;          // r NULL: no residual
  void *s, *y;                // s NULL: not kept
  const void *gain, *bias;    // NULL: ones, zeros
  float *mean, *rstd;         // NULL: not kept
  DropParams drop;
  int64_t rows, ldx, ldr, lds, ldy;
  int32_t d;
  float eps;
};
struct NormGradParams {
  const void *dy, *s, *ds;    // ds NULL: none
  const void* gain;           // NULL: ones
  const float *mean, *rstd;
  void *dx, *dr;              // NULL: not computed
  float* part;                // [workgroups][2][d]: dgain, dbias; NULL: not computed
  DropParams drop;
  int64_t rows, lddy, lds, ldds, lddx, lddr;
  int32_t d;
};
hipError_t launch_norm_forward(bool bf16, bool large, const NormParams& p, int grid, hipStream_t s);
hipError_t launch_norm_backward(bool bf16, bool large, const NormGradParams& p, int grid, hipStream_t s);
// parts partial sums of both -> dgain, dbias (either may be NULL)
hipError_t launch_norm_sums(const float* part, int parts, int d, float* dgain, float* dbias, hipStream_t s);

struct DropoutParams {
  const void *x, *r;
  void* y;
  DropParams drop;
  int64_t rows, ldx, ldr, ldy;
  int32_t d;
};
hipError_t launch_dropout(bool bf16, bool large, const DropoutParams& p, hipStream_t s);

struct QuantParams {
  const void* x;
  int8_t* codes;
  float* scale;
  int64_t rows, ldx, ldq;
  int32_t d;
};
hipError_t launch_quant(bool bf16, bool large, const QuantParams& p, int grid, hipStream_t s);

// ---- product of codes: tiles of ge_ffn_impl.h (FfnTile), sizes and pitches of X and W in 2-byte units ----
hipError_t launch_i8(int tile, const I8Launch& l, hipStream_t s);

// Up to kI8FewRows tokens: one pass over the weights (ge_i8_few.hip).
struct I8Few {
  const int8_t *X, *W;
  const void* R;              // residual, NULL: none
  void* Y;
  I8Epilogue ep;
  int64_t ldx, ldw, ldy, ldr;
  int32_t M, N, K;
  int32_t x_pitch;            // bytes between the tokens' codes in LDS
  int32_t cols;               // of a workgroup: kI8FewCols or half of them
};
constexpr int kI8FewRows = 32, kI8FewCols = 16, kI8FewWaves = 8;
constexpr int kI8FewStep = 512;               // codes of K a wave takes at a time
constexpr int kI8FewLd = kI8FewCols + 4;      // words between rows of the waves' sums in LDS
constexpr int64_t kI8FewLds = 160 * 1024;
// Pitch of the tokens' codes in LDS: whole loads of 1 KB, and 32 bytes, so that the 16 rows that one LDS pass
// reads lie on 16 different 16-byte columns of a 256-byte line.
inline int64_t i8_few_pitch(int64_t K) { return (K + 1023) / 1024 * 1024 + 32; }
// LDS of a workgroup: the tokens' codes, then in the same place the waves' sums.
inline int64_t i8_few_lds(int64_t M, int64_t K) {
  const int64_t sums = kI8FewWaves * (M <= 16 ? 16 : 32) * kI8FewLd * 4, codes = M * i8_few_pitch(K);
  return codes > sums ? codes : sums;
}
hipError_t launch_i8_few(const I8Few& p, hipStream_t s);

}  // namespace ge
