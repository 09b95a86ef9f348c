// Internal interface between the C-ABI of the transformer-block operators (block_api.cpp) and
// their HIP kernels.
#pragma once

#include "ge_internal.h"

namespace ge {

// ---- gated feed-forward block: its products ----
enum FfnMode : int {
  FFN_PAIR = 0,   // G = A B, U = A B2: Y = act(G) * U, optionally Y2 = G, Y3 = U
  FFN_DOWN = 1,   // Y = A B (+ E1)
  FFN_GRAD = 2,   // t = A B: Y = t * E2 * act'(E1) (dG), Y2 = t * act(E1) (dU), Y3 = act(E1) * E2 (H)
  FFN_DUAL = 3,   // Y = A B + A2 B2
  FFN_WGRAD = 4,  // Y = A B with both operands given contraction-major: A [K][M], B [K][N]
  FFN_MODES = 5
};
enum FfnTile : int { FFN_T256 = 0, FFN_T128 = 1, FFN_T64 = 2, FFN_TILES = 3 };

struct FfnProduct {
  const uint16_t *A, *A2, *B, *B2;
  const uint16_t *E1, *E2;      // residual (DOWN, may be NULL); G and U (GRAD)
  uint16_t *Y, *Y2, *Y3;
  int64_t lda, ldb, lde, ldy, ldy2;   // ldy2: Y2 and Y3
  int32_t M, N, K;
  int32_t tiles_m, tiles_n, tile0;    // tile0: first tile of this product in the launch
};
constexpr int kFfnMaxProducts = 3;
struct FfnLaunch {
  FfnProduct prod[kFfnMaxProducts];
  int32_t n, tiles;
  int32_t splits;             // workgroups that share a tile's contraction (1 with the 256-row tiles)
  float* part;                // splits > 1: partial sums [tile][split][bm * bn * operands]
  uint32_t* ctr;              // splits > 1: tickets per tile, zero between calls
};
constexpr uint32_t kFfnCtrStride = 16;       // 64 bytes between tickets
// A contraction is split only in launches of at most this many workgroups (three on every compute unit).
constexpr int kFfnMaxSplitGroups = 768;
// Every operator's workspace begins with the room of the most tickets and keeps its data behind it: a
// workspace may serve calls of several handles in turn, and what one leaves is never another's ticket.
constexpr size_t kTicketBytes = (size_t)kFfnMaxSplitGroups * kFfnCtrStride * 4;
static_assert(kTicketBytes % 256 == 0, "data behind the tickets is aligned");

struct FfnTileInfo { int bm, bn, bn_pair; };
inline FfnTileInfo ffn_tile_info(int tile) {
  return tile == FFN_T256 ? FfnTileInfo{256, 256, 128} : tile == FFN_T128 ? FfnTileInfo{128, 128, 128}
                                                                          : FfnTileInfo{64, 64, 64};
}

// Up to kFfnFewRows rows: products split over the contraction (ge_ffn_few.hip).
struct FfnFew {
  const uint16_t *A, *B, *B2, *E1;
  uint16_t *Y, *Y2, *Y3;
  float* part;                        // [tile][split][operand][kFfnFewRows][kFfnFewCols]
  uint32_t* ctr;                      // tickets per tile, zero between calls
  int64_t lda, ldb, lde, ldy, ldy2;
  int32_t M, N, K;
  int32_t tiles, splits;
};
constexpr int kFfnFewRows = 16;
constexpr int kFfnFewCols = 128;
constexpr int kFfnFewUnit = 64;              // K values a wave takes at a time
hipError_t launch_ffn_few(bool pair, int act, bool b_nk, const FfnFew& p, hipStream_t s);

// b_nk: B (and B2) given [N][K]; otherwise [K][N].  One translation unit per mode group.
hipError_t launch_ffn_pair(int tile, int act, bool b_nk, const FfnLaunch& l, hipStream_t s);
hipError_t launch_ffn_grad(int tile, int act, bool b_nk, const FfnLaunch& l, hipStream_t s);
hipError_t launch_ffn_plain(int mode, int tile, bool b_nk, const FfnLaunch& l, hipStream_t s);

// ---- query/key norm with rotation ----
struct QkParams {
  const void* x[2];           // q, k (forward, and backward with norm)
  void* y[2];                 // forward: outputs; backward: gradients of the inputs
  const void* dy[2];          // backward: gradients of the outputs
  const void* gain[2];
  const void* positions;
  const float* inv_freq;
  float* part;                // backward with norm: partial gain gradients [workgroups][2][head_dim]
  int64_t xt[2], xh[2], yt[2], yh[2], dt[2], dh[2];   // token and head strides of x, y, dy
  int64_t tokens;
  int64_t turns;              // runs of tokens_per_wg tokens, times head_splits
  int32_t heads[2];
  int32_t head_dim, rot_dim;
  int32_t group;              // lanes per head: a power of two, 8 values a lane
  int32_t tokens_per_wg;      // tokens of one turn of a workgroup
  int32_t head_splits;        // workgroups that share a token's heads: 1, or
  int32_t q_splits;           // q_splits for the queries' and the rest for the keys'
  int32_t workgroups;         // grid.x
  bool pos64;
  float eps, amplitude;
};
struct QkKind { bool bf16, wide, half, norm, backward; };
hipError_t launch_qk(const QkKind& kind, const QkParams& p, hipStream_t s);
hipError_t launch_qk_gains(const float* part, int rows, int head_dim, float* dgain_q, float* dgain_k, hipStream_t s);
constexpr int kQkThreads = 256;
constexpr int kQkMaxAngles = 256;       // angles of one turn kept in LDS (2 KB): at most one a thread
constexpr int kQkMaxBackwardGrid = 1024;

// ---- gradient norm and clipping ----
constexpr int kClipTensors = 128;       // tensors of one launch (its table travels as the argument)
constexpr int kClipPartials = 2048;     // workgroups of all norm launches of a call together
constexpr int kClipChunk = 16384;       // values of one workgroup's turn
struct ClipTable {
  const void* in[kClipTensors];
  void* out[kClipTensors];
  int64_t numel[kClipTensors];
  uint32_t chunk0[kClipTensors + 1];    // first chunk of each tensor; [n]: all chunks
  uint32_t fp32[kClipTensors / 32];     // bit t: tensor t is fp32
  int32_t n;
};
enum ClipPolicy : int { kClipCached = 0, kClipStoreThrough = 1, kClipStream = 2 };   // ge_clip.hip
inline int clip_policy(int64_t bytes) {
  return bytes > (int64_t(512) << 20) ? kClipStream : bytes > (int64_t(64) << 20) ? kClipStoreThrough : kClipCached;
}
hipError_t launch_clip_norm(const ClipTable& t, int grid, int policy, double* part, hipStream_t s);
// nparts partial sums -> *norm (if any)
hipError_t launch_clip_finish(const double* part, int nparts, float* norm, hipStream_t s);
hipError_t launch_clip_scale(const ClipTable& t, int grid, int policy, const double* part, int nparts, float max_norm,
                             float eps, float* norm, hipStream_t s);

}  // namespace ge
