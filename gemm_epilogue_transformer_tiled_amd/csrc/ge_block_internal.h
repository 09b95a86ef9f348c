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
};

struct FfnTileInfo { int bm, bn, bn_pair; };
inline FfnTileInfo ffn_tile_info(int tile) {
  return tile == FFN_T256 ? FfnTileInfo{256, 256, 128} : tile == FFN_T128 ? FfnTileInfo{128, 128, 128}
                                                                          : FfnTileInfo{64, 64, 64};
}

// b_nk: B (and B2) given [N][K]; otherwise [K][N].  One translation unit per mode group.
hipError_t launch_ffn_pair(int tile, int act, bool b_nk, const FfnLaunch& l, hipStream_t s);
hipError_t launch_ffn_grad(int tile, int act, bool b_nk, const FfnLaunch& l, hipStream_t s);
hipError_t launch_ffn_plain(int mode, int tile, bool b_nk, const FfnLaunch& l, hipStream_t s);

}  // namespace ge
