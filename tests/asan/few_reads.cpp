// Walks every load of the few-row kernels on the host: for ragged sizes, every split, wave, unit, lane,
// column block and half.  An address that the buffer's range check (offset < extent, the only guard
// the hardware gives) lets through has to be a whole 16-byte chunk of the matrix, outside its
// padding, and every weight has to be read exactly once.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../gemm_epilogue_transformer_tiled_amd/csrc/ge_block_internal.h"
#include "../../gemm_epilogue_transformer_tiled_amd/csrc/ge_ffn_few_addr.h"

#define CHECK(c)                                                                                              \
  do {                                                                                                        \
    if (!(c)) {                                                                                               \
      std::printf("outside: %s (line %d): M %d N %d K %d ld +%d, %s\n", #c, __LINE__, M, N, K, pad, nk ? "nk" : "kn"); \
      std::exit(1);                                                                                           \
    }                                                                                                         \
  } while (0)

static long g_loads = 0;

static void walk(int M, int N, int K, int pad, int splits, bool nk) {
  const int ldx = K + pad, ldb = (nk ? K : N) + pad;
  const uint32_t ldx2 = 2u * ldx, ldb2 = 2u * ldb;
  const int rows_b = nk ? N : K, cols_b = nk ? K : N;
  std::vector<int> seen((size_t)rows_b * cols_b, 0);
  const int units = (K + ge::kFfnFewUnit - 1) / ge::kFfnFewUnit, tiles = (N + ge::kFfnFewCols - 1) / ge::kFfnFewCols;
  // chunk at byte `from` + offset of a matrix: its row and column, if the range check lets it through
  auto at = [&](int64_t from, uint32_t offset, int extent, int ld, int rows, int cols, int* r, int* c) {
    ++g_loads;
    CHECK(extent >= 0);
    if (offset >= (uint32_t)extent) return false;
    CHECK(offset + 16u <= (uint32_t)extent);           // whole chunks only
    const int64_t e = from + offset / 2;
    CHECK(offset % 16 == 0);
    *r = (int)(e / ld);
    *c = (int)(e % ld);
    CHECK(*r < rows);
    CHECK(*c + 8 <= cols);
    return true;
  };
  for (int tile = 0; tile < tiles; ++tile) {
    const int n0 = tile * ge::kFfnFewCols, ncols = N - n0 < ge::kFfnFewCols ? N - n0 : ge::kFfnFewCols;
    for (int split = 0; split < splits; ++split) {
      const int u0 = (int)((int64_t)units * split / splits), u1 = (int)((int64_t)units * (split + 1) / splits);
      for (int u = u0; u <= u1; ++u)                   // u1: what a wave without a unit left asks for
        for (uint32_t lane = 0; lane < 64; ++lane) {
          const uint32_t l16 = lane & 15, q16 = lane >> 4;
          int r, c;
          for (int half = 0; half < 2; ++half) {
            // X: in one step of both halves ([N][K]), or in a step of its own per half ([K][N])
            const int k0 = u * ge::kFfnFewUnit + (nk ? 0 : 32 * half), left = u < u1 ? K - k0 : 0;
            const uint32_t xo = ge::few_x_offset(l16, q16, nk ? half : 0, left, ldx2);
            if (at(k0, xo, ge::few_row_extent(M, left, ldx2), ldx, M, K, &r, &c)) {
              CHECK(u < u1 && r == (int)l16 && c == u * ge::kFfnFewUnit + 32 * half + 8 * (int)q16);
            }
            for (int i = 0; i < 8; ++i) {
              if (nk) {
                const uint32_t wo = ge::few_nk_offset(ge::few_nk_column(l16, q16, i, ncols, ldb2), q16, half, left);
                if (!at((int64_t)n0 * ldb + k0, wo, ge::few_row_extent(ncols, left, ldb2), ldb, N, K, &r, &c)) continue;
                CHECK(u < u1 && r == n0 + 16 * i + (int)l16 && c == k0 + 32 * half + 8 * (int)q16);
              } else {
                const uint32_t wo = ge::few_kn_offset(l16, q16, i, ncols, ldb2);
                if (!at((int64_t)k0 * ldb + n0, wo, ge::few_kn_extent(ncols, left, ldb2), ldb, K, N, &r, &c)) continue;
                CHECK(u < u1 && r == k0 + 8 * (int)q16 + i && c == n0 + 8 * (int)l16);
              }
              for (int e = 0; e < 8; ++e) ++seen[(size_t)r * cols_b + c + e];
            }
          }
        }
    }
  }
  for (int s : seen) CHECK(s == 1);
}

int main() {
  for (int nk = 0; nk < 2; ++nk)
    for (int M : {1, 2, 7, 15, 16})
      for (int N : {8, 16, 40, 64, 104, 120, 128, 136, 168, 256, 264, 392})
        for (int K = 8; K <= 208; K += 8)
          for (int pad : {0, 8, 24})
            for (int splits : {1, 2, 3}) walk(M, N, K, pad, splits, nk != 0);
  std::printf("inside: %ld loads\n", g_loads);
  return 0;
}
