// Dropout of rows, with an optional residual add; its gradient is the same with the mask drawn again
// (gfx950).
//
// Memory-bound: every value is read once and written once, the mask is computed where it is needed.
// One Philox call serves a vector of eight values (its 20 products at a quarter of the adds' rate would cost as much as
// the memory with four).  Measured: 8192 x 11008 bf16, 361 MB, 57 us, 6.3 TB/s; its gradient the same; 8192 x 11007, rows at
// odd addresses, 64 us; 777 x 1021 fp32 with residual 3.5 us, a launch.
#include "ge_rows_common.h"

namespace ge {
namespace {

constexpr int kThreads = 256;
constexpr int kLarge = kRowsLoadsOnce | kRowsStoresThrough;

// FLAT: dense rows of whole vectors: block i is elements 8 i .. 8 i + 7.
template <class E, bool FLAT, bool TAIL, bool RES, int POLICY>
__global__ __launch_bounds__(kThreads) void dropout(DropoutParams p) {
  const DropKey key = drop_key(p.drop);
  const uint32_t blocks = (uint32_t)(p.d + 7) / 8u;
  const int64_t n = p.rows * blocks;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const uint32_t b = (uint32_t)i, row = FLAT ? 0u : b / blocks;
    const int col = FLAT ? 0 : (int)(8u * (b - row * blocks)), d = FLAT ? 8 : p.d;
    const E* x = (const E*)p.x + (FLAT ? 8 * i : (int64_t)row * p.ldx);
    const E* r = (const E*)p.r + (FLAT ? 8 * i : (int64_t)row * p.ldr);
    E* y = (E*)p.y + (FLAT ? 8 * i : (int64_t)row * p.ldy);
    Raw<E> rx = fetch<E, TAIL, POLICY>(x, col, d);
    Raw<E> rr;
    if constexpr (RES) rr = fetch<E, TAIL, POLICY>(r, col, d);
    const Words w = philox(b, p.drop.site, key);
    settle<TAIL>(rx, col, d);
    if constexpr (RES) settle<TAIL>(rr, col, d);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = dropped(get(rx, j), w, j, p.drop);
      if constexpr (RES) v[j] += get(rr, j);
    }
    put<E, TAIL, POLICY>(y, col, d, rounded(v, E()));
  }
}

template <class E, bool RES>
hipError_t go(bool large, const DropoutParams& p, hipStream_t s) {
  const int64_t n = p.rows * ((p.d + 7) / 8), groups = (n + kThreads - 1) / kThreads;
  // (57 us at 8192 x 11008 bf16; with 4096 workgroups, each longer in its loop, 62)
  const dim3 g((unsigned)(groups < 16384 ? groups : 16384)), b(kThreads);
  const bool flat = p.d % 8 == 0 && p.ldx == p.d && p.ldy == p.d && (!RES || p.ldr == p.d);
  if (flat && large) hipLaunchKernelGGL((dropout<E, true, false, RES, kLarge>), g, b, 0, s, p);
  else if (flat) hipLaunchKernelGGL((dropout<E, true, false, RES, 0>), g, b, 0, s, p);
  else if (p.d % 8) hipLaunchKernelGGL((dropout<E, false, true, RES, 0>), g, b, 0, s, p);
  else hipLaunchKernelGGL((dropout<E, false, false, RES, 0>), g, b, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(bool bf16, bool large, const DropoutParams& p, hipStream_t s) {
  if (p.rows <= 0 || p.d <= 0) return hipSuccess;
  if (bf16) return p.r ? go<uint16_t, true>(large, p, s) : go<uint16_t, false>(large, p, s);
  return p.r ? go<float, true>(large, p, s) : go<float, false>(large, p, s);
}

}  // namespace ge
