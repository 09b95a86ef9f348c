// Layer norm of rows, with dropout and residual add in front of it: the forward pass (gfx950).
//
// Memory-bound: X and R are read once, S and Y written once.  (In bf16 with dropout the vector instructions take 88 % of the
// issue slots at 16384 x 4096 as well.)  A row lies in the registers of 64 to 1024
// threads (RowShape) from its loads to its stores; its mean and the mean square of what is left are two
// sums over those threads, one after the other, so that rows far from zero lose nothing.  A workgroup takes
// one row and ends: with its loads out before anything else it hides more than workgroups that stay and loop do
// (105 us against 100).  Measured, with residual and dropout 0.1: 16384 x 4096 bf16, 537 MB, 90 us, 6.0 TB/s (a copy
// of 4 GB: 4.9), fp32 228 us, 4.7 TB/s; 8192 x 11008 bf16 145 us, 5.0 TB/s; 8192 x 4095 65 us.  16 x 4096 with residual 3.5
// us, a launch.  Ragged rows pay twice: 8192 x 11007 at a pitch of 11008 takes 204 us (masks that are kept in vector lanes,
// shifts, spills), dense 248, since every 16-byte access meets two lines (11008 at a pitch of 11009: 180).
#include "ge_rows_common.h"

namespace ge {
namespace {

constexpr int kLarge = kRowsLoadsOnce | kRowsStoresThrough;

// Waves that the registers have to leave room for on a SIMD: two workgroups of 512 threads a compute unit, and
// six of 256 with bf16 rows, where ragged rows would take a few registers more (8192 x 11007 bf16 with residual and dropout 247
// us against 289, 8192 x 2051 with residual 38 against 42).  Three ragged instances of 512 threads and four vectors spill at
// that: bf16 with dropout 36 bytes a thread, fp32 36, with dropout 108.  With more waves than these the others would too.
template <class E>
constexpr int waves_of(int threads, int vecs) {
  return threads == 512 && vecs > 2 ? 4 : threads == 256 && vecs == 2 && sizeof(E) == 2 ? 6 : 1;
}

template <class E, int TR, int V, bool TAIL, bool DROP, int POLICY>
__global__ __launch_bounds__(TR < 256 ? 256 : TR, waves_of<E>(TR, V)) void norm_forward(NormParams p) {
  constexpr int NT = TR < 256 ? 256 : TR, RPW = NT / TR;
  // Gain and bias are loaded with the row where registers are left for them, not after its sums (with residual, inputs in
  // the caches: 16 x 4096 bf16 3.8 us against 4.1, 2048 x 4096 12.3 against 12.8, 8192 x 1021 14.1 against 15.0; not in
  // large calls, 92 against 90.5, and not in long ragged rows, 8192 x 4095 90 against 64).
  constexpr bool EARLY = POLICY == 0 && V <= 2 && (!TAIL || TR == 64);
  __shared__ float red[2][NT / 64];
  const int t = (int)threadIdx.x % TR, sub = (int)threadIdx.x / TR, d = p.d;
  const uint32_t blocks = (uint32_t)(d + 7) / 8u;
  const float of_d = (float)d;
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);
  for (int64_t row = (int64_t)blockIdx.x * RPW + sub; row < p.rows; row += (int64_t)gridDim.x * RPW) {
    const E* x = (const E*)p.x + row * p.ldx;
    float v[V][8];
    Raw<E> raw[V], rr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) raw[i] = fetch<E, TAIL, POLICY>(x, 8 * (t + TR * i), d);
    if (p.r) {                                         // uniform
#pragma unroll
      for (int i = 0; i < V; ++i) rr[i] = fetch<E, TAIL, POLICY>((const E*)p.r + row * p.ldr, 8 * (t + TR * i), d);
    }
    Raw<E> gain[V], bias[V];
    if constexpr (EARLY) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (p.gain) gain[i] = fetch<E, TAIL>((const E*)p.gain, 8 * (t + TR * i), d);
        if (p.bias) bias[i] = fetch<E, TAIL>((const E*)p.bias, 8 * (t + TR * i), d);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      settle<TAIL>(raw[i], 8 * (t + TR * i), d);
      if (p.r) settle<TAIL>(rr[i], 8 * (t + TR * i), d);
      Words w{};
      if constexpr (DROP) w = philox((uint32_t)row * blocks + (uint32_t)(t + TR * i), p.drop.site, key);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = get(raw[i], j);
        if constexpr (DROP) v[i][j] = dropped(v[i][j], w, j, p.drop);
        if (p.r) v[i][j] += get(rr[i], j);
      }
      // the norm is that of the sum as it is kept
      const Raw<E> kept = rounded(v[i], E());
      if (p.s) put<E, TAIL, POLICY>((E*)p.s + row * p.lds, 8 * (t + TR * i), d, kept);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = get(kept, j);
        sum += v[i][j];
      }
    }
    const float mean = row_sum<TR>(sum, red[0]) / of_d;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = 8 * (t + TR * i) + j < d ? v[i][j] - mean : 0.0f;
        sq = fmaf(v[i][j], v[i][j], sq);
      }
    const float var = row_sum<TR>(sq, red[1]) / of_d, rstd = 1.0f / sqrtf(var + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 8 * (t + TR * i);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
      if (p.gain) {
        if constexpr (!EARLY) gain[i] = fetch<E, TAIL>((const E*)p.gain, col, d);
        settle<TAIL>(gain[i], col, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= get(gain[i], j);
      }
      if (p.bias) {
        if constexpr (!EARLY) bias[i] = fetch<E, TAIL>((const E*)p.bias, col, d);
        settle<TAIL>(bias[i], col, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += get(bias[i], j);
      }
      put<E, TAIL, POLICY>((E*)p.y + row * p.ldy, col, d, rounded(v[i], E()));
    }
  }
}

template <class E, int S, bool TAIL, int POLICY>
hipError_t go(const NormParams& p, int grid, hipStream_t s) {
  constexpr int TR = kRowShape[S].threads, V = kRowShape[S].vecs;
  const dim3 g((unsigned)grid), b(TR < 256 ? 256 : TR);
  if (p.drop.below) hipLaunchKernelGGL((norm_forward<E, TR, V, TAIL, true, POLICY>), g, b, 0, s, p);
  else hipLaunchKernelGGL((norm_forward<E, TR, V, TAIL, false, POLICY>), g, b, 0, s, p);
  return hipGetLastError();
}
template <class E, bool TAIL, int POLICY>
hipError_t by_shape(const NormParams& p, int grid, hipStream_t s) {
  switch (row_shape(p.d)) {
    case 0: return go<E, 0, TAIL, POLICY>(p, grid, s);
    case 1: return go<E, 1, TAIL, POLICY>(p, grid, s);
    case 2: return go<E, 2, TAIL, POLICY>(p, grid, s);
    case 3: return go<E, 3, TAIL, POLICY>(p, grid, s);
    case 4: return go<E, 4, TAIL, POLICY>(p, grid, s);
    case 5: return go<E, 5, TAIL, POLICY>(p, grid, s);
    default: return go<E, 6, TAIL, POLICY>(p, grid, s);
  }
}
template <class E>
hipError_t by_layout(bool large, const NormParams& p, int grid, hipStream_t s) {
  if (p.d % 8) return by_shape<E, true, 0>(p, grid, s);
  return large ? by_shape<E, false, kLarge>(p, grid, s) : by_shape<E, false, 0>(p, grid, s);
}

}  // namespace

hipError_t launch_norm_forward(bool bf16, bool large, const NormParams& p, int grid, hipStream_t s) {
  if (grid <= 0) return hipSuccess;
  return bf16 ? by_layout<uint16_t>(large, p, grid, s) : by_layout<float>(large, p, grid, s);
}

}  // namespace ge
