// int8 codes and a scale for every row (gfx950).
//
// Memory-bound: the row is read once, its largest magnitude found while it lies in registers, its codes
// written.  Measured: 8192 x 11008 bf16, 270 MB, 46 us, 5.8 TB/s, fp32 84 us, 5.4 TB/s; 8192 x 11007
// 66 us, fp32 88; 27 x 4096 3.4 us, a launch.
//
// A code is the exact quotient q = 127 x / a to the nearest integer, ties to even.  What is computed is
// x * (127 / a), off by two roundings, and then rounded to a grid that is coarser than that error and finer
// than the distance between a tie and any other quotient; so a tie lands on the tie, and nothing else does:
//   bf16   X and A the 8-bit integers of x and a: q = 127 X / (A 2^f), so q is a tie or at least
//          1 / (254 X) > 2^-16 of itself away from one.  fp32 product: off by less than 2^-23 (1 + 2^-20) of q;
//          grid: 20 bits after the leading one, half a step 2^-21
//   fp32   24-bit integers: at least 2^-32 of q away.  64-bit product: off by 127 * 2^-52 at most; grid: 2^-40
#include "ge_rows_common.h"

namespace ge {
namespace {

constexpr int kLarge = kRowsLoadsOnce | kRowsStoresThrough;

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}

// What the row's values are multiplied with.  Rows of values near the smallest normal one are scaled up
// first (exactly), so that 127 / a is finite.
struct Factor {
  float up, f;
  double f64;
};
template <class E>
__device__ __forceinline__ Factor factor_of(float a) {
  Factor q;
  q.up = a < 0x1p-60f ? 0x1p90f : 1.0f;
  const float b = a * q.up;
  if constexpr (sizeof(E) == 2) q.f = 127.0f / b;
  else q.f64 = 127.0 / (double)b;
  return q;
}
__device__ __forceinline__ int code(float x, const Factor& q, uint16_t) {
  const uint32_t t = __float_as_uint(x * q.up * q.f);
  return (int)__builtin_rintf(__uint_as_float((t + 4u) & ~7u));
}
__device__ __forceinline__ int code(float x, const Factor& q, float) {
  constexpr double grid = 0x1.8p12;                    // its unit in the last place: 2^-40
  const double t = (double)(x * q.up) * q.f64;
  return (int)__builtin_rint((t + grid) - grid);
}

template <class E, int TR, int V, bool TAIL, int POLICY>
__global__ __launch_bounds__(TR < 256 ? 256 : TR) void quant_rows(QuantParams p) {
  constexpr int NT = TR < 256 ? 256 : TR, RPW = NT / TR;
  __shared__ uint32_t top_of[2][NT / 64];
  const int t = (int)threadIdx.x % TR, sub = (int)threadIdx.x / TR, d = p.d;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPW + sub; row < p.rows; row += (int64_t)gridDim.x * RPW, turn ^= 1) {
    Raw<E> raw[V];
    uint32_t top = 0;                                  // magnitudes compare like their bits, NaN above all
#pragma unroll
    for (int i = 0; i < V; ++i) {
      raw[i] = fetch<E, TAIL, POLICY>((const E*)p.x + row * p.ldx, 8 * (t + TR * i), d);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      settle<TAIL>(raw[i], 8 * (t + TR * i), d);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(get(raw[i], j)) & 0x7FFFFFFFu);
    }
    top = wave_max(top);
    if constexpr (TR > 64) {
      if ((threadIdx.x & 63) == 0) top_of[turn][threadIdx.x >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TR / 64; ++w) top = max(top, top_of[turn][w]);
    }
    const float a = __uint_as_float(top);
    const bool sound = top < 0x7F800000u;
    if (t == 0) p.scale[row] = sound ? a / 127.0f : __uint_as_float(0x7FC00000u);
    const bool some = sound && top != 0u;
    const Factor q = factor_of<E>(some ? a : 1.0f);
    int8_t* const out = p.codes + row * p.ldq;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 8 * (t + TR * i);
      if (col >= d) continue;
      uint32_t w[2] = {0, 0};
      if (some)
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j >> 2] |= ((uint32_t)code(get(raw[i], j), q, E()) & 0xFFu) << (8 * (j & 3));
      if (!TAIL || col + 8 <= d) {
        typedef u32x2 Any8 __attribute__((aligned(1)));
        if constexpr ((POLICY & kRowsStoresThrough) != 0) __builtin_nontemporal_store(u32x2{w[0], w[1]}, (Any8*)(out + col));
        else *(Any8*)(out + col) = u32x2{w[0], w[1]};
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (col + j < d) out[col + j] = (int8_t)(w[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
}

template <class E, int S, bool TAIL, int POLICY>
hipError_t go(const QuantParams& p, int grid, hipStream_t s) {
  constexpr int TR = kRowShape[S].threads, V = kRowShape[S].vecs;
  hipLaunchKernelGGL((quant_rows<E, TR, V, TAIL, POLICY>), dim3((unsigned)grid), dim3(TR < 256 ? 256 : TR), 0, s, p);
  return hipGetLastError();
}
template <class E, bool TAIL, int POLICY>
hipError_t by_shape(const QuantParams& p, int grid, hipStream_t s) {
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
hipError_t by_layout(bool large, const QuantParams& p, int grid, hipStream_t s) {
  if (p.d % 8) return by_shape<E, true, 0>(p, grid, s);
  return large ? by_shape<E, false, kLarge>(p, grid, s) : by_shape<E, false, 0>(p, grid, s);
}

}  // namespace

hipError_t launch_quant(bool bf16, bool large, const QuantParams& p, int grid, hipStream_t s) {
  if (grid <= 0) return hipSuccess;
  return bf16 ? by_layout<uint16_t>(large, p, grid, s) : by_layout<float>(large, p, grid, s);
}

}  // namespace ge
