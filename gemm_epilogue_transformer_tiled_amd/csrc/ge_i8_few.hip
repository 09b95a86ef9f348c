// Product of int8 codes, few rows (decoding): one pass over the weights (gfx950).
//
// With few rows what bounds the product is how many of the weights' bytes are in flight.  A workgroup takes 16
// columns (weight rows), or 8 where that spreads better, and all of K, which its eight waves split; their int32 sums meet in LDS, so there
// are no partial sums in memory, no tickets and no workspace.  A wave loads the weights straight into
// registers, 512 codes of all 16 rows at a time (eight loads, whole cache lines), and multiplies them with the
// tokens' codes by v_mfma_i32_16x16x64_i8; lane l holds 16 codes, 16 (l / 16) .. + 15 of 64, of weight row
// (token) l % 16.  The tokens' codes are brought to LDS first, their loads ahead of the weights'.  So few registers are
// needed that three workgroups run on a compute unit, which hides more than a second buffer of loads
// in each (one token, weights from memory: 4096 x 11008 11.5 us against 12.9 with two buffers, 11008 x 4096 11.5
// against 14.3, 4096 x 4096 6.3 against 7.1; 32 or 64 columns, with or without splits of K: 7 to 20 % slower and
// more).  The scales, the bias and the residual are on their way from the start: read after the sums, cold, they
// cost 1.2 us.
#include "ge_ffn_act.h"
#include "ge_rows_internal.h"

namespace ge {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
constexpr int kWaves = kI8FewWaves, kUnits = kI8FewStep / 128;

// RB: blocks of 16 tokens.
template <int RB>
__global__ __launch_bounds__(64 * kWaves) void i8_few(I8Few p) {
  constexpr int ROWS = 16 * RB, LD = kI8FewLd;
  // the tokens' codes; afterwards the waves' sums
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t l16 = (uint32_t)(lane & 15), q16 = (uint32_t)(lane >> 4);
  const int n0 = (int)blockIdx.x * p.cols, K = p.K, M = p.M;
  const int ncols = min(p.N - n0, p.cols);

  // ---- what the outputs need besides the sums: thread t ends columns 4 (t % 4) .. + 3 of row t / 4 ----
  const int row = tid / 4, col = 4 * (tid % 4);
  const bool live = row < M && col < ncols;            // (N is a multiple of 8: all four columns or none)
  static_assert(ROWS * 4 <= 64 * kWaves, "a thread for every four outputs");
  // (range-checked loads without a branch, kept as they come: nothing waits for them before the weights' loads; of
  // bf16 values the first eight bytes count)
  const uint32_t size = p.ep.wide ? 4u : 2u;
  auto at = [&](const void* base, int64_t extent, uint32_t offset) {
    return __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(base, base ? extent : 0), live ? offset : kOOB, 0, 0);
  };
  const uint32_t sx = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(p.ep.x_scale, 4 * (int64_t)M), live ? 4u * (uint32_t)row : kOOB, 0, 0);
  const u32x4_t sw = at(p.ep.w_scale + n0, 4 * (int64_t)ncols, 4u * (uint32_t)col);
  const u32x4_t bias = at((const unsigned char*)p.ep.bias + (p.ep.bias ? (int64_t)n0 * size : 0), (int64_t)ncols * size, (uint32_t)col * size);
  const u32x4_t res = at((const unsigned char*)p.R + (p.R ? (int64_t)n0 * size : 0), ((int64_t)(M - 1) * p.ldr + ncols) * size,
                         (__umul24((uint32_t)row, (uint32_t)p.ldr) + (uint32_t)col) * size);

  // ---- the tokens' codes to LDS, a row's kilobyte a load; past K zeros ----
  const int steps = (K + kI8FewStep - 1) / kI8FewStep, pieces = (steps * kI8FewStep + 1023) / 1024, pitch = p.x_pitch;
  for (int i = wave; i < M * pieces; i += kWaves) {
    const int r = i / pieces, at = (i - r * pieces) * 1024;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.X + (int64_t)r * p.ldx + at, K > at ? K - at : 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (__attribute__((address_space(3))) void*)(lds + r * pitch + at), 16,
                                             16u * (uint32_t)lane, 0, 0, 0);
  }

  // ---- the weights; rows past the last one get an offset past every extent, which reads zeros ----
  const uint32_t ldw = (uint32_t)p.ldw;
  const unsigned char* const pw = (const unsigned char*)p.W + (int64_t)n0 * p.ldw;
  const uint32_t wrow = (int)l16 < ncols ? __umul24(l16, ldw) + 16u * q16 : kOOB;      // (pitches are below 2^22)
  // Each workgroup starts its steps at a place of its own: all rows have the same pitch, and if all walked
  // K in step, a power-of-two pitch would put what they read at a time on a few of the memory channels.
  const int turn = steps > 0 ? (int)((blockIdx.x * (unsigned)kWaves) % (unsigned)steps) : 0;
  auto place = [&](int i) { return (i + turn < steps ? i + turn : i + turn - steps) * kI8FewStep; };
  u32x4_t w[kUnits][2];
  auto load = [&](int i) {                             // step i, or zeros past the last one
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int k0 = i < steps ? place(i) + 128 * u : 0, left = i < steps ? K - k0 : 0;
      const __amdgpu_buffer_rsrc_t wr = make_rsrc(pw + k0, left > 0 ? (int64_t)(ncols - 1) * ldw + left : 0);
#pragma unroll
      for (int h = 0; h < 2; ++h)                      // (the next row's codes follow a row's last)
        w[u][h] = __builtin_amdgcn_raw_buffer_load_b128(wr, (int)(16u * q16) + 64 * h < left ? wrow + 64u * h : kOOB, 0, 0);
    }
  };
  i32x4_t acc[RB];
  uint32_t xrow[RB];                                   // (tokens past the last one: the last one's, not used)
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    acc[r] = i32x4_t{};
    xrow[r] = (uint32_t)(min(16 * r + (int)l16, M - 1) * pitch) + 16u * q16;
  }
  __builtin_amdgcn_sched_barrier(0);                   // (the wait counts on this order)
  load(wave);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * kUnits));   // this wave's loads to LDS, all issued before the weights'
  __syncthreads();
  for (int i = wave; i < steps; i += kWaves) {
    const unsigned char* x = lds + place(i);
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < RB; ++r)
          acc[r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, w[u][h]),
                                                         *(const i32x4_t*)(x + xrow[r] + 128 * u + 64 * h), acc[r], 0, 0, 0);
    if (i + kWaves < steps) load(i + kWaves);          // uniform
  }
  __syncthreads();                                     // every wave is done with the codes

  // ---- the waves' sums (exact: their order does not matter); a lane holds token 16 r + l16, columns 4 q16 .. + 3 ----
  int* const sums = (int*)lds;
#pragma unroll
  for (int r = 0; r < RB; ++r) *(i32x4_t*)(sums + (wave * ROWS + 16 * r + (int)l16) * LD + 4 * (int)q16) = acc[r];
  __syncthreads();
  if (!live) return;
  i32x4_t v = i32x4_t{};
#pragma unroll
  for (int k = 0; k < kWaves; ++k) v += *(const i32x4_t*)(sums + (k * ROWS + row) * LD + col);
  auto value = [&](const u32x4_t& raw, int e) {
    return p.ep.wide ? __uint_as_float(raw[e]) : (e & 1) ? bf16_hi(raw[e >> 1]) : bf16_lo(raw[e >> 1]);
  };
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float t = (float)v[e] * __uint_as_float(sx), c = __uint_as_float(sw[e]), b = value(bias, e);
    const float r = p.R ? value(res, e) : -0.0f;
    switch (p.ep.act) {                                // uniform
      case ACT_RELU: y[e] = i8_output<ACT_RELU>(t, c, b, r); break;
      case ACT_GELU_TANH: y[e] = i8_output<ACT_GELU_TANH>(t, c, b, r); break;
      case ACT_SILU: y[e] = i8_output<ACT_SILU>(t, c, b, r); break;
      default: y[e] = i8_output<ACT_NONE>(t, c, b, r); break;
    }
  }
  const int64_t to = (int64_t)row * p.ldy + n0 + col;
  if (p.ep.wide) *(f32x4_t*)((float*)p.Y + to) = f32x4_t{y[0], y[1], y[2], y[3]};
  else *(u32x2_t*)((uint16_t*)p.Y + to) = u32x2_t{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
}

}  // namespace

hipError_t launch_i8_few(const I8Few& p, hipStream_t s) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  if (p.M > kI8FewRows || i8_few_lds(p.M, p.K) > kI8FewLds) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((p.N + p.cols - 1) / p.cols)), block(64 * kWaves);
  const unsigned bytes = (unsigned)i8_few_lds(p.M, p.K);
  if (p.M <= 16) hipLaunchKernelGGL(i8_few<1>, grid, block, bytes, s, p);
  else hipLaunchKernelGGL(i8_few<2>, grid, block, bytes, s, p);
  return hipGetLastError();
}

}  // namespace ge
