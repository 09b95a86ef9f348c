// Gated feed-forward block, few rows (decoding): the gate/up pair and the down projection.
//
// With up to 16 rows the products are one pass over the weights: what bounds them is how many of the
// weights' bytes are in flight.  So a tile is 128 columns of weights, and the contraction is split
// over the eight waves of a workgroup and over several workgroups, at most one a compute unit (a second
// one on some of them only makes the others wait); each wave streams its part of the weights straight
// into registers, one step ahead, and multiplies it with the rows by v_mfma_f32_16x16x32_bf16.  One row
// at 4096 x 11008: 53 us for 270 MB, [in][out]; 58 us [out][in].  No LDS is used on the way:
//   [N][K] weights   a lane's 16 bytes are the eight K values of one column that the matrix core
//                    wants from it
//   [K][N] weights   a lane loads eight rows of eight columns; pairing the rows' halves (32 byte
//                    permutes for 64 values) gives the eight K values of each of its columns, and
//                    fragment c takes column c of every lane
// The waves' sums meet in LDS in wave order, the workgroups' in the workspace in split order (the
// last workgroup of a tile, found by a ticket, adds them up), so equal calls give equal bits.
#include "ge_block_internal.h"
#include "ge_ffn_act.h"
#include "ge_ffn_few_addr.h"
#include "ge_kernel_impl.h"

namespace ge {
namespace {

constexpr int kFewCols = kFfnFewCols;
// Cache policy of the [K][N] weights ("nt", bit 1): each line is read whole by one load and not again;
// 3-5 us of 58 on one token at 4096 x 11008.  [N][K] lines are read by two loads of one wave: there
// the policy loses the second half (39 -> 47 us for the pair).
constexpr int kStream = 2;

template <int ACT, bool PAIR, bool BNK>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2)))
void ffn_few(FfnFew p) {
  constexpr int NB = PAIR ? 2 : 1, ROWS = kFfnFewRows, LD = kFewCols + 4, WV = 8;
  __shared__ __attribute__((aligned(16))) float sums[WV * ROWS * LD];
  __shared__ uint32_t last;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t l16 = (uint32_t)(lane & 15), q16 = (uint32_t)(lane >> 4);

  const int tile = blockIdx.x / p.splits, split = blockIdx.x - tile * p.splits;
  const int n0 = tile * kFewCols;
  const int mrows = p.M, N = p.N, K = p.K;
  const int ncols = min(N - n0, kFewCols);
  // the contraction in units of UNIT values, dealt to the waves of the splits in turn
  constexpr int UNIT = kFfnFewUnit;
  const int units = (K + UNIT - 1) / UNIT;
  const int u0 = (int)((int64_t)units * split / p.splits), u1 = (int)((int64_t)units * (split + 1) / p.splits);

  const uint32_t ldx2 = (uint32_t)p.lda * 2u, ldb2 = (uint32_t)p.ldb * 2u;
  const uint16_t* const px = p.A;
  const int64_t b_at = BNK ? (int64_t)n0 * p.ldb : (int64_t)n0;
  const uint16_t* const pw[2] = {p.B + b_at, PAIR ? p.B2 + b_at : p.B + b_at};
  // block c of a lane: row l16; columns 16 c + 4 q16 + e ([N][K]), 32 q16 + 8 e + c ([K][N])
  f32x4_t acc[NB][8];
#pragma unroll
  for (int op = 0; op < NB; ++op)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[op][c] = f32x4_t{};
  auto mac = [&](const u32x4_t& w, const u32x4_t& x, f32x4_t& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, x), c, 0, 0, 0);
  };

  // the next step's loads go out before the wait for this one's: left to itself the compiler's
  // schedule waits first, which halves the bytes in flight
  auto keep_order = [] { __builtin_amdgcn_sched_barrier(0); };

  if constexpr (BNK) {
    // A unit is 64 K values of all 128 columns, in two steps of four 16-column blocks: a load takes
    // 64 bytes of 16 rows, the two loads of a block a whole cache line of each
    struct W { u32x4_t v[NB][4][2]; };
    struct X { u32x4_t v[2]; };
    uint32_t column[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) column[c] = few_nk_column(l16, q16, c, ncols, ldb2);
    auto load_x = [&](X& t, int u) {
      const int k0 = u * UNIT, lim = u < u1 ? K - k0 : 0;
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(px + k0, few_row_extent(mrows, lim, ldx2));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        t.v[j] = __builtin_amdgcn_raw_buffer_load_b128(rs, few_x_offset(l16, q16, j, lim, ldx2), 0, 0);
    };
    auto load_w = [&](W& t, int u, int cp) {
      const int k0 = u * UNIT, lim = u < u1 ? K - k0 : 0;
#pragma unroll
      for (int op = 0; op < NB; ++op) {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(pw[op] + k0, few_row_extent(ncols, lim, ldb2));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            t.v[op][i][j] = __builtin_amdgcn_raw_buffer_load_b128(rs, few_nk_offset(column[4 * cp + i], q16, j, lim), 0, 0);
      }
    };
    auto multiply = [&](const W& w, const X& x, auto cp_c) {
      constexpr int CP = decltype(cp_c)::value;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int op = 0; op < NB; ++op)
#pragma unroll
          for (int i = 0; i < 4; ++i) mac(w.v[op][i][j], x.v[j], acc[op][4 * CP + i]);
    };
    // Each tile starts its units at a place of its own: all rows have the same pitch, and if the tiles
    // walked K in step, a power-of-two pitch would put what they read at a time on a few of the
    // memory channels.
    const int n = u1 - u0, turn = n > 0 ? tile * WV % n : 0;
    auto unit = [&](int i) { return i >= n ? u1 : u0 + (i + turn < n ? i + turn : i + turn - n); };
    W a, b;
    X x, xn;
    int i = wave, u = unit(i);
    load_x(x, u);
    load_w(a, u, 0);
    for (; i < n; i += WV) {
      load_w(b, u, 1);
      keep_order();
      multiply(a, x, std::integral_constant<int, 0>{});
      keep_order();
      u = unit(i + WV);
      load_x(xn, u);
      load_w(a, u, 0);
      keep_order();
      multiply(b, x, std::integral_constant<int, 1>{});
      keep_order();
      x = xn;
    }
  } else {
    // A unit is two 32-deep steps; a lane's step is eight rows of eight columns.
    struct Step { u32x4_t w[NB][8], x; };
    uint32_t value[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) value[k] = few_kn_offset(l16, q16, k, ncols, ldb2);
    auto load = [&](Step& t, int u, int half) {
      const int k0 = u * UNIT + 32 * half, lim = u < u1 ? K - k0 : 0;      // past the split's end: zeros
      const __amdgpu_buffer_rsrc_t xr = make_rsrc(px + k0, few_row_extent(mrows, lim, ldx2));
      t.x = __builtin_amdgcn_raw_buffer_load_b128(xr, few_x_offset(l16, q16, 0, lim, ldx2), 0, 0);
#pragma unroll
      for (int op = 0; op < NB; ++op) {
        const __amdgpu_buffer_rsrc_t wr = make_rsrc((const unsigned char*)pw[op] + (uint64_t)(uint32_t)k0 * ldb2,
                                                    few_kn_extent(ncols, lim, ldb2));
#pragma unroll
        for (int k = 0; k < 8; ++k) t.w[op][k] = __builtin_amdgcn_raw_buffer_load_b128(wr, value[k], 0, kStream);
      }
    };
    auto multiply = [&](const Step& t) {
#pragma unroll
      for (int op = 0; op < NB; ++op)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          u32x4_t f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            f[j] = __builtin_amdgcn_perm(t.w[op][2 * j + 1][c >> 1], t.w[op][2 * j][c >> 1],
                                         (c & 1) ? 0x07060302u : 0x05040100u);
          mac(f, t.x, acc[op][c]);
        }
    };
    Step a, b;
    int u = u0 + wave;
    load(a, u, 0);
    for (; u < u1; u += WV) {
      load(b, u, 1);
      keep_order();
      multiply(a);
      keep_order();
      load(a, u + WV, 0);
      keep_order();
      multiply(b);
      keep_order();
    }
  }

  // ---- the waves' sums, one operand after the other, to registers of the thread that ends the
  // element: thread t takes columns 4 (t % 32) .. +3 of rows t / 32 + RS i ----
  constexpr int RS = 2 * WV, PER = ROWS / RS;          // rows a thread ends
  const int tc = 4 * (tid & 31), tr = tid >> 5;
  f32x4_t v[NB][PER];
#pragma unroll
  for (int op = 0; op < NB; ++op) {
    if (op > 0) __syncthreads();
    float* row = sums + (wave * ROWS + (int)l16) * LD;
    if constexpr (BNK) {
#pragma unroll
      for (int c = 0; c < 8; ++c) *(f32x4_t*)(row + 16 * c + 4 * (int)q16) = acc[op][c];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *(f32x4_t*)(row + 32 * (int)q16 + 8 * e + 4 * h) =
              f32x4_t{acc[op][4 * h][e], acc[op][4 * h + 1][e], acc[op][4 * h + 2][e], acc[op][4 * h + 3][e]};
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      f32x4_t t = *(const f32x4_t*)(sums + (tr + RS * i) * LD + tc);
#pragma unroll
      for (int w = 1; w < WV; ++w) t += *(const f32x4_t*)(sums + (w * ROWS + tr + RS * i) * LD + tc);
      v[op][i] = t;
    }
  }

  // ---- the splits' sums: partials and tickets go through device scope, as in ge_kernel_impl.h
  // (the partials are performed before the ticket; the last workgroup reads them after it) ----
  if (p.splits > 1) {
    typedef unsigned long long u64;
    u64* mine = (u64*)(p.part + ((int64_t)tile * p.splits + split) * (NB * ROWS * kFewCols));
#pragma unroll
    for (int op = 0; op < NB; ++op)
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (tr + RS * i < mrows) {
          u64* at = mine + ((op * ROWS + tr + RS * i) * kFewCols + tc) / 2;
          u64 w[2];
          __builtin_memcpy(w, &v[op][i], 16);
          __hip_atomic_store(at, w[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(at + 1, w[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    __builtin_amdgcn_s_waitcnt(kVmcnt0);
    __syncthreads();
    if (tid == 0) {
      uint32_t* ctr = p.ctr + (uint32_t)tile * kFfnCtrStride;
      const bool l = __hip_atomic_fetch_add(ctr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)p.splits - 1u;
      if (l) __hip_atomic_store(ctr, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = l ? 1u : 0u;
    }
    __syncthreads();
    if (!last) return;                                 // uniform
    // every element's partials of AHEAD splits are on their way at once, added in split order
    const u64* all = (const u64*)(p.part + (int64_t)tile * p.splits * (NB * ROWS * kFewCols));
    constexpr int AHEAD = 4;
#pragma unroll
    for (int op = 0; op < NB; ++op)
#pragma unroll
      for (int i = 0; i < PER; ++i) v[op][i] = f32x4_t{};
    for (int q0 = 0; q0 < p.splits; q0 += AHEAD) {
      u64 w[AHEAD][NB][PER][2];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q)
#pragma unroll
        for (int op = 0; op < NB; ++op)
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            w[q][op][i][0] = w[q][op][i][1] = 0;
            if (q0 + q < p.splits && tr + RS * i < mrows) {
              const u64* at = all + ((int64_t)(q0 + q) * (NB * ROWS * kFewCols) + (op * ROWS + tr + RS * i) * kFewCols + tc) / 2;
              w[q][op][i][0] = __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
              w[q][op][i][1] = __hip_atomic_load(at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
          }
#pragma unroll
      for (int q = 0; q < AHEAD; ++q)
#pragma unroll
        for (int op = 0; op < NB; ++op)
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            f32x4_t o;
            __builtin_memcpy(&o, w[q][op][i], 16);
            v[op][i] += o;
          }
    }
  }

  // ---- epilogue: 4 columns of PER rows a thread ----
  if (tc >= ncols) return;
  auto put = [&](uint16_t* base, int64_t ld, int row, const f32x4_t& y) {
    u32x2_t w;
    w[0] = pack_bf16x2(y[0], y[1]);
    w[1] = pack_bf16x2(y[2], y[3]);
    *(u32x2_t*)(base + (int64_t)row * ld + n0 + tc) = w;
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = tr + RS * i;
    if (row >= mrows) continue;
    if constexpr (PAIR) {
      f32x4_t h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = gate<ACT>(v[0][i][e]) * v[NB - 1][i][e];
      put(p.Y, p.ldy, row, h);
      if (p.Y2) {
        put(p.Y2, p.ldy2, row, v[0][i]);
        put(p.Y3, p.ldy2, row, v[NB - 1][i]);
      }
    } else {
      f32x4_t y = v[0][i];
      if (p.E1) {
        const u32x2_t w = *(const u32x2_t*)(p.E1 + (int64_t)row * p.lde + n0 + tc);
        y[0] += bf16_lo(w[0]);
        y[1] += bf16_hi(w[0]);
        y[2] += bf16_lo(w[1]);
        y[3] += bf16_hi(w[1]);
      }
      put(p.Y, p.ldy, row, y);
    }
  }
}

template <int ACT, bool PAIR, bool BNK>
hipError_t go(const FfnFew& p, hipStream_t s) {
  hipLaunchKernelGGL((ffn_few<ACT, PAIR, BNK>), dim3((unsigned)(p.tiles * p.splits)), dim3(512), 0, s, p);
  return hipGetLastError();
}

template <bool BNK>
hipError_t by_act(int act, const FfnFew& p, hipStream_t s) {
  switch (act) {
    case ACT_NONE: return go<ACT_NONE, true, BNK>(p, s);
    case ACT_RELU: return go<ACT_RELU, true, BNK>(p, s);
    case ACT_GELU_TANH: return go<ACT_GELU_TANH, true, BNK>(p, s);
    case ACT_SILU: return go<ACT_SILU, true, BNK>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_ffn_few(bool pair, int act, bool b_nk, const FfnFew& p, hipStream_t s) {
  if (p.tiles <= 0) return hipSuccess;
  if (pair) return b_nk ? by_act<true>(act, p, s) : by_act<false>(act, p, s);
  return b_nk ? go<ACT_NONE, false, true>(p, s) : go<ACT_NONE, false, false>(p, s);
}

}  // namespace ge
