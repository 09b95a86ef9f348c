#pragma once
// Products of the gated feed-forward block for MI355X (gfx950): kernel templates.
//
// Five products share one mainloop (FfnMode, ge_block_internal.h):
//   PAIR   G = X Wg, U = X Wu on one staged X tile; the epilogue writes H = act(G) * U and, for
//          training, G and U
//   DOWN   Y = H Wd (+ R)
//   GRAD   dH = dY Wd^T stays in registers; the epilogue reads G and U and writes dG, dU and H
//   DUAL   dX = dG Wg^T + dU Wu^T: one accumulator, the contraction runs over both products
//   WGRAD  dWg = X^T dG, dWu = X^T dU, dWd = H^T dY: one launch, both operands contraction-major
//
// Operand forms.  "Row" operands have the contraction contiguous ([rows][K]); they are staged as
// [rows][64] with 128-byte rows and read as fragments by plain 16-byte LDS reads.  "Column"
// operands are contraction-major ([K][cols]); they are staged as they lie, [k][cols], and read
// through transposing LDS reads.  Either side of the product can be either form, so no operand
// is ever transposed in memory: A is a row operand except for WGRAD; B follows the weight layout.
//
// Every step multiplies with v_mfma_f32_16x16x32_bf16 in ascending K, whatever the tile, so all
// tiles give the same bits for the same product.  Operands reach LDS by direct global->LDS loads.
// A step's buffer resource carries its K position: the base moves along K, the extent shrinks to
// the rows (columns) the tile has, and 16-byte chunks past K or past the last column get an
// offset outside the extent, which reads zeros -- ragged sizes take no branch, and no offset
// grows with the tensors (they stay below 256 rows of one leading dimension).
//
// Loops.  256-row tiles: 8 waves, two per SIMD, in two groups that alternate a memory phase
// (fragment reads, later steps' loads) and a matrix phase, as in ge_kernel_impl.h; every step carries
// 32 KB of loads.  128-row tiles: 8 waves, 64-row tiles: 4, a ring of NSLOT 64-deep slots, one barrier
// per slot; their contraction may be split over workgroups (few tiles, long contractions).
//
// What bounds them (8192 x 4096 x 11008, bf16): the matrix cores under the power limit.  Forward pair
// 1,060-1,110 us (1.33-1.39 PFLOP/s, with 540 MB of stores in the epilogue), down 509 us (1.45), input
// gradient 975 us (1.52), weight gradients 1,600-1,680 us (1.32-1.38); the gated gradient 670 us (1.10):
// its epilogue moves 900 MB (G, U in; dG, dU, H out) that the loop does not hide.
#include "ge_block_internal.h"
#include "ge_ffn_act.h"
#include "ge_kernel_impl.h"

namespace ge {
namespace {

template <int BM_, int BN_, int NB_, int WAVES_, int NSLOT_, bool PP_ = false>
struct FTile {
  static constexpr int BM = BM_, BN = BN_, NB = NB_, WAVES = WAVES_, NSLOT = NSLOT_;
  static constexpr bool PP = PP_;                     // two waves per SIMD, alternating phases
  static constexpr int NT = 64 * WAVES, WGN = WAVES / 2;
  static constexpr int WM = BM / 2, WN = BN / WGN;    // per-wave output: 2 x WGN waves
  static constexpr int FM = WM / 16, FN = WN / 16;
  static constexpr int A_SLOT = BM * 128;             // 64-deep slot of A
  static constexpr int B_OP = BN * 128;               // 64-deep slot of one B operand
  static constexpr int B_SLOT = NB * B_OP;
  static constexpr int LA = A_SLOT / 1024 / WAVES;    // 1-KB loads per wave per slot
  static constexpr int LB = B_SLOT / 1024 / WAVES;
  static constexpr int EP_LD = WN + 4;                // epilogue block: 32 rows, padded by 16 bytes
  static constexpr int EP_WAVE = 32 * EP_LD * 4;
  // the epilogue blocks lie in the operands' arrays: two-wave tiles EP_PER to each A array and the
  // last two in B's, the others half of them in each of the first two A arrays
  static constexpr int EP_PER = PP ? A_SLOT / EP_WAVE : WGN;
  static constexpr int A_ALLOC = A_SLOT > WGN * EP_WAVE || PP ? A_SLOT : WGN * EP_WAVE;
  static_assert(2 * EP_PER + 2 >= WAVES || !PP, "epilogue blocks");
  static_assert(A_SLOT % (1024 * WAVES) == 0 && B_SLOT % (1024 * WAVES) == 0, "loads divide over the waves");
  static_assert(WM % 32 == 0 && WN % 16 == 0, "epilogue blocks");
  static_assert(!PP || (WAVES == 8 && NSLOT == 2 && LB % 2 == 0), "two-wave loop: two slots");
  static_assert(NSLOT >= 2 && NSLOT <= 5, "slot arrays");
};

// Chunk swizzle of a row operand's staged row: chunk c of row r lies at c ^ (r & 6).  A 16-byte LDS
// read serves, in one pass, lanes 0-3, 12-15 and 20-27 (then 4-11, 16-19, 28-31; the same above 32): with
// K chunk c for lanes 0-15 and c ^ 1 for lanes 16-31, the even rows of the first set (0 2 12 14 at c, 4 6 8 10
// at c ^ 1) fall on the even, the others on the odd chunks, and no two on one bank.  (Measured:
// SQ_LDS_BANK_CONFLICT 1.4e8 of 2.7e8 LDS cycles on the two-row-operand product with a swizzle that
// separates lanes 0-15 instead.)
__device__ __forceinline__ uint32_t swz_row(uint32_t r) { return r & 6u; }

// Chunk swizzle of a column operand's staged row k (see swz_b16); rows of eight chunks have no
// fourth chunk bit to flip.
template <int CHUNKS>
__device__ __forceinline__ uint32_t swz_col(uint32_t k) {
  if constexpr (CHUNKS >= 16) return swz_b16<CHUNKS>(k);
  return swz_b<CHUNKS>(k) ^ ((k >> 3) & 1u);
}

// act(z) and act'(z) from one exponential and one reciprocal.  The GELU's cubic is taken where it
// still changes the sigmoid in fp32, so that squares of huge finite values do not turn 0 * inf into
// NaN (NaN arguments stay NaN).
template <int ACT>
__device__ __forceinline__ void act_and_slope(float z, float& a, float& s) {
  if constexpr (ACT == ACT_RELU) {
    a = relu_nan(z);
    s = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float c = z > 200.0f ? 200.0f : (z < -200.0f ? -200.0f : z), q = kGeluCubic * c * c;
    const float g = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(kGeluC * c * (1.0f + q)));
    a = z * g;
    s = g + 2.0f * 0.7978845608028654f * c * g * (1.0f - g) * (1.0f + 3.0f * q);
  } else if constexpr (ACT == ACT_SILU) {
    const float g = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
    a = z * g;
    s = g * (1.0f + z * (1.0f - g));
  } else {
    a = z;
    s = 1.0f;
  }
}

template <class T, int MODE, int ACT, bool AC, bool BC>
__global__ __launch_bounds__(T::NT) __attribute__((amdgpu_waves_per_eu(T::PP ? 2 : 1, T::PP ? 2 : 8)))
void ffn_product(FfnLaunch l) {
  constexpr bool PAIR = MODE == FFN_PAIR, DUAL = MODE == FFN_DUAL;
  constexpr int NB = T::NB;
  static_assert((NB == 2) == PAIR, "two B operands: the gate/up pair");
  constexpr int BST = T::B_SLOT / 2;                   // 32-deep stage of B (two-wave loop, column B)
  constexpr int B01 = (T::PP && BC) ? BST : T::B_SLOT;
  constexpr int B2B = (T::PP && BC) ? BST : (T::PP || T::NSLOT > 2 ? T::B_SLOT : 16);
  constexpr int B3B = (T::PP && BC) ? BST : (T::NSLOT > 3 ? T::B_SLOT : 16);
  constexpr int A2B = T::NSLOT > 2 ? T::A_SLOT : 16, A3B = T::NSLOT > 3 ? T::A_SLOT : 16;
  constexpr int A4B = T::NSLOT > 4 ? T::A_SLOT : 16, B4B = T::NSLOT > 4 ? T::B_SLOT : 16;
  // distinct arrays: the compiler can tell that a load into one does not alias reads of another
  __shared__ __attribute__((aligned(1024))) unsigned char a0[T::A_ALLOC];
  __shared__ __attribute__((aligned(1024))) unsigned char a1[T::A_ALLOC];
  __shared__ __attribute__((aligned(1024))) unsigned char a2[A2B];
  __shared__ __attribute__((aligned(1024))) unsigned char a3[A3B];
  __shared__ __attribute__((aligned(1024))) unsigned char a4[A4B];
  __shared__ __attribute__((aligned(1024))) unsigned char b0[B01];
  __shared__ __attribute__((aligned(1024))) unsigned char b1[B01];
  __shared__ __attribute__((aligned(1024))) unsigned char b2[B2B];
  __shared__ __attribute__((aligned(1024))) unsigned char b3[B3B];
  __shared__ __attribute__((aligned(1024))) unsigned char b4[B4B];
  static_assert(2 * T::A_ALLOC + A2B + A3B + A4B + 2 * B01 + B2B + B3B + B4B <= 160 * 1024 + 6 * 16, "LDS of a workgroup (16-byte arrays are unused ones)");
  auto a_arr = [&](auto i) -> unsigned char* {
    if constexpr (decltype(i)::value == 0) return a0;
    else if constexpr (decltype(i)::value == 1) return a1;
    else if constexpr (decltype(i)::value == 2) return a2;
    else if constexpr (decltype(i)::value == 3) return a3;
    else return a4;
  };
  auto b_arr = [&](auto i) -> unsigned char* {
    if constexpr (decltype(i)::value == 0) return b0;
    else if constexpr (decltype(i)::value == 1) return b1;
    else if constexpr (decltype(i)::value == 2) return b2;
    else if constexpr (decltype(i)::value == 3) return b3;
    else return b4;
  };
#define GE_I(n) std::integral_constant<int, (n)>{}

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave & 1) * T::WM, wn0 = (wave >> 1) * T::WN;
  const uint32_t l16 = (uint32_t)(lane & 15), q16 = (uint32_t)(lane >> 4);

  // ---- tile: contiguous runs per XCD (workgroups are dealt round-robin over the 8 dies), the
  // launch's products one after the other, tile rows walked in groups for L2 reuse ----
  int id;
  const int splits = T::PP ? 1 : l.splits;
  {
    const int total = l.tiles * splits, x = (int)blockIdx.x % kXCDs, loc = (int)blockIdx.x / kXCDs;
    const int per = (total + kXCDs - 1) / kXCDs;
    int tall = total % kXCDs;
    if (tall == 0) tall = kXCDs;
    id = x < tall ? x * per + loc : tall * per + (x - tall) * (per - 1) + loc;
  }
  const int split = T::PP ? 0 : id / l.tiles, tile_id = id - split * l.tiles;
  id = tile_id;
  int pi = 0;
  if (MODE == FFN_WGRAD) pi = (l.n > 1 && id >= l.prod[1].tile0) + (l.n > 2 && id >= l.prod[2].tile0);
  const FfnProduct& p = l.prod[pi];
  id -= p.tile0;
  const int span = kGroupM * p.tiles_n, grp_i = id / span;
  const int first_m = grp_i * kGroupM, gsize = min(p.tiles_m - first_m, kGroupM);
  const int m0 = (first_m + (id - grp_i * span) % gsize) * T::BM, n0 = ((id - grp_i * span) / gsize) * T::BN;
  const int M = p.M, N = p.N, K = p.K;
  const int mrows = min(M - m0, T::BM), ncols = min(N - n0, T::BN);

  // ---- step resources ----
  const uint32_t lda2 = (uint32_t)p.lda * 2u, ldb2 = (uint32_t)p.ldb * 2u;
  const int64_t a_at = AC ? (int64_t)m0 : (int64_t)m0 * p.lda, b_at = BC ? (int64_t)n0 : (int64_t)n0 * p.ldb;
  // contraction position of step j: DUAL runs through [0, K) twice, each pass padded to slots
  const int seg = 2 * ((K + 63) / 64);                 // steps of one pass, an even number
  const int nk = (DUAL ? 2 : 1) * seg;                 // 32-deep steps; those past the end read zeros
  // 64-deep slots of this workgroup's split
  const int slot0 = T::PP ? 0 : (int)((int64_t)(nk / 2) * split / splits);
  const int slot1 = T::PP ? nk / 2 : (int)((int64_t)(nk / 2) * (split + 1) / splits);
  auto second = [&](int j) { return DUAL && j >= seg; };
  auto kpos = [&](int j) { return (second(j) ? j - seg : j) * 32; };
  __amdgpu_buffer_rsrc_t ars, brs, brs2;
  int a_lim = 0, b_lim = 0;                            // row operands: K values left from the step's first
  // (32-bit byte extents: leading dimensions are below 2^22 elements, checked on the host)
  const uint16_t* const pa = p.A + a_at;
  const uint16_t* const pa2 = DUAL ? p.A2 + a_at : pa;
  const uint16_t* const pb = p.B + b_at;
  const uint16_t* const pb2 = (DUAL || PAIR) ? p.B2 + b_at : pb;
  auto extent = [](bool col, int lim, int rows, uint32_t ld2) -> int {
    const int whole = col ? (min(lim, 64) - 1) * (int)ld2 + rows * 2 : (rows - 1) * (int)ld2 + lim * 2;
    return lim > 0 ? whole : 0;
  };
  auto at_k = [](bool col, const uint16_t* base, int k0, uint32_t ld2) -> const void* {
    return (const unsigned char*)base + (col ? (uint64_t)(uint32_t)k0 * ld2 : (uint64_t)((uint32_t)k0 * 2u));
  };
  auto set_a = [&](int j) {
    const int k0 = kpos(j);
    a_lim = (T::PP || j < 2 * slot1) ? K - k0 : 0;
    ars = make_rsrc(at_k(AC, second(j) ? pa2 : pa, k0, lda2), extent(AC, a_lim, mrows, lda2));
  };
  auto set_b = [&](int j) {
    const int k0 = kpos(j);
    b_lim = (T::PP || j < 2 * slot1) ? K - k0 : 0;
    const int ext = extent(BC, b_lim, ncols, ldb2);
    brs = make_rsrc(at_k(BC, second(j) ? pb2 : pb, k0, ldb2), ext);
    if constexpr (PAIR) brs2 = make_rsrc(at_k(BC, pb2, k0, ldb2), ext);
  };

  // ---- direct loads: per-lane offsets, fixed for the whole loop ----
  // row operand, load u of a slot: rows 8u .. 8u+7, lane -> row lane / 8, physical chunk lane % 8
  // column operand, load u: rows u * RPL .. of the slot or stage, CHUNKS lanes per row
  const uint32_t r_x = (uint32_t)(lane & 7) ^ swz_row((uint32_t)(lane >> 3));     // its logical chunk
  constexpr int ACH = T::BM / 8, BCH = T::BN / 8;      // chunks per staged row of a column operand
  uint32_t a_voff[T::LA], b_voff[T::LB];
#pragma unroll
  for (int t = 0; t < T::LA; ++t) {
    const uint32_t u = (uint32_t)(wave * T::LA + t);
    if constexpr (AC) {
      const uint32_t row = u * (64 / ACH) + (uint32_t)lane / ACH, c = ((uint32_t)lane % ACH) ^ swz_col<ACH>(row);
      a_voff[t] = (int)(c * 8) < mrows ? row * lda2 + c * 16u : kOOB;
    } else {
      a_voff[t] = (8u * u + (uint32_t)(lane >> 3)) * lda2 + r_x * 16u;
    }
  }
  // loads of one B fill: a slot (LB per wave), or a 32-deep stage (LB / 2) in the two-wave loop
  constexpr bool BSTAGE = T::PP && BC;
  constexpr int LBF = BSTAGE ? T::LB / 2 : T::LB;
  constexpr int B_UNITS = (BSTAGE ? T::B_OP / 2 : T::B_OP) / 1024;   // loads per operand per fill
#pragma unroll
  for (int t = 0; t < LBF; ++t) {
    const uint32_t u = (uint32_t)(wave * LBF + t) % (uint32_t)B_UNITS;
    if constexpr (BC) {
      const uint32_t row = u * (64 / BCH) + (uint32_t)lane / BCH, c = ((uint32_t)lane % BCH) ^ swz_col<BCH>(row);
      b_voff[t] = (int)(c * 8) < ncols ? row * ldb2 + c * 16u : kOOB;
    } else {
      b_voff[t] = (8u * u + (uint32_t)(lane >> 3)) * ldb2 + r_x * 16u;
    }
  }
  // Row operands whose K is not a multiple of a slot: chunks past K get the out-of-range offset.
  // With K a multiple of 64 (WHOLE) a slot is inside K or its extent is empty: the loop without the
  // masks' vector instructions is up to 10 % faster on two row operands.
  auto issue_a = [&](auto whole, unsigned char* slot) {
    constexpr bool MASK = !AC && !decltype(whole)::value;
    const bool in_k = (int)(r_x * 8u) < a_lim;
#pragma unroll
    for (int t = 0; t < T::LA; ++t) {
      const uint32_t u = (uint32_t)(wave * T::LA + t);
      uint32_t off = a_voff[t];
      if constexpr (MASK) off = in_k ? off : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ars, (__attribute__((address_space(3))) void*)(slot + u * 1024), 16, off,
                                               0, 0, 0);
    }
  };
  auto issue_b = [&](auto whole, unsigned char* dst) {
    constexpr bool MASK = !BC && !decltype(whole)::value;
    const bool in_k = (int)(r_x * 8u) < b_lim;
#pragma unroll
    for (int t = 0; t < LBF; ++t) {
      const uint32_t g = (uint32_t)(wave * LBF + t);   // wave-uniform
      uint32_t off = b_voff[t];
      if constexpr (MASK) off = in_k ? off : kOOB;
      if (PAIR && g >= (uint32_t)B_UNITS)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(brs2, (__attribute__((address_space(3))) void*)(dst + g * 1024), 16, off,
                                                 0, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(brs, (__attribute__((address_space(3))) void*)(dst + g * 1024), 16, off,
                                                 0, 0, 0);
    }
  };

  // ---- fragments: a lane holds K 8 * (lane / 16) .. +7 of row (column) lane % 16 of a block ----
  // row operand: chunk 4h + lane / 16 of the staged row (h: which half of the slot); blocks of 16 rows
  // are immediate offsets
  uint32_t ar[2], br[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = ((4u * (uint32_t)h + q16) ^ swz_row(l16)) << 4;
    ar[h] = ((uint32_t)wm0 + l16) * 128u + c;
    br[h] = ((uint32_t)wn0 + l16) * 128u + c;
  }
  // column operand: in each group of 16 lanes, lane s points at rows 8 q + s / 4 (and + 4) and
  // columns nb + 4 (s % 4) .. +3, and receives column nb + s of the four rows
  const uint32_t k16 = 8u * q16 + (l16 >> 2);
  uint32_t ac[AC ? T::FM : 1], bc[BC ? T::FN : 1];
  if constexpr (AC) {
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
      const uint32_t col = (uint32_t)(wm0 + 16 * i) + 4u * (l16 & 3u);
      ac[i] = k16 * (T::BM * 2u) + (((col >> 3) ^ swz_col<ACH>(k16)) << 4) + (col & 7u) * 2u;
    }
  }
  if constexpr (BC) {
#pragma unroll
    for (int i = 0; i < T::FN; ++i) {
      const uint32_t col = (uint32_t)(wn0 + 16 * i) + 4u * (l16 & 3u);
      bc[i] = k16 * (T::BN * 2u) + (((col >> 3) ^ swz_col<BCH>(k16)) << 4) + (col & 7u) * 2u;
    }
  }
  typedef __attribute__((address_space(3))) v4bf16_t lds_v4bf16;
  auto tr_read = [](const unsigned char* q, int pitch) -> bf16x8_t {
    const v4bf16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4bf16*)(q));
    const v4bf16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4bf16*)(q + 4 * pitch));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  struct Frags {
    bf16x8_t a[T::FM], b[NB][T::FN];
  };
  // fragments of one 32-deep step: half h of the slots, or (staged B) the whole stage
  auto read_frags = [&](Frags& f, const unsigned char* as, const unsigned char* bs, int h) {
#pragma unroll
    for (int i = 0; i < T::FM; ++i) {
      if constexpr (AC) f.a[i] = tr_read(as + ac[i] + h * 32 * (T::BM * 2), T::BM * 2);
      else f.a[i] = *(const bf16x8_t*)(as + ar[h] + i * 16 * 128);
    }
#pragma unroll
    for (int op = 0; op < NB; ++op)
#pragma unroll
      for (int i = 0; i < T::FN; ++i) {
        if constexpr (BC) {
          constexpr int opb = BSTAGE ? T::B_OP / 2 : T::B_OP;
          f.b[op][i] = tr_read(bs + bc[i] + op * opb + (BSTAGE ? 0 : h * 32 * (T::BN * 2)), T::BN * 2);
        } else {
          f.b[op][i] = *(const bf16x8_t*)(bs + br[h] + i * 16 * 128 + op * T::B_OP);
        }
      }
  };
  // block (i, j): lane holds row 16 j + lane % 16, columns 16 i + 4 (lane / 16) .. +3
  f32x4_t acc[NB][T::FN][T::FM];
#pragma unroll
  for (int op = 0; op < NB; ++op)
#pragma unroll
    for (int i = 0; i < T::FN; ++i)
#pragma unroll
      for (int j = 0; j < T::FM; ++j) acc[op][i][j] = f32x4_t{};
  auto mfmas = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < T::FN; ++i)
#pragma unroll
      for (int j = 0; j < T::FM; ++j)
#pragma unroll
        for (int op = 0; op < NB; ++op)
          acc[op][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[op][i], f.a[j], acc[op][i][j], 0, 0, 0);
  };
  // a workgroup barrier that no LDS access moves across (the waits are explicit)
  auto barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  auto run = [&](auto whole) {
  if constexpr (T::PP) {
    // ---- two wave groups, one phase apart (ge_kernel_impl.h describes the phases) ----
    // Even steps j load the A slot of steps j+2, j+3; odd steps load B: a column B's stages of steps
    // j+2, j+3, a row B's slot of steps j+3, j+4 into the third of its arrays.  So every step moves
    // 32 KB, and a load has at least two phases to land.  (With two arrays for a row B its slot has to
    // come with A's, 64 KB on even steps: 1,140 us instead of 975 for the input gradient, 745 instead of
    // 670 for the gated gradient, at 8192 x 4096 x 11008.)
    const int grp = wave >> 2;
    Frags f;
    set_a(0);
    issue_a(whole, a0);
    if constexpr (BC) {
      set_b(0); issue_b(whole, b0);
      set_b(1); issue_b(whole, b1);
      set_b(2); issue_b(whole, b2);
    } else {
      set_b(0); issue_b(whole, b0);
      set_b(2); issue_b(whole, b1);
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(BC ? 2 * LBF : LBF));
    barrier();
    if (grp == 1) barrier();
    auto mem_phase = [&](auto s_c, int j) {
      constexpr int S = decltype(s_c)::value;          // step of the unrolled ring
      constexpr bool EVEN = S % 2 == 0;
      unsigned char* as = a_arr(GE_I(S / 2 % 2));
      unsigned char* bs = BC ? b_arr(GE_I(S % 4)) : b_arr(GE_I(S / 2 % 3));
      // this step's fragments before the later steps' loads: the phase waits for the reads
      read_frags(f, as, bs, S % 2);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (EVEN) {
        set_a(j + 2);
        issue_a(whole, a_arr(GE_I((S / 2 + 1) % 2)));
      } else if constexpr (BC) {
        set_b(j + 2);
        issue_b(whole, b_arr(GE_I((S + 2) % 4)));
        set_b(j + 3);
        issue_b(whole, b_arr(GE_I((S + 3) % 4)));
      } else {
        set_b(j + 3);
        issue_b(whole, b_arr(GE_I((S / 2 + 2) % 3)));
      }
      // loads younger than those of step j+1: column B, even steps -- the stage of j+2 that came with
      // j+1's, and A; odd steps -- this step's stages.  Row B: step j+1 of the same slot needs nothing new
      // (even); the next slot's A came a step ago and its B three, so all but this step's B (odd).
      constexpr int YOUNGER = BC ? (EVEN ? LBF + T::LA : 2 * LBF) : (EVEN ? LBF + T::LA : LBF);
      __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(YOUNGER));
      barrier();
    };
    auto mat_phase = [&]() {
      __builtin_amdgcn_s_setprio(1);
      mfmas(f);
      __builtin_amdgcn_s_setprio(0);
      barrier();
    };
    auto step = [&](auto s_c, int j) {
      mem_phase(s_c, j);
      mat_phase();
    };
    // whole rings: four steps (A and a column B), twelve with a row B's three arrays
    constexpr int RING = BC ? 4 : 12;
    for (int j = 0; j < nk; j += RING) {
      step(GE_I(0), j);
      step(GE_I(1), j + 1);
      step(GE_I(2), j + 2);
      step(GE_I(3), j + 3);
      if constexpr (RING == 12) {
        step(GE_I(4), j + 4);
        step(GE_I(5), j + 5);
        step(GE_I(6), j + 6);
        step(GE_I(7), j + 7);
        step(GE_I(8), j + 8);
        step(GE_I(9), j + 9);
        step(GE_I(10), j + 10);
        step(GE_I(11), j + 11);
      }
    }
    if (grp == 0) barrier();
  } else {
    // ---- ring of NSLOT slots: slot s is read while s+1 .. s+NSLOT-1 are on their way ----
    constexpr int NS = T::NSLOT, L = T::LA + LBF;
    auto fill = [&](auto i_c, int s) {
      set_a(2 * s);
      issue_a(whole, a_arr(i_c));
      set_b(2 * s);
      issue_b(whole, b_arr(i_c));
    };
    fill(GE_I(0), slot0);
    if constexpr (NS > 2) fill(GE_I(1), slot0 + 1);
    if constexpr (NS > 3) fill(GE_I(2), slot0 + 2);
    if constexpr (NS > 4) fill(GE_I(3), slot0 + 3);
    // the next slot has landed (this wave's part) and this wave is done reading this one: after the
    // barrier both hold for every wave, so the next slot may be read and this one refilled
    auto next = [&]() {
      __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm((NS - 2) * L));
      barrier();
    };
    next();
    // the fragments of a half are read while the other half's products run
    Frags f0, f1;
    read_frags(f0, a0, b0, 0);
    auto turn = [&](auto i_c, int s) {
      constexpr int I = decltype(i_c)::value;
      fill(GE_I((I + NS - 1) % NS), s + NS - 1);
      read_frags(f1, a_arr(GE_I(I)), b_arr(GE_I(I)), 1);
      mfmas(f0);
      next();
      read_frags(f0, a_arr(GE_I((I + 1) % NS)), b_arr(GE_I((I + 1) % NS)), 0);
      mfmas(f1);
    };
    // Whole rings (slots past the end read zeros): with an exit after every slot the compiler saw paths
    // on which a slot is read right after its loads were issued, and waited for all loads each ring.
    for (int s = slot0; s < slot1; s += NS) {
      turn(GE_I(0), s);
      turn(GE_I(1), s + 1);
      if constexpr (NS > 2) turn(GE_I(2), s + 2);
      if constexpr (NS > 3) turn(GE_I(3), s + 3);
      if constexpr (NS > 4) turn(GE_I(4), s + 4);
    }
  }
  };
  if (AC || K % 64 == 0) run(std::true_type{});         // (column operands need no masks)
  else run(std::false_type{});
#undef GE_I
  __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(0));      // loads past the end, last fragment reads
  __syncthreads();                                     // every wave is done with the slots

  // ---- a split contraction: every workgroup of the tile leaves its sums in the workspace, as the
  // lanes hold them, and takes a ticket; the one that draws the last adds all up in split order
  // (fixed, so equal calls give equal bits) and goes on to the epilogue.  Device-scope accesses
  // and their order are those of ge_kernel_impl.h's reductions: the stores are performed before
  // the ticket, the loads issued after it. ----
  if constexpr (!T::PP) {
    if (splits > 1) {                                  // uniform
      typedef unsigned long long u64;
      constexpr int BLOCKS = NB * T::FN * T::FM;
      u64* const tile_part = (u64*)l.part + (int64_t)tile_id * splits * (BLOCKS * T::NT * 2);
      u64* const mine = tile_part + (int64_t)split * (BLOCKS * T::NT * 2) + tid * 2;
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) {
        u64 w[2];
        __builtin_memcpy(w, &acc[b / (T::FN * T::FM)][b / T::FM % T::FN][b % T::FM], 16);
        __hip_atomic_store(mine + b * (T::NT * 2), w[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(mine + b * (T::NT * 2) + 1, w[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __builtin_amdgcn_s_waitcnt(kVmcnt0);
      __syncthreads();
      uint32_t* const flag = (uint32_t*)a0;
      if (tid == 0) {
        uint32_t* ctr = l.ctr + (uint32_t)tile_id * kFfnCtrStride;
        const bool last = __hip_atomic_fetch_add(ctr, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)splits - 1u;
        if (last) __hip_atomic_store(ctr, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *flag = last ? 1u : 0u;
      }
      __syncthreads();
      if (*flag == 0u) return;                         // uniform
      __syncthreads();
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) acc[b / (T::FN * T::FM)][b / T::FM % T::FN][b % T::FM] = f32x4_t{};
      for (int q = 0; q < splits; ++q) {
        const u64* from = tile_part + (int64_t)q * (BLOCKS * T::NT * 2) + tid * 2;
        u64 w[BLOCKS][2];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          w[b][0] = __hip_atomic_load(from + b * (T::NT * 2), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          w[b][1] = __hip_atomic_load(from + b * (T::NT * 2) + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          f32x4_t o;
          __builtin_memcpy(&o, w[b], 16);
          acc[b / (T::FN * T::FM)][b / T::FM % T::FN][b % T::FM] += o;
        }
      }
    }
  }

  // ---- epilogue, per 32-row block of the wave's tile ----
  // Registers hold four consecutive columns of a row per lane and block; each value set goes to a
  // wave-private fp32 block in LDS and is read back in row order (a wave's LDS accesses complete
  // in order), so loads and stores of bf16 rows are coalesced.
  constexpr int LPR = T::WN / 4, RPP = 64 / LPR, PASSES = 32 / RPP;
  const int ep_i = wave / T::EP_PER;
  float* ep = (float*)(ep_i == 0   ? a0 + wave * T::EP_WAVE
                       : ep_i == 1 ? a1 + (wave - T::EP_PER) * T::EP_WAVE
                       : wave == 2 * T::EP_PER ? b0 : b1);
  const int p2_row = lane / LPR, p2_col = 4 * (lane % LPR);
  const bool col_ok = wn0 + p2_col < ncols;
  const uint32_t col2 = (uint32_t)(wn0 + p2_col) * 2u;
  auto out_rs = [&](uint16_t* base, int64_t ld) {
    return make_rsrc(base + (int64_t)m0 * ld + n0, (int64_t)(uint32_t)(mrows - 1) * ld * 2 + ncols * 2);
  };
  auto offset = [&](int ml, int64_t ld) { return (ml < mrows && col_ok) ? (uint32_t)ml * ((uint32_t)ld * 2u) + col2 : kOOB; };
  auto stage = [&](int j, auto value) {                // value(i, block row, e) -> fp32
#pragma unroll
    for (int par = 0; par < 2; ++par)
#pragma unroll
      for (int i = 0; i < T::FN; ++i) {
        f32x4_t t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = value(i, 2 * j + par, e);
        *(f32x4_t*)(ep + (16 * par + (int)l16) * T::EP_LD + 16 * i + 4 * (int)q16) = t;
      }
  };
  auto staged = [&](int ps) { return *(const f32x4_t*)(ep + (ps * RPP + p2_row) * T::EP_LD + p2_col); };
  auto store = [&](const f32x4_t& y, __amdgpu_buffer_rsrc_t rs, uint32_t off) {
    u32x2_t w;
    w[0] = pack_bf16x2(y[0], y[1]);
    w[1] = pack_bf16x2(y[2], y[3]);
    __builtin_amdgcn_raw_buffer_store_b64(w, rs, off, 0, 0);
  };
  const __amdgpu_buffer_rsrc_t y_rs = out_rs(p.Y, p.ldy);

  if constexpr (PAIR) {
    const bool save = p.Y2 != nullptr;
    const __amdgpu_buffer_rsrc_t g_rs = save ? out_rs(p.Y2, p.ldy2) : y_rs, u_rs = save ? out_rs(p.Y3, p.ldy2) : y_rs;
    auto write = [&](int j, __amdgpu_buffer_rsrc_t rs, int64_t ld) {
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) store(staged(ps), rs, offset(wm0 + 32 * j + ps * RPP + p2_row, ld));
    };
#pragma unroll
    for (int j = 0; j < T::FM / 2; ++j) {
      stage(j, [&](int i, int r, int e) { return gate<ACT>(acc[0][i][r][e]) * acc[NB - 1][i][r][e]; });
      write(j, y_rs, p.ldy);
      if (save) {
        stage(j, [&](int i, int r, int e) { return acc[0][i][r][e]; });
        write(j, g_rs, p.ldy2);
        stage(j, [&](int i, int r, int e) { return acc[NB - 1][i][r][e]; });
        write(j, u_rs, p.ldy2);
      }
    }
  } else if constexpr (MODE == FFN_GRAD) {
    const __amdgpu_buffer_rsrc_t du_rs = out_rs(p.Y2, p.ldy2), h_rs = out_rs(p.Y3, p.ldy2);
    const __amdgpu_buffer_rsrc_t g_rs = out_rs(const_cast<uint16_t*>(p.E1), p.lde), u_rs = out_rs(const_cast<uint16_t*>(p.E2), p.lde);
    // the next block's G and U are on their way while this one is computed
    u32x2_t gb[2][PASSES], ub[2][PASSES];
    auto fetch = [&](int j) {
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) {
        const uint32_t off = offset(wm0 + 32 * j + ps * RPP + p2_row, p.lde);
        gb[j & 1][ps] = __builtin_amdgcn_raw_buffer_load_b64(g_rs, off, 0, 2);
        ub[j & 1][ps] = __builtin_amdgcn_raw_buffer_load_b64(u_rs, off, 0, 2);
      }
    };
    fetch(0);
#pragma unroll
    for (int j = 0; j < T::FM / 2; ++j) {
      if (j + 1 < T::FM / 2) fetch(j + 1);
      const u32x2_t (&gv)[PASSES] = gb[j & 1];
      const u32x2_t (&uv)[PASSES] = ub[j & 1];
      stage(j, [&](int i, int r, int e) { return acc[0][i][r][e]; });
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) {
        const int ml = wm0 + 32 * j + ps * RPP + p2_row;
        const f32x4_t t = staged(ps);
        f32x4_t dg, du, h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float g = (e & 1) ? bf16_hi(gv[ps][e >> 1]) : bf16_lo(gv[ps][e >> 1]);
          const float u = (e & 1) ? bf16_hi(uv[ps][e >> 1]) : bf16_lo(uv[ps][e >> 1]);
          float a, sl;
          act_and_slope<ACT>(g, a, sl);
          dg[e] = t[e] * u * sl;
          du[e] = t[e] * a;
          h[e] = a * u;
        }
        store(dg, y_rs, offset(ml, p.ldy));
        store(du, du_rs, offset(ml, p.ldy2));
        store(h, h_rs, offset(ml, p.ldy2));
      }
    }
  } else {
    const bool res = MODE == FFN_DOWN && p.E1 != nullptr;
    const __amdgpu_buffer_rsrc_t r_rs = res ? out_rs(const_cast<uint16_t*>(p.E1), p.lde) : y_rs;
#pragma unroll
    for (int j = 0; j < T::FM / 2; ++j) {
      u32x2_t rv[PASSES];
      if (res) {
#pragma unroll
        for (int ps = 0; ps < PASSES; ++ps)
          rv[ps] = __builtin_amdgcn_raw_buffer_load_b64(r_rs, offset(wm0 + 32 * j + ps * RPP + p2_row, p.lde), 0, 0);
      }
      stage(j, [&](int i, int r, int e) { return acc[0][i][r][e]; });
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) {
        f32x4_t y = staged(ps);
        if (res) {
          y[0] += bf16_lo(rv[ps][0]);
          y[1] += bf16_hi(rv[ps][0]);
          y[2] += bf16_lo(rv[ps][1]);
          y[3] += bf16_hi(rv[ps][1]);
        }
        store(y, y_rs, offset(wm0 + 32 * j + ps * RPP + p2_row, p.ldy));
      }
    }
  }
}

// The 128-row tiles run eight waves (two per SIMD, 64 x 32 each) with 96 KB of loads in flight, the
// 64-row ones four waves and two or three workgroups per CU.  Measured per 64-deep slot with every CU
// busy: 1.5 us (256), 0.45-0.6 us (128; with four waves 0.6-0.65), 0.21 us (64).
using F256 = FTile<256, 256, 1, 8, 2, true>;      // 128 x 64 per wave
using F256P = FTile<256, 128, 2, 8, 2, true>;     // 128 x 32 (x2: gate, up) per wave
using F128 = FTile<128, 128, 1, 8, 4>;            // 64 x 32 per wave
using F128P = FTile<128, 128, 2, 8, 3>;
using F64 = FTile<64, 64, 1, 4, 4>;               // 32 x 32 per wave
using F64P = FTile<64, 64, 2, 4, 3>;

template <class T, int MODE, int ACT, bool AC, bool BC>
hipError_t launch_product(const FfnLaunch& l, hipStream_t s) {
  if (l.tiles <= 0) return hipSuccess;
  hipLaunchKernelGGL((ffn_product<T, MODE, ACT, AC, BC>), dim3((unsigned)(l.tiles * (T::PP ? 1 : l.splits))),
                     dim3(T::NT), 0, s, l);
  return hipGetLastError();
}

}  // namespace
}  // namespace ge
