// Device helpers of the row operators: vectors of eight values, sums over the threads of a row, and
// dropout's random numbers.
#pragma once

#include "ge_rows_internal.h"

namespace ge {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// wide accesses at the elements' alignment: rows start anywhere
typedef u32x4 Any16 __attribute__((aligned(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const bf16x2 h = {(__bf16)a, (__bf16)b};      // round to nearest even
  return __builtin_bit_cast(uint32_t, h);
}

// Eight values as they lie in memory.
template <class E>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 w;
};
template <>
struct Raw<float> {
  u32x4 w, w2;
};

template <class E>
__device__ __forceinline__ Raw<E> zero() {
  Raw<E> r;
  r.w = u32x4{0, 0, 0, 0};
  if constexpr (sizeof(E) == 4) r.w2 = u32x4{0, 0, 0, 0};
  return r;
}

__device__ __forceinline__ float get(const Raw<uint16_t>& r, int j) { return (j & 1) ? hi(r.w[j >> 1]) : lo(r.w[j >> 1]); }
__device__ __forceinline__ float get(const Raw<float>& r, int j) { return __uint_as_float(j < 4 ? r.w[j] : r.w2[j - 4]); }
__device__ __forceinline__ Raw<uint16_t> rounded(const float (&v)[8], uint16_t) {
  Raw<uint16_t> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r.w[j] = pack2(v[2 * j], v[2 * j + 1]);
  return r;
}
__device__ __forceinline__ Raw<float> rounded(const float (&v)[8], float) {
  Raw<float> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.w[j] = __float_as_uint(v[j]);
    r.w2[j] = __float_as_uint(v[4 + j]);
  }
  return r;
}

// Cache policy of a call's accesses (kRows*, ge_rows_internal.h).
template <int POLICY>
__device__ __forceinline__ u32x4 get16(const void* p) {
  if constexpr ((POLICY & kRowsLoadsOnce) != 0) return __builtin_nontemporal_load((const Any16*)p);
  else return *(const Any16*)p;
}
template <int POLICY>
__device__ __forceinline__ void put16(void* p, u32x4 v) {
  if constexpr ((POLICY & kRowsStoresThrough) != 0) __builtin_nontemporal_store(v, (Any16*)p);
  else *(Any16*)p = v;
}

// Values col .. col + 7 of a row of d, zeros past its end.  TAIL: d is no multiple of eight.  The row's last vector is
// then loaded from its last eight values, and settle() shifts them to their places when they are used: nothing
// waits for a load when it is made.  (Value by value, and put together at once, the last vector held up its whole row:
// norm of 16432 x 1021 bf16 31 us against 25, its gradient 63 against 44.)
template <class E, bool TAIL, int POLICY = 0>
__device__ __forceinline__ Raw<E> fetch(const E* row, int col, int d) {
  Raw<E> r = zero<E>();
  if (col >= d) return r;
  if (!TAIL || d >= 8) {                               // (uniform)
    const E* at = row + (TAIL ? min(col, d - 8) : col);
    r.w = get16<POLICY>(at);
    if constexpr (sizeof(E) == 4) r.w2 = get16<POLICY>(at + 4);
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j) {
      const E v = row[min(j, d - 1)];
      if constexpr (sizeof(E) == 2) r.w[j >> 1] |= j < d ? (uint32_t)v << (16 * (j & 1)) : 0u;
      else if (j < 4) r.w[j] = j < d ? __float_as_uint(v) : 0u;
      else r.w2[j - 4] = j < d ? __float_as_uint(v) : 0u;
    }
  }
  return r;
}
template <bool TAIL>
__device__ __forceinline__ void settle(Raw<uint16_t>& r, int col, int d) {
  if (!TAIL || d < 8 || col >= d || col + 8 <= d) return;
  const int s = 16 * (8 - (d & 7));                    // bits; uniform
  uint64_t lo64 = (uint64_t)r.w[1] << 32 | r.w[0], hi64 = (uint64_t)r.w[3] << 32 | r.w[2];
  lo64 = s < 64 ? lo64 >> s | hi64 << (64 - s) : hi64 >> (s - 64);
  hi64 = s < 64 ? hi64 >> s : 0;
  r.w = u32x4{(uint32_t)lo64, (uint32_t)(lo64 >> 32), (uint32_t)hi64, (uint32_t)(hi64 >> 32)};
}
template <bool TAIL>
__device__ __forceinline__ void settle(Raw<float>& r, int col, int d) {
  if (!TAIL || d < 8 || col >= d || col + 8 <= d) return;
  const int s = 8 - (d & 7);                           // values; uniform
  if (s & 1) {
    r.w = u32x4{r.w[1], r.w[2], r.w[3], r.w2[0]};
    r.w2 = u32x4{r.w2[1], r.w2[2], r.w2[3], 0};
  }
  if (s & 2) {
    r.w = u32x4{r.w[2], r.w[3], r.w2[0], r.w2[1]};
    r.w2 = u32x4{r.w2[2], r.w2[3], 0, 0};
  }
  if (s & 4) {
    r.w = r.w2;
    r.w2 = u32x4{0, 0, 0, 0};
  }
}
template <class E, bool TAIL>
__device__ __forceinline__ Raw<E> fetch_settled(const E* row, int col, int d) {
  Raw<E> r = fetch<E, TAIL>(row, col, d);
  settle<TAIL>(r, col, d);
  return r;
}
// The last vector of a ragged row goes out in runs of four, two and one.
template <class E, bool TAIL, int POLICY = 0>
__device__ __forceinline__ void put(E* row, int col, int d, const Raw<E>& r) {
  typedef u32x2 Any8 __attribute__((aligned(2)));
  typedef uint32_t Any4 __attribute__((aligned(2)));
  if (col + (TAIL ? 8 : 1) <= d) {
    put16<POLICY>(row + col, r.w);
    if constexpr (sizeof(E) == 4) put16<POLICY>(row + col + 4, r.w2);
  } else if (TAIL && col < d) {
    const int n = d & 7;                               // uniform
    E* at = row + col;
    if constexpr (sizeof(E) == 2) {
      if (n & 4) *(Any8*)at = u32x2{r.w[0], r.w[1]};
      const uint32_t a = (n & 4) ? r.w[2] : r.w[0], b = (n & 4) ? r.w[3] : r.w[1];
      if (n & 2) *(Any4*)(at + (n & 4)) = a;
      if (n & 1) at[n & 6] = (uint16_t)((n & 2) ? b : a);
    } else {
      if (n & 4) *(Any16*)at = r.w;
      const u32x4 a = (n & 4) ? r.w2 : r.w;
      if (n & 2) *(Any8*)(at + (n & 4)) = u32x2{a[0], a[1]};
      if (n & 1) at[n & 6] = __uint_as_float((n & 2) ? a[2] : a[0]);
    }
  }
}

// Waits for a vector that was loaded earlier.
__device__ __forceinline__ void landed(Raw<uint16_t>& r) { asm volatile("" : "+v"(r.w)); }
__device__ __forceinline__ void landed(Raw<float>& r) { asm volatile("" : "+v"(r.w), "+v"(r.w2)); }

// Sum over a wave, the same bits in every lane: exchanges within 16 lanes are DPP operands of the adds
// (after the first two steps quads agree, so mirrored halves stand for the further ones).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0xB1>(v);       // quad: lanes 1 0 3 2
  v = dpp_add<0x4E>(v);       // quad: lanes 2 3 0 1
  v = dpp_add<0x141>(v);      // mirrored in 8
  v = dpp_add<0x140>(v);      // mirrored in 16
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
// Sum over the TR threads of a row.  `lds`: one word a wave; a place that alternates from call to call, so
// that one barrier is enough (a wave writes a place again only after the barrier of the other, which
// every wave reaches with its reads of the first done).
template <int TR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  v = wave_sum(v);
  if constexpr (TR == 64) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < TR / 64; ++w) v += lds[w];
  return v;
}

// ---- dropout ----
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): ten rounds of two 32 x 32 -> 64-bit products.  The
// products' rate is a quarter of the adds', so a value gets 16 bits, not 32: one call serves eight.
struct Words {
  uint32_t w[4];
};
struct DropKey {
  uint32_t k0, k1, o0, o1;    // seed, offset (uniform)
};
// (through the scalar cache: no vector load waits for them)
__device__ __forceinline__ DropKey drop_key(const DropParams& p) {
  typedef const __attribute__((address_space(4))) uint32_t* Constant;
  const Constant q = (Constant)(uintptr_t)p.rng;
  return DropKey{q[0], q[1], q[2], q[3]};
}
__device__ __forceinline__ Words philox(uint32_t block, uint32_t site, const DropKey& key) {
  uint32_t c0 = block, c1 = site, c2 = key.o0, c3 = key.o1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words{{c0, c1, c2, c3}};
}
// Value j of the block: 0 where dropped (a NaN too), times the factor elsewhere.
__device__ __forceinline__ float dropped(float v, const Words& w, int j, const DropParams& p) {
  const uint32_t h = (j & 1) ? w.w[j >> 1] >> 16 : w.w[j >> 1] & 0xFFFFu;
  return h < p.below ? 0.0f : v * p.factor;
}

}  // namespace
}  // namespace ge
