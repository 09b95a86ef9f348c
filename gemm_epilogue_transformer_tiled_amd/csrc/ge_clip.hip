// Global gradient norm over many tensors, and clipping (gfx950).
//
// Memory-bound: the norm reads every gradient once, the clipping reads it again and writes it.
// The tensors' table travels as the kernel argument, so a call needs no copy to the device and
// can be captured.  Each workgroup of the norm launch takes chunks of kClipChunk values in turn and
// leaves one partial sum; every workgroup of the clipping launch adds all partial sums itself, in
// the same order, so no third launch and no atomic is needed and the result does not depend on
// the order in which workgroups run.  Squares and sums are 64-bit: their range has no overflow or
// underflow for any bf16 or fp32 gradient, and the 64-bit rate is several times what the memory
// can feed.  The clipping launch walks the chunks backwards, so the last ones the norm read are
// met first, while the memory-side cache still holds them.
#include "ge_block_internal.h"

namespace ge {
namespace {

// 16-byte accesses at the elements' alignment: gradients packed one after another start anywhere
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 Any16 __attribute__((aligned(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Cache policy by the gradients' bytes (kClip*, ge_block_internal.h).  The clipped values are not
// read here again: past 64 MB they are stored "nt" (180 MB of gradients: 94 -> 85 us a call).  Past
// 512 MB the second read finds almost nothing in the 256 MB memory-side cache, and every access
// goes "nt" (2.2 GB: 1,205 -> 1,123 us; the norm alone then reads 6.9 TB/s instead of 6.1); below, that would
// lose what the cache keeps (180 MB: 85 -> 98 us).
template <int POLICY>
__device__ __forceinline__ u32x4 fetch(const void* p) {
  const Any16* q = (const Any16*)p;
  if constexpr (POLICY >= kClipStream) return __builtin_nontemporal_load(q);
  else return *q;
}
template <int POLICY>
__device__ __forceinline__ void put(void* p, u32x4 v) {
  Any16* q = (Any16*)p;
  if constexpr (POLICY >= kClipStoreThrough) __builtin_nontemporal_store(v, q);
  else *q = v;
}
constexpr int kThreads = 256;

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const bf16x2 h = {(__bf16)a, (__bf16)b};      // round to nearest even
  return __builtin_bit_cast(uint32_t, h);
}

// Values before the first 128-byte line of p: done one by one, so that the wide accesses that follow
// lie on whole lines (at odd addresses they met every line twice: 2.2 GB packed without padding,
// 1,323 us a call instead of 1,130).
template <class E>
__device__ __forceinline__ int head_of(const E* p, int n) {
  const int h = (int)((128u - ((uint32_t)reinterpret_cast<uintptr_t>(p) & 127u)) & 127u) / (int)sizeof(E);
  return h < n ? h : n;
}

// Index of the tensor that holds chunk c (chunk0 ascending, no empty tensors).
__device__ __forceinline__ int tensor_of(const ClipTable& t, uint32_t c) {
  int a = 0, b = t.n;
  while (b - a > 1) {
    const int m = (a + b) / 2;
    if (t.chunk0[m] <= c) a = m;
    else b = m;
  }
  return a;
}

__device__ __forceinline__ double block_sum(double s, double* lds) {
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

template <int POLICY>
__global__ __launch_bounds__(kThreads) void clip_norm(ClipTable t, double* part) {
  __shared__ double lds[4];
  double s = 0.0;
  const uint32_t chunks = t.chunk0[t.n];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.chunk0[k]) * kClipChunk, left = t.numel[k] - at;
    const int n = left < kClipChunk ? (int)left : kClipChunk;
    if ((t.fp32[k >> 5] >> (k & 31)) & 1u) {
      const float* x = (const float*)t.in[k] + at;
      const int h = head_of(x, n);
      if ((int)threadIdx.x < h) { const double v = (double)x[threadIdx.x]; s += v * v; }
      for (int i = h + 4 * threadIdx.x; i + 4 <= n; i += 4 * kThreads) {
        const u32x4 w = fetch<POLICY>(x + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) { const double v = (double)__uint_as_float(w[j]); s += v * v; }
      }
      const int i = h + ((n - h) & ~3) + (int)threadIdx.x;
      if (i < n) { const double v = (double)x[i]; s += v * v; }
    } else {
      const uint16_t* x = (const uint16_t*)t.in[k] + at;
      const int h = head_of(x, n);
      if ((int)threadIdx.x < h) { const double v = (double)lo(x[threadIdx.x]); s += v * v; }
      for (int i = h + 8 * threadIdx.x; i + 8 <= n; i += 8 * kThreads) {
        const u32x4 w = fetch<POLICY>(x + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const double a = (double)lo(w[j]), b = (double)hi(w[j]);
          s += a * a;
          s += b * b;
        }
      }
      const int i = h + ((n - h) & ~7) + (int)threadIdx.x;
      if (i < n) { const double v = (double)lo(x[i]); s += v * v; }
    }
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The sum of all partial sums, the same in every workgroup.
__device__ __forceinline__ double total(const double* part, int n, double* lds) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += part[i];
  return block_sum(s, lds);
}

__global__ __launch_bounds__(kThreads) void clip_finish(const double* part, int nparts, float* norm) {
  __shared__ double lds[4];
  const double s = total(part, nparts, lds);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

template <int POLICY>
__global__ __launch_bounds__(kThreads) void clip_scale(ClipTable t, const double* part, int nparts, float max_norm, float eps,
                                                       float* norm) {
  __shared__ double lds[4];
  const double nrm = sqrt(total(part, nparts, lds));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)nrm;
  const double ratio = (double)max_norm / (nrm + (double)eps);
  // The factor as m 2^e, m in [0.5, 1) rounded to fp32: gradients near the largest fp32 value have a
  // factor below the smallest normal one, whose 24 bits the plain fp32 factor would lose.
  const bool keep = ratio >= 1.0;                              // NaN: not kept
  int e = 0;
  const float f = keep ? 1.0f : (float)frexp(ratio, &e);
  const int e2 = (keep || !(ratio > 0.0)) ? 0 : e;             // (frexp leaves e open for NaN)
  auto scaled = [&](float x) { return __builtin_amdgcn_ldexpf(x * f, e2); };
  const uint32_t chunks = t.chunk0[t.n];
  for (uint32_t q = blockIdx.x; q < chunks; q += gridDim.x) {
    const uint32_t c = chunks - 1 - q;
    const int k = tensor_of(t, c);
    if (keep && t.in[k] == t.out[k]) continue;                 // uniform
    const int64_t at = (int64_t)(c - t.chunk0[k]) * kClipChunk, left = t.numel[k] - at;
    const int n = left < kClipChunk ? (int)left : kClipChunk;
    if ((t.fp32[k >> 5] >> (k & 31)) & 1u) {
      const float* x = (const float*)t.in[k] + at;
      float* y = (float*)t.out[k] + at;
      const int h = head_of(y, n);
      if ((int)threadIdx.x < h) y[threadIdx.x] = scaled(x[threadIdx.x]);
      for (int i = h + 4 * threadIdx.x; i + 4 <= n; i += 4 * kThreads) {
        u32x4 w = fetch<POLICY>(x + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(scaled(__uint_as_float(w[j])));
        put<POLICY>(y + i, w);
      }
      const int i = h + ((n - h) & ~3) + (int)threadIdx.x;
      if (i < n) y[i] = scaled(x[i]);
    } else {
      const uint16_t* x = (const uint16_t*)t.in[k] + at;
      uint16_t* y = (uint16_t*)t.out[k] + at;
      const int h = head_of(y, n);
      if ((int)threadIdx.x < h) y[threadIdx.x] = (uint16_t)(pack2(scaled(lo(x[threadIdx.x])), 0.0f) & 0xFFFFu);
      for (int i = h + 8 * threadIdx.x; i + 8 <= n; i += 8 * kThreads) {
        u32x4 w = fetch<POLICY>(x + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack2(scaled(lo(w[j])), scaled(hi(w[j])));
        put<POLICY>(y + i, w);
      }
      const int i = h + ((n - h) & ~7) + (int)threadIdx.x;
      if (i < n) y[i] = (uint16_t)(pack2(scaled(lo(x[i])), 0.0f) & 0xFFFFu);
    }
  }
}

}  // namespace

hipError_t launch_clip_norm(const ClipTable& t, int grid, int policy, double* part, hipStream_t s) {
  if (policy >= kClipStream) hipLaunchKernelGGL(clip_norm<kClipStream>, dim3((unsigned)grid), dim3(kThreads), 0, s, t, part);
  else hipLaunchKernelGGL(clip_norm<kClipCached>, dim3((unsigned)grid), dim3(kThreads), 0, s, t, part);
  return hipGetLastError();
}
hipError_t launch_clip_finish(const double* part, int nparts, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(clip_finish, dim3(1), dim3(kThreads), 0, s, part, nparts, norm);
  return hipGetLastError();
}
hipError_t launch_clip_scale(const ClipTable& t, int grid, int policy, const double* part, int nparts, float max_norm,
                             float eps, float* norm, hipStream_t s) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, t, part, nparts, max_norm, eps, norm);
  };
  if (policy == kClipCached) go(clip_scale<kClipCached>);
  else if (policy == kClipStoreThrough) go(clip_scale<kClipStoreThrough>);
  else go(clip_scale<kClipStream>);
  return hipGetLastError();
}

}  // namespace ge
