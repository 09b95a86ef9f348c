// Per-head norm of queries and keys with the position rotation, forward and backward (gfx950).
//
// Memory-bound: every value is read once and written once (backward: the gradient and, with the
// norm, the input are read).  A head lies on a group of lanes, eight values a lane, chosen so
// that both values of every rotation pair are in one lane: interleaved pairs are eight
// consecutive values, half pairs four consecutive values of each half.  So the rotation needs no
// exchange between lanes, a lane reads and writes the same elements (in place is safe), and only
// the norm's sums cross lanes.  Fused multiply-adds are written out: the kernels for aligned and for
// any layout give the same bits.
//
// The angle position * inv_freq and its reduction to a turn are computed in 64 bits (positions go
// past 2^24 turns' worth of fp32), its cosine and sine in 32, once per token and pair: a
// workgroup computes those of its tokens into LDS and all heads of the tokens read them there.
#include <type_traits>

#include "ge_block_internal.h"

namespace ge {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const bf16x2 h = {(__bf16)a, (__bf16)b};      // round to nearest even
  return __builtin_bit_cast(uint32_t, h);
}
__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)(pack2(v, 0.0f) & 0xFFFFu); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// The eight values of a lane: pair j is (a[j], b[j]).
struct Pairs {
  float a[4], b[4];
};

// Element offsets of pair j of a lane's slots slot .. slot + 3, of the head's head_dim / 2 pairs; the
// first rot_dim / 2 of them are turned.  The pairing of the others does not matter: half pairs take
// the lane's eight values as two runs of four where whole lanes are unturned (the same in the wide
// and the general kernels, so that both add up a head in the same order), and otherwise neighbours.
template <bool HALF>
__device__ __forceinline__ int offset_a(int slot, int j, int rot2, int d2) {
  if (HALF && slot + j < rot2) return slot + j;
  if (HALF && ((rot2 | d2) & 3) == 0) return 2 * slot + j;
  return 2 * (slot + j);
}
template <bool HALF>
__device__ __forceinline__ int offset_b(int slot, int j, int rot2, int d2) {
  if (HALF && slot + j < rot2) return slot + j + rot2;
  if (HALF && ((rot2 | d2) & 3) == 0) return 2 * slot + 4 + j;
  return 2 * (slot + j) + 1;
}

// WIDE: rot_dim / 2 and head_dim / 2 multiples of four and 16-byte aligned heads, so a lane's slots are
// all turned or all not, and its values are two runs of four (or one of eight).  Raw: the bytes as
// loaded, so that the next heads' loads can be on their way while one is computed.
template <class E, bool WIDE>
struct Raw {
  Pairs v;
};
template <>
struct Raw<uint16_t, true> {
  u32x4 v;
};

template <class E, bool WIDE, bool HALF>
__device__ __forceinline__ void load(Raw<E, WIDE>& raw, const E* head, int slot, int rot2, int d2) {
  if constexpr (WIDE) {
    // half pairs that are not turned: the pairing does not matter, take the runs as they come
    const int oa = HALF && slot < rot2 ? slot : 2 * slot, ob = HALF && slot < rot2 ? slot + rot2 : 2 * slot + 4;
    if constexpr (sizeof(E) == 2) {
      if constexpr (HALF) {
        const u32x2 x = *(const u32x2*)(head + oa), y = *(const u32x2*)(head + ob);
        raw.v = u32x4{x[0], x[1], y[0], y[1]};
      } else {
        raw.v = *(const u32x4*)(head + oa);
      }
    } else {
      const f32x4 x = *(const f32x4*)(head + oa), y = *(const f32x4*)(head + ob);
#pragma unroll
      for (int j = 0; j < 4; ++j) { raw.v.a[j] = x[j]; raw.v.b[j] = y[j]; }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool ok = slot + j < d2;
      raw.v.a[j] = ok ? one(head + offset_a<HALF>(slot, j, rot2, d2)) : 0.0f;
      raw.v.b[j] = ok ? one(head + offset_b<HALF>(slot, j, rot2, d2)) : 0.0f;
    }
  }
}
// Two runs of four to pairs: half pairs as they are, interleaved pairs neighbour by neighbour.
template <class E, bool WIDE, bool HALF>
__device__ __forceinline__ Pairs pairs_of(const Raw<E, WIDE>& raw) {
  if constexpr (!WIDE) {
    return raw.v;
  } else {
    float x[8];
    if constexpr (sizeof(E) == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) { x[2 * j] = lo(raw.v[j]); x[2 * j + 1] = hi(raw.v[j]); }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) { x[j] = raw.v.a[j]; x[4 + j] = raw.v.b[j]; }
    }
    Pairs v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v.a[j] = HALF ? x[j] : x[2 * j];
      v.b[j] = HALF ? x[4 + j] : x[2 * j + 1];
    }
    return v;
  }
}

template <class E, bool WIDE, bool HALF>
__device__ __forceinline__ void store(E* head, int slot, int rot2, int d2, const Pairs& v) {
  if constexpr (WIDE) {
    if constexpr (HALF) {
      const int oa = slot < rot2 ? slot : 2 * slot, ob = slot < rot2 ? slot + rot2 : 2 * slot + 4;
      if constexpr (sizeof(E) == 2) {
        *(u32x2*)(head + oa) = u32x2{pack2(v.a[0], v.a[1]), pack2(v.a[2], v.a[3])};
        *(u32x2*)(head + ob) = u32x2{pack2(v.b[0], v.b[1]), pack2(v.b[2], v.b[3])};
      } else {
        *(f32x4*)(head + oa) = f32x4{v.a[0], v.a[1], v.a[2], v.a[3]};
        *(f32x4*)(head + ob) = f32x4{v.b[0], v.b[1], v.b[2], v.b[3]};
      }
    } else if constexpr (sizeof(E) == 2) {
      *(u32x4*)(head + 2 * slot) = u32x4{pack2(v.a[0], v.b[0]), pack2(v.a[1], v.b[1]), pack2(v.a[2], v.b[2]),
                                         pack2(v.a[3], v.b[3])};
    } else {
      *(f32x4*)(head + 2 * slot) = f32x4{v.a[0], v.b[0], v.a[1], v.b[1]};
      *(f32x4*)(head + 2 * slot + 4) = f32x4{v.a[2], v.b[2], v.a[3], v.b[3]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (slot + j < d2) {
        put(head + offset_a<HALF>(slot, j, rot2, d2), v.a[j]);
        put(head + offset_b<HALF>(slot, j, rot2, d2), v.b[j]);
      }
  }
}

// Sum over the lanes of a group, the same bits in each: exchanges within 16 lanes are DPP operands
// of the adds (after the first two steps quads agree, so mirrored halves stand for the further ones).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float group_sum(float v, int G) {
  if (G >= 2) v = dpp_add<0xB1>(v);       // quad: lanes 1 0 3 2
  if (G >= 4) v = dpp_add<0x4E>(v);       // quad: lanes 2 3 0 1
  if (G >= 8) v = dpp_add<0x141>(v);      // mirrored in 8
  if (G >= 16) v = dpp_add<0x140>(v);     // mirrored in 16
  if (G >= 32) v += __shfl_xor(v, 16);
  if (G >= 64) v += __shfl_xor(v, 32);
  return v;
}

// 1 / sqrt(mean square + eps).  The hardware's takes a subnormal argument for zero; one is met only where
// eps itself is below the normal range (uniform): then small ones are scaled by 2^64 first.
__device__ __forceinline__ float inv_rms(float ss, float inv_d, float eps) {
  const float m = fmaf(ss, inv_d, eps);
  if (eps >= 0x1p-126f) return __builtin_amdgcn_rsqf(m);
  const bool tiny = m < 0x1p-64f;
  const float r = __builtin_amdgcn_rsqf(tiny ? m * 0x1p64f : m);
  return tiny ? r * 0x1p32f : r;
}

// Element offset of a head within a turn's tokens.  WIDE: 24-bit factors, 31-bit products (checked
// on the host), so the addresses take two full-rate multiplies.
template <bool WIDE>
__device__ __forceinline__ auto head_at(int t, int h, int64_t st, int64_t sh) {
  if constexpr (WIDE) return (uint32_t)(__umul24((uint32_t)t, (uint32_t)st) + __umul24((uint32_t)h, (uint32_t)sh));
  else return (int64_t)t * st + (int64_t)h * sh;
}

template <class E, bool WIDE, bool HALF, bool NORM, bool BWD>
__global__ __launch_bounds__(kQkThreads) void qk_rotary(QkParams p) {
  __shared__ __attribute__((aligned(16))) float turn_c[kQkMaxAngles], turn_s[kQkMaxAngles];
  __shared__ float gsum[BWD && NORM ? 2 * 8 * kQkThreads : 1];
  const int tid = threadIdx.x, G = p.group;
  const int gl = tid & (G - 1), ng = kQkThreads / G, grp = tid / G;
  const int slot = 4 * gl, rot2 = p.rot_dim / 2, d2 = p.head_dim / 2;
  const bool live = slot < d2;
  const float inv_d = 1.0f / (float)p.head_dim;

  Pairs gain[2];
  if constexpr (NORM) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool ok = p.heads[w] > 0 && slot + j < d2;
        gain[w].a[j] = ok ? one((const E*)p.gain[w] + offset_a<HALF>(slot, j, rot2, d2)) : 0.0f;
        gain[w].b[j] = ok ? one((const E*)p.gain[w] + offset_b<HALF>(slot, j, rot2, d2)) : 0.0f;
      }
  }
  Pairs dgain[2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int j = 0; j < 4; ++j) dgain[w].a[j] = dgain[w].b[j] = 0.0f;

  struct Item {
    Raw<E, WIDE> x, d;
  };
  const int tw = p.tokens_per_wg, hs = p.head_splits;
  // (a token's heads are split only where all heads of all tokens are few: 32-bit divisions)
  const int64_t turns = p.turns;
  for (int64_t it = blockIdx.x; it < turns; it += gridDim.x) {
    const int64_t t0 = hs == 1 ? it * tw : (int64_t)((uint32_t)it / (uint32_t)hs * (uint32_t)tw);
    const int part = hs == 1 ? 0 : (int)((uint32_t)it % (uint32_t)hs);
    const int nt = (int)(p.tokens - t0 < tw ? p.tokens - t0 : tw);
    // The heads of the queries, then those of the keys (or, with few tokens, only some of one of
    // them): which of the two is uniform.  One item (a head of a token) per group and step; the next
    // one is loaded before this one is computed.
    auto side = [&](auto w_c, bool angles, int part, int parts) {
      constexpr int w = decltype(w_c)::value;
      int h_lo = 0, nh = p.heads[w];
      if (parts > 1) {
        h_lo = (int)((uint32_t)p.heads[w] * (uint32_t)part / (uint32_t)parts);
        nh = (int)((uint32_t)p.heads[w] * (uint32_t)(part + 1) / (uint32_t)parts) - h_lo;
      }
      const E* const px = (const E*)p.x[w] + t0 * p.xt[w] + h_lo * p.xh[w];
      const E* const pd = (const E*)p.dy[w] + t0 * p.dt[w] + h_lo * p.dh[w];
      E* const py = (E*)p.y[w] + t0 * p.yt[w] + h_lo * p.yh[w];
      const int steps = nh > 0 ? (nt * nh + ng - 1) / ng : 0;          // uniform
      const int step_t = nh > 0 ? ng / nh : 0, step_h = ng - step_t * nh;
      int t = nh > 0 ? grp / nh : nt, h = nh > 0 ? grp - t * nh : 0;
      auto fetch = [&](Item& i) {
        if (t < nt && live) {
          if constexpr (!BWD || NORM) load<E, WIDE, HALF>(i.x, px + head_at<WIDE>(t, h, p.xt[w], p.xh[w]), slot, rot2, d2);
          if constexpr (BWD) load<E, WIDE, HALF>(i.d, pd + head_at<WIDE>(t, h, p.dt[w], p.dh[w]), slot, rot2, d2);
        }
      };
      auto work = [&](const Item& i, int t, int h) {
        Pairs x, d, o;
#pragma unroll
        for (int j = 0; j < 4; ++j) x.a[j] = x.b[j] = d.a[j] = d.b[j] = 0.0f;
        if (live) {
          if constexpr (!BWD || NORM) x = pairs_of<E, WIDE, HALF>(i.x);
          if constexpr (BWD) d = pairs_of<E, WIDE, HALF>(i.d);
        }
        float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (WIDE) {
          if (slot < rot2) {
            const f32x4 u = *(const f32x4*)(turn_c + t * rot2 + slot), v = *(const f32x4*)(turn_s + t * rot2 + slot);
#pragma unroll
            for (int j = 0; j < 4; ++j) { cs[j] = u[j]; sn[j] = v[j]; }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (slot + j < rot2) {
              cs[j] = turn_c[t * rot2 + slot + j];
              sn[j] = turn_s[t * rot2 + slot + j];
            }
        }
        if constexpr (!BWD) {
          if constexpr (NORM) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fmaf(x.a[j], x.a[j], fmaf(x.b[j], x.b[j], ss));
            const float r = inv_rms(group_sum(ss, G), inv_d, p.eps);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x.a[j] = x.a[j] * r * gain[w].a[j];
              x.b[j] = x.b[j] * r * gain[w].b[j];
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o.a[j] = fmaf(x.a[j], cs[j], -(x.b[j] * sn[j]));
            o.b[j] = fmaf(x.b[j], cs[j], x.a[j] * sn[j]);
          }
        } else {
          // the rotation's transpose, then the norm's derivative: with n = x r and e = dy * gain,
          // dx = r (e - n mean(e n)) and dgain += dy n
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o.a[j] = fmaf(d.a[j], cs[j], d.b[j] * sn[j]);
            o.b[j] = fmaf(d.b[j], cs[j], -(d.a[j] * sn[j]));
          }
          if constexpr (NORM) {
            float ss = 0.0f, ex = 0.0f;
            Pairs e;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              e.a[j] = o.a[j] * gain[w].a[j];
              e.b[j] = o.b[j] * gain[w].b[j];
              ss = fmaf(x.a[j], x.a[j], fmaf(x.b[j], x.b[j], ss));
              ex = fmaf(e.a[j], x.a[j], fmaf(e.b[j], x.b[j], ex));
            }
            ss = group_sum(ss, G);
            ex = group_sum(ex, G);
            const float r = inv_rms(ss, inv_d, p.eps);
            const float mean = ex * r * inv_d;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float na = x.a[j] * r, nb = x.b[j] * r;
              dgain[w].a[j] = fmaf(o.a[j], na, dgain[w].a[j]);
              dgain[w].b[j] = fmaf(o.b[j], nb, dgain[w].b[j]);
              o.a[j] = r * fmaf(-na, mean, e.a[j]);
              o.b[j] = r * fmaf(-nb, mean, e.b[j]);
            }
          }
        }
        if (live) store<E, WIDE, HALF>(py + head_at<WIDE>(t, h, p.yt[w], p.yh[w]), slot, rot2, d2, o);
      };
      Item now, next;
      fetch(now);
      if (angles && rot2 > 0) {                        // uniform
        __syncthreads();                               // the last turn's readers are done
        for (int i = tid; i < nt * rot2; i += kQkThreads) {
          const int q = i / rot2, f = i - q * rot2;
          const double pos =
              p.pos64 ? (double)((const int64_t*)p.positions)[t0 + q] : (double)((const int32_t*)p.positions)[t0 + q];
          double turns_of = pos * (double)p.inv_freq[f] * 0.15915494309189533577;     // angle / 2 pi
          turns_of -= __builtin_rint(turns_of);
          // the turn's rounding to fp32 (up to 9e-8 of angle, more than the sine's own error) is made good
          // to first order
          const float turn = (float)turns_of, rest = (float)(turns_of - (double)turn) * 6.283185307f;
          float s, c;
          sincospif(2.0f * turn, &s, &c);
          turn_c[i] = fmaf(-s, rest, c) * p.amplitude;
          turn_s[i] = fmaf(c, rest, s) * p.amplitude;
        }
        __syncthreads();
      }
      for (int k = 0; k < steps; ++k) {                // uniform
        const int t_now = t, h_now = h;
        t += step_t;
        h += step_h;
        if (h >= nh) {
          h -= nh;
          ++t;
        }
        fetch(next);
        if (t_now < nt) work(now, t_now, h_now);       // the same for a whole group
        now = next;
      }
    };
    const int qs = p.q_splits;
    if (hs == 1 || part < qs) side(std::integral_constant<int, 0>{}, true, part, hs == 1 ? 1 : qs);
    if (hs == 1 || part >= qs) side(std::integral_constant<int, 1>{}, hs > 1, hs == 1 ? 0 : part - qs, hs == 1 ? 1 : hs - qs);
  }

  if constexpr (BWD && NORM) {
    // the groups' sums meet in LDS and are added in group order
    const int D = p.head_dim;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (slot + j < d2) {
          gsum[(grp * 2 + w) * D + offset_a<HALF>(slot, j, rot2, d2)] = dgain[w].a[j];
          gsum[(grp * 2 + w) * D + offset_b<HALF>(slot, j, rot2, d2)] = dgain[w].b[j];
        }
    __syncthreads();
    for (int i = tid; i < 2 * D; i += kQkThreads) {
      float s = 0.0f;
      for (int g = 0; g < ng; ++g) s += gsum[g * 2 * D + i];
      p.part[(int64_t)blockIdx.x * 2 * D + i] = s;
    }
  }
}

// Sums the workgroups' partial gain gradients, 16 columns a workgroup, 64 threads a column, in a
// fixed order and in 64 bits.
__global__ __launch_bounds__(1024) void qk_gains(const float* part, int rows, int head_dim, float* dq, float* dk) {
  __shared__ double sums[64][17];
  const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4, col = blockIdx.x * 16 + c, cols = 2 * head_dim;
  double s = 0.0;
  if (col < cols) {
    int r = r0;
    for (; r + 192 < rows; r += 256) {                 // four loads on their way
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = part[(int64_t)(r + 64 * u) * cols + col];
#pragma unroll
      for (int u = 0; u < 4; ++u) s += (double)v[u];
    }
    for (; r < rows; r += 64) s += (double)part[(int64_t)r * cols + col];
  }
  sums[r0][c] = s;
  __syncthreads();
  if (r0 == 0 && col < cols) {
    double all = 0.0;
    for (int r = 0; r < 64; ++r) all += sums[r][c];
    float* out = col < head_dim ? dq : dk;
    if (out) out[col < head_dim ? col : col - head_dim] = (float)all;
  }
}

template <class E, bool WIDE, bool HALF>
hipError_t go(const QkKind& k, const QkParams& p, hipStream_t s) {
  const dim3 grid((unsigned)p.workgroups), block(kQkThreads);
  if (k.backward && k.norm) hipLaunchKernelGGL((qk_rotary<E, WIDE, HALF, true, true>), grid, block, 0, s, p);
  else if (k.backward) hipLaunchKernelGGL((qk_rotary<E, WIDE, HALF, false, true>), grid, block, 0, s, p);
  else if (k.norm) hipLaunchKernelGGL((qk_rotary<E, WIDE, HALF, true, false>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((qk_rotary<E, WIDE, HALF, false, false>), grid, block, 0, s, p);
  return hipGetLastError();
}
template <class E>
hipError_t go(const QkKind& k, const QkParams& p, hipStream_t s) {
  if (k.wide) return k.half ? go<E, true, true>(k, p, s) : go<E, true, false>(k, p, s);
  return k.half ? go<E, false, true>(k, p, s) : go<E, false, false>(k, p, s);
}

}  // namespace

hipError_t launch_qk(const QkKind& k, const QkParams& p, hipStream_t s) {
  if (p.workgroups <= 0) return hipSuccess;
  return k.bf16 ? go<uint16_t>(k, p, s) : go<float>(k, p, s);
}

hipError_t launch_qk_gains(const float* part, int rows, int head_dim, float* dq, float* dk, hipStream_t s) {
  hipLaunchKernelGGL(qk_gains, dim3((unsigned)((2 * head_dim + 15) / 16)), dim3(1024), 0, s, part, rows, head_dim, dq, dk);
  return hipGetLastError();
}

}  // namespace ge
