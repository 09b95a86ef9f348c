// Layer norm of rows: the backward pass with the sums of the gain's and the bias' gradients (gfx950).
//
// Memory-bound: dY, S (and dS) are read once, dX (and dR) written once.  A row lies in registers as in the
// forward pass; the sums behind mean(e) and mean(e n) are taken in one exchange.  A thread holds the same columns of every
// row, so it adds up dgain and dbias of its columns in registers over all rows of its workgroup, and
// a workgroup leaves one partial sum per column; a second launch adds these in 64 bits, in a fixed order.
// (Atomic adds would need no second launch, but their order changes the last bits.  A ticket, with the last workgroup
// adding the partial sums in their order, would keep them; that was not built.)  Measured: 16384 x 4096 bf16 with dropout
// 0.1, dS and dR, 671 MB, 114 us, 5.9 TB/s; 1001 x 1021 fp32 9.9 us; 4096 x 16384 bf16 with dS or dR 104 to 107 us, 5.1
// TB/s; 2048 x 32768 with both 132 us, 5.1 TB/s (with everything in registers, which spilled, 283 and 801 us).
#include "ge_rows_common.h"

namespace ge {
namespace {

constexpr int kLarge = kRowsLoadsOnce | kRowsStoresThrough;

template <class E, int TR, int V, bool TAIL, bool DROP, int POLICY>
__global__ __launch_bounds__(TR < 256 ? 256 : TR) void norm_backward(NormGradParams p) {
  constexpr int NT = TR < 256 ? 256 : TR, RPW = NT / TR;
  __shared__ float red[2][2][NT / 64];
  __shared__ f32x4 meet[RPW > 1 ? 4 * RPW * TR * V : 1];
  // WIDE: more than a vector a thread of the largest workgroup, which has 128 registers a thread.  dgain's sums then lie
  // in LDS, each thread's in places of its own, and e and c are taken again from dY and S after the exchange.  AHEAD: the
  // next row's loads have room.  LATE: the gain and dS are loaded where they are used.  TWICE: dY is loaded again for
  // its second use (fp32 rows past 16384; some registers still spill there, 1024 x 32768 with dS 173 to 178 us, 3.0 TB/s).
  constexpr bool WIDE = TR == 1024 && V > 1;
  constexpr int kHeld = V * (int)sizeof(E) * 2;        // registers of a row's dY
  constexpr bool AHEAD = !WIDE || kHeld <= 8, LATE = V > 2, TWICE = LATE && kHeld > 16;
  __shared__ f32x4 wide_sum[WIDE ? 2 * V * TR : 1];
  const int t = (int)threadIdx.x % TR, sub = (int)threadIdx.x / TR, d = p.d;
  const uint32_t blocks = (uint32_t)(d + 7) / 8u;
  const float of_d = (float)d;
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);
  float dgain[V][8], dbias[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dgain[i][j] = dbias[i][j] = 0.0f;
    if constexpr (WIDE) wide_sum[2 * i * TR + t] = wide_sum[(2 * i + 1) * TR + t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  Raw<E> gain[V];
  if constexpr (!LATE)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (p.gain) gain[i] = fetch_settled<E, TAIL>((const E*)p.gain, 8 * (t + TR * i), d);
  struct Row {
    Raw<E> dy[V], s[V], ds[V];
    float mean, rstd;
  };
  const int64_t step = (int64_t)gridDim.x * RPW;
  // The thread's number, for WIDE not known to be the same as before: no address is kept from row to row.
  auto place = [&] {
    int c = t;
    if constexpr (WIDE) {
      asm volatile("" : "+v"(c));
      c &= TR - 1;
    }
    return c;
  };
  auto load = [&](Row& q, int64_t row, int t) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 8 * (t + TR * i);
      q.dy[i] = fetch<E, TAIL, POLICY>((const E*)p.dy + row * p.lddy, col, d);
      q.s[i] = fetch<E, TAIL, POLICY>((const E*)p.s + row * p.lds, col, d);
      if (!LATE && p.ds) q.ds[i] = fetch<E, TAIL, POLICY>((const E*)p.ds + row * p.ldds, col, d);
    }
    q.mean = p.mean[row];
    q.rstd = p.rstd[row];
  };
  int turn = 0;
  int64_t row = (int64_t)blockIdx.x * RPW + sub;
  Row next{};
  if (AHEAD && row < p.rows) load(next, row, t);
  for (; row < p.rows; row += step, turn ^= 1) {
    const int t = place();
    Row q{};
    if constexpr (AHEAD) {
      q = next;
      if (row + step < p.rows) load(next, row + step, t);              // on its way while this row is computed
    } else {
      load(q, row, t);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      settle<TAIL>(q.dy[i], 8 * (t + TR * i), d);
      settle<TAIL>(q.s[i], 8 * (t + TR * i), d);
      if (!LATE && p.ds) settle<TAIL>(q.ds[i], 8 * (t + TR * i), d);
    }
    const float mean = q.mean, rstd = q.rstd;
    float e[V][8], c[V][8], se = 0.0f, sec = 0.0f;
    // e and c = s - mean of vector i.  The row's sum is that of e c, not of e n with n = c rstd: past the row's end, where
    // dy, e and s are 0, n can be too large for a number (rows of nearly equal values far from zero), and 0 times it is
    // none.  (What dgain gets of it there is not stored.)
    auto again = [&](int i, int t) {
      if constexpr (WIDE && !LATE) landed(gain[i]);    // (kept as it lies in memory)
      Raw<E> of = zero<E>();
      if constexpr (!LATE) of = gain[i];
      else if (p.gain) of = fetch_settled<E, TAIL>((const E*)p.gain, 8 * (t + TR * i), d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[i][j] = get(q.s[i], j) - mean;
        e[i][j] = p.gain ? get(q.dy[i], j) * get(of, j) : get(q.dy[i], j);
      }
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
      again(i, t);
      if constexpr (WIDE)
#pragma unroll
        for (int j = 0; j < 8; ++j) dgain[i][j] = wide_sum[(2 * i + j / 4) * TR + t][j % 4];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dy = get(q.dy[i], j);
        se += e[i][j];
        sec = fmaf(e[i][j], c[i][j], sec);
        dgain[i][j] = fmaf(dy, c[i][j] * rstd, dgain[i][j]);
        dbias[i][j] += dy;
      }
      if constexpr (WIDE)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wide_sum[(2 * i + h) * TR + t] = f32x4{dgain[i][4 * h], dgain[i][4 * h + 1], dgain[i][4 * h + 2], dgain[i][4 * h + 3]};
      if constexpr (WIDE) {                            // one vector after the other: less is held
        asm volatile("" : "+v"(se), "+v"(sec));
#pragma unroll
        for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(dbias[i][j]));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    se = wave_sum(se);
    sec = wave_sum(sec);
    if constexpr (TR > 64) {
      const int w = (int)threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
        red[turn][0][w] = se;
        red[turn][1][w] = sec;
      }
      __syncthreads();
      se = sec = 0.0f;
#pragma unroll
      for (int k = 0; k < TR / 64; ++k) {
        se += red[turn][0][k];
        sec += red[turn][1][k];
      }
    }
    const float me = se / of_d, mec = sec / of_d * rstd * rstd;
    // The next row has landed before this one's stores go out: a wait for loads behind stores would wait for
    // the stores too.
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        landed(next.dy[i]);
        landed(next.s[i]);
        landed(next.ds[i]);
      }
      asm volatile("" : "+v"(next.mean), "+v"(next.rstd));
    }
    const int u = place();
    if constexpr (WIDE)
#pragma unroll
      for (int i = 0; i < V; ++i) {                    // (not the e and c of before: they would be kept)
        if constexpr (!TWICE) landed(q.dy[i]);
        landed(q.s[i]);
      }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = 8 * (u + TR * i);
      if constexpr (TWICE) q.dy[i] = fetch_settled<E, TAIL>((const E*)p.dy + row * p.lddy, col, d);
      if constexpr (WIDE) again(i, u);
      Raw<E> ds = zero<E>();
      if constexpr (!LATE) ds = q.ds[i];
      else if (p.ds) ds = fetch_settled<E, TAIL>((const E*)p.ds + row * p.ldds, col, d);
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = rstd * fmaf(-c[i][j], mec, e[i][j] - me);
        if (p.ds) g[j] += get(ds, j);
      }
      if (p.dr) put<E, TAIL, POLICY>((E*)p.dr + row * p.lddr, col, d, rounded(g, E()));
      if (p.dx) {
        if constexpr (DROP) {
          const Words w = philox((uint32_t)row * blocks + (uint32_t)(u + TR * i), p.drop.site, key);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = dropped(g[j], w, j, p.drop);
        }
        put<E, TAIL, POLICY>((E*)p.dx + row * p.lddx, col, d, rounded(g, E()));
      }
      if constexpr (WIDE) __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (!p.part) return;                                 // uniform
  float* const out = p.part + (int64_t)blockIdx.x * 2 * d;
  if constexpr (WIDE)
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) dgain[i][j] = wide_sum[(2 * i + j / 4) * TR + t][j % 4];
  if constexpr (RPW > 1) {
    // the rows taken at once meet in LDS and are added in their order, a vector of columns a thread
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4* const at = meet + 4 * TR * V * sub + 2 * (t + TR * i) + h;
        at[0] = f32x4{dgain[i][4 * h], dgain[i][4 * h + 1], dgain[i][4 * h + 2], dgain[i][4 * h + 3]};
        at[2 * TR * V] = f32x4{dbias[i][4 * h], dbias[i][4 * h + 1], dbias[i][4 * h + 2], dbias[i][4 * h + 3]};
      }
    __syncthreads();
    for (int q = threadIdx.x; q < 2 * TR * V; q += NT) {
      f32x4 a = meet[2 * q], b = meet[2 * q + 1];
#pragma unroll
      for (int r = 1; r < RPW; ++r) {
        a += meet[4 * TR * V * r + 2 * q];
        b += meet[4 * TR * V * r + 2 * q + 1];
      }
      const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      const int which = q / (TR * V);
      put<float, TAIL>(out + which * d, 8 * (q - which * TR * V), d, rounded(v, float()));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      put<float, TAIL>(out, 8 * (t + TR * i), d, rounded(dgain[i], float()));
      put<float, TAIL>(out + d, 8 * (t + TR * i), d, rounded(dbias[i], float()));
    }
  }
}

// Adds the workgroups' partial sums, 32 columns a workgroup, 32 threads a column.
__global__ __launch_bounds__(1024) void norm_sums(const float* part, int parts, int d, float* dgain, float* dbias) {
  __shared__ double sums[32][33];
  const int c = threadIdx.x & 31, r0 = threadIdx.x >> 5, col = blockIdx.x * 32 + c, cols = 2 * d;
  double s = 0.0;
  if (col < cols) {
    int r = r0;
    for (; r + 96 < parts; r += 128) {                 // four loads on their way
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = part[(int64_t)(r + 32 * u) * cols + col];
#pragma unroll
      for (int u = 0; u < 4; ++u) s += (double)v[u];
    }
    for (; r < parts; r += 32) s += (double)part[(int64_t)r * cols + col];
  }
  sums[r0][c] = s;
  __syncthreads();
  if (r0 == 0 && col < cols) {
    double all = 0.0;
    for (int r = 0; r < 32; ++r) all += sums[r][c];
    float* out = col < d ? dgain : dbias;
    if (out) out[col < d ? col : col - d] = (float)all;
  }
}

template <class E, int S, bool TAIL, int POLICY>
hipError_t go(const NormGradParams& p, int grid, hipStream_t s) {
  constexpr int TR = kGradShape[S].threads, V = kGradShape[S].vecs;
  const dim3 g((unsigned)grid), b(TR < 256 ? 256 : TR);
  if (p.drop.below) hipLaunchKernelGGL((norm_backward<E, TR, V, TAIL, true, POLICY>), g, b, 0, s, p);
  else hipLaunchKernelGGL((norm_backward<E, TR, V, TAIL, false, POLICY>), g, b, 0, s, p);
  return hipGetLastError();
}
template <class E, bool TAIL, int POLICY>
hipError_t by_shape(const NormGradParams& p, int grid, hipStream_t s) {
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
hipError_t by_layout(bool large, const NormGradParams& p, int grid, hipStream_t s) {
  if (p.d % 8) return by_shape<E, true, 0>(p, grid, s);
  return large ? by_shape<E, false, kLarge>(p, grid, s) : by_shape<E, false, 0>(p, grid, s);
}

}  // namespace

hipError_t launch_norm_backward(bool bf16, bool large, const NormGradParams& p, int grid, hipStream_t s) {
  if (grid <= 0) return hipSuccess;
  return bf16 ? by_layout<uint16_t>(large, p, grid, s) : by_layout<float>(large, p, grid, s);
}

hipError_t launch_norm_sums(const float* part, int parts, int d, float* dgain, float* dbias, hipStream_t s) {
  hipLaunchKernelGGL(norm_sums, dim3((unsigned)((2 * d + 31) / 32)), dim3(1024), 0, s, part, parts, d, dgain, dbias);
  return hipGetLastError();
}

}  // namespace ge
