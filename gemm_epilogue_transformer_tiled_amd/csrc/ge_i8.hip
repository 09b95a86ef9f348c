// Product of int8 codes with scales per token and per channel: its tiles on the mainloop of
// ge_ffn_impl.h (gfx950).
//
// 128 codes lie where 64 bf16 values do, so staging, swizzles and waits are those of the bf16 products, and a step of
// v_mfma_i32_16x16x64_i8 takes the place of one of v_mfma_f32_16x16x32_bf16 with twice the products.  Sums are int32 and
// exact: tiles and splits of the contraction give equal bits.  Bound by the matrix cores under the power limit with many
// rows (8192 x 11008 x 4096, bias and SiLU: 292 to 297 us in a run of a second, 2.5 POP/s, matrix cores busy 73 % of the
// time; 310 to 330 us a launch on its own, up to 370 in the first ten after a pause; 8192^3 2.8 to 3.0 POP/s), by idle compute
// units or a second round of tiles and their epilogue with middle ones (777 x 2856 x 1040: 10.8 us; 512 x 4096 x 4096 15.7 us
// with its operands in the caches, 21.8 from memory), by the weights' way from memory and the tiles' latency with few
// (27 x 4096 x 11008: 13.0 to 13.3 us, 45 MB of weights).
#include "ge_ffn_impl.h"
#include "ge_rows_internal.h"

namespace ge {
namespace {

template <class T>
hipError_t go(const I8Launch& l, hipStream_t s) {
  hipLaunchKernelGGL((ffn_product<T, FFN_I8, ACT_NONE, false, false, I8Launch>),
                     dim3((unsigned)(l.tiles * (T::PP ? 1 : l.splits))), dim3(T::NT), 0, s, l);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8(int tile, const I8Launch& l, hipStream_t s) {
  if (l.tiles <= 0) return hipSuccess;
  switch (tile) {
    case FFN_T256: return go<F256>(l, s);
    case FFN_T128: return go<F128>(l, s);
    case FFN_T64: return go<F64>(l, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ge
