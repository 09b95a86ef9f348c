// Product of int8 codes with scales per token and per channel: its tiles on the mainloop of
// ge_ffn_impl.h (gfx950).
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
