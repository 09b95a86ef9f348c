// Gated feed-forward block: the down projection, the input gradient and the weight gradients.
#include "ge_ffn_impl.h"

namespace ge {
namespace {

template <class T>
hipError_t by_mode(int mode, bool b_nk, const FfnLaunch& l, hipStream_t s) {
  switch (mode) {
    case FFN_DOWN: return b_nk ? launch_product<T, FFN_DOWN, ACT_NONE, false, false>(l, s)
                               : launch_product<T, FFN_DOWN, ACT_NONE, false, true>(l, s);
    case FFN_DUAL: return b_nk ? launch_product<T, FFN_DUAL, ACT_NONE, false, false>(l, s)
                               : launch_product<T, FFN_DUAL, ACT_NONE, false, true>(l, s);
    case FFN_WGRAD: return launch_product<T, FFN_WGRAD, ACT_NONE, true, true>(l, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_ffn_plain(int mode, int tile, bool b_nk, const FfnLaunch& l, hipStream_t s) {
  switch (tile) {
    case FFN_T256: return by_mode<F256>(mode, b_nk, l, s);
    case FFN_T128: return by_mode<F128>(mode, b_nk, l, s);
    case FFN_T64: return by_mode<F64>(mode, b_nk, l, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ge
