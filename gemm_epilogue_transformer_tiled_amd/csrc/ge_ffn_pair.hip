// Gated feed-forward block: the gate/up pair, every activation.
#include "ge_ffn_impl.h"

namespace ge {
namespace {

template <class T, int MODE, bool BC>
hipError_t by_act(int act, const FfnLaunch& l, hipStream_t s) {
  switch (act) {
    case ACT_NONE: return launch_product<T, MODE, ACT_NONE, false, BC>(l, s);
    case ACT_RELU: return launch_product<T, MODE, ACT_RELU, false, BC>(l, s);
    case ACT_GELU_TANH: return launch_product<T, MODE, ACT_GELU_TANH, false, BC>(l, s);
    case ACT_SILU: return launch_product<T, MODE, ACT_SILU, false, BC>(l, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_ffn_pair(int tile, int act, bool b_nk, const FfnLaunch& l, hipStream_t s) {
  switch (tile) {
    case FFN_T256: return b_nk ? by_act<F256P, FFN_PAIR, false>(act, l, s) : by_act<F256P, FFN_PAIR, true>(act, l, s);
    case FFN_T128: return b_nk ? by_act<F128P, FFN_PAIR, false>(act, l, s) : by_act<F128P, FFN_PAIR, true>(act, l, s);
    case FFN_T64: return b_nk ? by_act<F64P, FFN_PAIR, false>(act, l, s) : by_act<F64P, FFN_PAIR, true>(act, l, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ge
