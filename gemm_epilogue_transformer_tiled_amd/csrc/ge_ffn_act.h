// Activations of the gated feed-forward block's kernels: those of the fused products, but a ReLU that
// keeps NaN (the hardware's maximum of NaN and 0 is 0, which would hide a broken gate).
#pragma once

#include "ge_kernel_impl.h"

namespace ge {

__device__ __forceinline__ float relu_nan(float z) { return z < 0.0f ? 0.0f : z; }

template <int ACT>
__device__ __forceinline__ float gate(float z) {
  if constexpr (ACT == ACT_RELU) return relu_nan(z);
  else return activate<ACT>(z);
}

// An output of the product of codes from its sum times the row's scale.  One function for all its kernels, and
// the residual never fused into the activation's last product: every tile gives the same bits.
template <int ACT>
__device__ __forceinline__ float i8_output(float sum, float w_scale, float bias, float residual) {
#pragma clang fp contract(off)
  const float y = gate<ACT>(__builtin_fmaf(sum, w_scale, bias));
  return y + residual;
}

}  // namespace ge
