// train.cuh -- device helpers of the training-step kernels.
#pragma once

#include "device_common.cuh"

namespace rwo {

// One element, by a load that is not moved and sees this kernel's own stores.
template <class D>
__device__ __forceinline__ float load1c(const void* p, int64_t i) {
  if constexpr (D::kBytes == 4) {
    return static_cast<const volatile float*>(p)[i];
  } else {
    const uint32_t b = static_cast<const volatile uint16_t*>(p)[i];
    if constexpr (D::kNegInfWord == BF16::kNegInfWord) return bf16_lo(b);
    else return f16_lo(b);
  }
}

// A value as the element type holds it.
template <class D>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (D::kBytes == 4) return v;
  else if constexpr (D::kNegInfWord == BF16::kNegInfWord) return bf16_lo(pack_bf16x2(v, 0.f));
  else return f16_lo(pack_f16x2(v, 0.f));
}

}  // namespace rwo
