// Device helpers of the state-space kernels (internal).
#pragma once

#include "device_common.h"
#include "selective_params.h"

namespace dcconv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// log(1 + e^v); above 20 the result rounds to v.  (A NaN takes the second form
// and stays one.)
__device__ __forceinline__ float softplus(float v) { return v > 20.0f ? v : log1pf(expf(v)); }

__device__ __forceinline__ float silu(float v) { return activate<DCCONV_ACT_SILU>(v); }

// The step of head `head` at element `at` of dt: bias and softplus applied, 32 bits.
template <typename Params>
__device__ __forceinline__ float load_step(const Params &p, int64_t at, int head) {
    float v = p.dt_f32 ? static_cast<const float *>(p.dt)[at]
                       : bf16_bits_to_f32(static_cast<const uint16_t *>(p.dt)[at]);
    if (p.dt_bias != nullptr) v += p.dt_bias[head];
    return p.dt_softplus ? softplus(v) : v;
}

}  // namespace
}  // namespace dcconv
