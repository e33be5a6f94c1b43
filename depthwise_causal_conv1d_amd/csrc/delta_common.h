// Device helpers of the gated delta rule's kernels (internal).
#pragma once

#include "delta_params.h"
#include "selective_common.h"

namespace dcconv {
namespace {

// Element `at` of a BF16 or F32 array.
__device__ __forceinline__ float load_either(const void *base, bool f32, int64_t at) {
    return f32 ? static_cast<const float *>(base)[at] : bf16_bits_to_f32(static_cast<const uint16_t *>(base)[at]);
}

// 1 / (1 + e^-v): within 2^-22 of itself; 0 and 1 at the ends.
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// The weight of a token's correction, from what memory holds.
__device__ __forceinline__ float weight_of(const DeltaParams &p, float v) { return p.beta_sigmoid ? sigmoid(v) : v; }

// 1 / sqrt(sum of squares + eps), or 1 where q and key are taken as they are.
__device__ __forceinline__ float unit_factor(const DeltaParams &p, float squares) {
    return p.l2norm ? rsqrtf(squares + p.eps) : 1.0f;
}

}  // namespace
}  // namespace dcconv
