// A lane's share of a state row, and sums over the lanes of a row (internal): what the
// one-token kernels of the recurrences have in common.
#pragma once

#include "selective_common.h"

namespace dcconv {
namespace {

constexpr int kRowLanes = 16;  // lanes that share a state row

// VEC neighbouring values of a state row, F32 or BF16 in memory.
template <bool F32, int VEC>
struct StateVec;
template <>
struct StateVec<true, 4> {
    u32x4 w;
    __device__ __forceinline__ void load(const void *s, int64_t at) {
        w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(static_cast<const float *>(s) + at));
    }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(w[i]); }
    __device__ __forceinline__ void set(int i, float v) { w[i] = __float_as_uint(v); }
    __device__ __forceinline__ void store(void *s, int64_t at) const {
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(static_cast<float *>(s) + at));
    }
};
template <>
struct StateVec<false, 8> {
    u32x4 w;
    float v[8];
    __device__ __forceinline__ void load(const void *s, int64_t at) {
        w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(s) + at));
    }
    __device__ __forceinline__ float get(int i) const { return (i & 1) ? hi_f32(w[i >> 1]) : lo_f32(w[i >> 1]); }
    __device__ __forceinline__ void set(int i, float x) { v[i] = x; }
    __device__ __forceinline__ void store(void *s, int64_t at) const {
        const u32x4 o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7])};
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(s) + at));
    }
};
template <bool F32>
struct StateVec<F32, 1> {
    float v;
    __device__ __forceinline__ void load(const void *s, int64_t at) {
        v = F32 ? static_cast<const float *>(s)[at] : bf16_bits_to_f32(static_cast<const uint16_t *>(s)[at]);
    }
    __device__ __forceinline__ float get(int) const { return v; }
    __device__ __forceinline__ void set(int, float x) { v = x; }
    __device__ __forceinline__ void store(void *s, int64_t at) const {
        if (F32)
            static_cast<float *>(s)[at] = v;
        else
            static_cast<uint16_t *>(s)[at] = f32_to_bf16_bits(v);
    }
};

// The sum over the 16 lanes of a row, in all of them.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum(float v) {
    v = dpp_add<0x128>(v);  // rotations of the row by 8, 4, 2 and 1
    v = dpp_add<0x124>(v);
    v = dpp_add<0x122>(v);
    return dpp_add<0x121>(v);
}

}  // namespace
}  // namespace dcconv
