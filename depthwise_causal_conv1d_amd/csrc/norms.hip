// The norms of a layer for gfx950: of the recurrence's output, times silu(z), and of the
// residual stream between two blocks.
//
//     gated:  out = x / rms(x) * (w + o) * silu(z),  or  y / rms(y) * (w + o), y = x * silu(z)
//     add:    y = x or x / rms(x) * (w' + o);  r += s * y * gate;  out = r / rms(r) * (w + o)
//
// with rms(v) = sqrt(mean of v^2 + eps).  A row is read once and stays in registers, eight
// values a lane and vector; 16, 32 or 64 lanes share a row of up to 1024 values, and a block
// of 256 threads one of up to 16384.  Everything is FP32; what is stored is rounded once, and
// the residual's norm is taken before that.  HBM bounds both.
//
// The widths follow from the registers: a row of up to 8192 values takes at most four vectors a lane, with the fewest
// lanes that hold a row, as each doubling of the lanes adds a step to every sum.  524288 rows of
// 128 with z: 75 to 79 us, 5.2 TB/s; 16384 rows of 4096 with an F32 residual, a gate and a
// first norm: 168 us, 5.6 TB/s; a large copy reaches 5.9.  Four rows: 3.0 and 3.6 us, launch and latency.
#include "delta_params.h"
#include "state_vec.h"

namespace dcconv {
namespace {

constexpr int kNormBlock = 256;

// Sums over the LANES threads that share a row, in all of them.  `part`: four floats of LDS
// that no sum since the last barrier has used (LANES = 256 alone).
template <int LANES>
__device__ __forceinline__ float sum_lanes(float v, float *part) {
    v = row_sum(v);
    if (LANES >= 32) v += __shfl_xor(v, 16);
    if (LANES >= 64) v += __shfl_xor(v, 32);
    if (LANES == kNormBlock) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0] + part[1] + part[2] + part[3];
    }
    return v;
}

// 1 / sqrt(mean of the row's squares + eps).  A sum of squares that leaves FP32's range is
// formed again from values scaled by a power of two; under 2^-80 only where eps is not far
// above the mean anyway.  Then the values are below 2^-40, and v is left scaled by 2^100, the result
// being for the scaled values: their own may be up to 2^149.  part: eight floats of LDS.
template <int LANES, int NV>
__device__ __forceinline__ float inverse_rms(float (&v)[NV][8], int d, float eps, float *part) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(v[i][j], v[i][j], sum);
    sum = sum_lanes<LANES>(sum, part);
    const float inv = 1.0f / (float)d;
    const bool large = !(sum < 0x1p+126f), small = sum < 0x1p-80f && eps < 0x1p-100f;
    if (!large && !small) return rsqrtf(__builtin_fmaf(sum, inv, eps));
    const float scale = large ? 0x1p-80f : 0x1p+100f;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float scaled = v[i][j] * scale;
            sum = __builtin_fmaf(scaled, scaled, sum);
            if (small) v[i][j] = scaled;
        }
    sum = sum_lanes<LANES>(sum, part + 4);
    const float f = rsqrtf(__builtin_fmaf(sum, inv, eps * scale * scale));
    return small ? f : scale * f;
}

// Sixteen bytes; ONCE: of an operand that nobody reads again soon, as streaming accesses, which leave
// the caches to the weights (16384 rows of 4096, loads and stores: 169 us, without 177).
template <bool ONCE>
__device__ __forceinline__ u32x4 load16(const void *at) {
    const u32x4 *p = static_cast<const u32x4 *>(at);
    return ONCE ? __builtin_nontemporal_load(p) : *p;
}
__device__ __forceinline__ void store16(void *at, u32x4 v) {
    __builtin_nontemporal_store(v, static_cast<u32x4 *>(at));
}

// Eight values from element `at` of a BF16 array, of which `count` exist (the rest: zeros).
template <bool WIDE, bool ONCE = true>
__device__ __forceinline__ void load8(const uint16_t *base, int64_t at, int count, float (&v)[8]) {
    if (WIDE) {
        u32x4 w = {0, 0, 0, 0};
        if (count > 0) w = load16<ONCE>(base + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (i & 1) ? hi_f32(w[i >> 1]) : lo_f32(w[i >> 1]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < count ? bf16_bits_to_f32(base[at + i]) : 0.0f;
}
template <bool WIDE, bool ONCE = true>
__device__ __forceinline__ void load8(const float *base, int64_t at, int count, float (&v)[8]) {
    if (WIDE) {
        u32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (count > 0) {
            a = load16<ONCE>(base + at);
            b = load16<ONCE>(base + at + 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]), v[4 + i] = __uint_as_float(b[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < count ? base[at + i] : 0.0f;
}
template <bool WIDE, bool ONCE>
__device__ __forceinline__ void load8(const void *base, bool f32, int64_t at, int count, float (&v)[8]) {
    if (f32)
        load8<WIDE, ONCE>(static_cast<const float *>(base), at, count, v);
    else
        load8<WIDE, ONCE>(static_cast<const uint16_t *>(base), at, count, v);
}
template <bool WIDE>
__device__ __forceinline__ void store8(uint16_t *base, int64_t at, int count, const float (&v)[8]) {
    if (WIDE) {
        if (count > 0)
            store16(base + at, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                     pack_bf16x2(v[6], v[7])});
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < count) base[at + i] = f32_to_bf16_bits(v[i]);
}
template <bool WIDE>
__device__ __forceinline__ void store8(float *base, int64_t at, int count, const float (&v)[8]) {
    if (WIDE) {
        if (count > 0) {
            store16(base + at, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
            store16(base + at + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < count) base[at + i] = v[i];
}

// row / size and what is left, by 32-bit division where that is enough.
__device__ __forceinline__ int64_t divide(int64_t row, int64_t size, int64_t *rest) {
    const int64_t q = ((row | size) >> 32) == 0 ? (int64_t)((uint32_t)row / (uint32_t)size) : row / size;
    *rest = row - q * size;
    return q;
}

template <int LANES, int NV, bool WIDE>
__global__ __launch_bounds__(kNormBlock) void gated_norm_kernel(const GatedNormParams p, int64_t rows, int64_t units) {
    constexpr int kRows = kNormBlock / LANES;
    __shared__ float part[8];
    const int sub = threadIdx.x % LANES;
    for_each_unit(units, [&](int64_t u) {
        const int64_t row = u * kRows + threadIdx.x / LANES;
        if (row >= rows) return;
        int64_t h, t;
        const int64_t nt = divide(row, p.h, &h), n = divide(nt, p.t, &t);
        const int64_t xa = n * p.xs_n + t * p.xs_t + h * p.xs_h, za = n * p.zs_n + t * p.zs_t + h * p.zs_h;
        float x[NV][8], gate[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * LANES + sub);
            load8<WIDE>(p.x, xa + c, p.d - c, x[i]);
            if (p.z != nullptr) load8<WIDE>(p.z, za + c, p.d - c, gate[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                gate[i][j] = p.z != nullptr ? activate<DCCONV_ACT_SILU>(gate[i][j]) : 1.0f;
                if (p.gate_first) x[i][j] *= gate[i][j], gate[i][j] = 1.0f;
            }
        const float f = inverse_rms<LANES, NV>(x, p.d, p.eps, part);
        const int64_t oa = n * p.os_n + t * p.os_t + h * p.os_h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * LANES + sub);
            float w[8];
            if (p.weight != nullptr) load8<WIDE, false>(p.weight, p.weight_f32, h * p.ws_h + c, p.d - c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[i][j] = x[i][j] * f * (p.weight != nullptr ? w[j] + p.offset : 1.0f) * gate[i][j];
            store8<WIDE>(p.out, oa + c, p.d - c, x[i]);
        }
        if (LANES == kNormBlock) __syncthreads();  // the next unit reuses `part`
    });
}

template <int LANES, int NV, bool F32, bool WIDE>
__global__ __launch_bounds__(kNormBlock) void add_norm_kernel(const AddNormParams p, int64_t rows, int64_t units) {
    constexpr int kRows = kNormBlock / LANES;
    __shared__ float part[16];
    const int sub = threadIdx.x % LANES;
    for_each_unit(units, [&](int64_t u) {
        const int64_t row = u * kRows + threadIdx.x / LANES;
        if (row >= rows) return;
        int64_t t;
        const int64_t n = divide(row, p.t, &t);
        const int64_t xa = n * p.xs_n + t * p.xs_t, ra = n * p.rs_n + t * p.rs_t, ga = n * p.gs_n + t * p.gs_t;
        float y[NV][8], r[NV][8], gate[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * LANES + sub);
            load8<WIDE>(p.x, xa + c, p.d - c, y[i]);
            load8<WIDE, true>(p.residual, F32, ra + c, p.d - c, r[i]);
            if (p.gate != nullptr) load8<WIDE>(p.gate, ga + c, p.d - c, gate[i]);
        }
        if (p.post != nullptr) {
            const float f = inverse_rms<LANES, NV>(y, p.d, p.eps, part);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = 8 * (i * LANES + sub);
                float w[8];
                load8<WIDE, false>(p.post, p.weight_f32, c, p.d - c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * f * (w[j] + p.offset);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * LANES + sub);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (p.gate != nullptr) y[i][j] *= gate[i][j];
                r[i][j] = __builtin_fmaf(p.residual_scale, y[i][j], r[i][j]);
            }
            if (F32)
                store8<WIDE>(static_cast<float *>(p.residual), ra + c, p.d - c, r[i]);
            else
                store8<WIDE>(static_cast<uint16_t *>(p.residual), ra + c, p.d - c, r[i]);
        }
        const float f = inverse_rms<LANES, NV>(r, p.d, p.eps, part + 8);
        const int64_t oa = n * p.os_n + t * p.os_t;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (i * LANES + sub);
            float w[8];
            load8<WIDE, false>(p.weight, p.weight_f32, c, p.d - c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * f * (w[j] + p.offset);
            store8<WIDE>(p.out, oa + c, p.d - c, r[i]);
        }
        if (LANES == kNormBlock) __syncthreads();  // the next unit reuses `part`
    });
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int LANES, int NV>
hipError_t launch_gated(const GatedNormParams &p, bool wide, hipStream_t stream) {
    const int64_t rows = p.n * p.t * p.h, units = (rows + kNormBlock / LANES - 1) / (kNormBlock / LANES);
    const dim3 grid((unsigned)(units < kMaxBlocks ? units : kMaxBlocks));
    if (wide)
        gated_norm_kernel<LANES, NV, true><<<grid, kNormBlock, 0, stream>>>(p, rows, units);
    else
        gated_norm_kernel<LANES, NV, false><<<grid, kNormBlock, 0, stream>>>(p, rows, units);
    return hipGetLastError();
}

template <int LANES, int NV>
hipError_t launch_add(const AddNormParams &p, bool wide, hipStream_t stream) {
    const int64_t rows = p.n * p.t, units = (rows + kNormBlock / LANES - 1) / (kNormBlock / LANES);
    const dim3 grid((unsigned)(units < kMaxBlocks ? units : kMaxBlocks));
    if (p.residual_f32) {
        if (wide)
            add_norm_kernel<LANES, NV, true, true><<<grid, kNormBlock, 0, stream>>>(p, rows, units);
        else
            add_norm_kernel<LANES, NV, true, false><<<grid, kNormBlock, 0, stream>>>(p, rows, units);
    } else {
        if (wide)
            add_norm_kernel<LANES, NV, false, true><<<grid, kNormBlock, 0, stream>>>(p, rows, units);
        else
            add_norm_kernel<LANES, NV, false, false><<<grid, kNormBlock, 0, stream>>>(p, rows, units);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_norm(const GatedNormParams &p, hipStream_t stream, const char **kernel_name) {
    const bool wide = p.d % 8 == 0 && aligned16(p.x) && aligned16(p.out) && (p.xs_n | p.xs_t | p.xs_h) % 8 == 0 &&
                      (p.os_n | p.os_t | p.os_h) % 8 == 0 &&
                      (p.z == nullptr || (aligned16(p.z) && (p.zs_n | p.zs_t | p.zs_h) % 8 == 0)) &&
                      (p.weight == nullptr || (aligned16(p.weight) && p.ws_h % 8 == 0));
    *kernel_name = wide ? "gated_norm" : "gated_norm_scalar";
    if (p.d <= 128) return launch_gated<16, 1>(p, wide, stream);
    if (p.d <= 256) return launch_gated<32, 1>(p, wide, stream);
    if (p.d <= 512) return launch_gated<64, 1>(p, wide, stream);
    if (p.d <= 1024) return launch_gated<64, 2>(p, wide, stream);
    if (p.d <= 2048) return launch_gated<256, 1>(p, wide, stream);
    if (p.d <= 4096) return launch_gated<256, 2>(p, wide, stream);
    if (p.d <= 8192) return launch_gated<256, 4>(p, wide, stream);
    return launch_gated<256, 8>(p, wide, stream);
}

hipError_t launch_add_norm(const AddNormParams &p, hipStream_t stream, const char **kernel_name) {
    const bool wide = p.d % 8 == 0 && aligned16(p.x) && aligned16(p.out) && aligned16(p.residual) &&
                      (p.xs_n | p.xs_t | p.rs_n | p.rs_t | p.os_n | p.os_t) % 8 == 0 &&
                      (p.gate == nullptr || (aligned16(p.gate) && (p.gs_n | p.gs_t) % 8 == 0)) &&
                      aligned16(p.weight) && aligned16(p.post);
    *kernel_name = wide ? "add_norm" : "add_norm_scalar";
    if (p.d <= 128) return launch_add<16, 1>(p, wide, stream);
    if (p.d <= 256) return launch_add<32, 1>(p, wide, stream);
    if (p.d <= 512) return launch_add<64, 1>(p, wide, stream);
    if (p.d <= 1024) return launch_add<64, 2>(p, wide, stream);
    if (p.d <= 2048) return launch_add<256, 1>(p, wide, stream);
    if (p.d <= 4096) return launch_add<256, 2>(p, wide, stream);
    if (p.d <= 8192) return launch_add<256, 4>(p, wide, stream);
    return launch_add<256, 8>(p, wide, stream);
}

}  // namespace dcconv
