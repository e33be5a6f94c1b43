// Products of a few rows with a 4-bit weight matrix for gfx950:
//
//     out[m, n] = sum_k x[m, k] * (q[n, k] - zero[k / group, n]) * scale[k / group, n] + bias[n]
//
// The weights are read once and are nearly all of the bytes, so HBM bounds the call
// as long as turning codes into operands costs less than reading them.  Three things
// keep it so.  The codes come in tiles of 16 outputs by 128 inputs in the order that
// lanes use them: one coalesced 16-byte load is a lane's share of four matrix
// instructions.  A code becomes a BF16 without a conversion: or-ed into the mantissa
// of 128 it reads 128 + q, exactly, two codes at a time (an and-or, and a shift for
// three of four), because a word's nibbles i and i + 4 hold neighbouring inputs.  And
// the matrix cores do the multiplying for one row of x as for sixteen; they also sum
// x itself against ones, and per group
//
//     sum x (q - zero) = sum x (128 + q) - (128 + zero) * sum x
//
// takes the offset out again in FP32 (it costs about 5 of FP32's 24 bits, of which a
// BF16 result keeps 8).  Products and sums are FP32 throughout; out is rounded once.
//
// A block owns NT tiles of outputs and its waves share out the inputs, 128 at a
// time; they are joined through LDS in the order of the waves.
#include "selective_common.h"

namespace dcconv {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTileN = 16, kTileK = 128;
constexpr int kMaxW4Waves = 16;

__device__ __forceinline__ f32x4_t mfma(u32x4 a, u32x4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

// Eight codes -> eight BF16 128 + q: nibbles i and i + 4 become word i.
__device__ __forceinline__ u32x4 expand(uint32_t w) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    return v;
}

// Up to eight consecutive values of a row, `count` of which exist: zeros behind.
template <bool WIDE>
__device__ __forceinline__ u32x4 load8(const uint16_t *s, int count) {
    u32x4 v = {0, 0, 0, 0};
    if (WIDE) {
        if (count > 0) v = *reinterpret_cast<const u32x4 *>(s);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) v[i >> 1] |= (uint32_t)s[i] << (16 * (i & 1));
    }
    return v;
}

// NT tiles of outputs, MT tiles of 16 rows of x; STEPS matrix instructions (of 32
// inputs) share a scale.
template <int NT, int MT, int STEPS, bool WIDE>
__global__ __launch_bounds__(kMaxW4Waves *kWave) void w4_matvec_kernel(const W4Params p) {
    extern __shared__ float joined[];  // [wave][NT][MT][16 x 16]
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int ktiles = (p.k + kTileK - 1) / kTileK, ntiles = (p.n + kTileN - 1) / kTileN;
    const int nt0 = blockIdx.x * NT;
    const int m0 = blockIdx.y * MT * 16;

    f32x4_t total[NT][MT];
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int b = 0; b < MT; ++b) total[a][b] = f32x4_t{0, 0, 0, 0};
    const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};

    for (int kt = wave; kt < ktiles; kt += waves) {
        u32x4 q[NT];
#pragma unroll
        for (int a = 0; a < NT; ++a)
            q[a] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p.q) +
                                              ((int64_t)min(nt0 + a, ntiles - 1) * ktiles + kt) * kWave + lane);
        float scale[NT][4 / STEPS], offset[NT][4 / STEPS];
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int s = 0; s < 4 / STEPS; ++s) {
                const int n = (nt0 + a) * kTileN + r, k = kt * kTileK + s * STEPS * 32;
                float sc = 0.0f, zero = 8.0f;
                if (n < p.n && k < p.k) {
                    const int64_t at = (int64_t)(k / p.group) * p.n + n;
                    sc = bf16_bits_to_f32(p.scales[at]);
                    if (p.zeros != nullptr) zero = (float)p.zeros[at];
                }
                scale[a][s] = sc;
                offset[a][s] = -sc * (128.0f + zero);
            }
        u32x4 x[MT][4];
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int m = m0 + 16 * b + r, k = kt * kTileK + 32 * s + 8 * g;
                x[b][s] = load8<WIDE>(p.x + (int64_t)m * p.xs_m + k, m < p.m ? p.k - k : 0);
            }
#pragma unroll
        for (int s = 0; s < 4 / STEPS; ++s) {
            f32x4_t sum[MT], acc[NT][MT];
#pragma unroll
            for (int b = 0; b < MT; ++b) {
                sum[b] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int a = 0; a < NT; ++a) acc[a][b] = f32x4_t{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
#pragma unroll
                for (int b = 0; b < MT; ++b) sum[b] = mfma(x[b][s * STEPS + i], ones, sum[b]);
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    const u32x4 w = expand(q[a][s * STEPS + i]);
#pragma unroll
                    for (int b = 0; b < MT; ++b) acc[a][b] = mfma(x[b][s * STEPS + i], w, acc[a][b]);
                }
            }
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int b = 0; b < MT; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        total[a][b][i] = __builtin_fmaf(offset[a][s], sum[b][i],
                                                        __builtin_fmaf(scale[a][s], acc[a][b][i], total[a][b][i]));
        }
    }

    // lane (r, g) holds output r, rows 4 g .. 4 g + 3 of each tile
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                joined[((wave * NT + a) * MT + b) * 256 + (4 * g + i) * 16 + r] = total[a][b][i];
    __syncthreads();
    for (int e = threadIdx.x; e < NT * MT * 256; e += blockDim.x) {
        const int n = (nt0 + (e >> 8) / MT) * kTileN + (e & 15), m = m0 + ((e >> 8) % MT) * 16 + ((e >> 4) & 15);
        if (n >= p.n || m >= p.m) continue;
        float v = p.bias != nullptr ? bf16_bits_to_f32(p.bias[n]) : 0.0f;
        for (int w = 0; w < waves; ++w) v += joined[w * NT * MT * 256 + e];
        p.out[(int64_t)m * p.os_m + n] = f32_to_bf16_bits(v);
    }
}

// One byte of the tiles a thread: byte 4 q + 2 u + v of lane 16 j + i holds output i
// and inputs 32 q + 8 j + 4 v + u (low half) and, two further, the high half.
__global__ __launch_bounds__(256) void w4_pack_kernel(const uint8_t *codes, int64_t n, int64_t k, int64_t ktiles,
                                                      int64_t bytes, uint8_t *out) {
    for_each_unit((bytes + 255) / 256, [&](int64_t unit) {
        const int64_t at = unit * 256 + threadIdx.x;
        if (at >= bytes) return;
        const int byte = (int)(at & 15), lane = (int)(at >> 4) & 63;
        const int64_t tile = at >> 10;
        const int64_t row = tile / ktiles * kTileN + (lane & 15);
        const int64_t col = tile % ktiles * kTileK + 32 * (byte >> 2) + 8 * (lane >> 4) + 4 * (byte & 1) + (byte >> 1 & 1);
        const int lo = row < n && col < k ? codes[row * k + col] & 15 : 8;
        const int hi = row < n && col + 2 < k ? codes[row * k + col + 2] & 15 : 8;
        out[at] = (uint8_t)(lo | hi << 4);
    });
}

// Waves of a block: as many as keep about this many on the card, with an input tile each.
constexpr int64_t kW4Waves = 4096;

template <int NT, int MT, int STEPS>
hipError_t launch_tiles(const W4Params &p, bool wide, hipStream_t stream) {
    const int64_t ktiles = (p.k + kTileK - 1) / kTileK;
    const int64_t blocks = ((p.n + kTileN - 1) / kTileN + NT - 1) / NT, rows = (p.m + 16 * MT - 1) / (16 * MT);
    int waves = 4;
    while (waves < kMaxW4Waves && blocks * rows * waves < kW4Waves) waves *= 2;
    while (waves > 1 && waves > ktiles) waves /= 2;
    if (rows > 65535) return hipErrorInvalidConfiguration;
    const size_t lds = (size_t)waves * NT * MT * 256 * 4;
    const dim3 grid((unsigned)blocks, (unsigned)rows);
    if (wide)
        w4_matvec_kernel<NT, MT, STEPS, true><<<grid, waves * kWave, lds, stream>>>(p);
    else
        w4_matvec_kernel<NT, MT, STEPS, false><<<grid, waves * kWave, lds, stream>>>(p);
    return hipGetLastError();
}

template <int STEPS>
hipError_t launch_steps(const W4Params &p, bool wide, hipStream_t stream) {
    if (p.m <= 16) return launch_tiles<1, 1, STEPS>(p, wide, stream);
    if (p.m <= 32) return launch_tiles<1, 2, STEPS>(p, wide, stream);
    return launch_tiles<1, 4, STEPS>(p, wide, stream);
}

}  // namespace

hipError_t launch_w4_matvec(const W4Params &p, hipStream_t stream, const char **kernel_name) {
    const bool wide = p.k % 8 == 0 && p.xs_m % 8 == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0;
    *kernel_name = wide ? "w4_matvec" : "w4_matvec_scalar";
    if (p.group % 128 == 0) return launch_steps<4>(p, wide, stream);
    if (p.group % 64 == 0) return launch_steps<2>(p, wide, stream);
    return launch_steps<1>(p, wide, stream);
}

hipError_t launch_w4_pack(const uint8_t *codes, int64_t n, int64_t k, uint8_t *q, hipStream_t stream) {
    const int64_t ktiles = (k + kTileK - 1) / kTileK;
    const int64_t bytes = (n + kTileN - 1) / kTileN * ktiles * 1024, units = (bytes + 255) / 256;
    w4_pack_kernel<<<dim3((unsigned)(units < kMaxBlocks ? units : kMaxBlocks)), 256, 0, stream>>>(codes, n, k, ktiles,
                                                                                                bytes, q);
    return hipGetLastError();
}

}  // namespace dcconv
