// Products of a few rows with a 4-bit weight matrix for gfx950:
//
//     out[m, n] = sum_k x[m, k] * (q[n, k] - zero[k / group, n]) * scale[k / group, n] + bias[n]
//
// The weights are read once and are nearly all of the bytes, so HBM bounds the call
// as long as turning codes into operands costs less than reading them.  Three things
// keep it so.  The codes come in tiles of 16 outputs by 128 inputs in the order that
// lanes use them: one coalesced 16-byte load is a lane's share of four matrix
// instructions.  A code becomes a BF16 without a conversion: or-ed into the mantissa
// of s = 2^-8 it reads s (1 + q / 128), exactly, two codes at a time (an and-or, and a
// shift for three of four), because a word's nibbles i and i + 4 hold neighbouring
// inputs.  And the matrix cores do the multiplying for one row of x as for sixteen; they
// also sum x itself times s, and per group
//
//     s sum x (q - zero) / 128 = sum x s (1 + q / 128) - (1 + zero / 128) * sum x s
//
// takes the offset out again in FP32 (it costs about 5 of FP32's 24 bits, of which a
// BF16 result keeps 8).  The factor s / 128 = 2^-15, undone when the waves are joined,
// leaves room for a group's sum of the largest x, which a small scale may bring back into
// range; sums of x below 2^-117 lose bits to it.  Products and sums are FP32 throughout;
// out is rounded once.
//
// A block owns a tile of outputs and its waves share out the inputs, 128 at a
// time; they are joined through LDS in the order of the waves.
//
// One row of x, 14432 x 4096 weights in groups of 128: 8.8 us, 30.5 MB at 3.5 TB/s; with
// 7200 waves of four tiles each, the launch, the first loads' latency and the join are
// the rest.  13 rows, 4096 x 6144 in groups of 64 with zero points: 9.2 us, 14 MB
// at 1.5 TB/s: one block a CU, whose sixteen waves take three tiles one after the other,
// load scales and zero points two bytes and one at a time, sum x again in every block
// and are joined by a quarter of the threads; x comes through the L2s (41 MB in all, about
// 1 us).  (Reading two or four tiles ahead was slower.)
#include "selective_common.h"

namespace dcconv {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTileN = 16, kTileK = 128;
constexpr int kMaxW4Waves = 16;
constexpr uint32_t kUnit = 0x3b80;  // 2^-8 as BF16
constexpr float kBack = 32768.0f;   // a code's step there is 2^-15

__device__ __forceinline__ f32x4_t mfma(u32x4 a, u32x4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

// Eight codes -> eight BF16 2^-8 (1 + q / 128): nibbles i and i + 4 become word i.
__device__ __forceinline__ u32x4 expand(uint32_t w) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ((w >> (4 * i)) & 0x000f000fu) | kUnit * 0x10001u;
    return v;
}

constexpr uint32_t kNowhere = 0x80000000u;  // past the end of every buffer

// What a wave reads: eight values of its lanes' rows of x from input k on, and the scale
// and zero point of group `gr` for its lanes' outputs.  WIDE goes through buffers, which
// leaves one compare and select a load to the vector units; otherwise element by element.
template <bool WIDE>
struct Operands {
    const W4Params &p;
    int n, g;
    Buffer xbuf, sbuf, zbuf;
    __device__ __forceinline__ Operands(const W4Params &p, int n, int g) : p(p), n(n), g(g) {
        if (!WIDE) return;
        const int groups = (p.k + p.group - 1) / p.group;
        xbuf = make_buffer(p.x, (uint32_t)(2 * ((p.m - 1) * p.xs_m + p.k)));
        sbuf = make_buffer(p.scales, 2u * (uint32_t)groups * (uint32_t)p.n);
        zbuf = make_buffer(p.zeros, p.zeros != nullptr ? (uint32_t)groups * (uint32_t)p.n : 0u);
    }
    // row: the byte offset of the lane's row and inner position, or kNowhere
    __device__ __forceinline__ u32x4 x(uint32_t row, int m, int k) const {
        if (WIDE) return buffer_load<kCached>(xbuf, k + 8 * g < p.k ? row + 2u * (uint32_t)k : kNowhere);
        u32x4 v = {0, 0, 0, 0};
        const uint16_t *s = p.x + (int64_t)m * p.xs_m + k + 8 * g;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (m < p.m && k + 8 * g + i < p.k) v[i >> 1] |= (uint32_t)s[i] << (16 * (i & 1));
        return v;
    }
    // (a scale of zero past the last output and the last group)
    __device__ __forceinline__ uint16_t scale(int gr, bool there) const {
        if (WIDE)
            return __builtin_amdgcn_raw_buffer_load_b16(sbuf, there && n < p.n ? 2u * (uint32_t)n : kNowhere,
                                                        there ? 2 * gr * p.n : 0, kCached);
        return there && n < p.n ? p.scales[(int64_t)gr * p.n + n] : 0;
    }
    __device__ __forceinline__ uint8_t zero(int gr, bool there) const {
        if (p.zeros == nullptr) return 8;
        if (WIDE)
            return __builtin_amdgcn_raw_buffer_load_b8(zbuf, there && n < p.n ? (uint32_t)n : kNowhere,
                                                       there ? gr * p.n : 0, kCached);
        return there && n < p.n ? p.zeros[(int64_t)gr * p.n + n] : 0;
    }
};

// MT tiles of 16 rows of x; STEPS matrix instructions (of 32 inputs) share a scale, and
// with ONE so many inputs are a whole group.
template <int MT, int STEPS, bool ONE, bool WIDE>
__global__ __launch_bounds__(kMaxW4Waves *kWave) void w4_matvec_kernel(const W4Params p) {
    constexpr int kScales = 4 / STEPS;
    extern __shared__ float joined[];  // [wave][MT][16 x 16]
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int ktiles = (p.k + kTileK - 1) / kTileK;
    // Blocks are dealt to the eight XCDs in turn; eight neighbouring tiles, whose scales
    // share cache lines, go to the same one.
    const int ntiles = (p.n + kTileN - 1) / kTileN, in64 = blockIdx.x & 63;
    const int nt = blockIdx.x - in64 + (in64 & 7) * 8 + (in64 >> 3), m0 = blockIdx.y * MT * 16;
    if (nt >= ntiles) return;
    const Operands<WIDE> in(p, nt * kTileN + r, g);

    f32x4_t total[MT];
    uint32_t row[MT];
#pragma unroll
    for (int b = 0; b < MT; ++b) {
        total[b] = f32x4_t{0, 0, 0, 0};
        const int m = m0 + 16 * b + r;
        row[b] = m < p.m ? 2u * ((uint32_t)m * (uint32_t)p.xs_m + 8u * (uint32_t)g) : kNowhere;
    }
    const u32x4 units = {kUnit * 0x10001u, kUnit * 0x10001u, kUnit * 0x10001u, kUnit * 0x10001u};
    const u32x4 *tiles = reinterpret_cast<const u32x4 *>(p.q) + (int64_t)nt * ktiles * kWave;

    for (int kt = wave; kt < ktiles; kt += waves) {
        const u32x4 q = tiles[(int64_t)kt * kWave + lane];
        uint16_t scale[kScales];
        uint8_t zero[kScales];
#pragma unroll
        for (int s = 0; s < kScales; ++s) {
            const int block = kt * kScales + s;
            const int gr = ONE ? block : __builtin_amdgcn_readfirstlane(block * (STEPS * 32) / p.group);
            scale[s] = in.scale(gr, block * (STEPS * 32) < p.k);
            zero[s] = in.zero(gr, block * (STEPS * 32) < p.k);
        }
        u32x4 x[MT][4];
#pragma unroll
        for (int b = 0; b < MT; ++b)
#pragma unroll
            for (int s = 0; s < 4; ++s) x[b][s] = in.x(row[b], m0 + 16 * b + r, kt * kTileK + 32 * s);
#pragma unroll
        for (int s = 0; s < kScales; ++s) {
            f32x4_t sum[MT], acc[MT];
#pragma unroll
            for (int b = 0; b < MT; ++b) sum[b] = acc[b] = f32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const u32x4 w = expand(q[s * STEPS + i]);
#pragma unroll
                for (int b = 0; b < MT; ++b) {
                    sum[b] = mfma(x[b][s * STEPS + i], units, sum[b]);
                    acc[b] = mfma(x[b][s * STEPS + i], w, acc[b]);
                }
            }
            const float sc = bf16_bits_to_f32(scale[s]), offset = -1.0f - (float)zero[s] * 0x1p-7f;
#pragma unroll
            for (int b = 0; b < MT; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    total[b][i] = __builtin_fmaf(sc, __builtin_fmaf(offset, sum[b][i], acc[b][i]), total[b][i]);
        }
    }

    // lane (r, g) holds output r, rows 4 g .. 4 g + 3 of each tile
#pragma unroll
    for (int b = 0; b < MT; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) joined[(wave * MT + b) * 256 + (4 * g + i) * 16 + r] = total[b][i];
    __syncthreads();
    for (int e = threadIdx.x; e < MT * 256; e += blockDim.x) {
        const int col = nt * kTileN + (e & 15), m = m0 + (e >> 4);
        if (col >= p.n || m >= p.m) continue;
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += joined[w * MT * 256 + e];
        v = __builtin_fmaf(v, kBack, p.bias != nullptr ? bf16_bits_to_f32(p.bias[col]) : 0.0f);
        p.out[(int64_t)m * p.os_m + col] = f32_to_bf16_bits(v);
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

// Waves of a block: as many as keep about this many on the card, with an input tile each
// (2048 and 8192 were slower on 14432 x 4096 and on 4096 x 6144).
constexpr int64_t kW4Waves = 4096;

template <int MT, int STEPS, bool ONE>
hipError_t launch_tiles(const W4Params &p, bool wide, hipStream_t stream) {
    const int64_t ktiles = (p.k + kTileK - 1) / kTileK;
    const int64_t blocks = (p.n + kTileN - 1) / kTileN, rows = (p.m + 16 * MT - 1) / (16 * MT);
    int waves = 4;
    while (waves < kMaxW4Waves && blocks * rows * waves < kW4Waves) waves *= 2;
    while (waves > 1 && waves > ktiles) waves /= 2;
    if (rows > 65535) return hipErrorInvalidConfiguration;
    const size_t lds = (size_t)waves * MT * 256 * 4;
    const dim3 grid((unsigned)((blocks + 63) / 64 * 64), (unsigned)rows);
    if (wide)
        w4_matvec_kernel<MT, STEPS, ONE, true><<<grid, waves * kWave, lds, stream>>>(p);
    else
        w4_matvec_kernel<MT, STEPS, ONE, false><<<grid, waves * kWave, lds, stream>>>(p);
    return hipGetLastError();
}

template <int STEPS, bool ONE>
hipError_t launch_steps(const W4Params &p, bool wide, hipStream_t stream) {
    if (p.m <= 16) return launch_tiles<1, STEPS, ONE>(p, wide, stream);
    if (p.m <= 32) return launch_tiles<2, STEPS, ONE>(p, wide, stream);
    return launch_tiles<4, STEPS, ONE>(p, wide, stream);
}

}  // namespace

hipError_t launch_w4_matvec(const W4Params &p, hipStream_t stream, const char **kernel_name) {
    // 16-byte rows, and offsets of 32 bits
    const int64_t groups = (p.k + p.group - 1) / p.group, most = (int64_t)1 << 31;
    const bool wide = p.k % 8 == 0 && p.xs_m % 8 == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
                      p.xs_m < most / 2 && 2 * ((p.m - 1) * p.xs_m + p.k) < most && 2 * groups * p.n < most;
    *kernel_name = wide ? "w4_matvec" : "w4_matvec_scalar";
    switch (p.group) {
        case 128: return launch_steps<4, true>(p, wide, stream);
        case 64: return launch_steps<2, true>(p, wide, stream);
        case 32: return launch_steps<1, true>(p, wide, stream);
    }
    if (p.group % 128 == 0) return launch_steps<4, false>(p, wide, stream);
    return launch_steps<1, false>(p, wide, stream);
}

hipError_t launch_w4_pack(const uint8_t *codes, int64_t n, int64_t k, uint8_t *q, hipStream_t stream) {
    const int64_t ktiles = (k + kTileK - 1) / kTileK;
    const int64_t bytes = (n + kTileN - 1) / kTileN * ktiles * 1024, units = (bytes + 255) / 256;
    w4_pack_kernel<<<dim3((unsigned)(units < kMaxBlocks ? units : kMaxBlocks)), 256, 0, stream>>>(codes, n, k, ktiles,
                                                                                                bytes, q);
    return hipGetLastError();
}

}  // namespace dcconv
