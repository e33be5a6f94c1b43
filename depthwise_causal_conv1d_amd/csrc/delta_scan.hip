// The gated delta rule over whole sequences for gfx950.
//
// Per head, with g_t = softplus(dt_t + dt_bias) a, b_t = sigmoid(beta_t), and the head's
// group holding q and k (of length one if asked for):
//
//     S_t = e^{g_t} S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,   out_t = scale S_t q_t
//
// Chunks of C = 64 tokens (32 where keys are longer than 128) turn this into matrix
// products.  With c_t the prefix sum of g_t inside the chunk, S the state ahead of it and
// u_t the correction that token t adds along its key,
//
//     (I + A) u = b (v - e^c S k),    A_tu = b_t e^{c_t - c_u} k_t.k_u for u < t
//     U   = T R,   T = (I + A)^-1 diag(b),   R_t = v_t - e^{c_t} S k_t
//     out = scale (e^{c_t} S q_t + sum_{u <= t} e^{c_t - c_u} q_t.k_u U_u)
//     S'  = e^{c_C} S + sum_u e^{c_C - c_u} U_u k_u^T
//
// T and P = e^{c_t - c_u} q_t.k_u do not depend on the state: a block's second four waves
// prepare them for the next chunk while its first four, which hold the state, run the
// chain S -> R -> U -> S'.
//
// The first four waves: each owns 16 or 32 rows p of a head's state and all of its k,
// in FP32 accumulators for the whole sequence, already in the lane order in which the next
// products read it (below).  The second four: the triangular inverse in blocks of 16, whose
// diagonal blocks come by substitution, one column a lane, and whose other blocks by FP32
// matrix instructions (a series in A would need terms that grow like binomials where keys
// repeat; substitution does not).
//
// Three barriers a chunk.  While the first four waves form R (1), U (2) and then the outputs
// and S' (3) of chunk j, the second put chunk j + 1's q and k into LDS, request chunk j + 2's
// and join T of chunk j (1); form A of chunk j + 1 and P of chunk j (2); and invert A's
// diagonal blocks (3).
//
// Layouts.  v_mfma_f32_16x16x32_bf16 takes, in lane l with r = l & 15 and g = l >> 4, row
// (column) r of an operand at inner indices 8 g .. 8 g + 7, and leaves column r, rows
// 4 g .. 4 g + 3 of the result.  The order of an operand's rows is free, and so is the inner
// indices' if both operands agree: so a result's tiles 2 m and 2 m + 1 are together an
// operand as they are, against rows in LDS whose inner order is 4 g .. of the first and of
// the second 16 of 32 (T and P are written so, and the transposing loads of k read so), or,
// for the state, whose columns interleave by four (tile 2 m + f, row 4 g + i is column 32 m +
// 8 g + 4 f + i), against rows of k and q as they are.
//
// Precision.  q, k and v are BF16 as given: a key's length enters as an FP32 factor.  Sums,
// states, A and its inverse are FP32, prefix sums 64 bits and their differences 48.  An
// operand that is no BF16 value is split into PARTS BF16 values, whose products are added
// up: with an F32 state, S, R, T and U are (PARTS = 3: all 24 bits); with a BF16 state S, R and
// the U that enters the state are rounded, T has two parts.  P, and the copy of the state that q reads, are
// rounded to BF16, and the U that P multiplies has two parts, in every case: what is left is about the
// output's own rounding.
//
// What is not finite.  An infinity or NaN of a later token must not meet the zeros above T's
// and P's diagonals.  A key, decay or weight that is not finite leaves A's entries out and
// makes R's factor NaN from there on; a channel of R or U with a value that is not finite is
// cut at its first such token: U is zero from there, and those outputs and the channel's
// state become NaN.
#include <type_traits>

#include "delta_common.h"

namespace dcconv {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kHalf = 4;                      // waves of each kind
constexpr int kHalfBlock = kHalf * kWave;
constexpr int kScanBlock = 2 * kHalfBlock;
constexpr int kAPitch = 20;                   // floats of a row of a 16 x 16 tile of A
constexpr float kNone = -65536.0f;            // log2 of a decay that counts as this: zero
constexpr uint32_t kNowhere = 0x80000000u;    // past the end of every buffer

// Per token of a chunk: the prefix sum of log2 decays in two floats, the weight, the factors
// of k and q; and from them what scales S k, S q and U.
enum { kSumHigh, kSumLow, kWeight, kUnitK, kUnitQ, kForK, kForQ, kForU, kTokenRows };

struct ScanPlan {
    int32_t tiles;  // blocks of a head
    int32_t each;   // blocks of a group
    bool runs;      // a group's blocks follow each other on one XCD
};

__device__ __forceinline__ f32x4_t mfma(u32x4 a, u32x4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
// The product of two 16 x 16 tiles in FP32: lane (r, g) gives a[r][4 g + s] and b[4 g + s][r].
__device__ __forceinline__ f32x4_t mfma_f32(f32x4_t a, f32x4_t b, f32x4_t c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ u32x4 lds16(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }
__device__ __forceinline__ f32x4_t lds4f(const float *p) { return *reinterpret_cast<const f32x4_t *>(p); }

// An operand whose inner index runs over rows in LDS: lane 4 q + j of the 16 that
// share g gives the address of its columns' piece j (four of them) in row 4 g + q, and
// gets column 4 q + j of rows 4 g .. 4 g + 3, and of the 16 rows further down.
__device__ __forceinline__ u32x4 load_columns(const uint16_t *at, int pitch) {
    typedef __attribute__((address_space(3))) s16x4_t *Lds;
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(s16x4_t *)at));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(s16x4_t *)(at + 16 * pitch)));
    return u32x4{a[0], a[1], b[0], b[1]};
}

__device__ __forceinline__ bool is_finite(float v) { return __builtin_fabsf(v) < __builtin_inff(); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Two result tiles as an operand of N parts: a BF16 value, and what each leaves.
template <int N>
__device__ __forceinline__ void split(f32x4_t a, f32x4_t b, u32x4 (&part)[N]) {
    float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            part[n][i] = h;
            if (n + 1 < N) {
                v[2 * i] -= lo_f32(h);
                v[2 * i + 1] -= hi_f32(h);
            }
        }
}

// The sum over the first lanes up to this one, in 64 bits.
template <int CTRL>
__device__ __forceinline__ double dpp_shift(double v) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    const u32x2 s = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, 0xf, 0xf, true),
                     (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, 0xf, 0xf, true)};
    return __builtin_bit_cast(double, s);
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    const u32x2 s = {(uint32_t)__builtin_amdgcn_readlane((int)w[0], lane),
                     (uint32_t)__builtin_amdgcn_readlane((int)w[1], lane)};
    return __builtin_bit_cast(double, s);
}
__device__ __forceinline__ double prefix_sum(double v, int lane) {
    v += dpp_shift<0x111>(v);
    v += dpp_shift<0x112>(v);
    v += dpp_shift<0x114>(v);
    v += dpp_shift<0x118>(v);
    const double r0 = lane_value(v, 15), r1 = lane_value(v, 31), r2 = lane_value(v, 47);
    return v + (lane >= 48 ? r0 + r1 + r2 : lane >= 32 ? r0 + r1 : lane >= 16 ? r0 : 0.0);
}

// The sum over 8, 16 or 32 neighbouring lanes, in all of them.
template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
    for (int s = 1; s < LANES; s *= 2) v += __shfl_xor(v, s);
    return v;
}

// One operand's rows of a chunk: a lane moves eight values from column col, of which
// `count` exist.  WIDE reads them at once (16 bytes) through a buffer that ends with the
// chunk's last row, so that what lies behind it reads as zeros.
template <bool WIDE>
struct Rows {
    const uint16_t *base;  // wave-uniform: the sequence's first row
    int64_t stride;
    int32_t row0, step, col, count, width;
    __device__ __forceinline__ Rows(const uint16_t *first, int64_t stride, int width, int row0, int step, int col)
        : base(first), stride(stride), row0(row0), step(step), col(col), count(width - col), width(width) {}
    // rows row0 + q * step of the chunk at token t0; n: the sequence's rows from there
    template <int N>
    __device__ __forceinline__ void load(u32x4 (&w)[N], int64_t t0, int n) const {
        const uint16_t *from = base + t0 * stride;
        if (WIDE) {
            const uint32_t pitch = 2u * (uint32_t)stride;
            n = min(n, N * step);  // the chunk's rows
            const Buffer buf = make_buffer(from, n > 0 ? (uint32_t)(n - 1) * pitch + 2u * (uint32_t)width : 0u);
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const int row = row0 + q * step;
                w[q] = buffer_load<kCached>(buf, row < n && count > 0 ? (uint32_t)row * pitch + 2u * (uint32_t)col : kNowhere);
            }
            return;
        }
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int row = row0 + q * step;
            w[q] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (row < n && i < count) w[q][i >> 1] |= (uint32_t)from[row * stride + col + i] << (16 * (i & 1));
        }
    }
};

// Four consecutive state values at element `at`, of which `count` exist.
__device__ __forceinline__ f32x4_t load_state4(const void *s, bool f32, bool wide, int64_t at, int count) {
    f32x4_t v = {0, 0, 0, 0};
    if (wide && count >= 4) {
        if (f32) return *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(s) + at);
        const u32x2 w = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(s) + at);
        return f32x4_t{lo_f32(w[0]), hi_f32(w[0]), lo_f32(w[1]), hi_f32(w[1])};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < count) v[i] = load_either(s, f32, at + i);
    return v;
}
__device__ __forceinline__ void store_state4(void *s, bool f32, bool wide, int64_t at, int count, f32x4_t v) {
    if (wide && count >= 4) {
        if (f32)
            *reinterpret_cast<f32x4_t *>(static_cast<float *>(s) + at) = v;
        else
            *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(s) + at) =
                u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < count) {
            if (f32)
                static_cast<float *>(s)[at + i] = v[i];
            else
                static_cast<uint16_t *>(s)[at + i] = f32_to_bf16_bits(v[i]);
        }
}

// The state column of row 4 g of the state's tile m.
__device__ __forceinline__ int column(int m, int g) { return 32 * (m >> 1) + 8 * g + 4 * (m & 1); }

// Reports a sequence table that is not 0 = starts[0] <= ... <= starts[n] = t.
__device__ __forceinline__ void check_table(const DeltaParams &p) {
    if (p.starts == nullptr || p.status == nullptr) return;
    bool bad = false;
    for (int i = threadIdx.x; i <= p.n; i += kScanBlock) {
        const int a = p.starts[i];
        bad |= a < 0 || a > p.t || (i == 0 && a != 0) || (i == p.n ? a != p.t : p.starts[i + 1] < a);
    }
    if (bad) atomicOr(p.status, DCCONV_DEV_BAD_SEQ);
}

// Sizes of a variant and its places in LDS (in bytes).  KS: keys' size, rounded up; C: tokens
// of a chunk; NT: tiles of 16 state rows a wave owns; PARTS: see above.
template <int KS, int C, int NT, int PARTS>
struct Sizes {
    static constexpr int kKeyPitch = KS + 16;  // of 16-bit values: 32 bytes more than a multiple of 64
    static constexpr int kRowsP = kHalf * 16 * NT;  // state rows of a block
    static constexpr int kVPitch = kRowsP + 8;
    static constexpr int kTPitch = C + 16;
    static constexpr int kTParts = PARTS == 1 ? 2 : PARTS;
    static constexpr int kBlocks = C / 16, kTiles = kBlocks * (kBlocks + 1) / 2;
    static constexpr int kKey = 0;                                   // [2][C][kKeyPitch]
    static constexpr int kQuery = kKey + 2 * C * kKeyPitch * 2;      // [2][C][kKeyPitch]
    static constexpr int kV = kQuery + 2 * C * kKeyPitch * 2;        // [C][kVPitch]
    static constexpr int kT = kV + C * kVPitch * 2;                  // [kTParts][C][kTPitch]
    static constexpr int kP = kT + kTParts * C * kTPitch * 2;        // [C][kTPitch]
    static constexpr int kA = kP + C * kTPitch * 2;                  // [kTiles][16][kAPitch] floats
    static constexpr int kToken = kA + kTiles * 16 * kAPitch * 4;    // [2][kTokenRows][C] floats
    static constexpr int kBytes = kToken + 2 * kTokenRows * C * 4;
    static_assert(kBytes <= 160 * 1024, "more LDS than a CU has");
};

template <int KS, int C, int NT, int PARTS, bool WIDE>
__global__ __launch_bounds__(kScanBlock, 2) void delta_scan_kernel(const DeltaParams p, const ScanPlan plan) {
    using Z = Sizes<KS, C, NT, PARTS>;
    constexpr int kB = Z::kBlocks, KP = Z::kKeyPitch, VP = Z::kVPitch, TP = Z::kTPitch, kSteps = KS / 32;
    constexpr int kTParts = Z::kTParts;
    extern __shared__ u32x4 smem[];
    char *lds = reinterpret_cast<char *>(smem);
    uint16_t *sk = reinterpret_cast<uint16_t *>(lds + Z::kKey), *sq = reinterpret_cast<uint16_t *>(lds + Z::kQuery);
    uint16_t *sv = reinterpret_cast<uint16_t *>(lds + Z::kV), *st = reinterpret_cast<uint16_t *>(lds + Z::kT);
    uint16_t *sp = reinterpret_cast<uint16_t *>(lds + Z::kP);
    float *sa = reinterpret_cast<float *>(lds + Z::kA), *tokens = reinterpret_cast<float *>(lds + Z::kToken);

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = uniform(tid >> 6);
    if (blockIdx.x == 0 && blockIdx.y == 0) check_table(p);

    // ---- this block's sequence, head and rows.  Blocks are dealt to the eight XCDs in turn:
    // a group's blocks, which read the same q and k, go to one of them.
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    int64_t ug;
    int member;
    if (plan.runs) {
        const int64_t turn = (block >> 3) / plan.each;
        ug = turn * 8 + (block & 7);
        member = uniform((int)((block >> 3) - turn * plan.each));
    } else {
        ug = block / plan.each;
        member = uniform((int)(block - ug * plan.each));
    }
    if (ug >= (int64_t)p.n * p.g) return;
    const int seq = uniform((int)(ug / p.g)), group = uniform((int)(ug - (int64_t)seq * p.g));
    const int which = uniform(member / plan.tiles);
    const int head = group * uniform(p.h / p.g) + which, p0 = (member - which * plan.tiles) * Z::kRowsP;
    int first = 0, len = p.t;
    if (p.starts != nullptr) {
        const int a = load_uniform(p.starts, seq), e = load_uniform(p.starts, seq + 1);
        if (a < 0 || a > e || e > p.t) return;
        first = a;
        len = e - a;
    }
    const int rows = min(Z::kRowsP, p.p - p0);  // of this block
    const int slot = uniform(route_row(p.idx, p.status, p.n, p.s, seq, lane));
    uint16_t *out = p.out + seq * p.os_n + (int64_t)first * p.os_t + head * p.os_h + p0;
    if (slot < 0) {  // a padding sequence: zeros, and no state moves
        for (int t = wave; t < len; t += 2 * kHalf)
            for (int c = lane; c < rows; c += kWave) out[t * p.os_t + c] = 0;
        return;
    }
    const int chunks = (len + C - 1) / C;

    // the tiles of T and P above the diagonal that products over 32 tokens read: zeros for good
    for (int i = tid; i < (kTParts + 1) * (kB / 2) * 16 * 4; i += kScanBlock) {
        const int piece = i & 3, row = (i >> 2) & 15, m = (i >> 6) % (kB / 2), part = (i >> 6) / (kB / 2);
        uint16_t *to = (part < kTParts ? st + part * C * TP : sp) + (32 * m + row) * TP + 32 * m + 8 * piece + 4;
        *reinterpret_cast<u32x2 *>(to) = u32x2{0, 0};
    }

    if (wave >= kHalf) {
        // ================================================== the waves that prepare T and P
        const int ptid = tid - kHalfBlock, pw = wave - kHalf;
        constexpr int kAcross = KS / 8, kRowsPer = kHalfBlock / kAcross, kMoves = C / kRowsPer;
        const int row0 = ptid / kAcross, col = ptid % kAcross * 8;
        const Rows<WIDE> rk(p.key + seq * p.ks_n + (int64_t)first * p.ks_t + group * p.ks_g, p.ks_t, p.k, row0, kRowsPer, col);
        const Rows<WIDE> rq(p.q + seq * p.qs_n + (int64_t)first * p.qs_t + group * p.qs_g, p.qs_t, p.k, row0, kRowsPer, col);
        u32x4 nk[kMoves], nq[kMoves];
        auto fetch = [&](int j) {
            rk.load(nk, (int64_t)j * C, len - j * C);
            rq.load(nq, (int64_t)j * C, len - j * C);
        };
        // q and k of chunk j into LDS, with the factors that make their rows of length one
        auto stage = [&](int j) {
            uint16_t *tk = sk + (j & 1) * C * KP, *tq = sq + (j & 1) * C * KP;
            float *tok = tokens + (j & 1) * kTokenRows * C;
#pragma unroll
            for (int q = 0; q < kMoves; ++q) {
                const int row = row0 + q * kRowsPer;
                *reinterpret_cast<u32x4 *>(tk + row * KP + col) = nk[q];
                *reinterpret_cast<u32x4 *>(tq + row * KP + col) = nq[q];
                float k2 = 0.0f, q2 = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    k2 = __builtin_fmaf(lo_f32(nk[q][i]), lo_f32(nk[q][i]), k2);
                    k2 = __builtin_fmaf(hi_f32(nk[q][i]), hi_f32(nk[q][i]), k2);
                    q2 = __builtin_fmaf(lo_f32(nq[q][i]), lo_f32(nq[q][i]), q2);
                    q2 = __builtin_fmaf(hi_f32(nq[q][i]), hi_f32(nq[q][i]), q2);
                }
                k2 = sum_lanes<kAcross>(k2);
                q2 = sum_lanes<kAcross>(q2);
                if (col == 0) {
                    tok[kUnitK * C + row] = is_finite(k2) ? unit_factor(p, k2) : __builtin_nanf("");
                    tok[kUnitQ * C + row] = p.scale * unit_factor(p, q2);
                }
            }
        };
        // ---- decays and weights of a chunk's tokens, a lane each (as they are in memory:
        // converting them here would wait for them)
        const float rate = p.a[head] * kLog2e, bias = p.dt_bias != nullptr ? p.dt_bias[head] : 0.0f;
        const int64_t dt0 = seq * p.ds_n + (int64_t)first * p.ds_t + head, beta0 = seq * p.es_n + (int64_t)first * p.es_t + head;
        uint32_t dt_raw = 0, beta_raw = 0;
        auto fetch_gates = [&](int j) {
            const int64_t t = (int64_t)j * C + lane;
            dt_raw = beta_raw = 0;
            if (lane < C && t < len) {
                dt_raw = p.dt_f32 ? static_cast<const uint32_t *>(p.dt)[dt0 + t * p.ds_t]
                                  : (uint32_t)static_cast<const uint16_t *>(p.dt)[dt0 + t * p.ds_t] << 16;
                beta_raw = p.beta_f32 ? static_cast<const uint32_t *>(p.beta)[beta0 + t * p.es_t]
                                      : (uint32_t)static_cast<const uint16_t *>(p.beta)[beta0 + t * p.es_t] << 16;
            }
        };
        auto put_gates = [&](int j) {
            float d = __uint_as_float(dt_raw) + bias;
            if (p.dt_softplus) d = softplus(d);
            float decay = d * rate, weight = weight_of(p, __uint_as_float(beta_raw));
            if (lane >= C || j * C + lane >= len) decay = weight = 0.0f;
            if (decay < kNone) decay = kNone;
            if (!is_finite(weight)) decay = __builtin_nanf(""), weight = 0.0f;
            const double c = prefix_sum((double)decay, lane);
            const float high = (float)c;
            float *tok = tokens + (j & 1) * kTokenRows * C + lane;
            if (lane < C) {
                tok[kSumHigh * C] = high;
                tok[kSumLow * C] = (float)(c - (double)high);
                tok[kWeight * C] = weight;
            }
        };
        // what the state's waves scale their products by
        auto put_scales = [&](int j) {
            if (lane >= C) return;
            float *tok = tokens + (j & 1) * kTokenRows * C;
            const float high = tok[kSumHigh * C + lane], low = tok[kSumLow * C + lane];
            const float e = __builtin_amdgcn_exp2f(high + low);
            const float behind =
                __builtin_amdgcn_exp2f((tok[kSumHigh * C + C - 1] - high) + (tok[kSumLow * C + C - 1] - low));
            const float unit = tok[kUnitK * C + lane];
            tok[kForK * C + lane] = e * unit;
            tok[kForQ * C + lane] = e * tok[kUnitQ * C + lane];
            tok[kForU * C + lane] = behind * unit;
        };
        // ---- tiles of A of chunk j + 1 (transposed: row u, column t) and of P of chunk j
        auto grams = [&](int ja, bool with_a, bool with_p) {
            for (int it = with_a ? pw : Z::kTiles + pw; it < (with_p ? 2 : 1) * Z::kTiles; it += kHalf) {
                const bool is_p = it >= Z::kTiles;
                const int e = is_p ? it - Z::kTiles : it;
                const int bt = e >= 6 ? 3 : e >= 3 ? 2 : e >= 1 ? 1 : 0, bu = e - bt * (bt + 1) / 2;
                const int j = is_p ? ja - 1 : ja;
                const uint16_t *km = sk + (j & 1) * C * KP, *tm = is_p ? sq + (j & 1) * C * KP : km;
                const float *tok = tokens + (j & 1) * kTokenRows * C;
                f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
                for (int m = 0; m < kSteps; ++m) {
                    const u32x4 u = lds16(km + (16 * bu + r) * KP + 32 * m + 8 * g);
                    const u32x4 t = lds16(tm + (16 * bt + r) * KP + 32 * m + 8 * g);
                    acc = is_p ? mfma(u, t, acc) : mfma(t, u, acc);
                }
                float v[4];
                if (is_p) {  // lane: column t = r, rows u
                    const int t = 16 * bt + r, u0 = 16 * bu + 4 * g;
                    const f32x4_t uh = lds4f(tok + kSumHigh * C + u0), ul = lds4f(tok + kSumLow * C + u0);
                    const f32x4_t uk = lds4f(tok + kUnitK * C + u0);
                    const float th = tok[kSumHigh * C + t], tl = tok[kSumLow * C + t], tq = tok[kUnitQ * C + t];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = u0 + i <= t ? acc[i] * tq * uk[i] * __builtin_amdgcn_exp2f((th - uh[i]) + (tl - ul[i])) : 0.0f;
                    *reinterpret_cast<u32x2 *>(sp + t * TP + 32 * (bu >> 1) + 8 * g + 4 * (bu & 1)) =
                        u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                } else {  // lane: column u = r, rows t
                    const int u = 16 * bu + r, t0 = 16 * bt + 4 * g;
                    const f32x4_t th = lds4f(tok + kSumHigh * C + t0), tl = lds4f(tok + kSumLow * C + t0);
                    const f32x4_t tk = lds4f(tok + kUnitK * C + t0), tb = lds4f(tok + kWeight * C + t0);
                    const float uh = tok[kSumHigh * C + u], ul = tok[kSumLow * C + u], uk = tok[kUnitK * C + u];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = acc[i] * (tk[i] * tb[i]) * uk * __builtin_amdgcn_exp2f((th[i] - uh) + (tl[i] - ul));
                        if (!(u < t0 + i && is_finite(v[i]))) v[i] = 0.0f;
                    }
                    *reinterpret_cast<f32x4_t *>(sa + (e * 16 + r) * kAPitch + 4 * g) = f32x4_t{v[0], v[1], v[2], v[3]};
                }
            }
        };
        // ---- the inverses of I + A's diagonal blocks, a column a lane, in place (transposed)
        auto invert = [&]() {
            const int blk = g;
            if (blk >= kB) return;
            float *tile = sa + (blk * (blk + 1) / 2 + blk) * 16 * kAPitch;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = i == r ? 1.0f : 0.0f;
#pragma unroll
            for (int u = 0; u < 15; ++u) {
#pragma unroll
                for (int q = (u + 1) / 4; q < 4; ++q) {
                    const f32x4_t a = lds4f(tile + u * kAPitch + 4 * q);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * q + i > u) x[4 * q + i] = __builtin_fmaf(-a[i], x[u], x[4 * q + i]);
                }
            }
            wave_lds_sync();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4_t *>(tile + r * kAPitch + 4 * q) = f32x4_t{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
        };
        // ---- block row I of T: T_ij = -(sum_{j < k <= i} T_ik A_kj) T_jj, transposed throughout
        auto join = [&](auto row_constant, int j) {
            constexpr int I = decltype(row_constant)::value;
            const float *weight = tokens + ((j & 1) * kTokenRows + kWeight) * C;
            f32x4_t y[I + 1];
            const float *diag = sa + (I * (I + 1) / 2 + I) * 16 * kAPitch;
#pragma unroll
            for (int s = 0; s < 4; ++s) y[I][s] = diag[(4 * g + s) * kAPitch + r];
#pragma unroll
            for (int b = I - 1; b >= 0; --b) {
                f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
                for (int k = I; k > b; --k)
                    acc = mfma_f32(lds4f(sa + ((k * (k + 1) / 2 + b) * 16 + r) * kAPitch + 4 * g), y[k], acc);
                const f32x4_t zero = {0, 0, 0, 0};
                y[b] = -mfma_f32(lds4f(sa + ((b * (b + 1) / 2 + b) * 16 + r) * kAPitch + 4 * g), acc, zero);
            }
#pragma unroll
            for (int b = 0; b <= I; ++b) {
                const f32x4_t w = lds4f(weight + 16 * b + 4 * g);
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = y[b][i] * w[i];
#pragma unroll
                for (int part = 0; part < kTParts; ++part) {
                    const uint32_t h0 = pack_bf16x2(v[0], v[1]), h1 = pack_bf16x2(v[2], v[3]);
                    *reinterpret_cast<u32x2 *>(st + part * C * TP + (16 * I + r) * TP + 32 * (b >> 1) + 8 * g + 4 * (b & 1)) =
                        u32x2{h0, h1};
                    v[0] -= lo_f32(h0), v[1] -= hi_f32(h0), v[2] -= lo_f32(h1), v[3] -= hi_f32(h1);
                }
            }
        };

        fetch(0);
        if (pw == 0) fetch_gates(0);
        stage(0);
        if (pw == 0) put_gates(0);
        fetch(1);
        if (pw == 0) fetch_gates(1);
        __syncthreads();
        grams(0, true, false);
        __syncthreads();
        if (pw == 0) invert();
        if (pw == 1) put_scales(0);
        __syncthreads();
        for (int j = 0; j < chunks; ++j) {
            const bool more = j + 1 < chunks;
            if (more) {
                stage(j + 1);
                if (pw == 0) put_gates(j + 1);
                fetch(j + 2);
                if (pw == 0) fetch_gates(j + 2);
            }
            if (pw == 0) join(std::integral_constant<int, 0>{}, j);
            if (pw == 1) join(std::integral_constant<int, 1>{}, j);
            if constexpr (kB > 2) {
                if (pw == 2) join(std::integral_constant<int, 2>{}, j);
                if (pw == 3) join(std::integral_constant<int, 3>{}, j);
            }
            __syncthreads();
            grams(j + 1, more, true);
            __syncthreads();
            if (more) {
                if (pw == 0) invert();
                if (pw == 1) put_scales(j + 1);
            }
            __syncthreads();
        }
        return;
    }

    // ====================================================== the waves that hold the state
    constexpr int kAcross = Z::kRowsP / 8, kRowsPer = kHalfBlock / kAcross, kMoves = C / kRowsPer;
    const int vrow = tid / kAcross, vcol = tid % kAcross * 8;
    const Rows<WIDE> rv(p.v + seq * p.vs_n + (int64_t)first * p.vs_t + head * p.vs_h + p0, p.vs_t, rows, vrow, kRowsPer, vcol);
    u32x4 nv[kMoves];
    auto fetch_v = [&](int j) { rv.load(nv, (int64_t)j * C, len - j * C); };
    auto stage_v = [&]() {
#pragma unroll
        for (int q = 0; q < kMoves; ++q) *reinterpret_cast<u32x4 *>(sv + (vrow + q * kRowsPer) * VP + vcol) = nv[q];
    };
    // Tile n's column r is row own(n, r) of the wave's, so that result rows 4 g .. of the
    // two tiles are eight neighbours.
    const int mine = wave * 16 * NT, left_rows = rows - mine;  // this wave's rows start at p0 + mine
    const auto own = [&](int n, int c) { return NT == 2 ? 8 * (c >> 2) + 4 * n + (c & 3) : c; };
    const bool busy = left_rows > 0;

    // ---- the state ahead: tile m, rows k = column(m, g) + i, columns p = own(n, r)
    f32x4_t hs[KS / 16][NT];
#pragma unroll
    for (int m = 0; m < KS / 16; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) hs[m][n] = f32x4_t{0, 0, 0, 0};
    const bool wide_state = p.k % 4 == 0 && p.ss_s % 4 == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0;
    const int64_t state_at = slot * p.ss_s + ((int64_t)head * p.p + p0 + mine) * p.k;
    if (p.state != nullptr && p.has_init != nullptr && p.has_init[seq] != 0)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (own(n, r) < left_rows)
#pragma unroll
                for (int m = 0; m < KS / 16; ++m)
                    hs[m][n] = load_state4(p.state, p.state_f32, wide_state,
                                           state_at + (int64_t)own(n, r) * p.k + column(m, g), p.k - column(m, g));

    fetch_v(0);
    stage_v();
    fetch_v(1);
    __syncthreads();
    __syncthreads();
    __syncthreads();
    for (int j = 0; j < chunks; ++j) {
        const uint16_t *km = sk + (j & 1) * C * KP, *qm = sq + (j & 1) * C * KP;
        const float *tok = tokens + (j & 1) * kTokenRows * C;
        int cut[NT];  // the first token whose R or U is not finite
#pragma unroll
        for (int n = 0; n < NT; ++n) cut[n] = C;
        f32x4_t d[kB][NT], o[kB][NT];
        // Zeros for the tokens of d from the first on that is not finite.
        auto cut_off = [&]() {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int tt = kB - 1; tt >= 0; --tt)
#pragma unroll
                    for (int i = 3; i >= 0; --i)
                        if (!is_finite(d[tt][n][i])) cut[n] = min(cut[n], 16 * tt + 4 * g + i);
                cut[n] = min(cut[n], __shfl_xor(cut[n], 16));
                cut[n] = min(cut[n], __shfl_xor(cut[n], 32));
#pragma unroll
                for (int tt = 0; tt < kB; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (16 * tt + 4 * g + i >= cut[n]) d[tt][n][i] = 0.0f;
            }
        };
        auto not_finite = [&]() {
            float probe = 0.0f;
#pragma unroll
            for (int tt = 0; tt < kB; ++tt)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) probe = __builtin_fmaf(d[tt][n][i], 0.0f, probe);
            return __any(probe != 0.0f);
        };
        bool bad = false;
        u32x4 rp[kB / 2][NT][PARTS];
        // ---- d = S k (columns p, rows t), o = S q (columns t, rows p), then d = R
        if (busy) {
#pragma unroll
            for (int tt = 0; tt < kB; ++tt)
#pragma unroll
                for (int n = 0; n < NT; ++n) d[tt][n] = o[tt][n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < kSteps; ++m) {
                u32x4 kf[kB], qf[kB];
#pragma unroll
                for (int tt = 0; tt < kB; ++tt) {
                    kf[tt] = lds16(km + (16 * tt + r) * KP + 32 * m + 8 * g);
                    qf[tt] = lds16(qm + (16 * tt + r) * KP + 32 * m + 8 * g);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    u32x4 hp[PARTS];
                    split<PARTS>(hs[2 * m][n], hs[2 * m + 1][n], hp);
#pragma unroll
                    for (int tt = 0; tt < kB; ++tt) {
#pragma unroll
                        for (int part = PARTS - 1; part >= 0; --part) d[tt][n] = mfma(kf[tt], hp[part], d[tt][n]);
                        o[tt][n] = mfma(hp[0], qf[tt], o[tt][n]);
                    }
                }
            }
            const uint16_t *va = sv + (4 * g + (r >> 2)) * VP + mine + (NT == 2 ? 8 : 4) * (r & 3);
#pragma unroll
            for (int m = 0; m < kB / 2; ++m) {
                const f32x4_t w0 = lds4f(tok + kForK * C + 32 * m + 4 * g), w1 = lds4f(tok + kForK * C + 32 * m + 16 + 4 * g);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const u32x4 v = load_columns(va + 32 * m * VP + 4 * n, VP);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[2 * m][n][i] = ((i & 1) ? hi_f32(v[i >> 1]) : lo_f32(v[i >> 1])) - w0[i] * d[2 * m][n][i];
                        d[2 * m + 1][n][i] = ((i & 1) ? hi_f32(v[2 + (i >> 1)]) : lo_f32(v[2 + (i >> 1)])) - w1[i] * d[2 * m + 1][n][i];
                    }
                }
            }
            if (not_finite()) {
                bad = true;
                cut_off();
            }
#pragma unroll
            for (int m = 0; m < kB / 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) split<PARTS>(d[2 * m][n], d[2 * m + 1][n], rp[m][n]);
        }
        __syncthreads();
        // ---- d = U = T R
        if (busy) {
#pragma unroll
            for (int tt = 0; tt < kB; ++tt) {
#pragma unroll
                for (int n = 0; n < NT; ++n) d[tt][n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int m = 0; m <= tt / 2; ++m)
#pragma unroll
                    for (int a = kTParts - 1; a >= 0; --a) {
                        const u32x4 tf = lds16(st + a * C * TP + (16 * tt + r) * TP + 32 * m + 8 * g);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int b = PARTS - 1; b >= 0; --b)
                                if (a + b < kTParts) d[tt][n] = mfma(tf, rp[m][n][b], d[tt][n]);
                    }
            }
            if (not_finite()) {
                bad = true;
                cut_off();
            } else if (bad) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int tt = 0; tt < kB; ++tt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (16 * tt + 4 * g + i >= cut[n]) d[tt][n][i] = 0.0f;
            }
        }
        if (j + 1 < chunks) {
            stage_v();
            fetch_v(j + 2);
        }
        __syncthreads();
        // ---- the outputs, and the state behind the chunk
        if (busy) {
            u32x4 up[kB / 2][NT][2];
#pragma unroll
            for (int m = 0; m < kB / 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) split<2>(d[2 * m][n], d[2 * m + 1][n], up[m][n]);
#pragma unroll
            for (int tt = 0; tt < kB; ++tt) {
                const float e = tok[kForQ * C + 16 * tt + r];
                u32x4 pf[kB / 2];
#pragma unroll
                for (int m = 0; m <= tt / 2; ++m) pf[m] = lds16(sp + (16 * tt + r) * TP + 32 * m + 8 * g);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[tt][n] *= e;
#pragma unroll
                    for (int m = 0; m <= tt / 2; ++m) {
                        o[tt][n] = mfma(up[m][n][1], pf[m], o[tt][n]);
                        o[tt][n] = mfma(up[m][n][0], pf[m], o[tt][n]);
                    }
                }
            }
            if (bad) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int from = __shfl(cut[n], 4 * g + i);
#pragma unroll
                        for (int tt = 0; tt < kB; ++tt)
                            if (16 * tt + r >= from) o[tt][n][i] = __builtin_nanf("");
                    }
            }
            const int left = len - j * C;
            uint16_t *to = out + (int64_t)j * C * p.os_t + mine + 4 * NT * g;
#pragma unroll
            for (int tt = 0; tt < kB; ++tt) {
                if (16 * tt + r >= left) continue;
                uint16_t *at = to + (int64_t)(16 * tt + r) * p.os_t;
                uint32_t w[2 * NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    w[2 * n] = pack_bf16x2(o[tt][n][0], o[tt][n][1]);
                    w[2 * n + 1] = pack_bf16x2(o[tt][n][2], o[tt][n][3]);
                }
                if (WIDE) {
                    if (4 * NT * g < left_rows) {
                        if constexpr (NT == 2)
                            *reinterpret_cast<u32x4 *>(at) = u32x4{w[0], w[1], w[2], w[3]};
                        else
                            *reinterpret_cast<u32x2 *>(at) = u32x2{w[0], w[1]};
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4 * NT; ++i)
                        if (4 * NT * g + i < left_rows) at[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                }
            }
            const float dec =
                __builtin_amdgcn_exp2f(tok[kSumHigh * C + C - 1] + tok[kSumLow * C + C - 1]);
            u32x4 wp[kB / 2][NT][PARTS];
#pragma unroll
            for (int m = 0; m < kB / 2; ++m) {
                const f32x4_t w0 = lds4f(tok + kForU * C + 32 * m + 4 * g), w1 = lds4f(tok + kForU * C + 32 * m + 16 + 4 * g);
#pragma unroll
                for (int n = 0; n < NT; ++n) split<PARTS>(d[2 * m][n] * w0, d[2 * m + 1][n] * w1, wp[m][n]);
            }
            const uint16_t *ka = km + (4 * g + (r >> 2)) * KP + 8 * (r & 3);
#pragma unroll
            for (int t = 0; t < KS / 16; ++t) {
                u32x4 kt[kB / 2];
#pragma unroll
                for (int m = 0; m < kB / 2; ++m) kt[m] = load_columns(ka + 32 * m * KP + 32 * (t >> 1) + 4 * (t & 1), KP);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    hs[t][n] *= dec;
#pragma unroll
                    for (int m = 0; m < kB / 2; ++m)
#pragma unroll
                        for (int part = PARTS - 1; part >= 0; --part) hs[t][n] = mfma(kt[m], wp[m][n][part], hs[t][n]);
                }
            }
            if (bad) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (cut[n] < C)
#pragma unroll
                        for (int t = 0; t < KS / 16; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) hs[t][n][i] = __builtin_nanf("");
            }
        }
        __syncthreads();
    }

    // ---- the state behind the sequence
    if (p.state == nullptr) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
        if (own(n, r) < left_rows)
#pragma unroll
            for (int m = 0; m < KS / 16; ++m)
                store_state4(p.state, p.state_f32, wide_state, state_at + (int64_t)own(n, r) * p.k + column(m, g),
                             p.k - column(m, g), hs[m][n]);
}

// Lets a kernel use a CU's whole LDS; once for each device, whose bit of *done is
// then set.
hipError_t allow_lds(const void *kernel, uint64_t *done) {
    int dev = 0;
    const hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (__atomic_load_n(done, __ATOMIC_RELAXED) & bit) return hipSuccess;
    const hipError_t set = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    if (set == hipSuccess) __atomic_fetch_or(done, bit, __ATOMIC_RELAXED);
    return set;
}

template <int KS, int C, int NT, int PARTS, bool WIDE>
uint64_t lds_allowed = 0;

template <int KS, int C, int NT, int PARTS, bool WIDE>
hipError_t launch(const DeltaParams &p, hipStream_t stream) {
    using Z = Sizes<KS, C, NT, PARTS>;
    ScanPlan plan;
    plan.tiles = (p.p + Z::kRowsP - 1) / Z::kRowsP;
    plan.each = p.h / p.g * plan.tiles;
    const int64_t groups = (int64_t)p.n * p.g;
    plan.runs = groups >= 32;
    const int64_t units = (plan.runs ? (groups + 7) / 8 * 8 : groups) * plan.each;
    auto kernel = delta_scan_kernel<KS, C, NT, PARTS, WIDE>;
    const hipError_t allowed = allow_lds(reinterpret_cast<const void *>(kernel), &lds_allowed<KS, C, NT, PARTS, WIDE>);
    if (allowed != hipSuccess) return allowed;
    const int64_t across = units < kMaxBlocks ? units : kMaxBlocks, deep = (units + across - 1) / across;
    if (deep > 65535) return hipErrorInvalidConfiguration;
    kernel<<<dim3((unsigned)across, (unsigned)deep), kScanBlock, Z::kBytes, stream>>>(p, plan);
    return hipGetLastError();
}

template <int KS, int C, int NT>
hipError_t launch_parts(const DeltaParams &p, bool wide, hipStream_t stream) {
    if (p.state != nullptr && p.state_f32)
        return wide ? launch<KS, C, NT, 3, true>(p, stream) : launch<KS, C, NT, 3, false>(p, stream);
    return wide ? launch<KS, C, NT, 1, true>(p, stream) : launch<KS, C, NT, 1, false>(p, stream);
}

// Whether rows at p with the given element strides start on 16 bytes, and a chunk's rows
// (b elements apart) span less than 2^31 bytes.
bool rows16(const void *p, int64_t a, int64_t b, int64_t c) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a % 8 == 0 && b % 8 == 0 && c % 8 == 0 && b < (1 << 23);
}

constexpr int64_t kEnoughBlocks = 256;

}  // namespace

hipError_t launch_delta_scan(const DeltaParams &p, hipStream_t stream, const char **kernel_name) {
    const bool wide = p.p % 8 == 0 && p.k % 8 == 0 && rows16(p.q, p.qs_n, p.qs_t, p.qs_g) &&
                      rows16(p.key, p.ks_n, p.ks_t, p.ks_g) && rows16(p.v, p.vs_n, p.vs_t, p.vs_h) &&
                      rows16(p.out, p.os_n, p.os_t, p.os_h);
    *kernel_name = wide ? "delta_scan" : "delta_scan_scalar";
    const bool two = (int64_t)p.n * p.h * ((p.p + 127) / 128) >= kEnoughBlocks && p.p > 64;
    if (p.k <= 64) return two ? launch_parts<64, 64, 2>(p, wide, stream) : launch_parts<64, 64, 1>(p, wide, stream);
    if (p.k <= 128) return two ? launch_parts<128, 64, 2>(p, wide, stream) : launch_parts<128, 64, 1>(p, wide, stream);
    return launch_parts<256, 32, 1>(p, wide, stream);
}

}  // namespace dcconv
