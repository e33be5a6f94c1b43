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
// (I + A)^-1 is taken 32 tokens at a time: U_0 = T_0 R_0 for the chunk's first half, and then
// U_1 = T_1 (R_1 - A_10 U_0), so that T needs no products over the whole chunk.
//
// T, A_10 and P = e^{c_t - c_u} q_t.k_u do not depend on the state: a block's second four waves
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
// Three phases a chunk, a barrier behind each.  Chunk j:
//
//     waves with the state                      the other four
//     1  S k, S q, R                            request q and k of j + 2; A of j + 1
//     2  U                                      request v of j + 1; invert A of j + 1 (one wave)
//                                               and form P of j (three); wait for the tiles
//     3  outputs, S'                            T of j + 1; factors of j + 1; gates and key
//                                               lengths of j + 2
//
// q, k and v go from memory to LDS without passing registers, q and k into one of three places
// each, in pieces of 16 bytes whose order within a row differs from row to row so that neither the rows
// nor the transposing loads meet on a bank by their layout.  (Some accesses do: conflicts take 15.4e6 of the 98.3e6
// cycles in which CUs are busy, in the case below.)  64-token chunks of 128-value keys take 154 to 160 KiB of
// LDS: one block a CU.
//
// Few heads leave CUs idle.  Then sequences are cut into segments: what a segment does to a
// state is S' = S M + B, with M and B from the same kernel (OUT = false), which takes the
// identity's rows without v for M; a join passes over the segments' M and B, and the output pass
// starts each segment from its state.  It is three times the work, and taken where a model of the
// times says so (make_plan).  Packed sequences that are not cut are started longest first.
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
// operand that is no BF16 value is split into parts, BF16 values whose products are added
// up, the smallest first.  With an F32 state R, T, A_10, U and S for S k have three parts (PARTS = 3), all 24
// bits: the state is off by what token-by-token FP32 is off by, 1e-7 to 7e-7 of its size over thousands of tokens.
// (S in two parts: packed sequences 179 us beside 188, but 1.4e-6 to 3e-6 where decay is slow.)  With a BF16
// state, or none, they have two (PARTS = 2), as S for S q, P and the U that P multiplies have in every case: outputs
// and BF16 states are off by their one rounding, 0.0017 of their size.  What fewer parts take and lose: P in one
// 180 us in the case below beside 184, packed sequences 195 beside 199, outputs 0.0017 to 0.0023; S for S q in one as well,
// packed 188, outputs 0.0023 to 0.0029; S for S k and the U that enters the state in one too, where states are BF16 or
// not given, 151 us, outputs 0.0024 to 0.004, states 0.0021 to 0.0042, the most without decay and with weights up to two.
//
// What is not finite.  An infinity or NaN of a later token must not meet the zeros above T's
// and P's diagonals.  An entry of A that is not finite, from operands that are not or from finite
// ones (decays that rise between two tokens, large weights and keys), makes its row of T so, and
// with it U at that token: the substitution takes a row from those ahead of it alone; between a
// half's two tiles the entry is left out of the product with T_11, and NaN put in its row of T; and
// A_10 between halves enters R row by row.  A channel of R or U with a value that is not finite is
// cut at its first such token: U is zero from there, and those outputs and the channel's
// state become NaN.
//
// What bounds it, at 8 x 2048 tokens, 32 heads of 128 x 128 in 16 groups, BF16 states (one block a CU, 32
// chunks): 183 to 190 us, 2.7 times its bytes' time.  A chunk takes about 12000 cycles.  Both kinds of waves wait
// for their own chain of reads, products and conversions, with two waves a SIMD to cover for each other (matrix
// units 37 % busy, vector instructions 52 % of the issue slots); 32 more matrix instructions a wave and chunk (512
// cycles) add 9 to 12 us.  What did not help there: 64 rows a block, twice the blocks (255 us, since T and P are
// prepared twice); S k and S q in one loop that splits S once (180), a part of S q in the second phase (178 to 180,
// or spills); loads of q and k by the waves with the state, a higher priority for the waves that prepare (both slower
// by 7 %); reading all of A's columns ahead of the substitution (spills).  What did: chunks in two halves rather
// than T over all 64 tokens, tiles straight to LDS, and no spilled register.  (Kernels whose rows are no whole 16
// bytes spill up to 16 of 256, and the join for keys above 128 fifty: a wave holds 2 x 64 of M's values there.)
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

// How a call is cut up; the same on the host and in every kernel.
struct ScanPlan {
    int32_t seg;    // tokens of a segment (a multiple of a chunk's)
    int32_t nseg;   // segments of a sequence (batch form)
    int32_t slots;  // segments in all; packed: an upper bound, some empty
    bool split;     // some sequence may have more than one segment
    bool two;       // blocks of 128 state rows, not 64
};
// One kernel's blocks.
struct ScanGrid {
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
// v, not known to be the same as anywhere else: addresses formed from it are formed where they
// are used, instead of being kept in registers through a loop.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

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

// acc + 0 times each of a word's two BF16 values: a NaN where one is not finite.
__device__ __forceinline__ float add_zeros(uint32_t w, float acc) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), __builtin_bit_cast(bf16x2_t, 0u), acc, false);
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

// log(1 + e^v) and 1 / (1 + e^-v) with the hardware's exponential, logarithm and reciprocal, each within
// 2^-21 of itself (down to 2^-126): by way of t = e^-|v|, whose exponent's rounding is made good, and with what
// 1 + t loses of t put back behind the logarithm; a series where t is small.
__device__ __forceinline__ float exp_minus_abs(float v) {
    const float a = __builtin_fabsf(v) > 128.0f ? 128.0f : __builtin_fabsf(v);  // (a NaN stays one)
    const float h = -a * kLog2e, low = __builtin_fmaf(-a, kLog2e, -h) - a * 1.9259629911266175e-8f;  // log2 e - kLog2e
    const float t = __builtin_amdgcn_exp2f(h);
    return __builtin_fmaf(t, low * 0.6931471805599453f, t);
}
__device__ __forceinline__ float softplus_near(float v) {
    const float t = exp_minus_abs(v), w = 1.0f + t;
    const float series = t * (1.0f + t * (-0.5f + t * (1.0f / 3.0f + t * (-0.25f + t * 0.2f))));
    const float far = __builtin_fmaf(__builtin_amdgcn_logf(w), 0.6931471805599453f, (t - (w - 1.0f)) * __builtin_amdgcn_rcpf(w));
    return (v > 0.0f ? v : 0.0f) + (t > 0x1p-5f ? far : series);
}
__device__ __forceinline__ float sigmoid_near(float v) {
    const float t = exp_minus_abs(v), s = __builtin_amdgcn_rcpf(1.0f + t);
    return v < 0.0f ? t * s : s;
}

// The place of 16-byte piece i of row `row` in a tile of rows of ACROSS pieces is i ^ swap: what
// sixteen lanes read at a time, a piece of 16 rows or four of four rows, then lies on banks of its own.
template <int ACROSS>
__device__ __forceinline__ int swap_of(int row) {
    return ACROSS == 8 ? ((row >> 1 & 1) << 2) | (row >> 2 & 3) : ((row & 3) << 2) | (row >> 2 & 3);
}

// One operand's tile of ROWS tokens in LDS, brought there by four waves.  WIDE: straight from
// memory, 64 pieces of 16 bytes an instruction, through a buffer that ends with the chunk's last
// row (what lies behind reads as zeros); the caller waits for them.
template <int ACROSS, int ROWS, bool WIDE>
struct Tile {
    static constexpr int kLoads = ROWS * ACROSS / kHalfBlock;
    const uint16_t *base;  // wave-uniform: the sequence's first row
    int64_t stride;
    int32_t width;
    // rows of the chunk at token t0; n: the sequence's rows from there
    __device__ __forceinline__ void load(uint16_t *to, int64_t t0, int n, int wave, int lane) const {
        typedef __attribute__((address_space(3))) void *Lds;
        const uint16_t *from = base + t0 * stride;
        n = min(n, ROWS);
        const uint32_t pitch = 2u * (uint32_t)stride;
        const Buffer buf = make_buffer(from, WIDE && n > 0 ? (uint32_t)(n - 1) * pitch + 2u * (uint32_t)width : 0u);
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int first = (wave * kLoads + q) * kWave, row = (first + lane) / ACROSS;
            const int piece = (first + lane) % ACROSS ^ swap_of<ACROSS>(row);
            if (WIDE) {
                const uint32_t at = row < n && 8 * piece < width ? (uint32_t)row * pitch + 16u * (uint32_t)piece : kNowhere;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (Lds)(to + 8 * first), 16, at, 0, 0, 0);
                continue;
            }
            u32x4 w = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (row < n && 8 * piece + i < width)
                    w[i >> 1] |= (uint32_t)from[row * stride + 8 * piece + i] << (16 * (i & 1));
            *reinterpret_cast<u32x4 *>(to + 8 * (first + lane)) = w;
        }
    }
};
__device__ __forceinline__ void wait_for_tiles() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// All waves' LDS accesses up to here done, tiles on their way or not (__syncthreads waits for those).
__device__ __forceinline__ void block_sync() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Four consecutive state values, F32 or BF16, from byte offset `at` of a buffer, of which
// `count` exist; WIDE: in one access.
template <bool F32, bool WIDE>
__device__ __forceinline__ f32x4_t load_state4(Buffer buf, uint32_t at, int count) {
    if (WIDE) {
        at = count > 0 ? at : kNowhere;
        if (F32) return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(buf, at, 0, kCached));
        const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(buf, at, 0, kCached);
        return f32x4_t{lo_f32(w[0]), hi_f32(w[0]), lo_f32(w[1]), hi_f32(w[1])};
    }
    f32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t to = i < count ? at + (F32 ? 4u : 2u) * i : kNowhere;
        v[i] = F32 ? __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buf, to, 0, kCached))
                   : bf16_bits_to_f32(__builtin_amdgcn_raw_buffer_load_b16(buf, to, 0, kCached));
    }
    return v;
}
template <bool F32, bool WIDE>
__device__ __forceinline__ void store_state4(Buffer buf, uint32_t at, int count, f32x4_t v) {
    if (WIDE) {
        at = count > 0 ? at : kNowhere;
        if (F32)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), buf, at, 0, kCached);
        else
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}, buf, at, 0, kCached);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t to = i < count ? at + (F32 ? 4u : 2u) * i : kNowhere;
        if (F32)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), buf, to, 0, kCached);
        else
            __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_bits(v[i]), buf, to, 0, kCached);
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

struct Segment {
    int seq, first, last, index, count;  // tokens [first, last) of sequence seq; segment `index` of `count`
    int token0;                          // the sequence's first token on the t axis
    bool ok;
};

// The segment at position u: sequence i has positions i * nseg .. in the batch form, and
// starts[i] / seg + i .. in the packed form (which leaves room for every sequence's last,
// partial segment).  A segment's position is its place in the workspace too.
__device__ __forceinline__ Segment find_segment(const DeltaParams &p, const ScanPlan &plan, int u) {
    Segment s;
    int len;
    if (p.starts == nullptr) {
        s.seq = uniform(u / plan.nseg);
        s.index = u - s.seq * plan.nseg;
        s.token0 = 0;
        len = p.t;
    } else if (!plan.split && p.n <= kWave) {
        // whole sequences, the longest first: those that come last are short ones
        const int lane = threadIdx.x & 63, i = min(lane, p.n - 1);
        const int a = p.starts[i], e = p.starts[i + 1];
        const int mine = lane < p.n ? (a >= 0 && a <= e && e <= p.t ? e - a : -1) : -2;
        int longer = 0;  // sequences ahead of this lane's
        for (int q = 0; q < p.n; ++q) {
            const int other = __builtin_amdgcn_readlane(mine, q);
            longer += other > mine || (other == mine && q < lane);
        }
        const uint64_t found = __ballot(lane < p.n && longer == u);  // (none at a position past the last)
        s.seq = found != 0 ? uniform(__builtin_ctzll(found)) : 0;
        len = found != 0 ? __builtin_amdgcn_readlane(mine, s.seq) : -1;
        s.token0 = len >= 0 ? __builtin_amdgcn_readlane(a, s.seq) : 0;
        s.index = 0;
    } else {
        int lo = 0, hi = p.n;  // the last i with starts[i] / seg + i <= u
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (uniform(load_uniform(p.starts, mid) / plan.seg) + mid <= u)
                lo = mid;
            else
                hi = mid;
        }
        s.seq = lo;
        const int a = load_uniform(p.starts, lo), e = load_uniform(p.starts, lo + 1);
        len = (a >= 0 && a <= e && e <= p.t) ? e - a : -1;
        s.token0 = len >= 0 ? a : 0;
        s.index = u - uniform(s.token0 / plan.seg) - lo;
    }
    s.count = len > 0 ? uniform((len - 1) / plan.seg) + 1 : 1;
    s.ok = len >= 0 && s.index >= 0 && s.index < s.count;
    s.first = s.ok ? s.index * plan.seg : 0;
    s.last = s.ok ? s.first + min(len - s.first, plan.seg) : 0;
    return s;
}

// A place of the workspace: for each head a segment's [p, k] and [k, k] floats.
__device__ __forceinline__ int64_t place_floats(const DeltaParams &p) { return (int64_t)p.h * (p.p + p.k) * p.k; }

// Sizes of a variant and its places in LDS (in bytes).  KS: keys' size, rounded up; C: tokens
// of a chunk; NT: tiles of 16 state rows a wave owns; PARTS: see above.
template <int KS, int C, int NT, int PARTS>
struct Sizes {
    static constexpr int kRowsP = kHalf * 16 * NT;  // state rows of a block
    static constexpr int kPPitch = C, kTPitch = 32;
    static constexpr int kBlocks = C / 16, kHalves = C / 32;
    static constexpr int kKey = 0;                                   // [3][C][KS]
    static constexpr int kQuery = kKey + 3 * C * KS * 2;             // [3][C][KS]
    static constexpr int kV = kQuery + 3 * C * KS * 2;               // [C][kRowsP]
    static constexpr int kT = kV + C * kRowsP * 2;                   // [PARTS][C][kTPitch]
    static constexpr int kOff = kT + PARTS * C * kTPitch * 2;      // [PARTS][C - 32][kTPitch]
    static constexpr int kP = kOff + PARTS * (C - 32) * kTPitch * 2;  // [2][C][kPPitch]
    static constexpr int kA = kP + 2 * C * kPPitch * 2;              // [3 kHalves][16][kAPitch] floats
    static constexpr int kToken = kA + 3 * kHalves * 16 * kAPitch * 4;  // [3][kTokenRows][C] floats
    static constexpr int kBytes = kToken + 3 * kTokenRows * C * 4;
    static_assert(kBytes <= 160 * 1024, "more LDS than a CU has");
};

// OUT: the outputs and final states.  Otherwise what a segment (any but a sequence's last) does
// to a state: S' = S M + B, with B from no state and M, row by row, from the unit rows and no v.
template <int KS, int C, int NT, int PARTS, bool OUT, bool WIDE>
__global__ __launch_bounds__(kScanBlock, 2) void delta_scan_kernel(const DeltaParams p, const ScanPlan plan,
                                                                   const ScanGrid grid) {
    using Z = Sizes<KS, C, NT, PARTS>;
    constexpr int kB = Z::kBlocks, VP = Z::kRowsP, TP = Z::kTPitch, PP = Z::kPPitch, kSteps = KS / 32;
    extern __shared__ u32x4 smem[];
    char *lds = reinterpret_cast<char *>(smem);
    uint16_t *sk = reinterpret_cast<uint16_t *>(lds + Z::kKey), *sq = reinterpret_cast<uint16_t *>(lds + Z::kQuery);
    uint16_t *sv = reinterpret_cast<uint16_t *>(lds + Z::kV), *st = reinterpret_cast<uint16_t *>(lds + Z::kT);
    uint16_t *sp = reinterpret_cast<uint16_t *>(lds + Z::kP), *so = reinterpret_cast<uint16_t *>(lds + Z::kOff);
    float *sa = reinterpret_cast<float *>(lds + Z::kA), *tokens = reinterpret_cast<float *>(lds + Z::kToken);

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = uniform(tid >> 6);
    if (OUT && blockIdx.x == 0 && blockIdx.y == 0) check_table(p);

    // ---- this block's sequence, head and rows.  Blocks are dealt to the eight XCDs in turn:
    // a group's blocks, which read the same q and k, go to one of them.
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    int64_t ug;
    int member;
    if (grid.runs) {
        const int64_t turn = (block >> 3) / grid.each;
        ug = turn * 8 + (block & 7);
        member = uniform((int)((block >> 3) - turn * grid.each));
    } else {
        ug = block / grid.each;
        member = uniform((int)(block - ug * grid.each));
    }
    if (ug >= (int64_t)plan.slots * p.g) return;
    const int place = uniform((int)(ug / p.g)), group = uniform((int)(ug - (int64_t)place * p.g));
    const Segment segment = find_segment(p, plan, place);
    if (!segment.ok || (!OUT && segment.index == segment.count - 1)) return;
    const int seq = segment.seq, which = uniform(member / grid.tiles), tile = member - which * grid.tiles;
    const int head = group * uniform(p.h / p.g) + which;
    const int first = segment.token0 + segment.first, len = segment.last - segment.first;
    // M's rows behind B's, in tiles of their own
    const int own_tiles = OUT ? grid.tiles : (p.p + Z::kRowsP - 1) / Z::kRowsP;
    const bool units = !OUT && tile >= own_tiles;
    const int p0 = (units ? tile - own_tiles : tile) * Z::kRowsP;
    const int rows = min(Z::kRowsP, (units ? p.k : p.p) - p0);  // of this block
    const int slot = uniform(route_row(p.idx, p.status, p.n, p.s, seq, lane));
    uint16_t *out = p.out + seq * p.os_n + (int64_t)first * p.os_t + head * p.os_h + p0;
    if (slot < 0) {  // a padding sequence: zeros, and no state moves
        if (OUT)
            for (int t = wave; t < len; t += 2 * kHalf)
                for (int c = lane; c < rows; c += kWave) out[t * p.os_t + c] = 0;
        return;
    }
    const int chunks = (len + C - 1) / C;

    // Where piece i of row r of a 16-row tile of T or A_10 (four pieces of eight inner indices), and of P, begins: sixteen
    // lanes that read a piece of 16 rows find banks of their own.
    const auto t_place = [](int r, int i) { return r * TP + 8 * (i ^ (r >> 2 & 3)); };
    const auto p_place = [](int r, int i) { return r * PP + 8 * (i ^ (C == 64 ? r >> 1 & 7 : r >> 2 & 3)); };

    // the tiles of T and P above the diagonal that products over 32 tokens read: zeros for good
    for (int i = tid; i < (PARTS + 2) * (kB / 2) * 16 * 4; i += kScanBlock) {
        const int piece = i & 3, row = (i >> 2) & 15, m = (i >> 6) % (kB / 2), part = (i >> 6) / (kB / 2);
        uint16_t *to = part < PARTS ? st + (part * C + 32 * m) * TP + t_place(row, piece)
                                    : sp + ((part - PARTS) * C + 32 * m) * PP + p_place(row, 4 * m + piece);
        *reinterpret_cast<u32x2 *>(to + 4) = u32x2{0, 0};
    }

    // Where a lane reads its share of k or q: row r's inner indices 32 m + 8 g .. of the state's
    // columns, and, with tokens as the inner index, columns 16 t ..
    constexpr int kAcross = KS / 8;
    const auto row_place = [](int m, int r, int g) {
        return r * KS + 8 * ((4 * (m & 3) + g) ^ swap_of<kAcross>(r)) + 128 * (m >> 2);
    };
    const auto column_place = [](int t, int r, int g) {
        const int row = 4 * g + (r >> 2);
        return row * KS + 8 * ((4 * (t >> 1 & 3) + (r & 3)) ^ swap_of<kAcross>(row)) + 128 * (t >> 3) + 4 * (t & 1);
    };
    const auto row_at = [&](int m) { return row_place(m, r, g); };

    if (wave >= kHalf) {
        // ================================================== the waves that prepare T and P
        if (chunks == 0) return;
        const int pw = wave - kHalf;
        const Tile<kAcross, C, WIDE> keys = {p.key + seq * p.ks_n + (int64_t)first * p.ks_t + group * p.ks_g, p.ks_t, p.k};
        const Tile<kAcross, C, WIDE> queries = {p.q + seq * p.qs_n + (int64_t)first * p.qs_t + group * p.qs_g, p.qs_t, p.k};
        const Tile<Z::kRowsP / 8, C, WIDE> values = {p.v + seq * p.vs_n + (int64_t)first * p.vs_t + head * p.vs_h + p0,
                                                     p.vs_t, rows};
        auto fetch = [&](int j) {
            keys.load(sk + j % 3 * C * KS, (int64_t)j * C, len - j * C, pw, lane);
            queries.load(sq + j % 3 * C * KS, (int64_t)j * C, len - j * C, pw, lane);
        };
        auto fetch_v = [&](int j) { values.load(sv, (int64_t)j * C, units ? 0 : len - j * C, pw, lane); };
        // ---- decays and weights of a chunk's tokens, a lane each (as they are in memory:
        // converting them here would wait for them)
        const float rate = p.a[head] * kLog2e, bias = p.dt_bias != nullptr ? p.dt_bias[head] : 0.0f;
        const int64_t dt0 = seq * p.ds_n + (int64_t)first * p.ds_t + head, beta0 = seq * p.es_n + (int64_t)first * p.es_t + head;
        uint32_t dt_raw = 0, beta_raw = 0;
        auto fetch_gates = [&](int j) {  // (behind the end: the last token's, which put_gates leaves out)
            const int64_t t = min(j * C + lane, len - 1);
            const int64_t d = dt0 + t * p.ds_t, e = beta0 + t * p.es_t;
            dt_raw = p.dt_f32 ? static_cast<const uint32_t *>(p.dt)[d] : static_cast<const uint16_t *>(p.dt)[d];
            beta_raw = p.beta_f32 ? static_cast<const uint32_t *>(p.beta)[e] : static_cast<const uint16_t *>(p.beta)[e];
        };
        auto put_gates = [&](int j) {
            float d = __uint_as_float(p.dt_f32 ? dt_raw : dt_raw << 16) + bias;
            if (p.dt_softplus) d = softplus_near(d);
            float decay = d * rate, weight = __uint_as_float(p.beta_f32 ? beta_raw : beta_raw << 16);
            if (p.beta_sigmoid) weight = sigmoid_near(weight);
            if (lane >= min(C, len - j * C)) decay = weight = 0.0f;
            if (decay < kNone) decay = kNone;
            if (!is_finite(weight)) decay = __builtin_nanf(""), weight = 0.0f;
            const double c = prefix_sum((double)decay, lane);
            const float high = (float)c;
            float *tok = tokens + j % 3 * kTokenRows * C + lane;
            if (lane < C) {
                tok[kSumHigh * C] = high;
                tok[kSumLow * C] = (float)(c - (double)high);
                tok[kWeight * C] = weight;
            }
        };
        // what the state's waves scale S k, S q and U by
        auto put_scales = [&](int j) {
            if (lane >= C) return;
            float *tok = tokens + j % 3 * kTokenRows * C;
            const float high = tok[kSumHigh * C + lane], low = tok[kSumLow * C + lane];
            const float end = tok[kSumHigh * C + C - 1], end_low = tok[kSumLow * C + C - 1];
            const float unit = tok[kUnitK * C + lane], e = __builtin_amdgcn_exp2f(high + low);
            tok[kForK * C + lane] = e * unit;
            tok[kForQ * C + lane] = e * tok[kUnitQ * C + lane];
            tok[kForU * C + lane] = __builtin_amdgcn_exp2f((end - high) + (end_low - low)) * unit;
        };
        // ---- the factors that make rows of length one, from the diagonals of the rows'
        // products with themselves (that of row r in lanes g = r >> 2)
        auto put_units = [&](int j) {
            if (pw >= kB) return;
            const uint16_t *km = sk + (j % 3 * C + 16 * pw) * KS, *qm = sq + (j % 3 * C + 16 * pw) * KS;
            f32x4_t k2 = {0, 0, 0, 0}, q2 = {0, 0, 0, 0};
            u32x4 kf[kSteps], qf[kSteps];
#pragma unroll
            for (int m = 0; m < kSteps; ++m) kf[m] = lds16(km + row_at(m)), qf[m] = lds16(qm + row_at(m));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < kSteps; ++m) k2 = mfma(kf[m], kf[m], k2), q2 = mfma(qf[m], qf[m], q2);
            const float k0 = r & 1 ? k2[1] : k2[0], k1 = r & 1 ? k2[3] : k2[2], kk = r & 2 ? k1 : k0;
            const float q0 = r & 1 ? q2[1] : q2[0], q1 = r & 1 ? q2[3] : q2[2], qq = r & 2 ? q1 : q0;
            float *tok = tokens + j % 3 * kTokenRows * C + 16 * pw + r;
            if (g == r >> 2) {
                tok[kUnitK * C] = is_finite(kk) ? unit_factor(p, kk) : __builtin_nanf("");
                tok[kUnitQ * C] = p.scale * unit_factor(p, qq);
            }
        };
        // Four values as PARTS parts, and put `apart` values apart.
        auto to_parts = [&](float (&v)[4], u32x2 (&parts)[PARTS]) {
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                const uint32_t h0 = pack_bf16x2(v[0], v[1]), h1 = pack_bf16x2(v[2], v[3]);
                parts[part] = u32x2{h0, h1};
                v[0] -= lo_f32(h0), v[1] -= hi_f32(h0), v[2] -= lo_f32(h1), v[3] -= hi_f32(h1);
            }
        };
        auto put_parts = [&](float (&v)[4], uint16_t *to, int apart) {
            u32x2 parts[PARTS];
            to_parts(v, parts);
#pragma unroll
            for (int part = 0; part < PARTS; ++part) *reinterpret_cast<u32x2 *>(to + part * apart) = parts[part];
        };
        // ---- block row I of P of chunk j
        auto form_p = [&](auto row_constant, int j) {
            constexpr int I = decltype(row_constant)::value;
            const uint16_t *km = sk + j % 3 * C * KS, *qm = sq + j % 3 * C * KS;
            const float *tok = tokens + j % 3 * kTokenRows * C;
            u32x4 tf[kSteps], f[I + 1][kSteps];
            f32x4_t acc[I + 1], uh[I + 1], ul[I + 1], uk[I + 1];
#pragma unroll
            for (int m = 0; m < kSteps; ++m) {
                tf[m] = lds16(qm + 16 * I * KS + row_at(m));
#pragma unroll
                for (int b = 0; b <= I; ++b) f[b][m] = lds16(km + 16 * b * KS + row_at(m));
            }
            const int t = 16 * I + r;
            const float th = tok[kSumHigh * C + t], tl = tok[kSumLow * C + t], unit = tok[kUnitQ * C + t];
            float ref = 0, ref_low = 0;
            if (I > 0) ref = tok[kSumHigh * C + 16 * I - 1], ref_low = tok[kSumLow * C + 16 * I - 1];
#pragma unroll
            for (int b = 0; b <= I; ++b) {
                const int u0 = 16 * b + 4 * g;
                uh[b] = lds4f(tok + kSumHigh * C + u0), ul[b] = lds4f(tok + kSumLow * C + u0);
                uk[b] = lds4f(tok + kUnitK * C + u0);
                acc[b] = f32x4_t{0, 0, 0, 0};
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < kSteps; ++m)
#pragma unroll
                for (int b = 0; b <= I; ++b) acc[b] = mfma(f[b][m], tf[m], acc[b]);
            // lane: column t = r, rows u; decays by way of the block's start
            const float ft = unit * __builtin_amdgcn_exp2f((th - ref) + (tl - ref_low));
#pragma unroll
            for (int b = 0; b <= I; ++b) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (b < I)
                        v[i] = acc[b][i] * ft * uk[b][i] * __builtin_amdgcn_exp2f((ref - uh[b][i]) + (ref_low - ul[b][i]));
                    else
                        v[i] = 4 * g + i <= r ? acc[b][i] * unit * uk[b][i] *
                                                    __builtin_amdgcn_exp2f((th - uh[b][i]) + (tl - ul[b][i]))
                                              : 0.0f;
                }
                uint16_t *to = sp + 16 * I * PP + p_place(r, 4 * (b >> 1) + g) + 4 * (b & 1);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const uint32_t h0 = pack_bf16x2(v[0], v[1]), h1 = pack_bf16x2(v[2], v[3]);
                    *reinterpret_cast<u32x2 *>(to + part * C * PP) = u32x2{h0, h1};
                    v[0] -= lo_f32(h0), v[1] -= hi_f32(h0), v[2] -= lo_f32(h1), v[3] -= hi_f32(h1);
                }
            }
        };
        // ---- A of chunk j, tile by tile.  Tiles inside a half of 32 tokens are kept in FP32,
        // transposed (row u, column t); the others, negative and without the weight, as P.
        struct Log {
            float high, low;
            __device__ __forceinline__ float to(const Log &u) const {  // e^{this - u}
                return __builtin_amdgcn_exp2f((high - u.high) + (low - u.low));
            }
        };
        auto log_at = [&](const float *tok, int t) { return Log{tok[kSumHigh * C + t], tok[kSumLow * C + t]}; };
        struct Logs {
            f32x4_t high, low;
        };
        auto logs_at = [&](const float *tok, int t) {
            return Logs{lds4f(tok + kSumHigh * C + t), lds4f(tok + kSumLow * C + t)};
        };
        u32x2 off[2][PARTS];  // what this wave has formed of the tiles between halves
        auto form_a = [&](auto wave_constant, int j) {
            // wave W's tiles: diagonal block W, and: blocks (2, W) and (3, W) for W = 0, 1, block
            // (1, 0) for W = 2 and (3, 2) for W = 3.  (Two blocks: (0, 0), and (1, 1) and (1, 0).)
            constexpr int W = decltype(wave_constant)::value;
            constexpr bool kOff = kB > 2 && W < 2, kSide = kB > 2 ? W >= 2 : W == 1;
            constexpr int S = kB > 2 && W == 3 ? 3 : 1;  // the block beside it: (S, S - 1)
            const uint16_t *km = sk + j % 3 * C * KS;
            const float *tok = tokens + j % 3 * kTokenRows * C;
            u32x4 f[kSteps], x[kSteps], y[kSteps];
#pragma unroll
            for (int m = 0; m < kSteps; ++m) {
                f[m] = lds16(km + 16 * W * KS + row_at(m));
                if (kOff) x[m] = lds16(km + 32 * KS + row_at(m)), y[m] = lds16(km + 48 * KS + row_at(m));
                if (kSide) y[m] = lds16(km + 16 * (S - 1) * KS + row_at(m));
                if (kSide && S != W) x[m] = lds16(km + 16 * S * KS + row_at(m));
            }
            const int t0 = 16 * W + 4 * g, s0 = 16 * S + 4 * g;
            const Logs tl = logs_at(tok, t0);
            const f32x4_t tw = lds4f(tok + kWeight * C + t0), tu = lds4f(tok + kUnitK * C + t0);
            const Log ul = log_at(tok, 16 * W + r);
            const float uu = tok[kUnitK * C + 16 * W + r];
            Logs sl = tl;
            f32x4_t sw = tw, su = tu;
            Log vl = {0, 0}, ref = {0, 0}, xl = {0, 0}, yl = {0, 0};
            float vu = 0, xu = 0, yu = 0;
            if (kSide) {
                vl = log_at(tok, 16 * (S - 1) + r), vu = tok[kUnitK * C + 16 * (S - 1) + r];
                if (S != W) sl = logs_at(tok, s0), sw = lds4f(tok + kWeight * C + s0), su = lds4f(tok + kUnitK * C + s0);
            }
            if (kOff) {
                ref = log_at(tok, 31), xl = log_at(tok, 32 + r), yl = log_at(tok, 48 + r);
                xu = tok[kUnitK * C + 32 + r], yu = tok[kUnitK * C + 48 + r];
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x4_t self = {0, 0, 0, 0}, a0 = {0, 0, 0, 0}, a1 = {0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < kSteps; ++m) {
                self = mfma(f[m], f[m], self);
                if (kOff) a0 = mfma(f[m], x[m], a0), a1 = mfma(f[m], y[m], a1);  // columns t, rows u
                if (kSide) a0 = mfma(S != W ? x[m] : f[m], y[m], a0);           // columns u, rows t
            }
            float *tile = sa + (3 * (W >> 1) + (W & 1)) * 16 * kAPitch + r * kAPitch + 4 * g;
            f32x4_t v;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = self[i] * (tw[i] * tu[i]) * uu * Log{tl.high[i], tl.low[i]}.to(ul);
                if (!(r < 4 * g + i)) v[i] = 0.0f;
            }
            *reinterpret_cast<f32x4_t *>(tile) = v;
            if (kSide) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = a0[i] * (sw[i] * su[i]) * vu * Log{sl.high[i], sl.low[i]}.to(vl);
                *reinterpret_cast<f32x4_t *>(sa + (3 * (S >> 1) + 2) * 16 * kAPitch + r * kAPitch + 4 * g) = v;
            }
            if (kOff) {  // decays by way of the second half's start
                f32x4_t fu;
#pragma unroll
                for (int i = 0; i < 4; ++i) fu[i] = -tu[i] * ref.to(Log{tl.high[i], tl.low[i]});
                const float fx = xu * xl.to(ref), fy = yu * yl.to(ref);
                float v0[4], v1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v0[i] = a0[i] * fx * fu[i], v1[i] = a1[i] * fy * fu[i];
                }
                to_parts(v0, off[0]);
                to_parts(v1, off[1]);
            }
        };
        // (written once the state's waves have done with the chunk before)
        auto put_off = [&](int w) {
            if (kB == 2 || w >= 2) return;
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                uint16_t *to = so + part * (C - 32) * TP + t_place(r, g) + 4 * w;
                *reinterpret_cast<u32x2 *>(to) = off[0][part];
                *reinterpret_cast<u32x2 *>(to + 16 * TP) = off[1][part];
            }
        };
        // ---- the inverses of I + A's diagonal blocks, a column a lane, in place (transposed)
        auto invert = [&]() {
            if (g >= kB) return;
            float *tile = sa + (3 * (g >> 1) + (g & 1)) * 16 * kAPitch;
            // (a group of A's columns read while the one before is worked off)
            f32x4_t a[2][4][4];
            auto read_columns = [&](int u0) {
#pragma unroll
                for (int u = u0; u < u0 + 4 && u < 15; ++u)
#pragma unroll
                    for (int q = (u + 1) / 4; q < 4; ++q) a[u0 >> 2 & 1][u - u0][q] = lds4f(tile + u * kAPitch + 4 * q);
            };
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = i == r ? 1.0f : 0.0f;
            read_columns(0);
#pragma unroll
            for (int u0 = 0; u0 < 15; u0 += 4) {
                read_columns(u0 + 4);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int u = u0; u < u0 + 4 && u < 15; ++u)
#pragma unroll
                    for (int i = u + 1; i < 16; ++i)
                        x[i] = __builtin_fmaf(-a[u0 >> 2 & 1][u - u0][i / 4][i % 4], x[u], x[i]);
            }
            wave_lds_sync();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4_t *>(tile + r * kAPitch + 4 * q) = f32x4_t{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
        };
        // ---- block row I of its half's T: the diagonal block's inverse, and in the second row
        // T_10 = -T_11 A_10 T_00, all transposed; times the weights, in parts
        auto join = [&](auto row_constant, int j) {
            constexpr int I = decltype(row_constant)::value;
            const float *weight = tokens + (j % 3 * kTokenRows + kWeight) * C + 16 * (I & ~1) + 4 * g;
            const float *half = sa + 3 * (I >> 1) * 16 * kAPitch;
            uint16_t *to = st + 16 * I * TP + t_place(r, g);
            const float *diag = half + (I & 1) * 16 * kAPitch;
            f32x4_t y, a, t, w0 = lds4f(weight), w1;
#pragma unroll
            for (int s = 0; s < 4; ++s) y[s] = diag[(4 * g + s) * kAPitch + r];
            if constexpr ((I & 1) == 0) {
                y *= w0;
                float v[4] = {y[0], y[1], y[2], y[3]};
                put_parts(v, to, C * TP);
            } else {
                a = lds4f(half + (2 * 16 + r) * kAPitch + 4 * g), t = lds4f(half + r * kAPitch + 4 * g);
                w1 = lds4f(weight + 16);
                const f32x4_t zero = {0, 0, 0, 0};
                // a row of A_10 that is not finite: left out of the product, where it would meet T_11's
                // zeros in the rows ahead, and NaN in T
                bool lost = false;
                if (__any(!is_finite((a[0] + a[1]) + (a[2] + a[3])))) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const bool bad = !is_finite(a[s]);
                        const uint64_t rows = __ballot(bad);  // that of row 4 q + s: in the lanes g = q
                        if (bad) a[s] = 0.0f;
                        if ((r & 3) == s) lost = (rows >> (16 * (r >> 2)) & 0xffff) != 0;
                    }
                }
                f32x4_t x = mfma_f32(t, mfma_f32(a, y, zero), zero) * w0;
                if (lost) x[0] = __builtin_nanf("");
                y *= w1;
                float v0[4] = {-x[0], -x[1], -x[2], -x[3]}, v1[4] = {y[0], y[1], y[2], y[3]};
                put_parts(v1, to + 4, C * TP);
                put_parts(v0, to, C * TP);
            }
        };

        // body(block row) for the block row of this wave
        auto by_row = [&](int row, auto &&body) {
            if (row == 0) body(std::integral_constant<int, 0>{});
            if (row == 1) body(std::integral_constant<int, 1>{});
            if constexpr (kB > 2) {
                if (row == 2) body(std::integral_constant<int, 2>{});
                if (row == 3) body(std::integral_constant<int, 3>{});
            }
        };
        // the rows of P, for the waves beside the one that inverts
        auto form_p_shared = [&](int j) {
            if constexpr (kB > 2) {
                if (pw == 1) form_p(std::integral_constant<int, 3>{}, j);
                if (pw == 2) form_p(std::integral_constant<int, 2>{}, j);
                if (pw == 3) form_p(std::integral_constant<int, 1>{}, j), form_p(std::integral_constant<int, 0>{}, j);
            } else {
                if (pw == 1) form_p(std::integral_constant<int, 1>{}, j);
                if (pw == 2) form_p(std::integral_constant<int, 0>{}, j);
            }
        };
        // (what a wave has to do beside its tiles goes to those that wait)
        const bool gates = pw == 2, scales = pw == 0;
        if (gates) fetch_gates(0);
        fetch(0);
        fetch_v(0);
        wait_for_tiles();
        block_sync();
        fetch(1);
        put_units(0);
        if (gates) put_gates(0), fetch_gates(1);
        block_sync();
        by_row(pw, [&](auto w) { form_a(w, 0); });
        block_sync();
        if (pw == 0) invert();
        if (gates) put_gates(1);
        wait_for_tiles();
        block_sync();
        by_row(pw, [&](auto row) { join(row, 0); });
        put_off(pw);
        if (scales) put_scales(0);
        put_units(1);
        block_sync();
        for (int j = 0; j < chunks; ++j) {
            const bool more = j + 1 < chunks;
            if (gates) fetch_gates(j + 2);
            if (j + 2 < chunks) fetch(j + 2);
            if (more) by_row(pw, [&](auto w) { form_a(w, j + 1); });
            block_sync();
            if (more) fetch_v(j + 1);
            if (more && pw == 0) invert();
            if constexpr (OUT) form_p_shared(j);
            wait_for_tiles();
            block_sync();
            if (more) {
                by_row(pw, [&](auto row) { join(row, j + 1); });
                put_off(pw);
                if (scales) put_scales(j + 1);
                if (gates) put_gates(j + 2);
                if (j + 2 < chunks) put_units(j + 2);
            }
            block_sync();
        }
        return;
    }

    // ====================================================== the waves that hold the state
    // Tile n's column r is row own(n, r) of the wave's, so that result rows 4 g .. of the
    // two tiles are eight neighbours.
    const int mine = wave * 16 * NT, left_rows = rows - mine;  // this wave's rows start at p0 + mine
    const auto own = [&](int n, int c) { return NT == 2 ? 8 * (c >> 2) + 4 * n + (c & 3) : c; };

    // Outputs of chunk j: a lane holds 4 NT neighbouring rows p of tokens 16 tt + r.
    auto put_out = [&](const f32x4_t(&o)[kB][NT], int j) {
        uint16_t *base = out + (int64_t)j * C * p.os_t;
        const int r = here(lane) & 15, g = here(lane) >> 4;
        const int left = min(len - j * C, C);
        const uint32_t pitch = 2u * (uint32_t)p.os_t;
        const Buffer buf = make_buffer(base, WIDE ? (uint32_t)(left - 1) * pitch + 2u * (uint32_t)rows : 0u);
        const uint32_t at = 4 * NT * g < left_rows ? (uint32_t)r * pitch + 2u * (uint32_t)(mine + 4 * NT * g) : kNowhere;
#pragma unroll
        for (int tt = 0; tt < kB; ++tt) {
            uint32_t w[2 * NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                w[2 * n] = pack_bf16x2(o[tt][n][0], o[tt][n][1]);
                w[2 * n + 1] = pack_bf16x2(o[tt][n][2], o[tt][n][3]);
            }
            const int t = 16 * tt + r;
            if (WIDE) {
                buffer_store_words<2 * NT, kCached>(w, buf, t < left ? at + 16u * (uint32_t)tt * pitch : kNowhere);
            } else if (t < left) {
                uint16_t *to = base + t * p.os_t + mine + 4 * NT * g;
#pragma unroll
                for (int i = 0; i < 4 * NT; ++i)
                    if (4 * NT * g + i < left_rows) to[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
        }
    };

    // ---- the state ahead: tile m, rows k = column(m, g) + i, columns p = own(n, r)
    f32x4_t hs[KS / 16][NT];
#pragma unroll
    for (int m = 0; m < KS / 16; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) hs[m][n] = f32x4_t{0, 0, 0, 0};
    // Where the state is from and where it goes: the pool's slot, or the workspace's place.
    // body(a tile's four values, their byte offset in the head's state, how many there are)
    constexpr bool kF32 = PARTS == 3;  // the pool's type, where there is a pool
    const bool wide_pool = p.k % 4 == 0 && p.ss_s % 4 == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0;
    const bool wide_place = p.k % 4 == 0;
    const auto in_pool = [&]() {
        const int64_t pk = (int64_t)p.p * p.k;
        return make_buffer(static_cast<const char *>(p.state) + (kF32 ? 4 : 2) * (slot * p.ss_s + head * pk),
                           (uint32_t)((kF32 ? 4 : 2) * pk));
    };
    const auto in_place = [&]() {
        const int64_t head_floats = (int64_t)(p.p + p.k) * p.k;
        return make_buffer(p.workspace + place * place_floats(p) + head * head_floats, (uint32_t)(4 * head_floats));
    };
    const auto each_state4 = [&](uint32_t bytes, auto &&body) {
        const int rr = here(r), gg = here(g);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t row = (uint32_t)((units ? p.p : 0) + p0 + mine + own(n, rr)) * (uint32_t)p.k;
            const int most = own(n, rr) < left_rows ? p.k : 0;
#pragma unroll
            for (int m = 0; m < KS / 16; ++m)
                body(hs[m][n], bytes * (row + (uint32_t)column(m, gg)), most - column(m, gg));
        }
    };
    if (!OUT) {
        if (units)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < KS / 16; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) hs[m][n][i] = column(m, g) + i == p0 + mine + own(n, r) ? 1.0f : 0.0f;
    } else if (segment.count > 1) {
        const Buffer buf = in_place();
        if (wide_place)
            each_state4(4, [&](f32x4_t &v, uint32_t at, int count) { v = load_state4<true, true>(buf, at, count); });
        else
            each_state4(4, [&](f32x4_t &v, uint32_t at, int count) { v = load_state4<true, false>(buf, at, count); });
    } else if (p.state != nullptr && p.has_init != nullptr && p.has_init[seq] != 0) {
        const Buffer buf = in_pool();
        if (wide_pool)
            each_state4(kF32 ? 4 : 2, [&](f32x4_t &v, uint32_t at, int count) { v = load_state4<kF32, true>(buf, at, count); });
        else
            each_state4(kF32 ? 4 : 2, [&](f32x4_t &v, uint32_t at, int count) { v = load_state4<kF32, false>(buf, at, count); });
    }

    if (chunks > 0)
        for (int i = 0; i < 5; ++i) block_sync();
    for (int j = 0; j < chunks; ++j) {
        const uint16_t *km = sk + j % 3 * C * KS, *qm = sq + j % 3 * C * KS;
        const float *tok = tokens + j % 3 * kTokenRows * C;
        f32x4_t d[kB][NT], o[kB][NT];
        u32x4 rp[NT][PARTS];
        // ---- d = S k (columns p, rows t), then R
        {
            const int lane_here = here(lane), r = lane_here & 15, g = lane_here >> 4;
#pragma unroll
            for (int tt = 0; tt < kB; ++tt)
#pragma unroll
                for (int n = 0; n < NT; ++n) d[tt][n] = f32x4_t{0, 0, 0, 0};
            // Rows of k, read ahead of their products; the next 32 columns of the state are split meanwhile.
            u32x4 f[2][kB], hp[2][NT][PARTS];
            auto read_rows = [&](int m) {
#pragma unroll
                for (int tt = 0; tt < kB; ++tt) f[m & 1][tt] = lds16(km + 16 * tt * KS + row_place(m, r, g));
            };
            auto split_state = [&](int m) {
#pragma unroll
                for (int n = 0; n < NT; ++n) split<PARTS>(hs[2 * m][n], hs[2 * m + 1][n], hp[m & 1][n]);
            };
            read_rows(0);
            split_state(0);
#pragma unroll
            for (int m = 0; m < kSteps; ++m) {
                if (m + 1 < kSteps) read_rows(m + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int tt = 0; tt < kB; ++tt) d[tt][n] = mfma(f[m & 1][tt], hp[m & 1][n][part], d[tt][n]);
                if (m + 1 < kSteps) {
                    split_state(m + 1);
                    // a product, and what the vector units do meanwhile
#pragma unroll
                    for (int i = 0; i < PARTS * NT * kB; ++i) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
                    }
                }
            }
            if constexpr (OUT) {
            // ---- o = S q (columns t, rows p)
#pragma unroll
            for (int tt = 0; tt < kB; ++tt)
#pragma unroll
                for (int n = 0; n < NT; ++n) o[tt][n] = f32x4_t{0, 0, 0, 0};
            u32x4 f[2][kB];
            auto read_rows = [&](int m) {
#pragma unroll
                for (int tt = 0; tt < kB; ++tt) f[m & 1][tt] = lds16(qm + 16 * tt * KS + row_place(m, r, g));
            };
            read_rows(0);
#pragma unroll
            for (int m = 0; m < kSteps; ++m) {
                if (m + 1 < kSteps) read_rows(m + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    u32x4 hp[2];
                    split<2>(hs[2 * m][n], hs[2 * m + 1][n], hp);
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int tt = 0; tt < kB; ++tt) o[tt][n] = mfma(hp[part], f[m & 1][tt], o[tt][n]);
                }
            }
            }
            const int vrow = 4 * g + (r >> 2), vpiece = NT == 2 ? 4 * wave + (r & 3) : 2 * wave + (r >> 1 & 1);
            const uint16_t *va = sv + vrow * VP + 8 * (vpiece ^ swap_of<VP / 8>(vrow)) + (NT == 2 ? 0 : 4 * (r & 1));
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
                    if (m == 0) split<PARTS>(d[0][n], d[1][n], rp[n]);
                }
            }
        }
        block_sync();
        // ---- d = U, half by half: U_0 = T_0 R_0, U_1 = T_1 (R_1 - A_10 U_0)
        int cut[NT];  // the first token whose R or U is not finite
        bool bad = false;
        u32x4 up[kB / 2][NT][PARTS], wp[kB / 2][NT][PARTS];
        {
            const int lane_here = here(lane), r = lane_here & 15, g = lane_here >> 4;
#pragma unroll
            for (int n = 0; n < NT; ++n) cut[n] = C;
#pragma unroll
            for (int m = 0; m < kB / 2; ++m) {
                f32x4_t(&d0)[NT] = d[2 * m], (&d1)[NT] = d[2 * m + 1];
                if (m > 0) {
                    u32x4 af[2][PARTS];
#pragma unroll
                    for (int a = PARTS - 1; a >= 0; --a)
#pragma unroll
                        for (int tt = 0; tt < 2; ++tt) af[tt][a] = lds16(so + (a * (C - 32) + 16 * tt) * TP + t_place(r, g));
#pragma unroll
                    for (int a = PARTS - 1; a >= 0; --a)
#pragma unroll
                        for (int b = PARTS - 1; b >= 0; --b)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                if (a + b < PARTS) {
                                    d0[n] = mfma(af[0][a], up[0][n][b], d0[n]);
                                    d1[n] = mfma(af[1][a], up[0][n][b], d1[n]);
                                }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (bad && cut[n] < 32) d0[n] = d1[n] = f32x4_t{0, 0, 0, 0};
                        split<PARTS>(d0[n], d1[n], rp[n]);
                    }
                }
                u32x4 tf[2][PARTS];
#pragma unroll
                for (int a = PARTS - 1; a >= 0; --a)
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt) tf[tt][a] = lds16(st + (a * C + 32 * m + 16 * tt) * TP + t_place(r, g));
                const f32x4_t w0 = lds4f(tok + kForU * C + 32 * m + 4 * g), w1 = lds4f(tok + kForU * C + 32 * m + 16 + 4 * g);
                auto correct = [&]() {
#pragma unroll
                    for (int n = 0; n < NT; ++n) d0[n] = d1[n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                    for (int a = PARTS - 1; a >= 0; --a)
#pragma unroll
                        for (int b = PARTS - 1; b >= 0; --b)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                if (a + b < PARTS) {
                                    d0[n] = mfma(tf[0][a], rp[n][b], d0[n]);
                                    d1[n] = mfma(tf[1][a], rp[n][b], d1[n]);
                                }
                };
                correct();
#pragma unroll
                for (int n = 0; n < NT; ++n) split<PARTS>(d0[n], d1[n], up[m][n]);
                float probe[4] = {0, 0, 0, 0};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) probe[i] = add_zeros(up[m][n][0][i], probe[i]);
                if (__any((probe[0] + probe[1]) + (probe[2] + probe[3]) != 0.0f)) {
                    // zeros for R from the first token on where it is not finite, U anew, and the same for U
                    bad = true;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        int at = 32;  // of the half's tokens
#pragma unroll
                        for (int i = 7; i >= 0; --i)
                            if (!is_finite((i & 1) ? hi_f32(rp[n][0][i >> 1]) : lo_f32(rp[n][0][i >> 1])))
                                at = 16 * (i >> 2) + 4 * g + (i & 3);
                        at = min(at, __shfl_xor(at, 16));
                        at = min(at, __shfl_xor(at, 32));
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (16 * (i >> 2) + 4 * g + (i & 3) >= at)
#pragma unroll
                                for (int part = 0; part < PARTS; ++part)
                                    rp[n][part][i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
                        if (at < 32) cut[n] = min(cut[n], 32 * m + at);
                    }
                    correct();
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (!is_finite(d0[n][i])) cut[n] = min(cut[n], 32 * m + 4 * g + i);
                            if (!is_finite(d1[n][i])) cut[n] = min(cut[n], 32 * m + 16 + 4 * g + i);
                        }
                        cut[n] = min(cut[n], __shfl_xor(cut[n], 16));
                        cut[n] = min(cut[n], __shfl_xor(cut[n], 32));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (32 * m + 4 * g + i >= cut[n]) d0[n][i] = 0.0f;
                            if (32 * m + 16 + 4 * g + i >= cut[n]) d1[n][i] = 0.0f;
                        }
                        split<PARTS>(d0[n], d1[n], up[m][n]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) split<PARTS>(d0[n] * w0, d1[n] * w1, wp[m][n]);
            }
        }
        block_sync();
        // ---- the outputs, and the state behind the chunk
        {
            const int lane_here = here(lane), r = lane_here & 15, g = lane_here >> 4;
            u32x4 pf[2][kB][kB / 2], kt[3][kB / 2];
            float e[kB];
            auto read_keys = [&](int t) {
#pragma unroll
                for (int m = 0; m < kB / 2; ++m) kt[t % 3][m] = load_columns(km + 32 * m * KS + column_place(t, r, g), KS);
            };
            // a part of P's columns 32 m ..
            auto read_p = [&](int m, int part) {
#pragma unroll
                for (int tt = 2 * m; tt < kB; ++tt) pf[part][tt][m] = lds16(sp + (part * C + 16 * tt) * PP + p_place(r, 4 * m + g));
            };
            auto add_p = [&](int m, int u_part, int p_part) {
#pragma unroll
                for (int tt = 2 * m; tt < kB; ++tt)
#pragma unroll
                    for (int n = 0; n < NT; ++n) o[tt][n] = mfma(up[m][n][u_part], pf[p_part][tt][m], o[tt][n]);
            };
            if constexpr (OUT) {
#pragma unroll
                for (int tt = 0; tt < kB; ++tt) e[tt] = tok[kForQ * C + 16 * tt + r];
#pragma unroll
                for (int m = 0; m < kB / 2; ++m) read_p(m, 1);
            }
            const float dec = __builtin_amdgcn_exp2f(tok[kSumHigh * C + C - 1] + tok[kSumLow * C + C - 1]);
            read_keys(0);
            read_keys(1);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (OUT) {
#pragma unroll
            for (int tt = 0; tt < kB; ++tt)
#pragma unroll
                for (int n = 0; n < NT; ++n) o[tt][n] *= e[tt];
            // U's first part with P's second, whose places P's first then takes; and U's two with that
            add_p(0, 0, 1);
            __builtin_amdgcn_sched_barrier(0);
            read_p(0, 0);
            if constexpr (kB > 2) {
                add_p(1, 0, 1);
                __builtin_amdgcn_sched_barrier(0);
                read_p(1, 0);
            }
#pragma unroll
            for (int m = 0; m < kB / 2; ++m) add_p(m, 1, 0), add_p(m, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < KS / 16; ++t) {
                if (t + 2 < KS / 16) read_keys(t + 2);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = 0; n < NT; ++n) hs[t][n] *= dec;
#pragma unroll
                for (int m = 0; m < kB / 2; ++m)
#pragma unroll
                    for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                        for (int n = 0; n < NT; ++n) hs[t][n] = mfma(kt[t % 3][m], wp[m][n][part], hs[t][n]);
            }
            if (bad) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int from = __shfl(cut[n], 4 * g + i);
#pragma unroll
                        for (int tt = 0; tt < kB; ++tt)
                            if (16 * tt + r >= from) o[tt][n][i] = __builtin_nanf("");
                    }
                    if (cut[n] < C)
#pragma unroll
                        for (int t = 0; t < KS / 16; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) hs[t][n][i] = __builtin_nanf("");
                }
            }
            if constexpr (OUT) put_out(o, j);
        }
        block_sync();
    }

    // ---- the state behind the segment
    if (!OUT) {
        const Buffer buf = in_place();
        if (wide_place)
            each_state4(4, [&](f32x4_t &v, uint32_t at, int count) { store_state4<true, true>(buf, at, count, v); });
        else
            each_state4(4, [&](f32x4_t &v, uint32_t at, int count) { store_state4<true, false>(buf, at, count, v); });
        return;
    }
    if (p.state == nullptr || segment.index != segment.count - 1) return;
    const Buffer buf = in_pool();
    if (wide_pool)
        each_state4(kF32 ? 4 : 2, [&](f32x4_t &v, uint32_t at, int count) { store_state4<kF32, true>(buf, at, count, v); });
    else
        each_state4(kF32 ? 4 : 2, [&](f32x4_t &v, uint32_t at, int count) { store_state4<kF32, false>(buf, at, count, v); });
}

// The states ahead of every segment: S_0 the sequence's initial state, S_(i+1) = S_i M_i + B_i, in
// FP32.  A block has 16 rows p of a head and its waves share out the columns, two tiles each; S_i,
// which every wave needs whole, passes through LDS, and takes B_i's place in the workspace.
template <int KS>
__global__ __launch_bounds__(KS / 32 * kWave) void delta_join_kernel(const DeltaParams p, const ScanPlan plan, int ptiles) {
    constexpr int kTiles = KS / 16, kMine = 2, kPitch = KS + 4;
    __shared__ float ss[2][16 * kPitch];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, wave = uniform(threadIdx.x >> 6);
    // Blocks are dealt to the eight XCDs in turn: a head's, which read the same M, go to one of them.
    const int64_t heads = (int64_t)p.n * p.h;
    for_each_unit((heads + 7) / 8 * 8 * ptiles, [&](int64_t unit) {
        const int64_t turn = (unit >> 3) / ptiles, nh = turn * 8 + (unit & 7);
        if (nh >= heads) return;
        const int seq = uniform((int)(nh / p.h)), head = uniform((int)(nh - (int64_t)seq * p.h));
        const int p0 = uniform((int)((unit >> 3) - turn * ptiles)) * 16;
        int token0 = 0, len = p.t;
        if (p.starts != nullptr) {
            token0 = load_uniform(p.starts, seq);
            const int end = load_uniform(p.starts, seq + 1);
            if (token0 < 0 || token0 > end || end > p.t) return;
            len = end - token0;
        }
        if (len <= plan.seg) return;  // one segment
        const int count = uniform((len - 1) / plan.seg) + 1;
        const int place0 = p.starts != nullptr ? uniform(token0 / plan.seg) + seq : seq * plan.nseg;
        const int slot = uniform(route_row(p.idx, p.status, p.n, p.s, seq, lane));
        if (slot < 0) return;
        const bool init = p.state != nullptr && p.has_init != nullptr && p.has_init[seq] != 0;
        const int64_t head_floats = (int64_t)(p.p + p.k) * p.k;
        const bool mine = p0 + r < p.p;
        // tile t of this wave: columns k' = 16 (wave kMine + t) + 4 g + i of row p0 + r
        f32x4_t now[kMine];
#pragma unroll
        for (int t = 0; t < kMine; ++t) {
            const int c = 16 * (wave * kMine + t) + 4 * g;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                now[t][i] = init && mine && c + i < p.k
                                ? load_either(p.state, p.state_f32, slot * p.ss_s + ((int64_t)head * p.p + p0 + r) * p.k + c + i)
                                : 0.0f;
        }
        for (int j = 0; j < count; ++j) {
            const Buffer buf = make_buffer(p.workspace + (place0 + j) * place_floats(p) + head * head_floats,
                                           (uint32_t)(4 * head_floats));
            const bool more = j < count - 1;
            // this wave's columns of B and of M (row k = 16 m + 4 g + i, column r of the tile)
            f32x4_t next[kMine];
            float mm[kMine][kTiles][4];
            uint32_t at[kMine];
            int left[kMine];
#pragma unroll
            for (int t = 0; t < kMine; ++t) {
                const int c = 16 * (wave * kMine + t);
                at[t] = 4u * ((uint32_t)(p0 + r) * (uint32_t)p.k + (uint32_t)(c + 4 * g));
                left[t] = mine ? p.k - c - 4 * g : 0;
                next[t] = p.k % 4 == 0 ? load_state4<true, true>(buf, at[t], more ? left[t] : 0)
                                       : load_state4<true, false>(buf, at[t], more ? left[t] : 0);
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 16 * m + 4 * g + i;
                        const uint32_t from = more && row < p.k && c + r < p.k
                                                  ? 4u * ((uint32_t)(p.p + row) * (uint32_t)p.k + (uint32_t)(c + r)) : kNowhere;
                        mm[t][m][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buf, from, 0, kCached));
                    }
            }
            float *mat = ss[j & 1];
#pragma unroll
            for (int t = 0; t < kMine; ++t)
                *reinterpret_cast<f32x4_t *>(mat + r * kPitch + 16 * (wave * kMine + t) + 4 * g) = now[t];
            __syncthreads();
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
                const f32x4_t s = lds4f(mat + r * kPitch + 16 * m + 4 * g);
#pragma unroll
                for (int t = 0; t < kMine; ++t)
                    next[t] = mfma_f32(f32x4_t{mm[t][m][0], mm[t][m][1], mm[t][m][2], mm[t][m][3]}, s, next[t]);
            }
            // (in the place of B's columns, which this wave alone has read)
#pragma unroll
            for (int t = 0; t < kMine; ++t) {
                if (p.k % 4 == 0)
                    store_state4<true, true>(buf, at[t], left[t], now[t]);
                else
                    store_state4<true, false>(buf, at[t], left[t], now[t]);
                now[t] = next[t];
            }
        }
        __syncthreads();  // the next unit reuses the LDS arrays
    });
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

template <int KS, int C, int NT, int PARTS, bool OUT, bool WIDE>
uint64_t lds_allowed = 0;

template <int KS, int C, int NT, int PARTS, bool OUT, bool WIDE>
hipError_t launch(const DeltaParams &p, const ScanPlan &plan, hipStream_t stream) {
    using Z = Sizes<KS, C, NT, PARTS>;
    const auto tiles = [](int64_t rows) { return (rows + Z::kRowsP - 1) / Z::kRowsP; };
    ScanGrid grid;
    grid.tiles = (int32_t)(tiles(p.p) + (OUT ? 0 : tiles(p.k)));
    grid.each = p.h / p.g * grid.tiles;
    const int64_t groups = (int64_t)plan.slots * p.g;
    grid.runs = groups >= 32;
    const int64_t units = (grid.runs ? (groups + 7) / 8 * 8 : groups) * grid.each;
    auto kernel = delta_scan_kernel<KS, C, NT, PARTS, OUT, WIDE>;
    const hipError_t allowed =
        allow_lds(reinterpret_cast<const void *>(kernel), &lds_allowed<KS, C, NT, PARTS, OUT, WIDE>);
    if (allowed != hipSuccess) return allowed;
    const int64_t across = units < kMaxBlocks ? units : kMaxBlocks, deep = (units + across - 1) / across;
    if (deep > 65535) return hipErrorInvalidConfiguration;
    kernel<<<dim3((unsigned)across, (unsigned)deep), kScanBlock, Z::kBytes, stream>>>(p, plan, grid);
    return hipGetLastError();
}

template <int KS, int C, int NT, int PARTS, bool WIDE>
hipError_t launch_passes(const DeltaParams &p, const ScanPlan &plan, hipStream_t stream) {
    if (plan.split) {
        hipError_t err = launch<KS, C, NT, PARTS, false, WIDE>(p, plan, stream);
        if (err != hipSuccess) return err;
        const int ptiles = (p.p + 15) / 16;
        const int64_t units = ((int64_t)p.n * p.h + 7) / 8 * 8 * ptiles;
        delta_join_kernel<KS><<<dim3((unsigned)(units < kMaxBlocks ? units : kMaxBlocks)), KS / 32 * kWave, 0, stream>>>(p, plan, ptiles);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return launch<KS, C, NT, PARTS, true, WIDE>(p, plan, stream);
}

template <int KS, int C, int NT, bool WIDE>
hipError_t launch_state(const DeltaParams &p, const ScanPlan &plan, hipStream_t stream) {
    return p.state != nullptr && p.state_f32 ? launch_passes<KS, C, NT, 3, WIDE>(p, plan, stream)
                                             : launch_passes<KS, C, NT, 2, WIDE>(p, plan, stream);
}

// Whether rows at p with the given element strides start on 16 bytes, and a chunk's rows
// (b elements apart) span less than 2^31 bytes.
bool rows16(const void *p, int64_t a, int64_t b, int64_t c) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a % 8 == 0 && b % 8 == 0 && c % 8 == 0 && b < (1 << 23);
}

// How a call is cut up, by a model of its time: rounds of a block a CU, in which a chunk takes
// kChunkNs.  Blocks have 64 or 128 rows of a head's state (8 x 2048 tokens of 32 heads of 128: 255 us and 178;
// few heads fill more CUs with 64).  Where there are fewer blocks than CUs,
// cutting sequences into segments may save time: it takes a pass that makes M and B, with blocks
// for M's rows too and kStatesNs a chunk, a join of kJoinNs a segment, and two more launches, each
// with the latency of a block's first and last accesses, kCutNs.  (128 x 128, F32 states, cut into 5, 8
// and 16 segments, 128 rows a block: 16381 tokens of 16 heads 577, 380 and 322 us, where the whole took 1012 with 64 rows;
// into 4 and 8, 4096 tokens of 32 heads 207 and 183, whole 258; 1000 tokens of 32 heads into 4: 84, whole 71.)
constexpr int64_t kCus = 256;
constexpr int64_t kChunkNs[2] = {4200, 5000}, kStatesNs[2] = {4000, 4700}, kJoinNs = 2200, kCutNs = 40000;

ScanPlan make_plan(int64_t n, int64_t t, int64_t h, int64_t p, int64_t k, bool packed) {
    const int64_t c = k <= 128 ? 64 : 32;  // tokens of a chunk (64 of longer keys would take 192 KiB of LDS for q and k)
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    // (packed: of more than two sequences, the longest is taken for twice the mean)
    const int64_t whole = up(t, c) > 0 ? up(t, c) : 1, longest = packed && n > 2 ? up(2 * t, n * c) : up(t, c);
    const int64_t all = up(packed ? t : n * t, c);  // chunks in all
    ScanPlan plan;
    int64_t seg = whole, best = -1;
    for (int two = 0; two < (k <= 128 && p > 64 ? 2 : 1); ++two) {
        const int64_t tiles = up(p, two ? 128 : 64), key_tiles = up(k, two ? 128 : 64), rounds = up(n * h * tiles, kCus);
        const int64_t uncut = rounds * longest * kChunkNs[two];
        if (best < 0 || uncut < best) best = uncut, seg = whole, plan.two = two != 0;
        for (int64_t s = 2; rounds == 1 && s <= 64 && 4 * s <= longest; ++s) {
            const int64_t chunks = up(longest, s), pieces = up(all, chunks);
            const int64_t time = kCutNs + s * kJoinNs + chunks * (up(pieces * h * (tiles + key_tiles), kCus) * kStatesNs[two] +
                                                                  up(pieces * h * tiles, kCus) * kChunkNs[two]);
            if (time < best) best = time, seg = chunks, plan.two = two != 0;
        }
    }
    if (seg > whole) seg = whole;
    plan.seg = (int32_t)(seg * c);
    plan.nseg = (int32_t)up(whole, seg);
    plan.split = plan.nseg > 1;
    plan.slots = (int32_t)(packed ? t / (seg * c) + n : n * plan.nseg);
    return plan;
}

}  // namespace

int64_t delta_scan_workspace_floats(int64_t n, int64_t t, int64_t h, int64_t p, int64_t k, bool packed) {
    const ScanPlan plan = make_plan(n, t, h, p, k, packed);
    return plan.split ? plan.slots * (h * (p + k) * k) : 0;
}

hipError_t launch_delta_scan(const DeltaParams &p, hipStream_t stream, const char **kernel_name) {
    const ScanPlan plan = make_plan(p.n, p.t, p.h, p.p, p.k, p.starts != nullptr);
    const bool wide = p.p % 8 == 0 && p.k % 8 == 0 && rows16(p.q, p.qs_n, p.qs_t, p.qs_g) &&
                      rows16(p.key, p.ks_n, p.ks_t, p.ks_g) && rows16(p.v, p.vs_n, p.vs_t, p.vs_h) &&
                      rows16(p.out, p.os_n, p.os_t, p.os_h);
    *kernel_name = plan.split ? (wide ? "delta_scan_split" : "delta_scan_split_scalar")
                              : (wide ? "delta_scan" : "delta_scan_scalar");
    const bool two = plan.two;
    if (p.k <= 64) {
        if (two) return wide ? launch_state<64, 64, 2, true>(p, plan, stream) : launch_state<64, 64, 2, false>(p, plan, stream);
        return wide ? launch_state<64, 64, 1, true>(p, plan, stream) : launch_state<64, 64, 1, false>(p, plan, stream);
    }
    if (p.k <= 128) {
        if (two) return wide ? launch_state<128, 64, 2, true>(p, plan, stream) : launch_state<128, 64, 2, false>(p, plan, stream);
        return wide ? launch_state<128, 64, 1, true>(p, plan, stream) : launch_state<128, 64, 1, false>(p, plan, stream);
    }
    return wide ? launch_state<256, 32, 1, true>(p, plan, stream) : launch_state<256, 32, 1, false>(p, plan, stream);
}

}  // namespace dcconv
