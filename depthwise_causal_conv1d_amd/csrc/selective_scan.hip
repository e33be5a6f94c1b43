// The selective state-space recurrence over whole sequences for gfx950.
//
// Per head, with d_t = softplus(dt_t + dt_bias), a_t = d_t * a and the head's group
// holding B and C:
//
//     h_t = e^{a_t} h_{t-1} + d_t x_t B_t^T,   y_t = h_t C_t + D x_t,   out_t = y_t * silu(z_t)
//
// Chunks of Q = 32 tokens turn this into matrix products.  With c_t the prefix sum of
// a_t inside the chunk and H the state ahead of it,
//
//     Y  = (L o C B^T) X + e^{c} C H^T      L_tu = e^{c_t - c_u} d_u for u <= t, else 0
//     H' = e^{c_Q} H + (e^{c_Q - c_u} d_u X)^T B
//
// so a token and head cost about 32 (k + p) + 4 p k operations on the matrix cores
// instead of 5 p k on the vector units, and x, z and out move once.
//
// A wave owns 16 of a head's p and all of the state's k: H stays in its FP32
// accumulators for the whole sequence, already in the lane order that the next
// product reads it in (below).  A block is four such waves of one group (one head at
// p = 64), which share the chunk's B and C in LDS and the products C B^T: the lower
// triangle's three tiles, scaled for each head of the block, are shared out.  (Blocks of
// eight and twelve waves, which share more, took 344 and 244 us where four took 229.)
//
// Two barriers a chunk: waves finish chunk i (the product with X, H', the outputs); then
// they put chunk i + 1's x and z and chunk i + 2's B and C into LDS, request the chunk
// behind each, and start chunk i + 1 (C H^T, its tiles of C B^T).  So B and C are kept in
// two places in LDS, x, z (and the outputs, in z's place) and L o C B^T in one: 49 KiB
// at k = 128, and 150 registers, for three blocks a CU.  (Four blocks need 128 registers
// and spill: 410 to 440 us against 200.  Chunks of 64 tokens need more of both and took
// 286 us where 32 took 270.)  x, z and the outputs move in whole rows of the block, 128
// bytes at p = 64: a wave's own 32 bytes a row cost 256 us against 229.
//
// What bounds it.  8 x 2048 tokens of 96 heads, 64 x 128 in 8 groups, with BF16 states:
// 200 us, 687 MB at 3.4 TB/s and 64 GFLOP at 320 TFLOP/s, where the memory's rate would
// allow 117 us.  The vector units are busy for 54 % of the time, LDS for 44 %, the matrix
// cores for 15 %: a chunk is a chain of products, exponentials and LDS round trips, about
// 3.1 us long, with 290 vector, 122 scalar and 55 LDS instructions around a wave's 21
// products, and twelve waves a CU do not hide all of it.  16 packed sequences of up to
// 1967 tokens (60 heads, F32 states): 188 us, 427 MB at 2.3 TB/s, the longest sequence's
// chunks one after the other, and 10 us of state pass and join without a sequence to cut.  One sequence of 16381 tokens of 24 heads: 96 us, 119 MB, of
// them about 38 the segments' states and 10 the join.  37 tokens: 10.3 us, two chunks' latency and the launch.
//
// Layouts.  v_mfma_f32_16x16x32_bf16 takes, in lane l with r = l & 15 and g = l >> 4,
// row (column) r of an operand at inner indices 8 g .. 8 g + 7, and leaves column r,
// rows 4 g .. 4 g + 3 of the result.  The order of an operand's rows is free, and so is
// the inner indices' if both operands agree.  So the state columns of result tiles 2 m
// and 2 m + 1 interleave by four (tile 2 m + f, row 4 g + i is column 32 m + 8 g + 4 f
// + i): together the two tiles of H are an operand as they are, against C's rows read
// 16 bytes at a time.  B and x, needed with tokens as the inner index too, are read
// through the transposing load, four rows (tokens) at a time: there the inner order is
// 4 g .. of the first and of the second 16 of 32 tokens, and L o C B^T is written in
// that order.  LDS rows are 32 bytes longer than a multiple of 64: measured with
// sixteen waves, 16-byte row reads then take 4.5 cycles (32 at a pitch of 256 bytes)
// and transposing loads 4.2 (16).
//
// Precision: B, C and x are BF16 as given; sums, prefix sums, exponentials and H are
// FP32.  The scaled products L o C B^T and the copy of H that C reads are rounded to
// BF16 (each about as much as the BF16 output's own rounding).  The scaled x that
// enters H is split into SPLIT BF16 parts whose products are added up: three carry all
// 24 bits, for states that are handed out in FP32.  One part is what a BF16 state needs:
// against 64 bits the outputs' error is then 0.0023 of their size, 0.0019 with three and
// 0.0017 for the best rounding (two parts: 222 us where one took 209).  The lower parts may
// be zero or of the other sign, which makes a NaN of an infinity of B.  (Telling such
// chunks and adding their terms one by one, as for x, kept the infinity and took 196 to 202
// us where the packed sequences above take 187, and 98 to 103 where the long one takes 94.)
#include "selective_common.h"

namespace dcconv {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kChunk = 32;
constexpr int kScanWaves = 4;
constexpr int kScanBlock = kWave * kScanWaves;
constexpr int kUnitP = 16;           // p of a wave
constexpr int kBlockP = kScanWaves * kUnitP;  // p of a block
constexpr int kPPitch = kChunk + 16;   // LDS row pitches of L o C B^T,
constexpr int kXPitch = kBlockP + 8;   // and of x and z
constexpr int kStepRows = 4;         // per token and head: c, d, the weight into H, e^c

// How a call is cut up; the same on the host and in every kernel.
struct ScanPlan {
    int32_t seg;     // tokens of a segment (a multiple of kChunk)
    int32_t nseg;    // segments of a sequence (batch form)
    int32_t slots;   // segments in all; packed: an upper bound, some empty
    int32_t np;      // waves a head takes: ceil(p / 16)
    int32_t quads;   // blocks a group takes
    int32_t run;     // of them that follow each other on one XCD
    int32_t parts;   // runs a group takes
    int32_t heads;   // most heads of one block
    int32_t places;  // states in the workspace
    bool sparse;     // packed: see first_place
    bool split;      // some sequence may have more than one segment
};

__device__ __forceinline__ f32x4_t mfma(u32x4 a, u32x4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

__device__ __forceinline__ u32x4 lds16(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

// An operand whose inner index runs over rows in LDS: lane 4 q + j of the 16 that
// share g gives the address of its columns' piece j (four of them) in row 4 g + q, and
// gets column 4 q + j of rows 4 g .. 4 g + 3, and of the 16 rows further down.
__device__ __forceinline__ u32x4 load_columns(const uint16_t *at, int pitch) {
    typedef __attribute__((address_space(3))) s16x4_t *Lds;
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(s16x4_t *)at));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(s16x4_t *)(at + 16 * pitch)));
    return u32x4{a[0], a[1], b[0], b[1]};
}

constexpr float kHuge = 3.0e38f;
constexpr float kNone = -160.0f;
__device__ __forceinline__ bool is_finite(float v) { return __builtin_fabsf(v) < __builtin_inff(); }

// acc + the two BF16 values of w.
__device__ __forceinline__ float sum_pair(uint32_t w, float acc) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 ones = __builtin_bit_cast(bf16x2, 0x3f803f80u);
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), ones, acc, false);
}

// w with a value that is no number, or infinite, replaced by zero.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
    if (!is_finite(lo_f32(w))) w &= 0xffff0000u;
    if (!is_finite(hi_f32(w))) w &= 0x0000ffffu;
    return w;
}

// v, which all lanes of the wave agree on, in a scalar register.  What was divided by
// a run-time number has passed through vector registers; a buffer whose base depends
// on it would be loaded from in a loop over the lanes' bases.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

struct Segment {
    int seq, first, last, index, count;  // tokens [first, last) of sequence seq; segment `index` of `count`
    int token0;                          // the sequence's first token on the t axis
    int place;                           // of the workspace (count > 1)
    bool ok;
};

// The workspace's place for the first segment of sequence seq, which starts at token a and
// is cut; the others follow.  Batch form: that of the segment's position.  Packed, either
// likewise, with a place for each sequence's last, partial segment; or, where there are
// many sequences, 2 (a / seg): the sequence of c > 1 segments is more than (c - 1) seg
// tokens long, so the next cut one starts at 2 (c - 1) >= c places further or more.
__device__ __forceinline__ int first_place(const ScanPlan &plan, bool packed, int seq, int a) {
    if (!packed) return seq * plan.nseg;
    const int before = uniform(a / plan.seg);
    return plan.sparse ? 2 * before : before + seq;
}

// The segment at position u: sequence i has positions i * nseg .. in the batch
// form, and starts[i] / seg + i .. in the packed form (which leaves room for every
// sequence's last, partial segment).
__device__ __forceinline__ Segment find_segment(const SelectiveScanParams &p, const ScanPlan &plan, int u) {
    Segment s;
    int len;
    if (p.starts == nullptr) {
        s.seq = uniform(u / plan.nseg);
        s.index = u - s.seq * plan.nseg;
        s.token0 = 0;
        len = p.t;
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
    s.place = first_place(plan, p.starts != nullptr, s.seq, s.token0) + s.index;
    s.first = s.ok ? s.index * plan.seg : 0;
    s.last = s.ok ? s.first + min(len - s.first, plan.seg) : 0;
    return s;
}

// Reports a sequence table that is not 0 = starts[0] <= ... <= starts[n] = t.
__device__ __forceinline__ void check_table(const SelectiveScanParams &p) {
    if (p.starts == nullptr || p.status == nullptr) return;
    bool bad = false;
    for (int i = threadIdx.x; i <= p.n; i += kScanBlock) {
        const int a = p.starts[i];
        bad |= a < 0 || a > p.t || (i == 0 && a != 0) || (i == p.n ? a != p.t : p.starts[i + 1] < a);
    }
    if (bad) atomicOr(p.status, DCCONV_DEV_BAD_SEQ);
}

// Sums over the first 32 lanes of a wave: of the lanes up to this one, and of the lanes
// behind it (each formed from small to large distances, so that the decay of a
// recent token is not the difference of two long sums).
template <int CTRL>
__device__ __forceinline__ float dpp_shift(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
__device__ __forceinline__ void wave_sums(float v, int lane, float *upto, float *behind, float *total) {
    float u = v, b = v;  // inside each row of 16 lanes, by DPP shifts
    u += dpp_shift<0x111>(u), b += dpp_shift<0x101>(b);
    u += dpp_shift<0x112>(u), b += dpp_shift<0x102>(b);
    u += dpp_shift<0x114>(u), b += dpp_shift<0x104>(b);
    u += dpp_shift<0x118>(u), b += dpp_shift<0x108>(b);
    const float r0 = lane_value(u, 15), r1 = lane_value(u, 31);
    *upto = u + (lane >= 16 ? r0 : 0.0f);
    *total = r0 + r1;
    b = dpp_shift<0x101>(b);  // the lanes behind this one; zero for a row's last
    *behind = b + (lane < 16 ? r1 : 0.0f);
}

constexpr uint32_t kNowhere = 0x80000000u;  // past the end of every buffer

// One operand's rows of a chunk, `stride` elements apart and `width` long: a lane moves
// eight values, of which `count` exist, from column `col` of rows row0, row0 + step, ...
// WIDE moves them at once (16 bytes) through a buffer that ends with the chunk's last row, so that what lies
// behind it reads as zeros and is not written.
template <bool WIDE>
struct ChunkRows {
    const uint16_t *base;  // wave-uniform: the chunk's first row
    int64_t stride, col;
    int32_t step, row0, count, rows;
    uint32_t at0, hop, width;
    Buffer buf;
    __device__ __forceinline__ ChunkRows(const uint16_t *first, int64_t stride, int step, int64_t width, int row,
                                         int64_t col, int count)
        : base(first), stride(stride), col(col), step(step), row0(row), count(count), width(2u * (uint32_t)width) {
        const uint32_t bytes = 2u * (uint32_t)stride;
        at0 = count > 0 ? (uint32_t)row * bytes + 2u * (uint32_t)col : kNowhere;
        hop = (uint32_t)step * bytes;
    }
    __device__ __forceinline__ void begin(int n) {
        rows = n;
        if (WIDE) buf = make_buffer(base, n > 0 ? (uint32_t)(n - 1) * 2u * (uint32_t)stride + width : 0u);
    }
    __device__ __forceinline__ void advance() { base += kChunk * stride; }
    // eight values of row row0 + q * step
    __device__ __forceinline__ void load(uint32_t (&w)[4], int q) const {
        if (WIDE) {
            buffer_load_words<4, kCached>(buf, row0 + q * step < rows ? at0 + (uint32_t)q * hop : kNowhere, w);
            return;
        }
        const int row = row0 + q * step;
        const uint16_t *from = base + row * stride + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (row < rows && i < count) w[i >> 1] |= (uint32_t)from[i] << (16 * (i & 1));
    }
    __device__ __forceinline__ void store(uint32_t (&w)[4]) const {
        if (WIDE) {
            buffer_store_words<4, kCached>(w, buf, row0 < rows ? at0 : kNowhere);
            return;
        }
        if (row0 >= rows) return;
        uint16_t *to = const_cast<uint16_t *>(base) + row0 * stride + col;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) to[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
};

// v, not known to be the same as anywhere else: addresses formed from it are formed
// where they are used, instead of being kept in registers from outside of a loop.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The kernel's arguments, read again: what is used only once a loop is done need not
// occupy scalar registers throughout it.
__device__ __forceinline__ const SelectiveScanParams &reread(const SelectiveScanParams &p) {
    typedef const __attribute__((address_space(4))) SelectiveScanParams *Args;
    Args args = (Args)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(args));
    return *(const SelectiveScanParams *)args;
}

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
        if (i < count)
            v[i] = f32 ? static_cast<const float *>(s)[at + i]
                       : bf16_bits_to_f32(static_cast<const uint16_t *>(s)[at + i]);
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

// The state column of row 4 g of H's tile m.
__device__ __forceinline__ int column(int m, int g) { return 32 * (m >> 1) + 8 * g + 4 * (m & 1); }

// Whether the pool's rows of four state values start on whole 8 or 16 bytes.
__device__ __forceinline__ bool wide_state(const SelectiveScanParams &p) {
    return p.k % 4 == 0 && p.ss_s % 4 == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0;
}

// OUT: the outputs and final states.  Otherwise the state that each segment but a
// sequence's last builds up from zero, and its decay, for the join.
template <int KS, int SPLIT, bool OUT, bool WIDE>
__global__ __launch_bounds__(kScanBlock, KS <= 128 ? 3 : 2) void selective_scan_kernel(const SelectiveScanParams p,
                                                                                      const ScanPlan plan) {
    constexpr int kPitch = KS + 16;
    constexpr int kTiles = KS / 16, kSteps = KS / 32;
    constexpr int kAcross = KS / 8;  // 16-byte pieces of a row of B (of C)
    constexpr int kPieces = (kChunk * kAcross + kScanBlock - 1) / kScanBlock;  // of them a thread stages
    extern __shared__ u32x4 smem[];
    uint16_t *sb = reinterpret_cast<uint16_t *>(smem);            // [2][kChunk][kPitch]
    uint16_t *sc = sb + 2 * kChunk * kPitch;                      // [2][kChunk][kPitch]
    uint16_t *sx_all = sc + (OUT ? 2 * kChunk * kPitch : 0);      // [kChunk][kXPitch]
    uint16_t *sz_all = sx_all + kChunk * kXPitch;                 // likewise: z, and then the outputs
    float *steps = reinterpret_cast<float *>(sz_all + (OUT ? kChunk * kXPitch : 0));  // [2][heads][kStepRows][kChunk]
    uint16_t *sp = reinterpret_cast<uint16_t *>(steps + 2 * plan.heads * kStepRows * kChunk);  // [heads][kChunk][kPPitch]

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint16_t *sx = sx_all + wave * kUnitP;
    uint16_t *sz = sz_all + wave * kUnitP;
    const int per_group = uniform(p.h / p.g), units = per_group * plan.np;

    if (OUT && blockIdx.x == 0 && blockIdx.y == 0) check_table(p);
    // the tile above the diagonal that the product over 32 tokens reads: zeros for good
    if (OUT)
        for (int i = tid; i < plan.heads * 16 * 16; i += kScanBlock) {
            const int mat = i >> 8, row = (i >> 4) & 15, col = i & 15;
            sp[(mat * kChunk + row) * kPPitch + 8 * (col >> 2) + 4 + (col & 3)] = 0;
        }

    // Blocks are dealt to the eight XCDs in turn: a run of a group's blocks, which read
    // the same B and C, goes to one of them, whose L2 then fetches those once.
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int turn = uniform((int)((block >> 3) / plan.run));
    const int64_t run = (int64_t)turn * 8 + (block & 7);
    const int64_t ug = run / plan.parts;
    const int quad = uniform((int)((block >> 3) - (int64_t)turn * plan.run + (run - ug * plan.parts) * plan.run));
    const int u = uniform((int)(ug / p.g)), group = uniform((int)(ug - (int64_t)u * p.g));
    if (u >= plan.slots || quad >= plan.quads) return;
    const Segment seg = find_segment(p, plan, u);
    if (!seg.ok || (!OUT && seg.index == seg.count - 1)) return;

    const int last_unit = min(quad * kScanWaves + kScanWaves, units) - 1;
    const int mine = min(quad * kScanWaves + wave, last_unit);
    const bool valid = quad * kScanWaves + wave == mine;
    const int first_head = uniform(quad * kScanWaves / plan.np);
    const int heads = uniform(last_unit / plan.np) - first_head + 1;
    const int my_head = uniform(mine / plan.np);  // of the group
    const int head_slot = my_head - first_head;
    const int head = group * per_group + my_head;
    const int p0 = (mine - my_head * plan.np) * kUnitP;
    const int pcount = valid ? min(kUnitP, p.p - p0) : 0;

    const int slot = uniform(route_row(p.idx, p.status, p.n, p.s, seg.seq, lane));
    if (slot < 0) {  // a padding sequence: zeros, and no state moves
        if (OUT)
            for (int t = seg.first; t < seg.last; ++t)
                if (lane < pcount)
                    p.out[seg.seq * p.os_n + ((int64_t)seg.token0 + t) * p.os_t + head * p.os_h + p0 + lane] = 0;
        return;
    }

    // ---- the state ahead of the segment: tile m, rows k = column(m, g) + i, column p = r
    f32x4_t hs[kTiles];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) hs[m] = f32x4_t{0, 0, 0, 0};
    const bool from_ws = seg.count > 1;
    if (OUT && (from_ws || (p.state != nullptr && p.has_init != nullptr && p.has_init[seg.seq] != 0))) {
        const void *src = from_ws ? p.workspace + seg.place * (int64_t)p.h * p.p * p.k : p.state;
        const bool f32 = from_ws || p.state_f32, wide = from_ws ? p.k % 4 == 0 : wide_state(p);
        const int64_t at = (from_ws ? 0 : slot * p.ss_s) + ((int64_t)head * p.p + p0 + r) * p.k;
        if (r < pcount)
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
                hs[m] = load_state4(src, f32, wide, at + column(m, g), p.k - column(m, g));
    }

    // ---- the operands' rows, shared out over the block.  Eight threads move the 64
    // channels of a token that the block's waves own, two for a wave's 16.
    const int64_t tok = (int64_t)seg.token0 + seg.first;
    constexpr int kRowsPerPiece = kScanBlock / kAcross;
    ChunkRows<WIDE> rb(p.b + seg.seq * p.bs_n + tok * p.bs_t + group * p.bs_g, p.bs_t, kRowsPerPiece, p.k, tid / kAcross,
                       tid % kAcross * 8, p.k - tid % kAcross * 8);
    ChunkRows<WIDE> rc(p.c + seg.seq * p.cs_n + tok * p.cs_t + group * p.cs_g, p.cs_t, kRowsPerPiece, p.k, tid / kAcross,
                       tid % kAcross * 8, p.k - tid % kAcross * 8);
    constexpr int kMoves = kBlockP / 8;
    const int move_row = tid / kMoves, move_col = tid % kMoves * 8;
    const int theirs = min(quad * kScanWaves + move_col / kUnitP, last_unit), their_head = theirs / plan.np;
    const int their_p = (theirs - their_head * plan.np) * kUnitP + move_col % kUnitP;
    const int their_count = quad * kScanWaves + move_col / kUnitP == theirs ? max(p.p - their_p, 0) : 0;
    const auto mover = [&](const uint16_t *base, int64_t sn, int64_t st, int64_t sh) {
        return ChunkRows<WIDE>(base + seg.seq * sn + tok * st + group * per_group * sh, st, kChunk,
                               (per_group - 1) * sh + p.p, move_row, their_head * sh + their_p, their_count);
    };
    ChunkRows<WIDE> rx = mover(p.x, p.xs_n, p.xs_t, p.xs_h), rz = mover(p.z, p.zs_n, p.zs_t, p.zs_h);
    ChunkRows<WIDE> ro = mover(p.out, p.os_n, p.os_t, p.os_h);
    const float skip = OUT && p.d_skip != nullptr ? p.d_skip[head] : 0.0f;
    const bool gated = p.z != nullptr;

    // Every fetch is unconditional (of no rows behind the last chunk): registers that only
    // one of two paths loads are waited for where the paths join.
    uint32_t nb[kPieces][4], nc[kPieces][4], nx[4], nz[4];
    auto fetch_bc = [&](int left) {
        const int n = max(min(left, kChunk), 0);
        rb.begin(n);
#pragma unroll
        for (int q = 0; q < kPieces; ++q) rb.load(nb[q], q);
        rb.advance();
        if (OUT) {
            rc.begin(n);
#pragma unroll
            for (int q = 0; q < kPieces; ++q) rc.load(nc[q], q);
            rc.advance();
        }
    };
    auto stage_bc = [&](int slot2) {
        const int row = tid / kAcross, col = tid % kAcross * 8;
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            if (kChunk * kAcross < kScanBlock && row >= kChunk) break;
            const int to = (q * kRowsPerPiece + row) * kPitch + col;
            *reinterpret_cast<u32x4 *>(sb + slot2 * kChunk * kPitch + to) = u32x4{nb[q][0], nb[q][1], nb[q][2], nb[q][3]};
            if (OUT)
                *reinterpret_cast<u32x4 *>(sc + slot2 * kChunk * kPitch + to) = u32x4{nc[q][0], nc[q][1], nc[q][2], nc[q][3]};
        }
    };
    auto fetch_x = [&](int left) {
        rx.begin(max(min(left, kChunk), 0));
        rx.load(nx, 0);
        rx.advance();
    };
    auto stage_x = [&]() {
        *reinterpret_cast<u32x4 *>(sx_all + move_row * kXPitch + move_col) = u32x4{nx[0], nx[1], nx[2], nx[3]};
    };
    auto fetch_z = [&](int left) {
        if (!OUT || !gated) return;
        rz.begin(max(min(left, kChunk), 0));
        rz.load(nz, 0);
        rz.advance();
    };
    auto stage_z = [&]() {
        if (OUT && gated)
            *reinterpret_cast<u32x4 *>(sz_all + move_row * kXPitch + move_col) = u32x4{nz[0], nz[1], nz[2], nz[3]};
    };
    // the outputs that the waves have left in place of z
    auto put_out = [&](int rows) {
        if (!OUT) return;
        const u32x4 v = lds16(sz_all + move_row * kXPitch + move_col);
        uint32_t w[4] = {v[0], v[1], v[2], v[3]};
        ro.begin(rows);
        ro.store(w);
        ro.advance();
    };

    // ---- the steps of a head's chunk: the last waves (which have the fewest tiles of
    // C B^T) take a head each
    const int job = kScanWaves - 1 - wave;
    const bool has_job = job < heads;
    const int job_head = group * per_group + first_head + min(job, heads - 1);
    const float a2 = p.a[job_head] * kLog2e;
    const float dt_bias = p.dt_bias != nullptr ? p.dt_bias[job_head] : 0.0f;
    int64_t dt_at = seg.seq * p.ds_n + tok * p.ds_t + job_head;
    float decay_sum = 0.0f;
    // (as it is in memory: converting it here would wait for it)
    auto fetch_step = [&](int left) {
        uint32_t v = 0;
        const int l = here(lane);
        if (has_job && l < min(left, kChunk))
            v = p.dt_f32 ? static_cast<const uint32_t *>(p.dt)[dt_at + l * p.ds_t]
                         : static_cast<const uint16_t *>(p.dt)[dt_at + l * p.ds_t];
        dt_at += kChunk * p.ds_t;
        return v;
    };
    auto put_steps = [&](uint32_t v, int left, int s_slot) {
        float d = __uint_as_float(p.dt_f32 ? v : v << 16) + dt_bias;
        if (p.dt_softplus) d = softplus(d);
        if (lane >= min(left, kChunk)) d = 0.0f;
        // 2^kNone is zero: a step that decays more counts as that, so that the differences of
        // the sums of the steps behind it keep their bits (a NaN stays)
        float rate = d * a2;
        if (rate < kNone) rate = kNone;
        float upto, behind, total;
        wave_sums(rate, lane, &upto, &behind, &total);
        float *to = steps + ((s_slot * plan.heads + job) * kStepRows) * kChunk + lane;
        if (lane < kChunk) {
            to[0] = upto;
            to[kChunk] = d;
            to[2 * kChunk] = d * __builtin_amdgcn_exp2f(behind);
            to[3 * kChunk] = __builtin_amdgcn_exp2f(upto);
        }
        decay_sum += total;
    };

    // ---- the first half of a chunk: y = e^c C H^T, and this wave's tiles of L o C B^T
    f32x4_t y[2];
    auto start = [&](int slot2) {
        const uint16_t *bm = sb + slot2 * kChunk * kPitch, *cm = sc + slot2 * kChunk * kPitch;
        const float *st = steps + slot2 * plan.heads * kStepRows * kChunk;
        const uint16_t *ca = cm + r * kPitch + 8 * g;
        // (reads ahead of the products that use them: left to itself the compiler waits for
        // each read behind the product before)
        u32x4 cf[kSteps][2];
        float e[2];
#pragma unroll
        for (int m = 0; m < kSteps; ++m)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) cf[m][tt] = lds16(ca + 16 * tt * kPitch + 32 * m);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            e[tt] = st[(head_slot * kStepRows + 3) * kChunk + 16 * tt + r];
            y[tt] = f32x4_t{0, 0, 0, 0};
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < kSteps; ++m) {
            const f32x4_t h0 = hs[2 * m], h1 = hs[2 * m + 1];
            const u32x4 hb = {pack_bf16x2(h0[0], h0[1]), pack_bf16x2(h0[2], h0[3]), pack_bf16x2(h1[0], h1[1]),
                              pack_bf16x2(h1[2], h1[3])};
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) y[tt] = mfma(hb, cf[m][tt], y[tt]);
        }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) y[tt] *= e[tt];

        for (int it = wave; it < 3 * heads; it += kScanWaves) {
            const int hd = it / 3, e = it - 3 * hd;
            const int tt = e > 0, ut = e > 1;
            f32x4_t acc = {0, 0, 0, 0};
            u32x4 bf[kSteps], cf[kSteps];
#pragma unroll
            for (int m = 0; m < kSteps; ++m) {
                bf[m] = lds16(bm + (16 * ut + r) * kPitch + 32 * m + 8 * g);
                cf[m] = lds16(cm + (16 * tt + r) * kPitch + 32 * m + 8 * g);
            }
            const int t = 16 * tt + r, u0 = 16 * ut + 4 * g;
            const float *sh = st + hd * kStepRows * kChunk;
            const f32x4_t cu = *reinterpret_cast<const f32x4_t *>(sh + u0);
            const f32x4_t du = *reinterpret_cast<const f32x4_t *>(sh + kChunk + u0);
            const float ct = sh[t];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < kSteps; ++m) acc = mfma(bf[m], cf[m], acc);
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = u0 + i <= t ? acc[i] * __builtin_amdgcn_exp2f(ct - cu[i]) * du[i] : 0.0f;
            *reinterpret_cast<u32x2 *>(sp + (hd * kChunk + t) * kPPitch + 8 * g + 4 * ut) =
                u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
    };

    // ---- the second half: y += (L o C B^T) X, H' = e^{c_Q} H + (scaled x)^T B, and the outputs
    auto finish = [&](int slot2) {
        const uint16_t *bm = sb + slot2 * kChunk * kPitch;
        const uint16_t *pm = sp + head_slot * kChunk * kPPitch;
        const float *ss = steps + (slot2 * plan.heads + head_slot) * kStepRows * kChunk;
        u32x4 xf = load_columns(sx + (4 * g + (r >> 2)) * kXPitch + 4 * (r & 3), kXPitch);
        u32x4 pf[2];
        u32x2 xv[2], zv[2];
        if (OUT) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                pf[tt] = lds16(pm + (16 * tt + r) * kPPitch + 8 * g);
                xv[tt] = *reinterpret_cast<const u32x2 *>(sx + (16 * tt + r) * kXPitch + 4 * g);
                zv[tt] = *reinterpret_cast<const u32x2 *>(sz + (16 * tt + r) * kXPitch + 4 * g);
            }
        }
        const f32x4_t w0 = *reinterpret_cast<const f32x4_t *>(ss + 2 * kChunk + 4 * g);
        const f32x4_t w1 = *reinterpret_cast<const f32x4_t *>(ss + 2 * kChunk + 16 + 4 * g);
        const float dec = ss[3 * kChunk + kChunk - 1];
        const uint16_t *ba = bm + (4 * g + (r >> 2)) * kPitch + 8 * (r & 3);
        constexpr int kAhead = 2;  // tiles of B read at a time (4: 1 to 2 % slower, 8: 3 to 6 %)
        u32x4 bt[kAhead];
#pragma unroll
        for (int m = 0; m < kAhead && m < kTiles; ++m) bt[m] = load_columns(ba + 32 * (m >> 1) + 4 * (m & 1), kPitch);
        __builtin_amdgcn_sched_barrier(0);
        // An infinity or NaN of a later token must not meet the zeros of L: it is taken
        // out of the matrix products and its terms are added one by one.
        float probe = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) probe = sum_pair(xf[i], probe);
        const bool bad = __any(!(__builtin_fabsf(probe) < kHuge));
        if (bad) {
#pragma unroll
            for (int i = 0; i < 4; ++i) xf[i] = finite_pair(xf[i]);
        }
        if constexpr (OUT) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) y[tt] = mfma(xf, pf[tt], y[tt]);
            if (bad) {
                const int rr = here(r), gg = here(g);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
                    for (int q = 0; q <= 16 * tt + rr; ++q)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float v = bf16_bits_to_f32(sx[q * kXPitch + 4 * gg + i]);
                            if (!is_finite(v))
                                y[tt][i] += bf16_bits_to_f32(pm[(16 * tt + rr) * kPPitch + 2 * (q & 12) + ((q & 16) >> 2) + (q & 3)]) * v;
                        }
            }
        }
        u32x4 xw[SPLIT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v0 = lo_f32(xf[i]) * (i < 2 ? w0[2 * i] : w1[2 * i - 4]);
            float v1 = hi_f32(xf[i]) * (i < 2 ? w0[2 * i + 1] : w1[2 * i - 3]);
#pragma unroll
            for (int part = 0; part < SPLIT; ++part) {
                const uint32_t h = pack_bf16x2(v0, v1);
                xw[part][i] = h;
                v0 -= lo_f32(h);
                v1 -= hi_f32(h);
            }
        }
#pragma unroll
        for (int m0 = 0; m0 < kTiles; m0 += kAhead) {
            if (m0 > 0) {
#pragma unroll
                for (int m = 0; m < kAhead; ++m) bt[m] = load_columns(ba + 32 * ((m0 + m) >> 1) + 4 * (m & 1), kPitch);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int m = m0; m < m0 + kAhead && m < kTiles; ++m) {
                hs[m] *= dec;
#pragma unroll
                for (int part = SPLIT - 1; part >= 0; --part) hs[m] = mfma(bt[m - m0], xw[part], hs[m]);
            }
        }
        if (bad) {
            const int rr = here(r), gg = here(g);
            for (int q = 0; q < kChunk; ++q) {
                const float v = bf16_bits_to_f32(sx[q * kXPitch + rr]);
                if (is_finite(v)) continue;
                const float w = ss[2 * kChunk + q] * v;
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) hs[m][i] += w * bf16_bits_to_f32(bm[q * kPitch + column(m, gg) + i]);
            }
        }
        // skip and gate: four consecutive p of a token a lane, left in LDS where its z was
        if constexpr (OUT) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                float o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = __builtin_fmaf(skip, (i & 1) ? hi_f32(xv[tt][i >> 1]) : lo_f32(xv[tt][i >> 1]), y[tt][i]);
                if (gated) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] *= silu((i & 1) ? hi_f32(zv[tt][i >> 1]) : lo_f32(zv[tt][i >> 1]));
                }
                *reinterpret_cast<u32x2 *>(sz + (16 * tt + r) * kXPitch + 4 * g) =
                    u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
            }
        }
    };

    int left = seg.last - seg.first;  // tokens from the current chunk on
    {
        const uint32_t step0 = fetch_step(left), step1 = fetch_step(left - kChunk);
        fetch_bc(left);
        fetch_x(left);
        fetch_z(left);
        if (has_job) put_steps(step0, left, 0);
        stage_bc(0);
        stage_x();
        stage_z();
        fetch_bc(left - kChunk);
        fetch_x(left - kChunk);
        fetch_z(left - kChunk);
        if (has_job) put_steps(step1, left - kChunk, 1);
    }
    uint32_t step = fetch_step(left - 2 * kChunk);
    __syncthreads();
    if constexpr (OUT) start(0);
    stage_bc(1);
    fetch_bc(left - 2 * kChunk);
    __syncthreads();
    for (int b = 0; left > 0; left -= kChunk, b ^= 1) {
        // finishing a chunk, and putting the next into LDS, ahead of other blocks' starts
        // (3 to 6 % on the packed and the batch form)
        __builtin_amdgcn_s_setprio(1);
        finish(b);
        __syncthreads();  // chunk i's places are free
        put_out(min(left, kChunk));
        stage_x();  // of chunk i + 1
        stage_z();
        stage_bc(b);  // of chunk i + 2
        fetch_x(left - 2 * kChunk);
        fetch_z(left - 2 * kChunk);
        fetch_bc(left - 3 * kChunk);
        __builtin_amdgcn_s_setprio(0);
        if constexpr (OUT) start(b ^ 1);
        if (has_job) put_steps(step, left - 2 * kChunk, b);
        step = fetch_step(left - 3 * kChunk);
        __syncthreads();
    }

    // ---- the state behind the segment
    const SelectiveScanParams &late = reread(p);
    if (OUT && (late.state == nullptr || seg.index != seg.count - 1)) return;
    const int64_t hpk = (int64_t)late.h * late.p * late.k;
    void *to = OUT ? late.state : late.workspace;
    const bool f32 = !OUT || late.state_f32, wide = OUT ? wide_state(late) : late.k % 4 == 0;
    const int64_t at = (OUT ? slot * late.ss_s : (seg.place + 1) * hpk) + ((int64_t)head * late.p + p0 + here(r)) * late.k;
    const int gg = here(g);
    if (r < pcount)
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
            store_state4(to, f32, wide, at + column(m, gg), late.k - column(m, gg), hs[m]);
    if (!OUT && has_job && lane == 0)
        late.workspace[plan.places * hpk + (int64_t)(seg.place + 1) * late.h + job_head] = __builtin_amdgcn_exp2f(decay_sum);
}

// The states ahead of every segment, in place: the workspace's place behind a segment's
// holds what that segment built up from zero and its decay.  A thread carries VEC
// neighbouring values along a sequence's segments, and reads kJoinAhead segments at a
// time: as the values it writes lie in the same array, reads one by one would each wait
// for the write before (the whole call on 16381 tokens of 24 heads: 98.1 us reading one,
// 94.8 four, 94.5 eight, 95.4 sixteen).
constexpr int kJoinBlock = 256;
constexpr int kJoinAhead = 8;
template <int VEC>
__global__ __launch_bounds__(kJoinBlock) void selective_join_kernel(const SelectiveScanParams p, const ScanPlan plan,
                                                                    int blocks_per_seq) {
    const int64_t hpk = (int64_t)p.h * p.p * p.k, pk = (int64_t)p.p * p.k;
    for_each_unit((int64_t)p.n * blocks_per_seq, [&](int64_t unit) {
        const int seq = uniform((int)(unit / blocks_per_seq)), part = (int)(unit - (int64_t)seq * blocks_per_seq);
        int first = 0, len = p.t;
        if (p.starts != nullptr) {
            first = load_uniform(p.starts, seq);
            const int end = load_uniform(p.starts, seq + 1);
            if (first < 0 || first > end || end > p.t) return;
            len = end - first;
        }
        if (len <= plan.seg) return;  // one segment
        const int count = (len - 1) / plan.seg + 1, u0 = first_place(plan, p.starts != nullptr, seq, first);
        const int slot = route_row(p.idx, nullptr, p.n, p.s, seq, threadIdx.x & 63);
        const bool init = slot >= 0 && p.state != nullptr && p.has_init != nullptr && p.has_init[seq] != 0;
        for (int64_t e = ((int64_t)part * kJoinBlock + threadIdx.x) * VEC; e < hpk;
             e += (int64_t)blocks_per_seq * kJoinBlock * VEC) {
            float run[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                run[i] = !init ? 0.0f
                         : p.state_f32 ? static_cast<const float *>(p.state)[slot * p.ss_s + e + i]
                                       : bf16_bits_to_f32(static_cast<const uint16_t *>(p.state)[slot * p.ss_s + e + i]);
            typedef float fvec __attribute__((ext_vector_type(VEC)));
            fvec *ws = reinterpret_cast<fvec *>(p.workspace + u0 * hpk + e);
            const float *dec = p.workspace + plan.places * hpk + (int64_t)u0 * p.h + e / pk;
            for (int j0 = 0; j0 < count; j0 += kJoinAhead) {
                fvec v[kJoinAhead];
                float d[kJoinAhead];
#pragma unroll
                for (int q = 0; q < kJoinAhead; ++q) {
                    const int j = min(j0 + q, count - 1);
                    v[q] = ws[j * (hpk / VEC)];
                    d[q] = dec[(int64_t)j * p.h];
                }
#pragma unroll
                for (int q = 0; q < kJoinAhead; ++q) {
                    const int j = j0 + q;
                    if (j >= count) break;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        if (j > 0) run[i] = __builtin_fmaf(run[i], d[q], v[q][i]);
                        v[q][i] = run[i];
                    }
                    ws[j * (hpk / VEC)] = v[q];
                }
            }
        }
    });
}

// Three blocks a CU fill the card.  With fewer than one a CU, sequences are cut into
// segments, as many as fill it (16381 tokens of 24 heads: 94 us; with 640 and 512 blocks
// 106 and 111) but not below kMinSegment tokens (with 64, 96, 128 and 256: 400 tokens of
// 24 heads 25, 27, 29 and 39 us, 1000 tokens 38, 36, 34 and 43).  Packed sequences, whose
// lengths the host does not know, are cut where they are longer than kLongSequence even
// if there are enough of them, so that one does not outlast the rest (16 of up to 1967
// tokens, 60 heads: 186 us whole, 254 to 270 cut at 768 to 1536).
constexpr int64_t kFullGrid = 768;
constexpr int64_t kEnoughBlocks = 256;
constexpr int64_t kMinSegment = 96;
constexpr int64_t kLongSequence = 2048;
// Runs of blocks that share B and C, at least: 8 x 2048 tokens of 96 heads take 200 us
// with 16, 32 and 64, and 224 with every block a run.
constexpr int64_t kRuns = 32;
constexpr int64_t kJoinBlocks = 2048;  // of the join, over all sequences

// Whether cutting the longest sequence at `seg` saves time: a chunk takes about 1.9 us,
// and 0.6 of that again in the pass that builds up the segments' states, which costs two
// more launches and moves each state four times (24 heads of 64 x 128, whole and cut: 320
// tokens 25 and 26 us, 400 tokens 31 and 27, 1000 tokens 66 and 36; 8 x 400 tokens 32 and
// 50, 8 x 700 tokens 49 and 56).
constexpr int64_t kChunkNs = 1900, kCutNs = 10000, kCutChunkNs = kChunkNs * 8 / 5, kStatesPerNs = 312;
bool cut_pays(int64_t longest, int64_t seg, int64_t slots, int64_t state) {
    const auto chunks = [](int64_t tokens) { return (tokens + kChunk - 1) / kChunk; };
    return kChunkNs * chunks(longest) > kCutNs + kCutChunkNs * chunks(seg) + slots * state / kStatesPerNs;
}

ScanPlan make_plan(int64_t n, int64_t t, int64_t h, int64_t p, int64_t g, int64_t k, bool packed) {
    ScanPlan plan;
    plan.np = (int32_t)((p + kUnitP - 1) / kUnitP);
    plan.quads = (int32_t)((h / g * plan.np + kScanWaves - 1) / kScanWaves);
    // heads that successive waves of a group can belong to
    plan.heads = kScanWaves % plan.np == 0 ? kScanWaves / plan.np : (kScanWaves - 2) / plan.np + 2;
    const int64_t per_slot = g * plan.quads, blocks = n * per_slot;
    const int64_t tokens = packed ? t : n * t;  // the whole call's
    int64_t seg;
    if (blocks >= kEnoughBlocks) {
        seg = packed ? (tokens * per_slot / kFullGrid > kLongSequence ? tokens * per_slot / kFullGrid : kLongSequence) : t;
    } else {
        const int64_t each = kFullGrid / ((packed ? 1 : n) * per_slot);  // segments of the t axis
        seg = each > 1 ? (t + each - 1) / each : t;
        if (seg < kMinSegment) seg = kMinSegment;
        // (packed: the longest of n is taken for twice the mean)
        if (!cut_pays(packed && n > 2 ? 2 * t / n : t, seg, packed ? t / seg + n : n * ((t + seg - 1) / seg), h * p * k)) seg = t;
    }
    seg = (seg + kChunk - 1) / kChunk * kChunk;
    if (seg >= t) seg = (t + kChunk - 1) / kChunk * kChunk;
    if (seg < kChunk) seg = kChunk;
    plan.seg = (int32_t)seg;
    plan.nseg = (int32_t)(t > 0 ? (t + seg - 1) / seg : 1);
    plan.split = plan.nseg > 1;
    plan.slots = (int32_t)(packed ? t / seg + n : n * plan.nseg);
    // sparse places end at 2 (nseg - 1), as one of c segments starts (c - 1) seg tokens ahead of t's last
    const int64_t cut = 2 * ((int64_t)plan.nseg - 1);
    plan.sparse = packed && cut < plan.slots;
    plan.places = plan.sparse ? (int32_t)cut : plan.slots;
    // the longest runs of which there are still kRuns (of equal length: packed
    // sequences would leave some XCDs with more to do than others)
    const int64_t run = packed ? 1 : plan.slots * per_slot / kRuns;
    plan.run = (int32_t)(run < 1 ? 1 : run > plan.quads ? plan.quads : run);
    plan.parts = (plan.quads + plan.run - 1) / plan.run;
    return plan;
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

template <int KS, int SPLIT, bool OUT, bool WIDE>
uint64_t lds_allowed = 0;

template <int KS, int SPLIT, bool OUT, bool WIDE>
hipError_t launch_pass(const SelectiveScanParams &p, const ScanPlan &plan, hipStream_t stream) {
    const int64_t units = ((int64_t)plan.slots * p.g * plan.parts + 7) / 8 * 8 * plan.run;
    const size_t lds = (size_t)(OUT ? 4 : 2) * kChunk * (KS + 16) * 2 + (size_t)(OUT ? 2 : 1) * kChunk * kXPitch * 2 +
                       (size_t)2 * plan.heads * kStepRows * kChunk * 4 +
                       (OUT ? (size_t)plan.heads * kChunk * kPPitch * 2 : 0);
    auto kernel = selective_scan_kernel<KS, SPLIT, OUT, WIDE>;
    const hipError_t allowed = allow_lds(reinterpret_cast<const void *>(kernel), &lds_allowed<KS, SPLIT, OUT, WIDE>);
    if (allowed != hipSuccess) return allowed;
    const int64_t across = units < kMaxBlocks ? units : kMaxBlocks, deep = (units + across - 1) / across;
    if (deep > 65535) return hipErrorInvalidConfiguration;
    kernel<<<dim3((unsigned)across, (unsigned)deep), kScanBlock, lds, stream>>>(p, plan);
    return hipGetLastError();
}

template <int KS, int SPLIT, bool WIDE>
hipError_t launch_passes(const SelectiveScanParams &p, const ScanPlan &plan, hipStream_t stream) {
    if (plan.split) {
        hipError_t err = launch_pass<KS, SPLIT, false, WIDE>(p, plan, stream);
        if (err != hipSuccess) return err;
        const bool vec = (int64_t)p.p * p.k % 4 == 0;
        const int64_t need = ((int64_t)p.h * p.p * p.k / (vec ? 4 : 1) + kJoinBlock - 1) / kJoinBlock;
        const int64_t spread = p.n < kJoinBlocks ? kJoinBlocks / p.n : 1, per_seq = need < spread ? need : spread;
        const int64_t units = per_seq * p.n;
        const dim3 grid((unsigned)(units < kMaxBlocks ? units : kMaxBlocks));
        if (vec)
            selective_join_kernel<4><<<grid, kJoinBlock, 0, stream>>>(p, plan, (int)per_seq);
        else
            selective_join_kernel<1><<<grid, kJoinBlock, 0, stream>>>(p, plan, (int)per_seq);
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return launch_pass<KS, SPLIT, true, WIDE>(p, plan, stream);
}

template <int KS>
hipError_t launch_ks(const SelectiveScanParams &p, const ScanPlan &plan, bool wide, hipStream_t stream) {
    const bool exact = p.state != nullptr && p.state_f32;
    if (wide) return exact ? launch_passes<KS, 3, true>(p, plan, stream) : launch_passes<KS, 1, true>(p, plan, stream);
    return exact ? launch_passes<KS, 3, false>(p, plan, stream) : launch_passes<KS, 1, false>(p, plan, stream);
}

// Whether rows at p with the given element strides start on 16 bytes, and 32 tokens
// (b elements apart) of `heads` heads (c apart) span less than 2^31 bytes.
bool rows16(const void *p, int64_t a, int64_t b, int64_t c, int64_t heads) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a % 8 == 0 && b % 8 == 0 && c % 8 == 0 && b < (1 << 23) &&
           c < (1 << 28) / heads;
}

}  // namespace

int64_t selective_scan_workspace_floats(int64_t n, int64_t t, int64_t h, int64_t p, int64_t g, int64_t k, bool packed) {
    const ScanPlan plan = make_plan(n, t, h, p, g, k, packed);
    return plan.split ? plan.places * (h * p * k + h) : 0;
}

hipError_t launch_selective_scan(const SelectiveScanParams &p, hipStream_t stream, const char **kernel_name) {
    const ScanPlan plan = make_plan(p.n, p.t, p.h, p.p, p.g, p.k, p.starts != nullptr);
    const int64_t heads = p.h / p.g;
    const bool wide = p.p % 8 == 0 && p.k % 8 == 0 && rows16(p.x, p.xs_n, p.xs_t, p.xs_h, heads) &&
                      rows16(p.b, p.bs_n, p.bs_t, p.bs_g, 1) && rows16(p.c, p.cs_n, p.cs_t, p.cs_g, 1) &&
                      (p.z == nullptr || rows16(p.z, p.zs_n, p.zs_t, p.zs_h, heads)) &&
                      rows16(p.out, p.os_n, p.os_t, p.os_h, heads);
    *kernel_name = plan.split ? (wide ? "selective_scan_split" : "selective_scan_split_scalar")
                              : (wide ? "selective_scan" : "selective_scan_scalar");
    if (p.k <= 64) return launch_ks<64>(p, plan, wide, stream);
    if (p.k <= 128) return launch_ks<128>(p, plan, wide, stream);
    return launch_ks<256>(p, plan, wide, stream);
}

}  // namespace dcconv
