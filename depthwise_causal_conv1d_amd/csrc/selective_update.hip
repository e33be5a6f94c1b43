// One token of the selective state-space recurrence for gfx950, with or without
// the causal convolution ahead of it.
//
// For row n, head i (its B and C belong to group i / (h/g)) and the slot the row
// selects, with d = softplus(dt + dt_bias):
//
//     state[p, k] = exp(d * a[i]) * state[p, k] + d * x[p] * B[k]
//     out[p]      = (sum_k state[p, k] * C[k] + D[i] * x[p]) * silu(z[p])
//
// The state is read and written once and everything else is a few percent of it:
// HBM bounds the call.  An item is up to 32 rows p of one head's state; a block takes
// several items of a group one after the other, with the next one's rows in flight
// while it computes.  Sixteen lanes share a row, so the sum over k is four DPP steps.
// The small operands (x, B, C, z, dt: 2 bytes each, any strides) are brought into LDS
// for all of the block's items at once, as FP32.  All arithmetic is FP32; a BF16 state
// is rounded when it is stored, after C has read the unrounded value.
//
// 256 rows of 96 heads, 64 x 128, F32 states: 258 us, 1621 MB at 6.3 TB/s (a plain copy
// reaches 5.9).  61 rows of 30 heads, 80 x 72, BF16 states: 14.4 us, 38 MB at 2.7 TB/s:
// items of 4.6 KiB, whose rows of 144 bytes fill neither the 16 lanes nor a cache line.  4 rows of 24
// heads: 5 us, a launch and one item's latency.
//
// The fused form computes x, B and C as the width-4 convolution of its channels
// (kept in FP32, not rounded to BF16 between the two operators).  Every block of
// a group needs the group's B and C channels (several items a block make that cheap),
// and the convolution state of those is advanced in place: each block counts itself in
// `arrivals[row, group]` once it has read them, and the block that completes the count
// writes their state and sets the count back to zero.  Nothing waits on the count.
// 256 rows of 96 heads with BF16 states: 155 us, 841 MB at 5.4 TB/s.  64 rows of 60
// heads in one group, F32 states, some padding: 54.7 us, 225 MB at 4.1 TB/s, as the group's
// B and C are convolved by 30 blocks a row.  One row of 24 heads: 7.8 us, the loads of the
// taps, the count and then the state's items behind the launch.
#include "state_vec.h"

namespace dcconv {
namespace {

constexpr int kUpdateBlock = 256;
constexpr int kGroups = kUpdateBlock / kRowLanes;    // rows a block holds at a time
constexpr int kMaxK = 256;

// Channel `ch` of the fused form: the convolution of its history and this token.
// The three newest values and x are left in `taps` for the state's advance.
__device__ __forceinline__ float conv_channel(const SelectiveUpdateParams &p, int row, int64_t base, int seen, int ch,
                                              uint16_t (&taps)[4]) {
    const uint16_t *st = p.conv_state + base + (int64_t)ch * p.st_d;
    if (p.seqlens == nullptr) {
#pragma unroll
        for (int j = 0; j < 3; ++j) taps[j] = st[(int64_t)(p.l - 3 + j) * p.st_l];
    } else {
        const int at = seen % p.l;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            int q = at - 3 + j;
            if (q < 0) q += p.l;
            taps[j] = st[(int64_t)q * p.st_l];
        }
    }
    taps[3] = p.xbc[(int64_t)row * p.xbcs_n + ch];
    float w[4];
    if (reinterpret_cast<uintptr_t>(p.weight) % 8 == 0) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(p.weight + (int64_t)ch * 4);
        w[0] = lo_f32(v[0]), w[1] = hi_f32(v[0]), w[2] = lo_f32(v[1]), w[3] = hi_f32(v[1]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = bf16_bits_to_f32(p.weight[(int64_t)ch * 4 + j]);
    }
    float acc = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_fmaf(bf16_bits_to_f32(taps[j]), w[j], acc);
    if (p.bias != nullptr) acc += bf16_bits_to_f32(p.bias[ch]);
    return p.silu ? silu(acc) : acc;
}

// Advances channel ch's convolution state by the token in taps[3].
__device__ __forceinline__ void conv_advance(const SelectiveUpdateParams &p, int64_t base, int seen, int ch,
                                             const uint16_t (&taps)[4]) {
    uint16_t *st = p.conv_state + base + (int64_t)ch * p.st_d;
    if (p.seqlens != nullptr) {
        st[(int64_t)(seen % p.l) * p.st_l] = taps[3];
        return;
    }
    for (int j = 0; j < p.l - 3; ++j) st[j * p.st_l] = st[(j + 1) * p.st_l];
#pragma unroll
    for (int j = 0; j < 3; ++j) st[(int64_t)(p.l - 3 + j) * p.st_l] = taps[j + 1];
}

constexpr int kMaxItems = 8;  // of a block

// How a call is cut up: items of `16 * ROWS` rows p, `chunk` of a group's to a block.
struct UpdatePlan {
    int32_t ptiles;  // items of a head
    int32_t chunk, blocks;  // items of a block; blocks of a group
};

// ROWS rows of the state per 16-lane group and item, NV vectors of VEC elements per
// lane and row (16 * VEC * NV >= k).
template <bool F32, int VEC, int NV, int ROWS, bool CONV>
__global__ __launch_bounds__(kUpdateBlock) void selective_update_kernel(const SelectiveUpdateParams p,
                                                                        const UpdatePlan plan) {
    constexpr int kItemRows = ROWS * kGroups;
    __shared__ float s_x[kMaxItems * kItemRows], s_gate[kMaxItems * kItemRows], s_b[kMaxK], s_c[kMaxK];
    __shared__ float s_step[kMaxItems], s_decay[kMaxItems], s_skip[kMaxItems];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63, sub = tid & (kRowLanes - 1), grp = tid / kRowLanes;
    const int per_group = p.h / p.g, group_items = per_group * plan.ptiles;
    for_each_unit((int64_t)p.n * p.g * plan.blocks, [&](int64_t u) {
        const int64_t rg = u / plan.blocks;
        const int first = (int)(u - rg * plan.blocks) * plan.chunk, items = min(plan.chunk, group_items - first);
        const int row = __builtin_amdgcn_readfirstlane((int)(rg / p.g));
        const int group = __builtin_amdgcn_readfirstlane((int)(rg - (int64_t)row * p.g));
        int slot = route_row(p.idx, p.status, p.n, p.s, row, lane);
        int seen = 0;
        if (CONV && p.seqlens != nullptr) {
            seen = p.seqlens[row];
            if (seen < 0) {
                if (p.status != nullptr && tid == 0) atomicOr(p.status, DCCONV_DEV_BAD_SEQLEN);
                slot = -1;
            }
        }
        // item i's head and first row
        auto place = [&](int i, int *head, int *p0) {
            const int t = __builtin_amdgcn_readfirstlane((first + i) / plan.ptiles);
            *head = group * per_group + t;
            *p0 = (first + i - t * plan.ptiles) * kItemRows;
        };
        int head, p0;
        if (slot < 0) {  // a padding row: zeros, and no state moves
            for (int i = 0; i < items; ++i) {
                place(i, &head, &p0);
                for (int q = p0 + tid; q < min(p.p, p0 + kItemRows); q += kUpdateBlock)
                    p.out[(int64_t)row * p.os_n + (int64_t)head * p.os_h + q] = 0;
            }
            return;
        }

        // an item's state rows, all in flight at once
        StateVec<F32, VEC> st[ROWS][NV];
        auto fetch = [&](int i) {
            int fh, fp;
            place(i, &fh, &fp);
            const int64_t base = (int64_t)slot * p.ss_s + (int64_t)fh * p.p * p.k;
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int pr = fp + r * kGroups + grp, k0 = (v * kRowLanes + sub) * VEC;
                    if (pr < p.p && k0 < p.k) st[r][v].load(p.state, base + (int64_t)pr * p.k + k0);
                }
        };
        fetch(0);

        // the small operands of all items, through LDS
        if (tid < items) {
            const int h = group * per_group + (first + tid) / plan.ptiles;
            const float step = load_step(p, (int64_t)row * p.ds_n + h, h);
            s_step[tid] = step;
            s_decay[tid] = expf(step * p.a[h]);
            s_skip[tid] = p.d_skip != nullptr ? p.d_skip[h] : 0.0f;
        }
        const int64_t cbase = CONV ? (int64_t)slot * p.st_s : 0;
        for (int e = tid; e < items * kItemRows; e += kUpdateBlock) {
            const int i = e / kItemRows, t = (first + i) / plan.ptiles, h = group * per_group + t;
            const int q = (first + i - t * plan.ptiles) * kItemRows + e % kItemRows;
            if (q >= p.p) continue;
            if constexpr (CONV) {
                uint16_t taps[4];
                s_x[e] = conv_channel(p, row, cbase, seen, h * p.p + q, taps);
                conv_advance(p, cbase, seen, h * p.p + q, taps);  // this block's alone
            } else {
                s_x[e] = bf16_bits_to_f32(p.x[(int64_t)row * p.xs_n + (int64_t)h * p.xs_h + q]);
            }
            s_gate[e] = p.z != nullptr ? silu(bf16_bits_to_f32(p.z[(int64_t)row * p.zs_n + (int64_t)h * p.zs_h + q])) : 1.0f;
        }
        if constexpr (CONV) {
            uint16_t bt[4], ct[4];
            const int bch = p.h * p.p + group * p.k + tid, cch = bch + p.g * p.k;
            if (tid < p.k) {
                s_b[tid] = conv_channel(p, row, cbase, seen, bch, bt);
                s_c[tid] = conv_channel(p, row, cbase, seen, cch, ct);
            }
            __syncthreads();  // every lane has read its channels' history
            if (tid == 0) {
                int32_t *count = p.arrivals + (int64_t)row * p.g + group;
                const int before = __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                s_last = before == plan.blocks - 1;
                if (s_last) __hip_atomic_store(count, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            __syncthreads();
            if (s_last && tid < p.k) {
                conv_advance(p, cbase, seen, bch, bt);
                conv_advance(p, cbase, seen, cch, ct);
            }
        } else {
            if (tid < p.k) {
                s_b[tid] = bf16_bits_to_f32(p.b[(int64_t)row * p.bs_n + (int64_t)group * p.bs_g + tid]);
                s_c[tid] = bf16_bits_to_f32(p.c[(int64_t)row * p.cs_n + (int64_t)group * p.cs_g + tid]);
            }
            __syncthreads();
        }

        float bv[NV][VEC], cv[NV][VEC];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int k0 = (v * kRowLanes + sub) * VEC;
                bv[v][e] = k0 < p.k ? s_b[k0 + e] : 0.0f;
                cv[v][e] = k0 < p.k ? s_c[k0 + e] : 0.0f;
            }
        for (int i = 0; i < items; ++i) {
            StateVec<F32, VEC> now[ROWS][NV];
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int v = 0; v < NV; ++v) now[r][v] = st[r][v];
            if (i + 1 < items) fetch(i + 1);
            place(i, &head, &p0);
            const int64_t base = (int64_t)slot * p.ss_s + (int64_t)head * p.p * p.k;
            uint16_t *out = p.out + (int64_t)row * p.os_n + (int64_t)head * p.os_h;
            const float step = s_step[i], decay = s_decay[i], skip = s_skip[i];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int at = r * kGroups + grp, pr = p0 + at;
                if (pr >= p.p) continue;
                const float xv = s_x[i * kItemRows + at], xd = step * xv;
                float y = 0.0f;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int k0 = (v * kRowLanes + sub) * VEC;
                    if (k0 >= p.k) continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float s = __builtin_fmaf(xd, bv[v][e], now[r][v].get(e) * decay);
                        y = __builtin_fmaf(s, cv[v][e], y);
                        now[r][v].set(e, s);
                    }
                    now[r][v].store(p.state, base + (int64_t)pr * p.k + k0);
                }
                y = row_sum(y);
                if (sub == 0) {
                    y = __builtin_fmaf(skip, xv, y);
                    if (p.z != nullptr) y *= s_gate[i * kItemRows + at];
                    out[pr] = f32_to_bf16_bits(y);
                }
            }
        }
        __syncthreads();  // the next unit reuses the LDS arrays
    });
}

// Items of 32 rows while there are this many, else of 16.  A block takes items worth
// kBlockState bytes of state, or kFusedBlockState in the fused form, where each block
// convolves its group's B and C; but no more than leave kUpdateBlocks blocks.  (256 rows
// of 96 heads, 64 x 128: F32 states with 16, 32 and 64 KiB a block 295, 257 and 285 us,
// BF16 147 at 16 and 136 at 32 KiB; fused, BF16 states, 201, 160 and 154 us at 16, 32
// and 64 KiB, eight items; F32 states, four items in 64 KiB, were not measured at others.)
constexpr int64_t kMinLargeItems = 2048;
constexpr int64_t kUpdateBlocks = 768;
constexpr int64_t kBlockState = 32 * 1024, kFusedBlockState = 64 * 1024;

template <bool F32, int VEC, int NV>
hipError_t launch_rows(const SelectiveUpdateParams &p, hipStream_t stream) {
    const int64_t heads = (int64_t)p.n * p.h;
    const bool large = heads * ((p.p + 31) / 32) >= kMinLargeItems;
    const int rows = large ? 32 : 16;
    UpdatePlan plan;
    plan.ptiles = (p.p + rows - 1) / rows;
    const int64_t in_group = (int64_t)(p.h / p.g) * plan.ptiles;
    int64_t chunk = (p.conv ? kFusedBlockState : kBlockState) / ((int64_t)rows * p.k * (F32 ? 4 : 2));
    if (chunk > heads * plan.ptiles / kUpdateBlocks) chunk = heads * plan.ptiles / kUpdateBlocks;
    plan.chunk = (int32_t)(chunk < 1 ? 1 : chunk > kMaxItems ? kMaxItems : chunk);
    plan.blocks = (int32_t)((in_group + plan.chunk - 1) / plan.chunk);
    plan.chunk = (int32_t)((in_group + plan.blocks - 1) / plan.blocks);  // even shares
    plan.blocks = (int32_t)((in_group + plan.chunk - 1) / plan.chunk);
    const int64_t units = (int64_t)p.n * p.g * plan.blocks;
    const dim3 grid((unsigned)(units < kMaxBlocks ? units : kMaxBlocks));
    if (p.conv) {
        if (large)
            selective_update_kernel<F32, VEC, NV, 2, true><<<grid, kUpdateBlock, 0, stream>>>(p, plan);
        else
            selective_update_kernel<F32, VEC, NV, 1, true><<<grid, kUpdateBlock, 0, stream>>>(p, plan);
    } else {
        if (large)
            selective_update_kernel<F32, VEC, NV, 2, false><<<grid, kUpdateBlock, 0, stream>>>(p, plan);
        else
            selective_update_kernel<F32, VEC, NV, 1, false><<<grid, kUpdateBlock, 0, stream>>>(p, plan);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_selective_update(const SelectiveUpdateParams &p, hipStream_t stream, const char **kernel_name) {
    const int vec = p.state_f32 ? 4 : 8;
    const bool wide = p.k % vec == 0 && p.ss_s % vec == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0;
    if (!wide) {
        *kernel_name = p.conv ? "selective_update_conv_scalar" : "selective_update_scalar";
        return p.state_f32 ? launch_rows<true, 1, 16>(p, stream) : launch_rows<false, 1, 16>(p, stream);
    }
    if (p.state_f32) {
        *kernel_name = p.conv ? "selective_update_conv<f32>" : "selective_update<f32>";
        if (p.k <= 64) return launch_rows<true, 4, 1>(p, stream);
        return p.k <= 128 ? launch_rows<true, 4, 2>(p, stream) : launch_rows<true, 4, 4>(p, stream);
    }
    *kernel_name = p.conv ? "selective_update_conv<bf16>" : "selective_update<bf16>";
    return p.k <= 128 ? launch_rows<false, 8, 1>(p, stream) : launch_rows<false, 8, 2>(p, stream);
}

}  // namespace dcconv
