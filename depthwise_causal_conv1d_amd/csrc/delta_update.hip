// One token of the gated delta rule for gfx950.
//
// For row n, head i (its q and k belong to group i / (h/g)) and the slot the row selects,
// with d = softplus(dt + dt_bias), b = sigmoid(beta) and k, q of length one if asked for:
//
//     S[p, :] = exp(d * a[i]) * S[p, :]
//     u[p]    = b * (v[p] - S[p, :] k)
//     S[p, :] = S[p, :] + u[p] k
//     out[p]  = scale * S[p, :] q
//
// A row p of the state is read and written once and needs no other row, and everything
// else is a few percent of it: HBM bounds the call.  An item is up to 32 rows p of one
// head's state; a block takes several items of a group one after the other, with the next
// one's rows in flight while it computes.  Sixteen lanes share a row: its two sums over k
// are four DPP steps each.  q, k (as F32, made to length one once for all of the block's
// heads), v and the heads' factors pass through LDS.  All arithmetic is FP32; a BF16 state
// is rounded when it is stored, after q has read the unrounded value.
//
// 256 rows, 32 heads of 128 x 128, F32 states: 176 us, 6.1 TB/s of state, where a large copy
// reaches 5.9.  61 rows, 9 heads of 80 x 72, BF16 states: 8.5 us for 11 MB; rows of 144
// bytes fill nine of sixteen lanes.  4 rows, 8 heads: 5.0 us, launch and one item's latency.
#include "delta_common.h"
#include "state_vec.h"

namespace dcconv {
namespace {

constexpr int kUpdateBlock = 256;
constexpr int kGroups = kUpdateBlock / kRowLanes;  // rows a block holds at a time
constexpr int kMaxK = 256;
constexpr int kMaxItems = 8;  // of a block

// How a call is cut up: items of `16 * ROWS` rows p, `chunk` of a group's to a block.
struct UpdatePlan {
    int32_t ptiles;         // items of a head
    int32_t chunk, blocks;  // items of a block; blocks of a group
};

// The sum of v over the block's four waves, in all of its threads.
__device__ __forceinline__ float block_sum(float v, float *part, int tid) {
    v = row_sum(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    if ((tid & 63) == 0) part[tid >> 6] = v;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}

// ROWS rows of the state per 16-lane group and item, NV vectors of VEC elements per lane
// and row (16 * VEC * NV >= k).
template <bool F32, int VEC, int NV, int ROWS>
__global__ __launch_bounds__(kUpdateBlock) void delta_update_kernel(const DeltaParams p, const UpdatePlan plan) {
    constexpr int kItemRows = ROWS * kGroups;
    __shared__ float s_v[kMaxItems * kItemRows], s_q[kMaxK], s_k[kMaxK], s_part[2][4];
    __shared__ float s_weight[kMaxItems], s_decay[kMaxItems];
    const int tid = threadIdx.x, lane = tid & 63, sub = tid & (kRowLanes - 1), grp = tid / kRowLanes;
    const int per_group = p.h / p.g, group_items = per_group * plan.ptiles;
    for_each_unit((int64_t)p.n * p.g * plan.blocks, [&](int64_t u) {
        const int64_t rg = u / plan.blocks;
        const int first = (int)(u - rg * plan.blocks) * plan.chunk, items = min(plan.chunk, group_items - first);
        const int row = __builtin_amdgcn_readfirstlane((int)(rg / p.g));
        const int group = __builtin_amdgcn_readfirstlane((int)(rg - (int64_t)row * p.g));
        const int slot = route_row(p.idx, p.status, p.n, p.s, row, lane);
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
            s_weight[tid] = weight_of(p, load_either(p.beta, p.beta_f32, (int64_t)row * p.es_n + h));
            s_decay[tid] = expf(load_step(p, (int64_t)row * p.ds_n + h, h) * p.a[h]);
        }
        for (int e = tid; e < items * kItemRows; e += kUpdateBlock) {
            const int i = e / kItemRows, t = (first + i) / plan.ptiles, h = group * per_group + t;
            const int q = (first + i - t * plan.ptiles) * kItemRows + e % kItemRows;
            if (q < p.p) s_v[e] = bf16_bits_to_f32(p.v[(int64_t)row * p.vs_n + (int64_t)h * p.vs_h + q]);
        }
        float qe = 0.0f, ke = 0.0f;
        if (tid < p.k) {
            qe = bf16_bits_to_f32(p.q[(int64_t)row * p.qs_n + (int64_t)group * p.qs_g + tid]);
            ke = bf16_bits_to_f32(p.key[(int64_t)row * p.ks_n + (int64_t)group * p.ks_g + tid]);
        }
        float qf = p.scale, kf = 1.0f;
        if (p.l2norm) {
            qf *= unit_factor(p, block_sum(qe * qe, s_part[0], tid));
            kf = unit_factor(p, block_sum(ke * ke, s_part[1], tid));
        }
        if (tid < p.k) {
            s_q[tid] = qe * qf;
            s_k[tid] = ke * kf;
        }
        __syncthreads();

        float qv[NV][VEC], kv[NV][VEC];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int k0 = (v * kRowLanes + sub) * VEC;
                qv[v][e] = k0 < p.k ? s_q[k0 + e] : 0.0f;
                kv[v][e] = k0 < p.k ? s_k[k0 + e] : 0.0f;
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
            const float weight = s_weight[i], decay = s_decay[i];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int at = r * kGroups + grp, pr = p0 + at;
                if (pr >= p.p) continue;
                float told = 0.0f;  // what the state says of k
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if ((v * kRowLanes + sub) * VEC >= p.k) continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) told = __builtin_fmaf(now[r][v].get(e) * decay, kv[v][e], told);
                }
                const float u = weight * (s_v[i * kItemRows + at] - row_sum(told));
                float y = 0.0f;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int k0 = (v * kRowLanes + sub) * VEC;
                    if (k0 >= p.k) continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float s = __builtin_fmaf(u, kv[v][e], now[r][v].get(e) * decay);
                        y = __builtin_fmaf(s, qv[v][e], y);
                        now[r][v].set(e, s);
                    }
                    now[r][v].store(p.state, base + (int64_t)pr * p.k + k0);
                }
                y = row_sum(y);
                if (sub == 0) out[pr] = f32_to_bf16_bits(y);
            }
        }
        __syncthreads();  // the next unit reuses the LDS arrays
    });
}

// Items of 32 rows while there are this many, else of 16; a block takes items worth
// kBlockState bytes of state, but no more than leave kUpdateBlocks blocks: the figures
// that the state-space update measured, whose traffic is the same.
constexpr int64_t kMinLargeItems = 2048;
constexpr int64_t kUpdateBlocks = 768;
constexpr int64_t kBlockState = 32 * 1024;

template <bool F32, int VEC, int NV>
hipError_t launch_rows(const DeltaParams &p, hipStream_t stream) {
    const int64_t heads = (int64_t)p.n * p.h;
    const bool large = heads * ((p.p + 31) / 32) >= kMinLargeItems;
    const int rows = large ? 32 : 16;
    UpdatePlan plan;
    plan.ptiles = (p.p + rows - 1) / rows;
    const int64_t in_group = (int64_t)(p.h / p.g) * plan.ptiles;
    int64_t chunk = kBlockState / ((int64_t)rows * p.k * (F32 ? 4 : 2));
    if (chunk > heads * plan.ptiles / kUpdateBlocks) chunk = heads * plan.ptiles / kUpdateBlocks;
    plan.chunk = (int32_t)(chunk < 1 ? 1 : chunk > kMaxItems ? kMaxItems : chunk);
    plan.blocks = (int32_t)((in_group + plan.chunk - 1) / plan.chunk);
    plan.chunk = (int32_t)((in_group + plan.blocks - 1) / plan.blocks);  // even shares
    plan.blocks = (int32_t)((in_group + plan.chunk - 1) / plan.chunk);
    const int64_t units = (int64_t)p.n * p.g * plan.blocks;
    const dim3 grid((unsigned)(units < kMaxBlocks ? units : kMaxBlocks));
    if (large)
        delta_update_kernel<F32, VEC, NV, 2><<<grid, kUpdateBlock, 0, stream>>>(p, plan);
    else
        delta_update_kernel<F32, VEC, NV, 1><<<grid, kUpdateBlock, 0, stream>>>(p, plan);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_update(const DeltaParams &p, hipStream_t stream, const char **kernel_name) {
    const int vec = p.state_f32 ? 4 : 8;
    const bool wide = p.k % vec == 0 && p.ss_s % vec == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0;
    if (!wide) {
        *kernel_name = "delta_update_scalar";
        return p.state_f32 ? launch_rows<true, 1, 16>(p, stream) : launch_rows<false, 1, 16>(p, stream);
    }
    if (p.state_f32) {
        *kernel_name = "delta_update<f32>";
        if (p.k <= 64) return launch_rows<true, 4, 1>(p, stream);
        return p.k <= 128 ? launch_rows<true, 4, 2>(p, stream) : launch_rows<true, 4, 4>(p, stream);
    }
    *kernel_name = "delta_update<bf16>";
    return p.k <= 128 ? launch_rows<false, 8, 1>(p, stream) : launch_rows<false, 8, 2>(p, stream);
}

}  // namespace dcconv
