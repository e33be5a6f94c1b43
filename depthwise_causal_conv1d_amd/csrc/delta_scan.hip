// The gated delta rule over whole sequences for gfx950, token by token.
//
// A block holds 16 rows p of one head's state in registers, sixteen lanes a row, and steps
// through its sequence: each token's q and k pass through LDS.  All arithmetic is FP32.
#include "delta_common.h"
#include "state_vec.h"

namespace dcconv {
namespace {

constexpr int kScanBlock = 256;
constexpr int kRows = kScanBlock / kRowLanes;
constexpr int kMaxK = 256;
constexpr int kLaneK = kMaxK / kRowLanes;

__device__ __forceinline__ float block_sum(float v, float *part, int tid) {
    v = row_sum(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    if ((tid & 63) == 0) part[tid >> 6] = v;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}

__global__ __launch_bounds__(kScanBlock) void delta_scan_kernel(const DeltaParams p, int ptiles) {
    __shared__ float s_q[kMaxK], s_k[kMaxK], s_part[2][4];
    const int tid = threadIdx.x, sub = tid & (kRowLanes - 1), grp = tid / kRowLanes;
    if (blockIdx.x == 0 && p.starts != nullptr && p.status != nullptr) {
        bool bad = false;
        for (int i = tid; i <= p.n; i += kScanBlock) {
            const int a = p.starts[i];
            bad |= a < 0 || a > p.t || (i == 0 && a != 0) || (i == p.n ? a != p.t : p.starts[i + 1] < a);
        }
        if (bad) atomicOr(p.status, DCCONV_DEV_BAD_SEQ);
    }
    for_each_unit((int64_t)p.n * p.h * ptiles, [&](int64_t u) {
        const int64_t nh = u / ptiles;
        const int seq = __builtin_amdgcn_readfirstlane((int)(nh / p.h));
        const int head = __builtin_amdgcn_readfirstlane((int)(nh - (int64_t)seq * p.h));
        const int group = head / (p.h / p.g), pr = (int)(u - nh * ptiles) * kRows + grp;
        const bool mine = pr < p.p;
        int64_t tok = 0;
        int len = p.t;
        if (p.starts != nullptr) {
            const int a = p.starts[seq], e = p.starts[seq + 1];
            if (a < 0 || a > e || e > p.t) return;
            tok = a;
            len = e - a;
        }
        const int slot = route_row(p.idx, p.status, p.n, p.s, seq, tid & 63);
        uint16_t *out = p.out + seq * p.os_n + tok * p.os_t + head * p.os_h;
        if (slot < 0) {
            for (int t = 0; t < len; ++t)
                if (mine && sub == 0) out[t * p.os_t + pr] = 0;
            return;
        }
        float st[kLaneK];
        const int64_t at = slot * p.ss_s + ((int64_t)head * p.p + pr) * p.k;
        const bool init = p.state != nullptr && p.has_init != nullptr && p.has_init[seq] != 0;
#pragma unroll
        for (int e = 0; e < kLaneK; ++e) {
            const int kk = e * kRowLanes + sub;
            st[e] = init && mine && kk < p.k ? load_either(p.state, p.state_f32, at + kk) : 0.0f;
        }
        for (int t = 0; t < len; ++t) {
            const int64_t now = tok + t;
            float qe = 0.0f, ke = 0.0f;
            if (tid < p.k) {
                qe = bf16_bits_to_f32(p.q[seq * p.qs_n + now * p.qs_t + group * p.qs_g + tid]);
                ke = bf16_bits_to_f32(p.key[seq * p.ks_n + now * p.ks_t + group * p.ks_g + tid]);
            }
            float qf = p.scale, kf = 1.0f;
            if (p.l2norm) {
                qf *= unit_factor(p, block_sum(qe * qe, s_part[0], tid));
                kf = unit_factor(p, block_sum(ke * ke, s_part[1], tid));
            }
            s_q[tid] = qe * qf;
            s_k[tid] = ke * kf;
            __syncthreads();
            const float decay = expf(load_step(p, seq * p.ds_n + now * p.ds_t + head, head) * p.a[head]);
            const float weight = weight_of(p, load_either(p.beta, p.beta_f32, seq * p.es_n + now * p.es_t + head));
            const float vv = mine ? bf16_bits_to_f32(p.v[seq * p.vs_n + now * p.vs_t + head * p.vs_h + pr]) : 0.0f;
            float told = 0.0f, y = 0.0f;
#pragma unroll
            for (int e = 0; e < kLaneK; ++e) {
                st[e] *= decay;
                told = __builtin_fmaf(st[e], s_k[e * kRowLanes + sub], told);
            }
            const float w = weight * (vv - row_sum(told));
#pragma unroll
            for (int e = 0; e < kLaneK; ++e) {
                st[e] = __builtin_fmaf(w, s_k[e * kRowLanes + sub], st[e]);
                y = __builtin_fmaf(st[e], s_q[e * kRowLanes + sub], y);
            }
            y = row_sum(y);
            if (mine && sub == 0) out[t * p.os_t + pr] = f32_to_bf16_bits(y);
            __syncthreads();
        }
        if (p.state == nullptr || !mine) return;
#pragma unroll
        for (int e = 0; e < kLaneK; ++e) {
            const int kk = e * kRowLanes + sub;
            if (kk >= p.k) continue;
            if (p.state_f32)
                static_cast<float *>(p.state)[at + kk] = st[e];
            else
                static_cast<uint16_t *>(p.state)[at + kk] = f32_to_bf16_bits(st[e]);
        }
    });
}

}  // namespace

hipError_t launch_delta_scan(const DeltaParams &p, hipStream_t stream, const char **kernel_name) {
    *kernel_name = "delta_scan_recurrent";
    const int ptiles = (p.p + kRows - 1) / kRows;
    const int64_t units = (int64_t)p.n * p.h * ptiles;
    delta_scan_kernel<<<dim3((unsigned)(units < kMaxBlocks ? units : kMaxBlocks)), kScanBlock, 0, stream>>>(p, ptiles);
    return hipGetLastError();
}

}  // namespace dcconv
