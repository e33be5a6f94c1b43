// Internal interface between the C-ABI front end of the gated delta rule and of the
// norms (delta_abi.hip) and their kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dcconv {

// The gated delta rule over whole sequences (batch or packed), or over one token of n
// rows (t = 1, the _t strides unused), validated on the host.
struct DeltaParams {
    const uint16_t *q, *key;  // BF16 [n, t, g, k], or packed [t, g, k]
    int64_t qs_n, qs_t, qs_g, ks_n, ks_t, ks_g;
    const uint16_t *v;  // BF16 [n, t, h, p]
    int64_t vs_n, vs_t, vs_h;
    const void *dt, *beta;  // BF16 or F32 [n, t, h], unit head stride
    int64_t ds_n, ds_t, es_n, es_t;
    const float *dt_bias, *a;  // F32 [h]; dt_bias may be null
    const int32_t *starts;     // int32 [n+1] or null (batch form)
    void *state;               // F32 or BF16 [s, h, p, k], dense behind the slot, or null
    int64_t ss_s;
    const int32_t *idx;
    const uint8_t *has_init;
    int32_t *status;
    uint16_t *out;  // BF16 [n, t, h, p]
    int64_t os_n, os_t, os_h;
    float *workspace;
    int32_t n, t, h, p, g, k, s;
    float eps, scale;
    bool dt_f32, dt_softplus, beta_f32, beta_sigmoid, l2norm, state_f32;
};

hipError_t launch_delta_update(const DeltaParams &p, hipStream_t stream, const char **kernel_name);
// Floats of workspace a scan needs (0: none).
int64_t delta_scan_workspace_floats(int64_t n, int64_t t, int64_t h, int64_t p, int64_t k, bool packed);

hipError_t launch_delta_scan(const DeltaParams &p, hipStream_t stream, const char **kernel_name);

// Rows [n, t, h] of d values, normed and gated.
struct GatedNormParams {
    const uint16_t *x, *z;  // BF16; z may be null
    int64_t xs_n, xs_t, xs_h, zs_n, zs_t, zs_h;
    const void *weight;  // BF16 or F32 [h, d] with row stride ws_h, or null
    int64_t ws_h;
    uint16_t *out;
    int64_t os_n, os_t, os_h;
    int64_t n, t, h;
    int32_t d;
    float offset, eps;
    bool weight_f32, gate_first;
};

hipError_t launch_gated_norm(const GatedNormParams &p, hipStream_t stream, const char **kernel_name);

// Rows [n, t] of d values, added to the residual stream and its norm taken.
struct AddNormParams {
    const uint16_t *x, *gate;  // BF16; gate may be null
    int64_t xs_n, xs_t, gs_n, gs_t;
    void *residual;  // F32 or BF16
    int64_t rs_n, rs_t;
    const void *post, *weight;  // BF16 or F32 [d]; post may be null
    uint16_t *out;
    int64_t os_n, os_t;
    int64_t n, t;
    int32_t d;
    float residual_scale, offset, eps;
    bool weight_f32, residual_f32;
};

hipError_t launch_add_norm(const AddNormParams &p, hipStream_t stream, const char **kernel_name);

}  // namespace dcconv
