// Internal interface between the C-ABI front end of the state-space operators
// (selective_abi.hip) and their kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dcconv {

// One token of n rows through the recurrence, validated on the host.  With
// `conv` set, x, b and c come from the convolution fields instead.
struct SelectiveUpdateParams {
    const uint16_t *x;  // BF16 [n, h, p]
    int64_t xs_n, xs_h;
    const uint16_t *b, *c;  // BF16 [n, g, k]
    int64_t bs_n, bs_g, cs_n, cs_g;
    const void *dt;  // BF16 or F32 [n, h], unit head stride
    int64_t ds_n;
    const float *dt_bias, *a, *d_skip;  // F32 [h]; dt_bias and d_skip may be null
    const uint16_t *z;                  // BF16 [n, h, p] or null
    int64_t zs_n, zs_h;
    void *state;  // F32 or BF16 [s, h, p, k], dense behind the slot
    int64_t ss_s;
    const int32_t *idx;
    int32_t *status;
    uint16_t *out;  // BF16 [n, h, p]
    int64_t os_n, os_h;
    int32_t n, h, p, g, k, s;
    bool dt_f32, dt_softplus, state_f32;

    // the convolution of the fused form
    bool conv;
    const uint16_t *xbc;  // BF16 [n, h*p + 2*g*k], unit channel stride
    int64_t xbcs_n;
    uint16_t *conv_state;  // BF16 [s, h*p + 2*g*k, l]
    int64_t st_s, st_d, st_l;
    const uint16_t *weight, *bias;
    const int32_t *seqlens;
    int32_t *arrivals;  // int32 [n*g], zero between calls
    int32_t l;
    bool silu;
};

hipError_t launch_selective_update(const SelectiveUpdateParams &p, hipStream_t stream, const char **kernel_name);

// Whole sequences through the recurrence, validated on the host.
struct SelectiveScanParams {
    const uint16_t *x;  // BF16 [n, t, h, p], or packed [t, h, p]
    int64_t xs_n, xs_t, xs_h;
    const uint16_t *b, *c;  // BF16 [n, t, g, k]
    int64_t bs_n, bs_t, bs_g, cs_n, cs_t, cs_g;
    const void *dt;  // BF16 or F32 [n, t, h], unit head stride
    int64_t ds_n, ds_t;
    const float *dt_bias, *a, *d_skip;
    const uint16_t *z;
    int64_t zs_n, zs_t, zs_h;
    const int32_t *starts;  // int32 [n+1] or null (batch form)
    void *state;            // F32 or BF16 [s, h, p, k], or null
    int64_t ss_s;
    const int32_t *idx;
    const uint8_t *has_init;
    int32_t *status;
    uint16_t *out;
    int64_t os_n, os_t, os_h;
    float *workspace;
    int32_t n, t, h, p, g, k, s;
    bool dt_f32, dt_softplus, state_f32;
};

// Floats of workspace a call needs (0: none).
int64_t selective_scan_workspace_floats(int64_t n, int64_t t, int64_t h, int64_t p, int64_t g, int64_t k, bool packed);

hipError_t launch_selective_scan(const SelectiveScanParams &p, hipStream_t stream, const char **kernel_name);

// A few rows against a 4-bit weight matrix, validated on the host.
struct W4Params {
    const uint16_t *x;  // BF16 [m, k], row stride xs_m
    int64_t xs_m;
    const uint8_t *q;  // tiles [ceil(n/16), ceil(k/128), 64, 16]
    const uint16_t *scales;  // BF16 [ceil(k/group), n]
    const uint8_t *zeros;    // [ceil(k/group), n] or null (8)
    const uint16_t *bias;    // BF16 [n] or null
    uint16_t *out;           // BF16 [m, n], row stride os_m
    int64_t os_m;
    int32_t m, n, k, group;
};

hipError_t launch_w4_matvec(const W4Params &p, hipStream_t stream, const char **kernel_name);

// Codes [n, k] (one a byte) -> the tiles of W4Params.q.
hipError_t launch_w4_pack(const uint8_t *codes, int64_t n, int64_t k, uint8_t *q, hipStream_t stream);

}  // namespace dcconv
