// C-ABI front end of the gated delta rule and of the layer's norms: host-side
// validation and dispatch, under the same rules as the other entry points (metadata
// only, nothing allocated, nothing synchronised, nothing enqueued on an error).
#include <math.h>
#include <stdint.h>

#include "delta_params.h"
#include "operand_checks.h"

using namespace dcconv::abi;

namespace {

constexpr int64_t kMaxKey = 256;       // key size k
constexpr int64_t kMaxNorm = 16384;    // values of a normed row
constexpr int64_t kMaxNormRows = (int64_t)1 << 40;

// What the scan and the update share: sizes, types and options.
int check_delta(int64_t n, int64_t h, int64_t p, int64_t g, int64_t k, int dt_dtype, int beta_dtype, int qk_l2norm,
                float l2norm_eps, float scale, int state_dtype, int64_t s, int64_t ss_s, bool has_indices,
                bool stateless) {
    if (n < 0) return fail(DCCONV_EINVAL, "n must be >= 0, got %lld", (long long)n);
    if (h < 1 || p < 1 || g < 1 || k < 1)
        return fail(DCCONV_EINVAL, "h, p, g and k must be >= 1, got %lld, %lld, %lld, %lld", (long long)h,
                    (long long)p, (long long)g, (long long)k);
    if (h % g != 0)
        return fail(DCCONV_EINVAL, "h=%lld heads do not divide into g=%lld groups", (long long)h, (long long)g);
    if (!known_dtype(dt_dtype) || !known_dtype(beta_dtype) || !known_dtype(state_dtype))
        return fail(DCCONV_EINVAL,
                    "dt_dtype, beta_dtype and state_dtype must be DCCONV_DTYPE_BF16 (0) or DCCONV_DTYPE_F32 (1)");
    if (qk_l2norm && !(l2norm_eps > 0.0f && isfinite(l2norm_eps)))
        return fail(DCCONV_EINVAL, "l2norm_eps must be positive and finite, got %g", (double)l2norm_eps);
    if (!isfinite(scale)) return fail(DCCONV_EINVAL, "scale must be finite, got %g", (double)scale);
    if (s < 0 || ss_s < 0) return fail(DCCONV_EINVAL, "s and ss_s must be >= 0");
    if (k > kMaxKey)
        return fail(DCCONV_EUNSUPPORTED, "key sizes above %lld are not served, got k=%lld", (long long)kMaxKey,
                    (long long)k);
    if (n > kI32Max - (1 << 24) || s > kI32Max || h > (1 << 20) || p > (1 << 20) || h * p > (1 << 26) || g * k > (1 << 26))
        return fail(DCCONV_EUNSUPPORTED,
                    "sizes beyond n < 2^31 - 2^24, s < 2^31, h, p <= 2^20 and h*p, g*k <= 2^26 are not served");
    if (!stateless) {
        if (s > 1 && ss_s < h * p * k)
            return fail(DCCONV_EINVAL, "state slots overlap: stride %lld, %lld elements", (long long)ss_s,
                        (long long)(h * p * k));
        if (!has_indices && s < n)
            return fail(DCCONV_EINVAL, "without state_indices row r uses slot r, so s=%lld must be >= n=%lld",
                        (long long)s, (long long)n);
    }
    return DCCONV_OK;
}

// Spans, addresses and overlaps of a call with `rows` rows of t tokens (n sequences), and its launch.
int run_delta(const dcconv::DeltaParams &q, int64_t rows, int64_t slots, int64_t workspace_bytes, bool scan, void *stream) {
    const int64_t n = q.n, t = q.t, h = q.h, p = q.p, g = q.g, k = q.k;
    if (t > 0 && !rows_distinct({rows, t, h}, {q.os_n, q.os_t, q.os_h}, p))
        return fail(DCCONV_EINVAL, "out strides (%lld, %lld, %lld, 1) give two elements the same address",
                    (long long)q.os_n, (long long)q.os_t, (long long)q.os_h);
    const int64_t dt_bytes = q.dt_f32 ? 4 : 2, beta_bytes = q.beta_f32 ? 4 : 2, state_bytes = q.state_f32 ? 4 : 2;
    int64_t qb, kb, vb, db, eb, sb, ob;
    if (!extent({rows, t, g}, {q.qs_n, q.qs_t, q.qs_g}, k, 2, &qb) ||
        !extent({rows, t, g}, {q.ks_n, q.ks_t, q.ks_g}, k, 2, &kb) ||
        !extent({rows, t, h}, {q.vs_n, q.vs_t, q.vs_h}, p, 2, &vb) ||
        !extent({rows, t, 1}, {q.ds_n, q.ds_t, 0}, h, dt_bytes, &db) ||
        !extent({rows, t, 1}, {q.es_n, q.es_t, 0}, h, beta_bytes, &eb) ||
        !extent({slots, 1, 1}, {q.ss_s, 0, 0}, h * p * k, state_bytes, &sb) ||
        !extent({rows, t, h}, {q.os_n, q.os_t, q.os_h}, p, 2, &ob))
        return fail(DCCONV_EINVAL, "strides span more than 2^47 bytes");
    const Operand ops[] = {{"out", q.out, ob, 2, true},
                           {"state", q.state, sb, state_bytes, true},
                           {"workspace", q.workspace, workspace_bytes, 16, true},
                           {"dev_status", q.status, 4, 4, true},
                           {"q", q.q, qb, 2, false},
                           {"key", q.key, kb, 2, false},
                           {"v", q.v, vb, 2, false},
                           {"dt", q.dt, db, dt_bytes, false},
                           {"dt_bias", q.dt_bias, 4 * h, 4, false},
                           {"a", q.a, 4 * h, 4, false},
                           {"beta", q.beta, eb, beta_bytes, false},
                           {"seq_starts", q.starts, 4 * (n + 1), 4, false},
                           {"state_indices", q.idx, 4 * n, 4, false},
                           {"has_initial_state", q.has_init, n, 1, false}};
    const int rc = check_operands(ops);
    if (rc != DCCONV_OK) return rc;
    const char *name = "";
    const hipError_t err = scan ? dcconv::launch_delta_scan(q, static_cast<hipStream_t>(stream), &name)
                                : dcconv::launch_delta_update(q, static_cast<hipStream_t>(stream), &name);
    if (err != hipSuccess) return fail(DCCONV_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return succeed(name);
}

}  // namespace

extern "C" int dcconv_gated_delta_update(const void *q, const void *key, const void *v, int64_t n, int64_t h,
                                         int64_t p, int64_t g, int64_t k, int64_t qs_n, int64_t qs_g, int64_t ks_n,
                                         int64_t ks_g, int64_t vs_n, int64_t vs_h, const void *dt, int dt_dtype,
                                         int64_t ds_n, const float *dt_bias, int dt_softplus, const float *a,
                                         const void *beta, int beta_dtype, int64_t es_n, int beta_sigmoid,
                                         int qk_l2norm, float l2norm_eps, float scale, void *state, int state_dtype,
                                         int64_t s, int64_t ss_s, const int32_t *state_indices, void *out,
                                         int64_t os_n, int64_t os_h, int32_t *dev_status, void *stream) {
    const int rc = check_delta(n, h, p, g, k, dt_dtype, beta_dtype, qk_l2norm, l2norm_eps, scale, state_dtype, s, ss_s,
                               state_indices != nullptr, false);
    if (rc != DCCONV_OK) return rc;
    if (any_negative({qs_n, qs_g, ks_n, ks_g, vs_n, vs_h, ds_n, es_n, os_n, os_h}))
        return fail(DCCONV_EINVAL, "strides must be non-negative");
    if (n == 0) return succeed("");
    if (!q || !key || !v || !dt || !a || !beta || !out || (!state && s > 0))
        return fail(DCCONV_EINVAL, "q, key, v, dt, a, beta, out (and state when s > 0) must be non-NULL when n > 0");
    dcconv::DeltaParams c = {};
    c.q = static_cast<const uint16_t *>(q);
    c.key = static_cast<const uint16_t *>(key);
    c.v = static_cast<const uint16_t *>(v);
    c.qs_n = qs_n, c.qs_g = qs_g, c.ks_n = ks_n, c.ks_g = ks_g, c.vs_n = vs_n, c.vs_h = vs_h;
    c.dt = dt, c.beta = beta, c.ds_n = ds_n, c.es_n = es_n;
    c.dt_bias = dt_bias, c.a = a;
    c.state = state, c.ss_s = ss_s, c.idx = state_indices, c.status = dev_status;
    c.out = static_cast<uint16_t *>(out);
    c.os_n = os_n, c.os_h = os_h;
    c.n = (int32_t)n, c.t = 1, c.h = (int32_t)h, c.p = (int32_t)p, c.g = (int32_t)g, c.k = (int32_t)k;
    c.s = (int32_t)s;
    c.eps = l2norm_eps, c.scale = scale;
    c.dt_f32 = dt_dtype == DCCONV_DTYPE_F32, c.beta_f32 = beta_dtype == DCCONV_DTYPE_F32;
    c.state_f32 = state_dtype == DCCONV_DTYPE_F32;
    c.dt_softplus = dt_softplus != 0, c.beta_sigmoid = beta_sigmoid != 0, c.l2norm = qk_l2norm != 0;
    return run_delta(c, n, s, 0, false, stream);
}

extern "C" int64_t dcconv_gated_delta_scan_workspace(int64_t n, int64_t t, int64_t h, int64_t p, int64_t g, int64_t k,
                                                     int packed) {
    if (n < 1 || t < 1 || h < 1 || p < 1 || g < 1 || k < 1 || h % g != 0 || n > kI32Max - (1 << 24) || t > kI32Max - 1024 ||
        h > (1 << 20) || p > (1 << 20) || h * p > (1 << 26) || k > kMaxKey)
        return 0;
    return 4 * dcconv::delta_scan_workspace_floats(n, t, h, p, k, packed != 0);
}

extern "C" int dcconv_gated_delta_scan(const void *q, const void *key, const void *v, int64_t n, int64_t t, int64_t h,
                                       int64_t p, int64_t g, int64_t k, int64_t qs_n, int64_t qs_t, int64_t qs_g,
                                       int64_t ks_n, int64_t ks_t, int64_t ks_g, int64_t vs_n, int64_t vs_t,
                                       int64_t vs_h, const void *dt, int dt_dtype, int64_t ds_n, int64_t ds_t,
                                       const float *dt_bias, int dt_softplus, const float *a, const void *beta,
                                       int beta_dtype, int64_t es_n, int64_t es_t, int beta_sigmoid, int qk_l2norm,
                                       float l2norm_eps, float scale, const int32_t *seq_starts, void *state,
                                       int state_dtype, int64_t s, int64_t ss_s, const int32_t *state_indices,
                                       const uint8_t *has_initial_state, void *out, int64_t os_n, int64_t os_t,
                                       int64_t os_h, void *workspace, int64_t workspace_bytes, int32_t *dev_status,
                                       void *stream) {
    const bool stateless = state == nullptr && s == 0;
    if (stateless && (has_initial_state != nullptr || state_indices != nullptr))
        return fail(DCCONV_EINVAL, "has_initial_state and state_indices need a state");
    const int rc = check_delta(n, h, p, g, k, dt_dtype, beta_dtype, qk_l2norm, l2norm_eps, scale, state_dtype, s, ss_s,
                               state_indices != nullptr, stateless);
    if (rc != DCCONV_OK) return rc;
    if (t < 0) return fail(DCCONV_EINVAL, "t (tokens) must be >= 0, got %lld", (long long)t);
    if (t > kI32Max - 1024) return fail(DCCONV_EUNSUPPORTED, "t >= 2^31 - 1024 tokens is not served");
    if (any_negative({qs_n, qs_t, qs_g, ks_n, ks_t, ks_g, vs_n, vs_t, vs_h, ds_n, ds_t, es_n, es_t, os_n, os_t, os_h,
                      workspace_bytes}))
        return fail(DCCONV_EINVAL, "strides and workspace_bytes must be non-negative");
    if (n == 0 || (t == 0 && stateless)) return succeed("");
    if (!a || (!state && s > 0) || (t > 0 && (!q || !key || !v || !dt || !beta || !out)))
        return fail(DCCONV_EINVAL, "q, key, v, dt, a, beta, out (and state when s > 0) must be non-NULL");
    const bool packed = seq_starts != nullptr;
    dcconv::DeltaParams c = {};
    c.q = static_cast<const uint16_t *>(q);
    c.key = static_cast<const uint16_t *>(key);
    c.v = static_cast<const uint16_t *>(v);
    c.qs_n = packed ? 0 : qs_n, c.qs_t = qs_t, c.qs_g = qs_g;
    c.ks_n = packed ? 0 : ks_n, c.ks_t = ks_t, c.ks_g = ks_g;
    c.vs_n = packed ? 0 : vs_n, c.vs_t = vs_t, c.vs_h = vs_h;
    c.dt = dt, c.beta = beta;
    c.ds_n = packed ? 0 : ds_n, c.ds_t = ds_t, c.es_n = packed ? 0 : es_n, c.es_t = es_t;
    c.dt_bias = dt_bias, c.a = a, c.starts = seq_starts;
    c.state = state, c.ss_s = ss_s, c.idx = state_indices, c.has_init = has_initial_state, c.status = dev_status;
    c.out = static_cast<uint16_t *>(out);
    c.os_n = packed ? 0 : os_n, c.os_t = os_t, c.os_h = os_h;
    c.n = (int32_t)n, c.t = (int32_t)t, c.h = (int32_t)h, c.p = (int32_t)p, c.g = (int32_t)g, c.k = (int32_t)k;
    c.s = (int32_t)s;
    c.eps = l2norm_eps, c.scale = scale;
    c.dt_f32 = dt_dtype == DCCONV_DTYPE_F32, c.beta_f32 = beta_dtype == DCCONV_DTYPE_F32;
    c.state_f32 = state_dtype == DCCONV_DTYPE_F32;
    c.dt_softplus = dt_softplus != 0, c.beta_sigmoid = beta_sigmoid != 0, c.l2norm = qk_l2norm != 0;
    const int64_t need = dcconv_gated_delta_scan_workspace(n, t, h, p, g, k, packed);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(DCCONV_EINVAL, "workspace of %lld bytes needed, got %lld", (long long)need,
                    (long long)(workspace ? workspace_bytes : 0));
    c.workspace = need > 0 ? static_cast<float *>(workspace) : nullptr;
    return run_delta(c, packed ? 1 : n, s, need, true, stream);
}

namespace {

int check_norm(int64_t rows[3], int64_t d, int weight_dtype, float weight_offset, float eps) {
    for (int i = 0; i < 3; ++i)
        if (rows[i] < 0) return fail(DCCONV_EINVAL, "n, t and h must be >= 0, got %lld", (long long)rows[i]);
    if (d < 1) return fail(DCCONV_EINVAL, "d must be >= 1, got %lld", (long long)d);
    if (!known_dtype(weight_dtype))
        return fail(DCCONV_EINVAL, "weight_dtype must be DCCONV_DTYPE_BF16 (0) or DCCONV_DTYPE_F32 (1)");
    if (!(eps >= 0.0f && isfinite(eps))) return fail(DCCONV_EINVAL, "eps must be finite and >= 0, got %g", (double)eps);
    if (!isfinite(weight_offset))
        return fail(DCCONV_EINVAL, "weight_offset must be finite, got %g", (double)weight_offset);
    if (d > kMaxNorm)
        return fail(DCCONV_EUNSUPPORTED, "rows of more than %lld values are not served, got d=%lld", (long long)kMaxNorm,
                    (long long)d);
    int64_t all = 1;
    for (int i = 0; i < 3; ++i) {
        if (rows[i] > kMaxNormRows || (rows[i] > 0 && all > kMaxNormRows / rows[i]))
            return fail(DCCONV_EUNSUPPORTED, "more than 2^40 rows are not served");
        all *= rows[i];
    }
    return DCCONV_OK;
}

}  // namespace

extern "C" int dcconv_gated_rms_norm(const void *x, int64_t n, int64_t t, int64_t h, int64_t d, int64_t xs_n,
                                     int64_t xs_t, int64_t xs_h, const void *z, int64_t zs_n, int64_t zs_t,
                                     int64_t zs_h, int gate_first, const void *weight, int weight_dtype, int64_t ws_h,
                                     float weight_offset, float eps, void *out, int64_t os_n, int64_t os_t,
                                     int64_t os_h, void *stream) {
    int64_t rows[3] = {n, t, h};
    int rc = check_norm(rows, d, weight_dtype, weight_offset, eps);
    if (rc != DCCONV_OK) return rc;
    if (any_negative({xs_n, xs_t, xs_h, zs_n, zs_t, zs_h, ws_h, os_n, os_t, os_h}))
        return fail(DCCONV_EINVAL, "strides must be non-negative");
    if (n == 0 || t == 0 || h == 0) return succeed("");
    if (!x || !out) return fail(DCCONV_EINVAL, "x and out must be non-NULL");
    if (!rows_distinct({n, t, h}, {os_n, os_t, os_h}, d))
        return fail(DCCONV_EINVAL, "out strides (%lld, %lld, %lld, 1) give two elements the same address",
                    (long long)os_n, (long long)os_t, (long long)os_h);
    int64_t xb, zb, wb, ob;
    if (!extent({n, t, h}, {xs_n, xs_t, xs_h}, d, 2, &xb) || !extent({n, t, h}, {zs_n, zs_t, zs_h}, d, 2, &zb) ||
        !extent({h, 1, 1}, {ws_h, 0, 0}, d, dtype_bytes(weight_dtype), &wb) ||
        !extent({n, t, h}, {os_n, os_t, os_h}, d, 2, &ob))
        return fail(DCCONV_EINVAL, "strides span more than 2^47 bytes");
    const Operand ops[] = {{"out", out, ob, 2, true},
                           {"x", x, xb, 2, false},
                           {"z", z, zb, 2, false},
                           {"weight", weight, wb, dtype_bytes(weight_dtype), false}};
    rc = check_operands(ops);
    if (rc != DCCONV_OK) return rc;
    dcconv::GatedNormParams q = {};
    q.x = static_cast<const uint16_t *>(x);
    q.z = static_cast<const uint16_t *>(z);
    q.xs_n = xs_n, q.xs_t = xs_t, q.xs_h = xs_h, q.zs_n = zs_n, q.zs_t = zs_t, q.zs_h = zs_h;
    q.weight = weight, q.ws_h = ws_h, q.weight_f32 = weight_dtype == DCCONV_DTYPE_F32;
    q.out = static_cast<uint16_t *>(out);
    q.os_n = os_n, q.os_t = os_t, q.os_h = os_h;
    q.n = n, q.t = t, q.h = h, q.d = (int32_t)d;
    q.offset = weight_offset, q.eps = eps, q.gate_first = gate_first != 0;
    const char *name = "";
    const hipError_t err = dcconv::launch_gated_norm(q, static_cast<hipStream_t>(stream), &name);
    if (err != hipSuccess) return fail(DCCONV_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return succeed(name);
}

extern "C" int dcconv_add_rms_norm(const void *x, int64_t n, int64_t t, int64_t d, int64_t xs_n, int64_t xs_t,
                                   void *residual, int residual_dtype, int64_t rs_n, int64_t rs_t, const void *gate,
                                   int64_t gs_n, int64_t gs_t, float residual_scale, const void *post_weight,
                                   const void *weight, int weight_dtype, float weight_offset, float eps, void *out,
                                   int64_t os_n, int64_t os_t, void *stream) {
    int64_t rows[3] = {n, t, 1};
    int rc = check_norm(rows, d, weight_dtype, weight_offset, eps);
    if (rc != DCCONV_OK) return rc;
    if (!known_dtype(residual_dtype))
        return fail(DCCONV_EINVAL, "residual_dtype must be DCCONV_DTYPE_BF16 (0) or DCCONV_DTYPE_F32 (1)");
    if (!isfinite(residual_scale))
        return fail(DCCONV_EINVAL, "residual_scale must be finite, got %g", (double)residual_scale);
    if (any_negative({xs_n, xs_t, rs_n, rs_t, gs_n, gs_t, os_n, os_t}))
        return fail(DCCONV_EINVAL, "strides must be non-negative");
    if (n == 0 || t == 0) return succeed("");
    if (!x || !residual || !weight || !out)
        return fail(DCCONV_EINVAL, "x, residual, weight and out must be non-NULL");
    if (!rows_distinct({n, t, 1}, {os_n, os_t, 0}, d) || !rows_distinct({n, t, 1}, {rs_n, rs_t, 0}, d))
        return fail(DCCONV_EINVAL, "out and residual strides must give every element its own address");
    const int64_t wsize = dtype_bytes(weight_dtype), rsize = dtype_bytes(residual_dtype);
    int64_t xb, rb, gb, ob;
    if (!extent({n, t, 1}, {xs_n, xs_t, 0}, d, 2, &xb) || !extent({n, t, 1}, {rs_n, rs_t, 0}, d, rsize, &rb) ||
        !extent({n, t, 1}, {gs_n, gs_t, 0}, d, 2, &gb) || !extent({n, t, 1}, {os_n, os_t, 0}, d, 2, &ob))
        return fail(DCCONV_EINVAL, "strides span more than 2^47 bytes");
    const Operand ops[] = {{"out", out, ob, 2, true},
                           {"residual", residual, rb, rsize, true},
                           {"x", x, xb, 2, false},
                           {"gate", gate, gb, 2, false},
                           {"post_weight", post_weight, wsize * d, wsize, false},
                           {"weight", weight, wsize * d, wsize, false}};
    rc = check_operands(ops);
    if (rc != DCCONV_OK) return rc;
    dcconv::AddNormParams q = {};
    q.x = static_cast<const uint16_t *>(x);
    q.gate = static_cast<const uint16_t *>(gate);
    q.xs_n = xs_n, q.xs_t = xs_t, q.gs_n = gs_n, q.gs_t = gs_t;
    q.residual = residual, q.rs_n = rs_n, q.rs_t = rs_t, q.residual_f32 = residual_dtype == DCCONV_DTYPE_F32;
    q.post = post_weight, q.weight = weight, q.weight_f32 = weight_dtype == DCCONV_DTYPE_F32;
    q.out = static_cast<uint16_t *>(out);
    q.os_n = os_n, q.os_t = os_t;
    q.n = n, q.t = t, q.d = (int32_t)d;
    q.residual_scale = residual_scale, q.offset = weight_offset, q.eps = eps;
    const char *name = "";
    const hipError_t err = dcconv::launch_add_norm(q, static_cast<hipStream_t>(stream), &name);
    if (err != hipSuccess) return fail(DCCONV_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return succeed(name);
}
