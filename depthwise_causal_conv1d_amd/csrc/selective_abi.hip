// C-ABI front end of the state-space operators: host-side validation and dispatch,
// under the same rules as the convolution's entry points (metadata only, nothing
// allocated, nothing synchronised, nothing enqueued on an error).
#include <stdint.h>

#include "abi_common.h"
#include "selective_params.h"

using namespace dcconv::abi;

namespace {

constexpr int64_t kMaxState = 256;  // state size k

// Bytes from an array's first element to its last: extents e at element strides
// st, `inner` dense elements behind them.  False when that passes 2^47 bytes.
bool extent(const int64_t (&e)[3], const int64_t (&st)[3], int64_t inner, int64_t elem, int64_t *bytes) {
    *bytes = 0;
    int64_t last = 0;
    const int64_t most = ((int64_t)1 << 47) / elem;
    if (inner <= 0) return true;
    if (inner > most) return false;
    for (int i = 0; i < 3; ++i)
        if (e[i] <= 0) return true;
    for (int i = 0; i < 3; ++i) {
        int64_t term;
        if (__builtin_mul_overflow(e[i] - 1, st[i], &term) || term > most) return false;
        last += term;
        if (last > most) return false;
    }
    if (last + inner > most) return false;
    *bytes = elem * (last + inner);
    return true;
}

// Whether rows of `inner` dense elements at extents e and strides st are disjoint.
bool rows_distinct(const int64_t (&e)[3], const int64_t (&st)[3], int64_t inner) {
    int order[3] = {0, 1, 2};
    for (int i = 1; i < 3; ++i)
        for (int j = i; j > 0 && st[order[j]] < st[order[j - 1]]; --j) {
            const int t = order[j];
            order[j] = order[j - 1];
            order[j - 1] = t;
        }
    int64_t below = inner;
    for (int i = 0; i < 3; ++i) {
        const int q = order[i];
        if (e[q] <= 1) continue;
        if (st[q] < below) return false;
        below += st[q] * (e[q] - 1);
    }
    return true;
}

struct Operand {
    const char *name;
    const void *ptr;
    int64_t bytes, align;
    bool written;
};

// Alignment of every operand, and none written that overlaps another.
template <int N>
int check_operands(const Operand (&ops)[N]) {
    for (const Operand &o : ops)
        if (o.ptr != nullptr && !aligned(o.ptr, (uintptr_t)o.align))
            return fail(DCCONV_EINVAL, "%s must be %lld-byte aligned", o.name, (long long)o.align);
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j)
            if (i != j && ops[i].written &&
                overlaps(span(ops[i].name, ops[i].ptr, ops[i].bytes), span(ops[j].name, ops[j].ptr, ops[j].bytes)))
                return fail(DCCONV_EINVAL, "%s overlaps %s", ops[i].name, ops[j].name);
    return DCCONV_OK;
}

bool known_dtype(int dtype) { return dtype == DCCONV_DTYPE_BF16 || dtype == DCCONV_DTYPE_F32; }
int64_t dtype_bytes(int dtype) { return dtype == DCCONV_DTYPE_F32 ? 4 : 2; }

// Shapes shared by the scan and the updates.  `stateless` calls have no pool.
int check_shapes(int64_t n, int64_t h, int64_t p, int64_t g, int64_t k, int dt_dtype, int state_dtype, int64_t s,
                 int64_t ss_s, bool has_indices, bool stateless) {
    if (n < 0) return fail(DCCONV_EINVAL, "n must be >= 0, got %lld", (long long)n);
    if (h < 1 || p < 1 || g < 1 || k < 1)
        return fail(DCCONV_EINVAL, "h, p, g and k must be >= 1, got %lld, %lld, %lld, %lld", (long long)h,
                    (long long)p, (long long)g, (long long)k);
    if (h % g != 0)
        return fail(DCCONV_EINVAL, "h=%lld heads do not divide into g=%lld groups", (long long)h, (long long)g);
    if (!known_dtype(dt_dtype) || !known_dtype(state_dtype))
        return fail(DCCONV_EINVAL, "dt_dtype and state_dtype must be DCCONV_DTYPE_BF16 (0) or DCCONV_DTYPE_F32 (1)");
    if (s < 0 || ss_s < 0) return fail(DCCONV_EINVAL, "s and ss_s must be >= 0");
    if (k > kMaxState)
        return fail(DCCONV_EUNSUPPORTED, "state sizes above %lld are not served, got k=%lld", (long long)kMaxState,
                    (long long)k);
    if (n > kI32Max - 1 || s > kI32Max || h > (1 << 20) || p > (1 << 20) || h * p > (1 << 26) || g * k > (1 << 26))
        return fail(DCCONV_EUNSUPPORTED, "sizes beyond n, s < 2^31, h, p <= 2^20 and h*p, g*k <= 2^26 are not served");
    if (!stateless) {
        if (s > 1 && ss_s < h * p * k)
            return fail(DCCONV_EINVAL, "ssm_state slots overlap: stride %lld, %lld elements", (long long)ss_s,
                        (long long)(h * p * k));
        if (!has_indices && s < n)
            return fail(DCCONV_EINVAL, "without state_indices row r uses slot r, so s=%lld must be >= n=%lld",
                        (long long)s, (long long)n);
    }
    return DCCONV_OK;
}

template <int N>
bool any_negative(const int64_t (&v)[N]) {
    for (int64_t x : v)
        if (x < 0) return true;
    return false;
}

// A slot stride, h*p*k elements behind it; false past 2^47 bytes.
bool state_extent(int64_t s, int64_t ss_s, int64_t inner, int dtype, int64_t *bytes) {
    return extent({s, 1, 1}, {ss_s, 0, 0}, inner, dtype_bytes(dtype), bytes);
}

}  // namespace

extern "C" int dcconv_selective_update(const void *x, int64_t n, int64_t h, int64_t p, int64_t xs_n, int64_t xs_h,
                                       const void *dt, int dt_dtype, int64_t ds_n, const float *dt_bias,
                                       int dt_softplus, const float *a, const void *b, const void *c, int64_t g,
                                       int64_t k, int64_t bs_n, int64_t bs_g, int64_t cs_n, int64_t cs_g,
                                       const float *d_skip, const void *z, int64_t zs_n, int64_t zs_h,
                                       void *ssm_state, int state_dtype, int64_t s, int64_t ss_s,
                                       const int32_t *state_indices, void *out, int64_t os_n, int64_t os_h,
                                       int32_t *dev_status, void *stream) {
    int rc = check_shapes(n, h, p, g, k, dt_dtype, state_dtype, s, ss_s, state_indices != nullptr, false);
    if (rc != DCCONV_OK) return rc;
    if (any_negative({xs_n, xs_h, ds_n, bs_n, bs_g, cs_n, cs_g, zs_n, zs_h, os_n, os_h}))
        return fail(DCCONV_EINVAL, "strides must be non-negative");
    if (n == 0) return succeed("");
    if (!x || !dt || !a || !b || !c || !out || (!ssm_state && s > 0))
        return fail(DCCONV_EINVAL, "x, dt, a, b, c, out (and ssm_state when s > 0) must be non-NULL when n > 0");
    if (!rows_distinct({n, h, 1}, {os_n, os_h, 0}, p))
        return fail(DCCONV_EINVAL, "out strides (%lld, %lld, 1) give two elements the same address", (long long)os_n,
                    (long long)os_h);
    int64_t xb, db, bb, cb, zb, sb, ob;
    if (!extent({n, h, 1}, {xs_n, xs_h, 0}, p, 2, &xb) || !extent({n, 1, 1}, {ds_n, 0, 0}, h, dtype_bytes(dt_dtype), &db) ||
        !extent({n, g, 1}, {bs_n, bs_g, 0}, k, 2, &bb) || !extent({n, g, 1}, {cs_n, cs_g, 0}, k, 2, &cb) ||
        !extent({n, h, 1}, {zs_n, zs_h, 0}, p, 2, &zb) || !state_extent(s, ss_s, h * p * k, state_dtype, &sb) ||
        !extent({n, h, 1}, {os_n, os_h, 0}, p, 2, &ob))
        return fail(DCCONV_EINVAL, "strides span more than 2^47 bytes");
    const Operand ops[] = {{"out", out, ob, 2, true},
                           {"ssm_state", ssm_state, sb, dtype_bytes(state_dtype), true},
                           {"dev_status", dev_status, 4, 4, true},
                           {"x", x, xb, 2, false},
                           {"dt", dt, db, dtype_bytes(dt_dtype), false},
                           {"dt_bias", dt_bias, 4 * h, 4, false},
                           {"a", a, 4 * h, 4, false},
                           {"b", b, bb, 2, false},
                           {"c", c, cb, 2, false},
                           {"d_skip", d_skip, 4 * h, 4, false},
                           {"z", z, zb, 2, false},
                           {"state_indices", state_indices, 4 * n, 4, false}};
    rc = check_operands(ops);
    if (rc != DCCONV_OK) return rc;

    dcconv::SelectiveUpdateParams q = {};
    q.x = static_cast<const uint16_t *>(x);
    q.xs_n = xs_n;
    q.xs_h = xs_h;
    q.b = static_cast<const uint16_t *>(b);
    q.c = static_cast<const uint16_t *>(c);
    q.bs_n = bs_n;
    q.bs_g = bs_g;
    q.cs_n = cs_n;
    q.cs_g = cs_g;
    q.dt = dt;
    q.ds_n = ds_n;
    q.dt_bias = dt_bias;
    q.a = a;
    q.d_skip = d_skip;
    q.z = static_cast<const uint16_t *>(z);
    q.zs_n = zs_n;
    q.zs_h = zs_h;
    q.state = ssm_state;
    q.ss_s = ss_s;
    q.idx = state_indices;
    q.status = dev_status;
    q.out = static_cast<uint16_t *>(out);
    q.os_n = os_n;
    q.os_h = os_h;
    q.n = (int32_t)n;
    q.h = (int32_t)h;
    q.p = (int32_t)p;
    q.g = (int32_t)g;
    q.k = (int32_t)k;
    q.s = (int32_t)s;
    q.dt_f32 = dt_dtype == DCCONV_DTYPE_F32;
    q.dt_softplus = dt_softplus != 0;
    q.state_f32 = state_dtype == DCCONV_DTYPE_F32;
    const char *name = "";
    const hipError_t err = dcconv::launch_selective_update(q, static_cast<hipStream_t>(stream), &name);
    if (err != hipSuccess) return fail(DCCONV_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return succeed(name);
}

extern "C" int dcconv_conv_selective_update(const void *xbc, int64_t n, int64_t h, int64_t p, int64_t g, int64_t k,
                                            int64_t xbcs_n, void *conv_state, int64_t l, int64_t st_s, int64_t st_d,
                                            int64_t st_l, const void *weight, int64_t w, const void *bias,
                                            const int32_t *cache_seqlens, int activation, const void *dt,
                                            int dt_dtype, int64_t ds_n, const float *dt_bias, int dt_softplus,
                                            const float *a, const float *d_skip, const void *z, int64_t zs_n,
                                            int64_t zs_h, void *ssm_state, int state_dtype, int64_t s, int64_t ss_s,
                                            const int32_t *state_indices, void *out, int64_t os_n, int64_t os_h,
                                            int32_t *workspace, int32_t *dev_status, void *stream) {
    int rc = check_shapes(n, h, p, g, k, dt_dtype, state_dtype, s, ss_s, state_indices != nullptr, false);
    if (rc != DCCONV_OK) return rc;
    if (any_negative({xbcs_n, st_s, st_d, st_l, ds_n, zs_n, zs_h, os_n, os_h}))
        return fail(DCCONV_EINVAL, "strides must be non-negative");
    if (w < 1) return fail(DCCONV_EINVAL, "w (filter width) must be >= 1, got %lld", (long long)w);
    if (l < w - 1)
        return fail(DCCONV_EINVAL, "conv_state length l=%lld must be >= w-1=%lld", (long long)l, (long long)(w - 1));
    if (activation != DCCONV_ACT_IDENTITY && activation != DCCONV_ACT_SILU)
        return fail(DCCONV_EINVAL, "activation must be DCCONV_ACT_IDENTITY (0) or DCCONV_ACT_SILU (1), got %d",
                    activation);
    if (w != 4) return fail(DCCONV_EUNSUPPORTED, "only filter width w=4 is served, got w=%lld", (long long)w);
    if (l > 65536) return fail(DCCONV_EUNSUPPORTED, "l=%lld > 65536 is not served", (long long)l);
    const int64_t d = h * p + 2 * g * k;
    if (s > 0 && !rows_distinct({s, d, l}, {st_s, st_d, st_l}, 1))
        return fail(DCCONV_EINVAL, "conv_state strides (%lld, %lld, %lld) give two elements the same address",
                    (long long)st_s, (long long)st_d, (long long)st_l);
    if (n == 0) return succeed("");
    if (!xbc || !weight || !dt || !a || !out || !workspace || ((!ssm_state || !conv_state) && s > 0))
        return fail(DCCONV_EINVAL,
                    "xbc, weight, dt, a, out, workspace (and both states when s > 0) must be non-NULL when n > 0");
    if (!rows_distinct({n, h, 1}, {os_n, os_h, 0}, p))
        return fail(DCCONV_EINVAL, "out strides (%lld, %lld, 1) give two elements the same address", (long long)os_n,
                    (long long)os_h);
    int64_t xb, vb, db, zb, sb, ob;
    if (!extent({n, 1, 1}, {xbcs_n, 0, 0}, d, 2, &xb) || !extent({s, d, l}, {st_s, st_d, st_l}, 1, 2, &vb) ||
        !extent({n, 1, 1}, {ds_n, 0, 0}, h, dtype_bytes(dt_dtype), &db) ||
        !extent({n, h, 1}, {zs_n, zs_h, 0}, p, 2, &zb) || !state_extent(s, ss_s, h * p * k, state_dtype, &sb) ||
        !extent({n, h, 1}, {os_n, os_h, 0}, p, 2, &ob))
        return fail(DCCONV_EINVAL, "strides span more than 2^47 bytes");
    const Operand ops[] = {{"out", out, ob, 2, true},
                           {"ssm_state", ssm_state, sb, dtype_bytes(state_dtype), true},
                           {"conv_state", conv_state, vb, 2, true},
                           {"workspace", workspace, 4 * n * g, 4, true},
                           {"dev_status", dev_status, 4, 4, true},
                           {"xbc", xbc, xb, 2, false},
                           {"weight", weight, 8 * d, 2, false},
                           {"bias", bias, 2 * d, 2, false},
                           {"cache_seqlens", cache_seqlens, 4 * n, 4, false},
                           {"dt", dt, db, dtype_bytes(dt_dtype), false},
                           {"dt_bias", dt_bias, 4 * h, 4, false},
                           {"a", a, 4 * h, 4, false},
                           {"d_skip", d_skip, 4 * h, 4, false},
                           {"z", z, zb, 2, false},
                           {"state_indices", state_indices, 4 * n, 4, false}};
    rc = check_operands(ops);
    if (rc != DCCONV_OK) return rc;

    dcconv::SelectiveUpdateParams q = {};
    q.dt = dt;
    q.ds_n = ds_n;
    q.dt_bias = dt_bias;
    q.a = a;
    q.d_skip = d_skip;
    q.z = static_cast<const uint16_t *>(z);
    q.zs_n = zs_n;
    q.zs_h = zs_h;
    q.state = ssm_state;
    q.ss_s = ss_s;
    q.idx = state_indices;
    q.status = dev_status;
    q.out = static_cast<uint16_t *>(out);
    q.os_n = os_n;
    q.os_h = os_h;
    q.n = (int32_t)n;
    q.h = (int32_t)h;
    q.p = (int32_t)p;
    q.g = (int32_t)g;
    q.k = (int32_t)k;
    q.s = (int32_t)s;
    q.dt_f32 = dt_dtype == DCCONV_DTYPE_F32;
    q.dt_softplus = dt_softplus != 0;
    q.state_f32 = state_dtype == DCCONV_DTYPE_F32;
    q.conv = true;
    q.xbc = static_cast<const uint16_t *>(xbc);
    q.xbcs_n = xbcs_n;
    q.conv_state = static_cast<uint16_t *>(conv_state);
    q.st_s = st_s;
    q.st_d = st_d;
    q.st_l = st_l;
    q.weight = static_cast<const uint16_t *>(weight);
    q.bias = static_cast<const uint16_t *>(bias);
    q.seqlens = cache_seqlens;
    q.arrivals = workspace;
    q.l = (int32_t)l;
    q.silu = activation == DCCONV_ACT_SILU;
    const char *name = "";
    const hipError_t err = dcconv::launch_selective_update(q, static_cast<hipStream_t>(stream), &name);
    if (err != hipSuccess) return fail(DCCONV_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return succeed(name);
}

extern "C" int64_t dcconv_selective_scan_workspace(int64_t n, int64_t t, int64_t h, int64_t p, int64_t g, int64_t k,
                                                   int packed) {
    if (n < 1 || t < 1 || h < 1 || p < 1 || g < 1 || k < 1 || h % g != 0 || n > kI32Max - 1 || t > kI32Max ||
        h > (1 << 20) || p > (1 << 20) || h * p > (1 << 26) || k > kMaxState)
        return 0;
    return 4 * dcconv::selective_scan_workspace_floats(n, t, h, p, g, k, packed != 0);
}

extern "C" int dcconv_selective_scan(const void *x, int64_t n, int64_t t, int64_t h, int64_t p, int64_t xs_n,
                                     int64_t xs_t, int64_t xs_h, const void *dt, int dt_dtype, int64_t ds_n,
                                     int64_t ds_t, const float *dt_bias, int dt_softplus, const float *a,
                                     const void *b, const void *c, int64_t g, int64_t k, int64_t bs_n, int64_t bs_t,
                                     int64_t bs_g, int64_t cs_n, int64_t cs_t, int64_t cs_g, const float *d_skip,
                                     const void *z, int64_t zs_n, int64_t zs_t, int64_t zs_h,
                                     const int32_t *seq_starts, void *ssm_state, int state_dtype, int64_t s,
                                     int64_t ss_s, const int32_t *state_indices, const uint8_t *has_initial_state,
                                     void *out, int64_t os_n, int64_t os_t, int64_t os_h, void *workspace,
                                     int64_t workspace_bytes, int32_t *dev_status, void *stream) {
    const bool stateless = ssm_state == nullptr && s == 0;
    if (stateless && (has_initial_state != nullptr || state_indices != nullptr))
        return fail(DCCONV_EINVAL, "has_initial_state and state_indices need an ssm_state");
    int rc = check_shapes(n, h, p, g, k, dt_dtype, state_dtype, s, ss_s, state_indices != nullptr, stateless);
    if (rc != DCCONV_OK) return rc;
    if (t < 0) return fail(DCCONV_EINVAL, "t (tokens) must be >= 0, got %lld", (long long)t);
    if (t > kI32Max - 1024 || n > kI32Max - (1 << 24))
        return fail(DCCONV_EUNSUPPORTED, "t >= 2^31 - 1024 tokens or n >= 2^31 - 2^24 sequences is not served");
    if (any_negative({xs_n, xs_t, xs_h, ds_n, ds_t, bs_n, bs_t, bs_g, cs_n, cs_t, cs_g, zs_n, zs_t, zs_h, os_n, os_t,
                      os_h, workspace_bytes}))
        return fail(DCCONV_EINVAL, "strides and workspace_bytes must be non-negative");
    if (n == 0 || (t == 0 && stateless)) return succeed("");
    const bool packed = seq_starts != nullptr;
    const int64_t rows = packed ? 1 : n;
    if (!a || (!ssm_state && s > 0) || (t > 0 && (!x || !dt || !b || !c || !out)))
        return fail(DCCONV_EINVAL, "x, dt, a, b, c, out (and ssm_state when s > 0) must be non-NULL");
    if (t > 0 && !rows_distinct({rows, t, h}, {os_n, os_t, os_h}, p))
        return fail(DCCONV_EINVAL, "out strides (%lld, %lld, %lld, 1) give two elements the same address",
                    (long long)os_n, (long long)os_t, (long long)os_h);
    int64_t xb, db, bb, cb, zb, sb, ob;
    if (!extent({rows, t, h}, {xs_n, xs_t, xs_h}, p, 2, &xb) ||
        !extent({rows, t, 1}, {ds_n, ds_t, 0}, h, dtype_bytes(dt_dtype), &db) ||
        !extent({rows, t, g}, {bs_n, bs_t, bs_g}, k, 2, &bb) || !extent({rows, t, g}, {cs_n, cs_t, cs_g}, k, 2, &cb) ||
        !extent({rows, t, h}, {zs_n, zs_t, zs_h}, p, 2, &zb) || !state_extent(s, ss_s, h * p * k, state_dtype, &sb) ||
        !extent({rows, t, h}, {os_n, os_t, os_h}, p, 2, &ob))
        return fail(DCCONV_EINVAL, "strides span more than 2^47 bytes");
    const int64_t need = dcconv_selective_scan_workspace(n, t, h, p, g, k, packed);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(DCCONV_EINVAL, "workspace of %lld bytes needed, got %lld", (long long)need,
                    (long long)(workspace ? workspace_bytes : 0));
    const Operand ops[] = {{"out", out, ob, 2, true},
                           {"ssm_state", ssm_state, sb, dtype_bytes(state_dtype), true},
                           {"workspace", workspace, need, 16, true},
                           {"dev_status", dev_status, 4, 4, true},
                           {"x", x, xb, 2, false},
                           {"dt", dt, db, dtype_bytes(dt_dtype), false},
                           {"dt_bias", dt_bias, 4 * h, 4, false},
                           {"a", a, 4 * h, 4, false},
                           {"b", b, bb, 2, false},
                           {"c", c, cb, 2, false},
                           {"d_skip", d_skip, 4 * h, 4, false},
                           {"z", z, zb, 2, false},
                           {"seq_starts", seq_starts, 4 * (n + 1), 4, false},
                           {"state_indices", state_indices, 4 * n, 4, false},
                           {"has_initial_state", has_initial_state, n, 1, false}};
    rc = check_operands(ops);
    if (rc != DCCONV_OK) return rc;

    dcconv::SelectiveScanParams q = {};
    q.x = static_cast<const uint16_t *>(x);
    q.xs_n = packed ? 0 : xs_n;
    q.xs_t = xs_t;
    q.xs_h = xs_h;
    q.b = static_cast<const uint16_t *>(b);
    q.c = static_cast<const uint16_t *>(c);
    q.bs_n = packed ? 0 : bs_n;
    q.bs_t = bs_t;
    q.bs_g = bs_g;
    q.cs_n = packed ? 0 : cs_n;
    q.cs_t = cs_t;
    q.cs_g = cs_g;
    q.dt = dt;
    q.ds_n = packed ? 0 : ds_n;
    q.ds_t = ds_t;
    q.dt_bias = dt_bias;
    q.a = a;
    q.d_skip = d_skip;
    q.z = static_cast<const uint16_t *>(z);
    q.zs_n = packed ? 0 : zs_n;
    q.zs_t = zs_t;
    q.zs_h = zs_h;
    q.starts = seq_starts;
    q.state = ssm_state;
    q.ss_s = ss_s;
    q.idx = state_indices;
    q.has_init = has_initial_state;
    q.status = dev_status;
    q.out = static_cast<uint16_t *>(out);
    q.os_n = packed ? 0 : os_n;
    q.os_t = os_t;
    q.os_h = os_h;
    q.workspace = static_cast<float *>(workspace);
    q.n = (int32_t)n;
    q.t = (int32_t)t;
    q.h = (int32_t)h;
    q.p = (int32_t)p;
    q.g = (int32_t)g;
    q.k = (int32_t)k;
    q.s = (int32_t)s;
    q.dt_f32 = dt_dtype == DCCONV_DTYPE_F32;
    q.dt_softplus = dt_softplus != 0;
    q.state_f32 = state_dtype == DCCONV_DTYPE_F32;
    const char *name = "";
    const hipError_t err = dcconv::launch_selective_scan(q, static_cast<hipStream_t>(stream), &name);
    if (err != hipSuccess) return fail(DCCONV_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return succeed(name);
}

namespace {

// Shapes of a 4-bit weight matrix.
int check_w4(int64_t n, int64_t k) {
    if (n < 1 || k < 1)
        return fail(DCCONV_EINVAL, "n and k must be >= 1, got %lld and %lld", (long long)n, (long long)k);
    if (n > (1 << 24) || k > (1 << 24))
        return fail(DCCONV_EUNSUPPORTED, "n and k above 2^24 are not served, got %lld and %lld", (long long)n,
                    (long long)k);
    return DCCONV_OK;
}

int64_t w4_bytes(int64_t n, int64_t k) { return (n + 15) / 16 * ((k + 127) / 128) * 1024; }

}  // namespace

extern "C" int dcconv_w4_matvec(const void *x, int64_t m, int64_t k, int64_t xs_m, const void *qweight, int64_t n,
                                const void *scales, const uint8_t *zeros, int64_t group_size, const void *bias,
                                void *out, int64_t os_m, void *stream) {
    int rc = check_w4(n, k);
    if (rc != DCCONV_OK) return rc;
    if (m < 0) return fail(DCCONV_EINVAL, "m must be >= 0, got %lld", (long long)m);
    if (group_size < 1) return fail(DCCONV_EINVAL, "group_size must be >= 1, got %lld", (long long)group_size);
    if (xs_m < 0 || os_m < 0) return fail(DCCONV_EINVAL, "strides must be non-negative");
    if (group_size % 32 != 0 || group_size > (1 << 24))
        return fail(DCCONV_EUNSUPPORTED, "group_size must be a multiple of 32 up to 2^24, got %lld",
                    (long long)group_size);
    if (m > (1 << 20) - 64) return fail(DCCONV_EUNSUPPORTED, "m=%lld rows are not served", (long long)m);
    if (m == 0) return succeed("");
    if (!x || !qweight || !scales || !out)
        return fail(DCCONV_EINVAL, "x, qweight, scales and out must be non-NULL when m > 0");
    if (m > 1 && os_m < n)
        return fail(DCCONV_EINVAL, "out row stride %lld is smaller than n=%lld", (long long)os_m, (long long)n);
    int64_t xb, ob;
    if (!extent({m, 1, 1}, {xs_m, 0, 0}, k, 2, &xb) || !extent({m, 1, 1}, {os_m, 0, 0}, n, 2, &ob))
        return fail(DCCONV_EINVAL, "strides span more than 2^47 bytes");
    const int64_t groups = (k + group_size - 1) / group_size;
    const Operand ops[] = {{"out", out, ob, 2, true},
                           {"x", x, xb, 2, false},
                           {"qweight", qweight, w4_bytes(n, k), 16, false},
                           {"scales", scales, 2 * groups * n, 2, false},
                           {"zeros", zeros, groups * n, 1, false},
                           {"bias", bias, 2 * n, 2, false}};
    rc = check_operands(ops);
    if (rc != DCCONV_OK) return rc;

    dcconv::W4Params q = {};
    q.x = static_cast<const uint16_t *>(x);
    q.xs_m = xs_m;
    q.q = static_cast<const uint8_t *>(qweight);
    q.scales = static_cast<const uint16_t *>(scales);
    q.zeros = zeros;
    q.bias = static_cast<const uint16_t *>(bias);
    q.out = static_cast<uint16_t *>(out);
    q.os_m = os_m;
    q.m = (int32_t)m;
    q.n = (int32_t)n;
    q.k = (int32_t)k;
    q.group = (int32_t)group_size;
    const char *name = "";
    const hipError_t err = dcconv::launch_w4_matvec(q, static_cast<hipStream_t>(stream), &name);
    if (err != hipSuccess) return fail(DCCONV_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return succeed(name);
}

extern "C" int dcconv_w4_pack(const uint8_t *codes, int64_t n, int64_t k, void *qweight, void *stream) {
    int rc = check_w4(n, k);
    if (rc != DCCONV_OK) return rc;
    if (!codes || !qweight) return fail(DCCONV_EINVAL, "codes and qweight must be non-NULL");
    const Operand ops[] = {{"qweight", qweight, w4_bytes(n, k), 16, true}, {"codes", codes, n * k, 1, false}};
    rc = check_operands(ops);
    if (rc != DCCONV_OK) return rc;
    const hipError_t err =
        dcconv::launch_w4_pack(codes, n, k, static_cast<uint8_t *>(qweight), static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return fail(DCCONV_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return succeed("w4_pack");
}
