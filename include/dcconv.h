/*
 * dcconv.h -- C ABI of the MI355X (gfx950) depthwise causal conv1d library.
 *
 * The operation is the decode update described on the cuDNN FE-OSS page
 * "Causal Conv1d Decode Update" (docs.nvidia.com/cudnn/latest/fe-oss-apis/
 * causal_conv1d_update): for every decode row n, channel d and the cache slot s
 * the row selects,
 *
 *     history            = concat(conv_state[s, d, :], x[n, d])      (length L+1)
 *     conv_state[s, d, :] = newest L values of history
 *     out[n, d]          = act(sum_j history[L+1-W+j] * weight[d, j] + bias[d])
 *
 * (page section "Causal Conv1d Decode Update").  Sums are formed in FP32 and
 * rounded once to BF16 (round to nearest even).
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers (HIP device memory or memory the
 *    device can address), except where a comment says otherwise.
 *  - The caller owns every buffer.  The library allocates nothing, never
 *    synchronises, never reads device memory from the host and converts nothing,
 *    so a call may be captured into a HIP graph (stable pointers).
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream) and is
 *    asynchronous; results are visible after the stream is synchronised.
 *  - Metadata is validated on the host, in full, before anything is enqueued.
 *    A non-zero return means nothing was enqueued; dcconv_last_error() then
 *    describes the problem (thread-local, valid until the next call on the same
 *    thread).
 *  - Elements are BF16 carried as 16-bit patterns; indices are int32.
 */
#ifndef DCCONV_H
#define DCCONV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DCCONV_ABI_VERSION 1

/* Return codes.  The page distinguishes a contract violation (Python ValueError)
 * from a valid request the implementation does not serve (NotImplementedError);
 * section "Current native implementation". */
enum {
    DCCONV_OK = 0,
    DCCONV_EINVAL = 1,       /* contract violation: shape, stride, alignment, overlap, null */
    DCCONV_EUNSUPPORTED = 2, /* semantically valid but not served (e.g. W != 4) */
    DCCONV_EHIP = 3          /* the HIP runtime refused the launch (hipGetLastError) */
};

/* Activations (page section "Causal Conv1d Decode Update": None/"identity" and
 * "silu"/"swish").  Each is a separate compiled kernel; the identity kernel
 * contains no activation code. */
enum { DCCONV_ACT_IDENTITY = 0, DCCONV_ACT_SILU = 1 };

/* Element types where an operand may have either. */
enum { DCCONV_DTYPE_BF16 = 0, DCCONV_DTYPE_F32 = 1 };

/* Bits OR-ed into *dev_status by the device when a routing entry is rejected. */
enum {
    DCCONV_DEV_BAD_INDEX = 1, /* an index below -1, or not below S           */
    DCCONV_DEV_DUP_INDEX = 2, /* two rows of the batch select one real slot  */
    DCCONV_DEV_BAD_SEQ = 4,   /* dcconv_prefill, dcconv_selective_scan, dcconv_gated_delta_scan:
                                 seq_starts is not 0 = starts[0] <= starts[1] <= ... <= starts[n] = t */
    DCCONV_DEV_BAD_SEQLEN = 8 /* dcconv_update, dcconv_update_tokens and
                                 dcconv_conv_selective_update: a cache_seqlens entry below 0 */
};

/* The DCCONV_ABI_VERSION the library was built with. */
int dcconv_abi_version(void);

/* Message for the last non-OK return on the calling thread ("" if none). */
const char *dcconv_last_error(void);

/* Name of the kernel specialisation the last successful call on the calling
 * thread enqueued ("" if that call enqueued nothing).  Lets a benchmark prove
 * which route ran. */
const char *dcconv_last_kernel(void);

/*
 * dcconv_update -- one decode step, in place.
 * Defined by the page section "Causal Conv1d Decode Update" (update rule, bias
 * default, activations, slot routing, padding rows) and section "Semantic tensor
 * contract" (shapes, strides, alignment); the limits of the served subset follow
 * section "Current native implementation".
 *
 * x           BF16 [n, d], element (r, c) at x[r*ld_x + c].  ld_x == d, or
 *             ld_x > d with ld_x % 8 == 0 (16-byte aligned rows).  Columns
 *             d..ld_x-1 are never read.
 * n           decode rows, n >= 0.  n == 0 returns DCCONV_OK and enqueues nothing.
 * d           channels, d >= 1.
 * conv_state  BF16 [s, d, l], READ AND WRITTEN.  Element (slot, c, k) at
 *             conv_state[slot*st_s + c*st_d + k*st_l]; k = 0 is the oldest value.
 *             Accepted layouts: compact (st_d == l, st_l == 1, st_s >= d*l) and
 *             channel-last (st_d == 1, st_l == d, st_s >= l*d; the layout a
 *             full-sequence prefill hands over).
 * s           slots, s >= 0; without an index table s >= n (row r uses slot r).
 *             With s == 0 every row must be padding and conv_state may be NULL.
 * l           history length, l >= w - 1.
 * weight      BF16 [d, w] contiguous.  Only w == 4 is served.
 * bias        BF16 [d] or NULL (zero bias).
 * conv_state_indices  int32 [n] or NULL.  Row r uses slot conv_state_indices[r];
 *             -1 marks a padding row: its output is zero and no slot changes
 *             (repeated -1 is allowed).  Other values must lie in [0, s) and be
 *             unique within the call.  An entry below -1 or >= s makes that row
 *             behave as a padding row and sets DCCONV_DEV_BAD_INDEX.  When
 *             dev_status is non-NULL every row whose slot is shared with another
 *             row is also treated as padding (so that slot is left untouched)
 *             and DCCONV_DEV_DUP_INDEX is set; when dev_status is NULL duplicates
 *             are not detected and the result for the shared slot is unspecified
 *             (the page calls such an update "not transactional").
 * cache_seqlens  NULL, or int32 [n]: circular-buffer state, the use the page
 *             reserves this keyword for (section "Causal Conv1d Decode Update").
 *             c = cache_seqlens[r] is the number of tokens row r's slot has seen;
 *             the slot keeps token i at position i mod l (k is then a ring
 *             position, not an age).  The taps are tokens c-3, c-2, c-1, read at
 *             positions (c-3+k) mod l before any write, and x; x then replaces
 *             the oldest token at position c mod l, and no other value moves
 *             (one element per channel is written).  cache_seqlens is only read
 *             (the caller advances it).  An entry below 0 makes the row behave
 *             as padding and sets DCCONV_DEV_BAD_SEQLEN.  Read-only; 4-byte
 *             aligned; must not overlap anything the call writes.
 * activation  DCCONV_ACT_IDENTITY or DCCONV_ACT_SILU (SiLU(v) = v / (1 + e^-v)).
 * out         BF16 [n, d] contiguous, written.  Must not overlap any operand.
 * dev_status  NULL, or a device int32 the kernel ORs DCCONV_DEV_* bits into.
 *             It is never cleared by the library.
 * stream      hipStream_t to enqueue on; NULL = null stream.
 *
 * Alignment: every BF16 pointer 16-byte aligned, indices and dev_status 4-byte
 * aligned (page section "Current native implementation").  conv_state must not
 * overlap x, weight, bias, the index table, out or dev_status.
 *
 * Returns DCCONV_OK, DCCONV_EINVAL (contract violation), DCCONV_EUNSUPPORTED
 * (valid but not served), or DCCONV_EHIP (launch refused by the runtime).
 */
int dcconv_update(const void *x, int64_t n, int64_t d, int64_t ld_x,
                  void *conv_state, int64_t s, int64_t l,
                  int64_t st_s, int64_t st_d, int64_t st_l,
                  const void *weight, int64_t w,
                  const void *bias,
                  const int32_t *conv_state_indices,
                  const int32_t *cache_seqlens,
                  int activation,
                  void *out,
                  int32_t *dev_status,
                  void *stream);

/*
 * dcconv_update_tokens -- T successive decode steps on the same slots, in place.
 * The multi-token form the page reserves for x[N, D, Tstep] (section "Semantic
 * tensor contract": the state and weight meanings do not change): token t of
 * every row is applied, in order t = 0..T-1, by exactly the rule of
 * dcconv_update, and out[:, :, t] is that step's output.  One call reads and
 * writes each selected state once instead of T times.
 *
 * x           BF16, element (r, c, t) at x[r*xs_n + c*xs_d + t*xs_t]; strides >= 0.
 * n, d, t     rows, channels, tokens (t == 0 or n == 0: DCCONV_OK, nothing enqueued).
 * out         BF16, element (r, c, t) at out[r*os_n + c*os_d + t*os_t]; the strides
 *             must give every element its own address (no two (r, c, t) alias).
 * cache_seqlens  NULL, or int32 [n]: circular-buffer state as for
 * dcconv_update; token t of row r is the (cache_seqlens[r] + t)-th token its
 * slot sees: its taps are tokens c+t-3 .. c+t-1 (from the ring for the first
 * three, from x after that) and it lands at position (c + t) mod l.  Only the
 * last min(t, l) tokens remain in the ring; the count is only read.
 * conv_state, s, l, st_*, weight, w, bias, conv_state_indices,
 * activation, dev_status, stream: exactly as for dcconv_update (the routing of a
 * row is the same for all of its tokens; a padding or rejected row writes zeros
 * for every token and leaves the state untouched).
 *
 * Alignment: x, out and the other BF16 pointers 16-byte aligned.  The fast path
 * additionally needs unit channel strides and row/token strides that are
 * multiples of 8 elements; other strides are served by a per-element path.
 * Nothing the call writes may overlap any other operand.
 *
 * Returns DCCONV_OK, DCCONV_EINVAL, DCCONV_EUNSUPPORTED or DCCONV_EHIP, with the
 * same meanings as for dcconv_update.
 */
int dcconv_update_tokens(const void *x, int64_t n, int64_t d, int64_t t,
                         int64_t xs_n, int64_t xs_d, int64_t xs_t,
                         void *conv_state, int64_t s, int64_t l,
                         int64_t st_s, int64_t st_d, int64_t st_l,
                         const void *weight, int64_t w,
                         const void *bias,
                         const int32_t *conv_state_indices,
                         const int32_t *cache_seqlens,
                         int activation,
                         void *out, int64_t os_n, int64_t os_d, int64_t os_t,
                         int32_t *dev_status,
                         void *stream);

/*
 * dcconv_prefill -- full-sequence causal convolution (prefill), returning the
 * final state that dcconv_update continues.
 *
 * The decode page names this operation at its top (cudnn.ops.causal_conv1d, for
 * full sequences; its width-four final state is handed to the update, section
 * "Semantic tensor contract": an L=3 state from prefill is accepted in place).
 * Its own page is not among the sources; this follows the plainest reading the
 * decode page supports.  For sequence i (slot s) and channel c:
 *
 *     ext          = concat(init[0:L], x[i, c, 0:T_i])     init = slot s's state or zeros
 *     out[i, c, j] = act(sum_k ext[L + j - 3 + k] * weight[c, k] + bias[c])
 *     slot s       = ext[T_i : T_i + L]                     (the newest L values)
 *
 * Sequences -- two forms:
 *   seq_starts == NULL  n sequences of t tokens each; token j of sequence i,
 *                       channel c at x[i*xs_n + c*xs_d + j*xs_t] (out likewise).
 *   seq_starts != NULL  device int32 [n+1], 0 = starts[0] <= ... <= starts[n] = t:
 *                       sequence i is packed tokens starts[i] .. starts[i+1]-1,
 *                       token p at x[c*xs_d + p*xs_t]; xs_n and os_n are unused.
 *                       A table that breaks the ordering sets DCCONV_DEV_BAD_SEQ
 *                       in *dev_status; outputs and states are then unspecified
 *                       (every access still stays inside the operands).
 * State:
 *   conv_state == NULL  no initial and no final state (history starts at zero);
 *                       s must be 0, conv_state_indices and has_initial_state
 *                       NULL; l and st_* are ignored.
 *   conv_state != NULL  [s, d, l] at strides (st_s, st_d, st_l), compact or
 *                       channel-last as for dcconv_update (channel-last l = 3 is
 *                       the hand-off layout).  Sequence i uses slot
 *                       conv_state_indices[i] (or i); -1 is a padding sequence:
 *                       zero outputs, no slot touched; bad and duplicate indices
 *                       as for dcconv_update.  The final state replaces the slot.
 *   has_initial_state   device uint8 [n] or NULL.  Nonzero: sequence i continues
 *                       from its slot's state; zero or NULL: from zeros.
 * x, out           BF16 at element strides >= 0; out must give every element its
 *                  own address.  16-byte aligned; seq_starts 4-byte aligned.
 *                  Nothing the call writes may overlap any other operand.
 * weight, w, bias, activation, dev_status, stream: as for dcconv_update.
 *
 * t == 0 (or every sequence empty) still writes the final states (the initial
 * state unchanged, or zeros).  n == 0: DCCONV_OK, nothing enqueued.
 * The fast path needs d % 8 == 0, unit channel strides, token and row strides
 * that are multiples of 8 and 3 <= l <= 8; other shapes take a per-element path.
 *
 * Returns DCCONV_OK, DCCONV_EINVAL, DCCONV_EUNSUPPORTED or DCCONV_EHIP, with the
 * same meanings as for dcconv_update.
 */
int dcconv_prefill(const void *x, int64_t n, int64_t d, int64_t t,
                   int64_t xs_n, int64_t xs_d, int64_t xs_t,
                   const int32_t *seq_starts,
                   void *conv_state, int64_t s, int64_t l,
                   int64_t st_s, int64_t st_d, int64_t st_l,
                   const int32_t *conv_state_indices,
                   const uint8_t *has_initial_state,
                   const void *weight, int64_t w,
                   const void *bias,
                   int activation,
                   void *out, int64_t os_n, int64_t os_d, int64_t os_t,
                   int32_t *dev_status,
                   void *stream);

/* ---------------------------------------------------------------------------
 * The state-space recurrence behind the convolution.
 *
 * Heads i = 0..h-1 of p channels each; B and C of k values belong to the head's
 * group i / (h/g).  With d = softplus(dt + dt_bias[i]) (or dt + dt_bias[i]
 * without dt_softplus), a head's state H [p, k] and a token's x, B and C:
 *
 *     H    = exp(d * a[i]) * H + d * x B^T
 *     y    = H C + d_skip[i] * x
 *     out  = y * SiLU(z)                        (y without z)
 *
 * Sums, exponentials and the recurrence are FP32.  The one-token entry points round
 * out, and a BF16 state, once and nothing else; dcconv_selective_scan rounds some
 * operands of its matrix products besides (see there).  The decay has one rate per
 * head (a[i], usually negative).
 *
 * Operands of all three entry points:
 *  x, z, out   BF16, p unit-stride channels of a head; the other strides are given
 *              in elements, >= 0.  z may be NULL.  out must give every element its
 *              own address.
 *  b, c        BF16, k unit-stride values of a group.  1 <= k <= 256.
 *  dt          BF16 or F32 (dt_dtype), h unit-stride values of a token.
 *  dt_bias, a, d_skip  F32 [h]; dt_bias and d_skip may be NULL (zero).
 *  ssm_state   F32 or BF16 (state_dtype) [s, h, p, k], slots ss_s elements apart
 *              and dense inside, READ AND WRITTEN.
 *  state_indices, dev_status, stream: as conv_state_indices, dev_status and stream
 *              of dcconv_update: -1 is a padding row (zero output, no state moves);
 *              a bad index, and with dev_status a duplicate one, makes a row padding.
 * Operands are aligned to their elements; rows that start on 16 bytes (and sizes
 * that are multiples of 8) take 16-byte accesses.  Nothing that a call writes may
 * lie within the range another operand spans.
 * ------------------------------------------------------------------------ */

/*
 * dcconv_selective_update -- one token of n rows, in place.
 * x [n, h, p] (strides xs_n, xs_h), dt [n, h] (ds_n), b and c [n, g, k], z and out
 * [n, h, p].  n == 0 returns DCCONV_OK and enqueues nothing.
 * Returns DCCONV_OK, DCCONV_EINVAL, DCCONV_EUNSUPPORTED (k > 256, or sizes past
 * n, s < 2^31, h*p and g*k <= 2^26) or DCCONV_EHIP.
 */
int dcconv_selective_update(const void *x, int64_t n, int64_t h, int64_t p, int64_t xs_n, int64_t xs_h,
                            const void *dt, int dt_dtype, int64_t ds_n, const float *dt_bias, int dt_softplus,
                            const float *a, const void *b, const void *c, int64_t g, int64_t k,
                            int64_t bs_n, int64_t bs_g, int64_t cs_n, int64_t cs_g,
                            const float *d_skip, const void *z, int64_t zs_n, int64_t zs_h,
                            void *ssm_state, int state_dtype, int64_t s, int64_t ss_s,
                            const int32_t *state_indices, void *out, int64_t os_n, int64_t os_h,
                            int32_t *dev_status, void *stream);

/*
 * dcconv_conv_selective_update -- one token through the convolution and the
 * recurrence, both states in place, in one launch.
 * xbc         BF16 [n, d], d = h*p + 2*g*k channels ordered x | B | C, row stride
 *             xbcs_n.  Every channel passes the convolution of dcconv_update
 *             (weight [d, 4], bias [d] or NULL, activation), whose result enters the
 *             recurrence in FP32, without the rounding to BF16 between two calls.
 * conv_state  BF16 [s, d, l] at any strides that give every element its own address,
 *             l >= 3; with cache_seqlens (int32 [n] or NULL) a circular buffer, as
 *             for dcconv_update.  Both states use the same slots.
 * workspace   int32 [n*g] on the device, zero before the first call that uses it; a
 *             call leaves it zero.  Calls that may run at the same time need one each.
 * Returns as dcconv_selective_update; w != 4 is DCCONV_EUNSUPPORTED.
 */
int dcconv_conv_selective_update(const void *xbc, int64_t n, int64_t h, int64_t p, int64_t g, int64_t k,
                                 int64_t xbcs_n, void *conv_state, int64_t l, int64_t st_s, int64_t st_d,
                                 int64_t st_l, const void *weight, int64_t w, const void *bias,
                                 const int32_t *cache_seqlens, int activation,
                                 const void *dt, int dt_dtype, int64_t ds_n, const float *dt_bias, int dt_softplus,
                                 const float *a, const float *d_skip, const void *z, int64_t zs_n, int64_t zs_h,
                                 void *ssm_state, int state_dtype, int64_t s, int64_t ss_s,
                                 const int32_t *state_indices, void *out, int64_t os_n, int64_t os_h,
                                 int32_t *workspace, int32_t *dev_status, void *stream);

/*
 * dcconv_selective_scan -- whole sequences (prefill).
 * x, z, out [n, t, h, p], dt [n, t, h], b and c [n, t, g, k]; or, with seq_starts
 * (device int32 [n+1], as for dcconv_prefill), n packed sequences on one axis of t
 * tokens, the _n strides unused.
 * ssm_state   NULL (with s == 0, no indices and no has_initial_state: every sequence
 *             starts from zero and its final state is dropped), or the pool: sequence
 *             i starts from its slot's state where has_initial_state[i] (uint8 [n],
 *             NULL: nowhere) is nonzero, from zero elsewhere, and leaves its final
 *             state there.  An empty sequence leaves its initial state or zeros.
 * workspace   dcconv_selective_scan_workspace() bytes, 16-byte aligned; its contents
 *             need not be kept and are not read from one call to the next.
 * Precision   the state is carried in FP32.  Rounded to BF16 (by at most 2^-8 of a term
 *             of the sums they enter) are the copy of the state that c multiplies, the
 *             products of c and b with their decays, and, unless ssm_state is F32, the
 *             x that enters the state, scaled; an F32 state takes all of its 24 bits.
 *             Then out, and a BF16 state, once.  The outputs' error is 0.0019 (F32 state)
 *             to 0.0025 of their root mean square, where one rounding makes 0.0017.
 * A finite dt is assumed.  The outputs and state values that the recurrence takes an
 * infinity or NaN of x, B, C or z to are not finite, and no others are.  An infinity
 * may become a NaN there (the one-token entry points keep it): it is a term of matrix
 * products, whose other operand may be zero or split into parts of either sign.
 * Returns as dcconv_selective_update.
 */
int dcconv_selective_scan(const void *x, int64_t n, int64_t t, int64_t h, int64_t p,
                          int64_t xs_n, int64_t xs_t, int64_t xs_h,
                          const void *dt, int dt_dtype, int64_t ds_n, int64_t ds_t,
                          const float *dt_bias, int dt_softplus, const float *a,
                          const void *b, const void *c, int64_t g, int64_t k,
                          int64_t bs_n, int64_t bs_t, int64_t bs_g, int64_t cs_n, int64_t cs_t, int64_t cs_g,
                          const float *d_skip, const void *z, int64_t zs_n, int64_t zs_t, int64_t zs_h,
                          const int32_t *seq_starts, void *ssm_state, int state_dtype, int64_t s, int64_t ss_s,
                          const int32_t *state_indices, const uint8_t *has_initial_state,
                          void *out, int64_t os_n, int64_t os_t, int64_t os_h,
                          void *workspace, int64_t workspace_bytes, int32_t *dev_status, void *stream);

/* Bytes of workspace that dcconv_selective_scan needs for these sizes (0: none, the
 * pointer may be NULL).  `packed` is nonzero with seq_starts. */
int64_t dcconv_selective_scan_workspace(int64_t n, int64_t t, int64_t h, int64_t p, int64_t g, int64_t k,
                                        int packed);

/* ---------------------------------------------------------------------------
 * The gated delta rule behind the convolution.
 *
 * Heads i = 0..h-1 of p channels each; q and key of k values belong to the head's
 * group i / (h/g).  With d = softplus(dt + dt_bias[i]) (or dt + dt_bias[i] without
 * dt_softplus), b = sigmoid(beta) (or beta without beta_sigmoid), a head's state
 * S [p, k] and a token's q, key and v:
 *
 *     S    = exp(d * a[i]) * S
 *     u    = b * (v - S key)
 *     S    = S + u key^T
 *     out  = scale * S q
 *
 * With qk_l2norm, q and key are first multiplied by 1 / sqrt(sum of squares +
 * l2norm_eps).  Sums, exponentials and the recurrence are FP32.  The one-token entry
 * point rounds out, and a BF16 state, once and nothing else; dcconv_gated_delta_scan
 * keeps 16 bits or more of the operands of its matrix products besides (see there).
 *
 * Operands of both entry points:
 *  q, key      BF16, k unit-stride values of a group.  1 <= k <= 256.
 *  v, out      BF16, p unit-stride channels of a head.  Other strides are given in
 *              elements, >= 0; out must give every element its own address.
 *  dt, beta    BF16 or F32 (dt_dtype, beta_dtype), h unit-stride values of a token.
 *  dt_bias, a  F32 [h]; dt_bias may be NULL (zero).
 *  l2norm_eps  positive and finite with qk_l2norm, else unused; scale: finite.
 *  state       F32 or BF16 (state_dtype) [s, h, p, k], slots ss_s elements apart and
 *              dense inside, READ AND WRITTEN.
 *  state_indices, dev_status, stream: as conv_state_indices, dev_status and stream
 *              of dcconv_update: -1 is a padding row (zero output, no state moves);
 *              a bad index, and with dev_status a duplicate one, makes a row padding.
 * Operands are aligned to their elements; rows that start on 16 bytes (and sizes
 * that are multiples of 8) take 16-byte accesses.  Nothing that a call writes may
 * lie within the range another operand spans.  The sums of squares of a q and of a
 * key are assumed to be finite in FP32 (values below 2^59 are enough).
 * ------------------------------------------------------------------------ */

/*
 * dcconv_gated_delta_update -- one token of n rows, in place.
 * q and key [n, g, k] (strides qs_n, qs_g and ks_n, ks_g), v and out [n, h, p], dt and
 * beta [n, h] (ds_n and es_n).  n == 0 returns DCCONV_OK and enqueues nothing.
 * Returns DCCONV_OK, DCCONV_EINVAL, DCCONV_EUNSUPPORTED (k > 256, or sizes past
 * n, s < 2^31, h*p and g*k <= 2^26) or DCCONV_EHIP.
 */
int dcconv_gated_delta_update(const void *q, const void *key, const void *v, int64_t n, int64_t h, int64_t p,
                              int64_t g, int64_t k, int64_t qs_n, int64_t qs_g, int64_t ks_n, int64_t ks_g,
                              int64_t vs_n, int64_t vs_h,
                              const void *dt, int dt_dtype, int64_t ds_n, const float *dt_bias, int dt_softplus,
                              const float *a, const void *beta, int beta_dtype, int64_t es_n, int beta_sigmoid,
                              int qk_l2norm, float l2norm_eps, float scale,
                              void *state, int state_dtype, int64_t s, int64_t ss_s, const int32_t *state_indices,
                              void *out, int64_t os_n, int64_t os_h, int32_t *dev_status, void *stream);

/*
 * dcconv_gated_delta_scan -- whole sequences (prefill).
 * q and key [n, t, g, k], v and out [n, t, h, p], dt and beta [n, t, h]; or, with
 * seq_starts (device int32 [n+1], as for dcconv_prefill), n packed sequences on one
 * axis of t tokens, the _n strides unused.
 * state       NULL (with s == 0, no indices and no has_initial_state: every sequence
 *             starts from zero and its final state is dropped), or the pool: sequence
 *             i starts from its slot's state where has_initial_state[i] (uint8 [n],
 *             NULL: nowhere) is nonzero, from zero elsewhere, and leaves its final
 *             state there.  An empty sequence leaves its initial state or zeros.
 * workspace   dcconv_gated_delta_scan_workspace() bytes, 16-byte aligned; its contents
 *             need not be kept and are not read from one call to the next.  Calls that
 *             may run at the same time need one each.
 * Precision.  Tokens are taken 32 or 64 at a time as matrix products with BF16 operands
 * and FP32 sums; operands that are no BF16 values are split into two or three, 16 bits or more.
 * An F32 state is kept as exactly as FP32 products keep it (over thousands of tokens 1e-7 to 7e-7 of
 * its size off); out, and a BF16 state, are rounded when they are stored (0.0017 of their size in the
 * mean), and what they are off by besides is some 2^-16 of the terms they are sums of.  Decays below
 * 2^-126, a token's or several tokens' together, count as zero, and u and b are held to multiples of
 * 2^-133 at best.
 * What is not finite.  A NaN or infinity reaches what the recurrence lets it reach and
 * nothing else: no earlier token, no other sequence, and for v no other channel.  An
 * infinity may arrive as a NaN, and stays one.  Where states, u, or the factors that a token or
 * several together multiply a state by, exp(d * a) (1 - b key key^T), pass FP32's range (with positive
 * d * a, say, or b above 2), also where those would meet a state of zeros or later tokens take the
 * growth back, what follows is not finite either, or finite and as right as any other result.
 * Results do not depend on the run.  They may differ in their last bits between forms of the
 * same call: batched or packed, cut into segments or not (which the sizes decide).
 * Returns as dcconv_gated_delta_update.
 */
int dcconv_gated_delta_scan(const void *q, const void *key, const void *v, int64_t n, int64_t t, int64_t h, int64_t p,
                            int64_t g, int64_t k, int64_t qs_n, int64_t qs_t, int64_t qs_g,
                            int64_t ks_n, int64_t ks_t, int64_t ks_g, int64_t vs_n, int64_t vs_t, int64_t vs_h,
                            const void *dt, int dt_dtype, int64_t ds_n, int64_t ds_t, const float *dt_bias,
                            int dt_softplus, const float *a,
                            const void *beta, int beta_dtype, int64_t es_n, int64_t es_t, int beta_sigmoid,
                            int qk_l2norm, float l2norm_eps, float scale, const int32_t *seq_starts,
                            void *state, int state_dtype, int64_t s, int64_t ss_s, const int32_t *state_indices,
                            const uint8_t *has_initial_state,
                            void *out, int64_t os_n, int64_t os_t, int64_t os_h,
                            void *workspace, int64_t workspace_bytes, int32_t *dev_status, void *stream);

/* Bytes of workspace that dcconv_gated_delta_scan needs for these sizes (0: none, the pointer
 * may be NULL).  `packed` is nonzero with seq_starts. */
int64_t dcconv_gated_delta_scan_workspace(int64_t n, int64_t t, int64_t h, int64_t p, int64_t g, int64_t k,
                                          int packed);

/* ---------------------------------------------------------------------------
 * Norms of the layer: behind the recurrence, and between blocks.  All arithmetic is
 * FP32, and what is stored is rounded once.  weight_dtype (and post_weight's, the
 * same) is BF16 or F32; weight_offset is added to every weight (1 for weights that
 * are kept as their difference from one).  rms(v) = sqrt(mean of v^2 + eps) over the
 * d values of a row; the squares of all finite values are served, also where their
 * sum is not finite or zero in FP32 (what is normed is an FP32 value each, a sum or a
 * product x SiLU(z) too).  A row of zeros with eps 0 gives NaN.  1 <= d <= 16384.  x, z, gate and out are BF16 with
 * d unit-stride values of a row and other strides >= 0, in elements.  Nothing that a
 * call writes may lie within the range another operand spans.
 * ------------------------------------------------------------------------ */

/*
 * dcconv_gated_rms_norm -- rows x [n, t, h, d], each normed by itself, times SiLU(z):
 *
 *     out = x / rms(x) * (weight + weight_offset) * SiLU(z)
 *     out = y / rms(y) * (weight + weight_offset), y = x * SiLU(z)     (gate_first)
 *
 * z           as x, or NULL (no gate).
 * weight      [d] (ws_h == 0) or a row of d for each h, ws_h elements apart; or NULL
 *             (ones, and weight_offset is not added).
 * n, t, h     0 of any returns DCCONV_OK and enqueues nothing.
 * Returns DCCONV_OK, DCCONV_EINVAL, DCCONV_EUNSUPPORTED (d > 16384, or 2^40 rows) or
 * DCCONV_EHIP.
 */
int dcconv_gated_rms_norm(const void *x, int64_t n, int64_t t, int64_t h, int64_t d,
                          int64_t xs_n, int64_t xs_t, int64_t xs_h,
                          const void *z, int64_t zs_n, int64_t zs_t, int64_t zs_h, int gate_first,
                          const void *weight, int weight_dtype, int64_t ws_h, float weight_offset, float eps,
                          void *out, int64_t os_n, int64_t os_t, int64_t os_h, void *stream);

/*
 * dcconv_add_rms_norm -- the residual stream between two blocks, rows [n, t, d]:
 *
 *     y        = x, or x / rms(x) * (post_weight + weight_offset)
 *     residual = residual + residual_scale * y * gate
 *     out      = residual / rms(residual) * (weight + weight_offset)
 *
 * x           the block's output.
 * gate        [n, t, d] (strides of 0 share a row), or NULL (1).
 * post_weight, weight  [d]; post_weight NULL: x enters as it is.
 * residual    BF16 or F32 (residual_dtype), READ AND WRITTEN; its rows must not share
 *             addresses.  out is made from the sum before it is rounded to BF16.
 * n == 0 or t == 0 returns DCCONV_OK and enqueues nothing.
 * Returns as dcconv_gated_rms_norm.
 */
int dcconv_add_rms_norm(const void *x, int64_t n, int64_t t, int64_t d, int64_t xs_n, int64_t xs_t,
                        void *residual, int residual_dtype, int64_t rs_n, int64_t rs_t,
                        const void *gate, int64_t gs_n, int64_t gs_t, float residual_scale,
                        const void *post_weight, const void *weight, int weight_dtype, float weight_offset, float eps,
                        void *out, int64_t os_n, int64_t os_t, void *stream);

/*
 * dcconv_w4_matvec -- a few rows times a 4-bit weight matrix, as the projections
 * before and after the convolution and the recurrence:
 *
 *     out[r, i] = sum_j x[r, j] * (code[i, j] - zero[j / group_size, i])
 *                                * scale[j / group_size, i] + bias[i]
 *
 * in FP32, rounded once.
 *
 * x, out      BF16 [m, k] and [m, n], rows xs_m and os_m elements apart (rows of x
 *             that start on 16 bytes, with k a multiple of 8, are read 16 bytes wide).
 * qweight     codes 0..15 of n outputs by k inputs in tiles [ceil(n/16)][ceil(k/128)]
 *             of 64 lanes x 16 bytes, 16-byte aligned, as dcconv_w4_pack lays them
 *             out: byte 4q + 2u + v of lane 16j + i holds output i and inputs
 *             32q + 8j + 4v + u (low half) and 32q + 8j + 4v + 2 + u (high half) of
 *             the tile.  Codes past n and k are not used.
 * scales      BF16 [ceil(k/group_size), n]; zeros: uint8 likewise, or NULL (8).
 * group_size  a multiple of 32.
 * bias        BF16 [n] or NULL.
 * Any m is served; the kernel is made for decode batches (it takes 64 rows at a
 * time, and reads the weights again for the next 64).  An infinite x gives NaN.
 * m == 0 returns DCCONV_OK and enqueues nothing.
 * Returns DCCONV_OK, DCCONV_EINVAL, DCCONV_EUNSUPPORTED or DCCONV_EHIP.
 */
int dcconv_w4_matvec(const void *x, int64_t m, int64_t k, int64_t xs_m, const void *qweight, int64_t n,
                     const void *scales, const uint8_t *zeros, int64_t group_size, const void *bias,
                     void *out, int64_t os_m, void *stream);

/* dcconv_w4_pack -- codes (uint8 [n, k] contiguous, the low four bits of each) into
 * the tiles of dcconv_w4_matvec, ceil(n/16) * ceil(k/128) * 1024 bytes.  Once per
 * weight matrix, when it is loaded. */
int dcconv_w4_pack(const uint8_t *codes, int64_t n, int64_t k, void *qweight, void *stream);

/*
 * dcconv_stream_copy -- measurement control, not part of the operation.
 * The page "Composing multi-kernel blocks in Python" (section "Measuring a block
 * honestly") asks for a plain baseline timed in the same run as the block it
 * judges.  This copies `bytes` bytes from src to dst with the access pattern of
 * the update kernels (coalesced 16-byte non-temporal loads and stores, about
 * 2048 wavefronts for 16 MiB), so a benchmark can time what moving the update's
 * bytes costs with no arithmetic at all.
 *
 * dst, src  device pointers, 16-byte aligned, not overlapping.  The caller owns
 *           both; dst is written, src only read.
 * bytes     a multiple of 16, 0 <= bytes <= 2^47.  0 returns DCCONV_OK and
 *           enqueues nothing.
 * stream    hipStream_t (NULL = the null stream); asynchronous like every call.
 *
 * Returns DCCONV_OK, DCCONV_EINVAL (negative, unaligned or overlapping
 * arguments, or a size not a multiple of 16) or DCCONV_EHIP.
 */
int dcconv_stream_copy(void *dst, const void *src, int64_t bytes, void *stream);

/*
 * dcconv_busy_spin -- measurement control, not part of the operation.
 * Enqueues a kernel that keeps every SIMD of the current device busy with FP32
 * arithmetic for about `microseconds` (timed by the device's constant-rate wall
 * clock).  A benchmark puts it ahead of a timed region: the host enqueues the
 * region's launches meanwhile, and the region starts on a chip at its working
 * clocks.  (Behind a one-thread spin the chip idles, and the prefill, whose
 * arithmetic is a large part of its time, measured 3 % slower in the region.)
 *
 * microseconds  0 <= microseconds <= 1e6; 0 returns DCCONV_OK and enqueues
 *               nothing.
 * stream        hipStream_t (NULL = the null stream); asynchronous.
 *
 * Returns DCCONV_OK, DCCONV_EINVAL (out of range or NaN) or DCCONV_EHIP.
 */
int dcconv_busy_spin(double microseconds, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DCCONV_H */
