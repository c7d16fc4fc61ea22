/*
 * jamba_ssm_gated.h -- C ABI of the gated linear recurrence
 * (libjamba_ssm_gated.so, sm_100a): the scan over whole sequences, its
 * backward pass and the one-token update.
 *
 * The operation.  A recurrence of its own beside jamba_ssm.h's selective one
 * (h_t = Abar_t h_{t-1} + Bbar_t x_t, which is that of Jamba's layers): one state
 * per channel, whose decay and input weight come from one gate of the token and
 * add up to one:
 *     u_t   = rate[d] * sigmoid(g_t + bias[d])           (update rate)
 *     h_t   = h_{t-1} + u_t (x_t - h_{t-1})              = (1 - u_t) h_{t-1} + u_t x_t
 *     out_t = h_t * silu(z_t),  silu(z) = z / (1 + e^-z)   (no z: out_t = h_t)
 * rate, in [0, 1] (values are not checked), caps a channel's update rate and so
 * sets how long it remembers (about 1 / rate tokens).  The form h + u (x - h)
 * never rounds the decay 1 - u, and the scans join their runs of rows in the
 * same form, so a rate of 1e-6 still moves the state by the right amount and
 * leaves a state that has reached its input there.
 * A state that is not finite leaves every later step of its sequence not
 * finite.
 *
 * Conventions are those of jamba_ssm.h: device pointers owned by the caller,
 * nothing allocated, `stream` a cudaStream_t passed as void*, argument errors
 * returned before anything is enqueued, device-side conditions kept in a
 * status word (the first word of the workspace when the call was given one,
 * else this library's per-device word), no C++ exception across the interface,
 * JAMBA_SSM_SYNC_CHECK as there.  Every result is a fixed function of the
 * inputs and sizes: no atomics, every sum in a fixed order.
 */
#ifndef JAMBA_SSM_GATED_H
#define JAMBA_SSM_GATED_H

#include <stddef.h>
#include <stdint.h>

#include "jamba_ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define JAMBA_SSM_GATED_ABI_VERSION 1

/* Steps between two checkpoints of a sequence. */
#define JAMBA_SSM_GATED_CKPT_STEPS 64

/*
 * The scan.
 * Sizes: batch >= 0, seqlen >= 0, d_inner in [1, 2^20]; any width, no
 * alignment beyond the element's (even widths, strides and 2-element aligned
 * pointers take the kernels whose lanes hold two channels).  At most 2^30
 * token rows, 2^24 sequences, and 2^31 - 1 sequences times ceil(d_inner / 32)
 * (JAMBA_SSM_ERR_UNSUPPORTED beyond).  Packed sequences are cut by their mean
 * length: one that is much longer than three times the mean takes longer than
 * it would in a call of its own.
 * Pointers (device):
 *   x, g, z    [batch, seqlen, d_inner] io_dtype; z may be NULL.  Row r of x
 *              starts x_stride elements after row r - 1 (batches follow one
 *              another without a gap: sequence b starts at row b * seqlen), so
 *              the three may be column blocks of one projection's output.
 *              A stride of 0 means d_inner; others are >= d_inner.
 *   rate, bias [d_inner] fp32 or NULL (ones, zeros).
 *   h0         [batch, d_inner] fp32 or NULL (zeros).
 *   out        [batch, seqlen, d_inner] io_dtype, contiguous; must not overlap
 *              an input.
 *   h_final    [batch, d_inner] fp32 or NULL.  h_final == h0 is allowed.  An
 *              empty sequence copies its initial state.
 * Packed sequences: cu_seqlens (device int32 [batch + 1], NULL = batched) as in
 *   jamba_ssm_scan: rows cu_seqlens[b] .. cu_seqlens[b+1] - 1 of
 *   [total_tokens, d_inner]; offsets are clamped to [0, total_tokens]; rows
 *   that belong to no sequence are left as they were in out.
 * State slots: state_indices (device int32 [batch], NULL = row b): h0 and
 *   h_final are [num_slots, d_inner] caches; sequence b's final state goes to
 *   row state_indices[b], and its initial state is read from row
 *   initial_indices[b] (NULL: state_indices[b]).  A negative initial index
 *   means a zero initial state, a negative state index that no final state is
 *   written; an index >= num_slots is taken as negative and recorded as
 *   JAMBA_SSM_ERR_INVALID_ARG.  State indices must be distinct, and in a cache
 *   that is both h0 and h_final no sequence may read a row that another writes.
 * ckpt         fp32, jamba_ssm_gated_scan_ckpt_size bytes, 16-byte aligned, or
 *   NULL: receives each sequence's state before every 64th step, for
 *   jamba_ssm_gated_scan_bwd.
 * workspace    as in jamba_ssm_scan (JAMBA_SSM_STATUS_BYTES, zero-filled once,
 *   16-byte aligned) or NULL.
 */
typedef struct jamba_ssm_gated_scan_params {
    size_t struct_size;              /* = sizeof(jamba_ssm_gated_scan_params) */
    int64_t batch, seqlen, d_inner;
    int32_t io_dtype;                /* jamba_ssm_dtype */
    int32_t reserved;                /* 0 */
    const void *x, *g, *z;
    int64_t x_stride, g_stride, z_stride;
    const float *rate, *bias;
    const float *h0;
    void *out;
    float *h_final;
    const int32_t *cu_seqlens;
    int64_t total_tokens;
    const int32_t *state_indices;
    const int32_t *initial_indices;
    int64_t num_slots;
    float *ckpt;
    void *workspace;
    size_t workspace_bytes;
} jamba_ssm_gated_scan_params;

jamba_ssm_status jamba_ssm_gated_scan(const jamba_ssm_gated_scan_params *p, void *stream);

/* Bytes of the checkpoints of `batch` sequences over `rows` token rows in all
 * (batched: rows = batch * seqlen): (rows / 64 + batch) * d_inner * 4.
 * Sequence b's entry k is row (first row of b) / 64 + b + k.  0 for a negative
 * size. */
size_t jamba_ssm_gated_scan_ckpt_size(int64_t batch, int64_t rows, int64_t d_inner);

/*
 * The backward pass: gradients of a loss L given dout = dL/dout and,
 * optionally, dL/dh_final.  With gh_t = dL/dh_t, s = sigmoid(g + bias):
 *     gh_t = dout_t silu(z_t) + (1 - u_{t+1}) gh_{t+1},
 *     dx = u gh,  du = gh (x - h_{t-1}),  dg = du u (1 - s),
 *     dz = dout h silu'(z),  drate = sum du s,  dbias = sum dg,
 *     dh0 = (1 - u_0) gh_0.
 *   x, g, z, strides, rate, bias, h0, cu_seqlens, total_tokens: as given to the
 *              forward (no state slots: h0 is [batch, d_inner]).
 *   dout       [batch, seqlen, d_inner] io_dtype, contiguous.
 *   dh_final   [batch, d_inner] fp32 or NULL (zeros).
 *   dx, dg, dz as out, written (dz only with z); rows that belong to no
 *              sequence are left as they were.
 *   drate, dbias [d_inner] fp32, summed over all sequences, or NULL.
 *   dh0        [batch, d_inner] fp32 or NULL.
 *              Outputs must not overlap one another or an input.
 *   ckpt       the forward's checkpoints of the same inputs, or NULL: the
 *              backward then runs the recurrence once more to make them.
 *   workspace  jamba_ssm_gated_scan_bwd_workspace_size() bytes, 16-byte
 *              aligned (NULL where that is 0).  Scratch only: it needs no
 *              filling, and holds nothing between calls.  Calls that share one
 *              must not overlap on the GPU.
 */
typedef struct jamba_ssm_gated_scan_bwd_params {
    size_t struct_size;              /* = sizeof(jamba_ssm_gated_scan_bwd_params) */
    int64_t batch, seqlen, d_inner;
    int32_t io_dtype;
    int32_t reserved;                /* 0 */
    const void *x, *g, *z;
    int64_t x_stride, g_stride, z_stride;
    const float *rate, *bias;
    const float *h0;
    const void *dout;
    const float *dh_final;
    void *dx, *dg, *dz;
    float *drate, *dbias;
    float *dh0;
    const int32_t *cu_seqlens;
    int64_t total_tokens;
    const float *ckpt;
    void *workspace;
    size_t workspace_bytes;
} jamba_ssm_gated_scan_bwd_params;

/* has_ckpt: whether the call will be given the forward's checkpoints.  0 for a
 * negative size. */
size_t jamba_ssm_gated_scan_bwd_workspace_size(int64_t batch, int64_t rows, int64_t d_inner,
                                               int32_t has_ckpt);

jamba_ssm_status jamba_ssm_gated_scan_bwd(const jamba_ssm_gated_scan_bwd_params *p, void *stream);

/*
 * One token for each of `batch` requests: the state is overwritten in place.
 *   x, g, z, out [batch, d_inner] io_dtype, x / g / z with row strides as
 *              above, z may be NULL; out contiguous, overlapping no input.
 *   state      [batch, d_inner] fp32, or a [num_slots, d_inner] cache whose row
 *              state_indices[b] is request b's, read as it is: a new request's
 *              row has to be zero.  A negative index skips the
 *              request (its out row stays as it was); an index >= num_slots is
 *              skipped too and recorded as JAMBA_SSM_ERR_INVALID_ARG.  Indices
 *              of one call must be distinct.
 */
typedef struct jamba_ssm_gated_state_update_params {
    size_t struct_size;              /* = sizeof(jamba_ssm_gated_state_update_params) */
    int64_t batch, d_inner;
    int32_t io_dtype;
    int32_t reserved;                /* 0 */
    float *state;
    const void *x, *g, *z;
    int64_t x_stride, g_stride, z_stride;
    const float *rate, *bias;
    void *out;
    const int32_t *state_indices;
    int64_t num_slots;
    void *workspace;
    size_t workspace_bytes;
} jamba_ssm_gated_state_update_params;

jamba_ssm_status jamba_ssm_gated_state_update(const jamba_ssm_gated_state_update_params *p,
                                              void *stream);

/* As jamba_ssm_get_status, for this library's calls. */
jamba_ssm_status jamba_ssm_gated_get_status(void *workspace, void *stream);
int jamba_ssm_gated_last_cuda_error(void);
int jamba_ssm_gated_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* JAMBA_SSM_GATED_H */
