/*
 * jamba_ssm_serve.h -- C ABI of what a serving step needs around the scans
 * (libjamba_ssm_serve.so, sm_100a): the layer's large projections in 8-bit
 * integers, and the maps of a continuous batch made from its requests' lengths.
 *
 * Conventions are those of jamba_ssm.h: device pointers owned by the caller,
 * nothing allocated, `stream` a cudaStream_t passed as void*, argument errors
 * returned before anything is enqueued, no C++ exception across the interface.
 * Device-side conditions go to this library's per-device status word
 * (jamba_ssm_serve_get_status); JAMBA_SSM_SYNC_CHECK as there.
 */
#ifndef JAMBA_SSM_SERVE_H
#define JAMBA_SSM_SERVE_H

#include <stddef.h>
#include <stdint.h>

#include "jamba_ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define JAMBA_SSM_SERVE_ABI_VERSION 1

/* Rows of an 8-bit matrix are this many bytes apart: K rounded up to 16, the
 * columns behind K zero. */
#define JAMBA_SSM_I8_PITCH(k) ((((int64_t)(k)) + 15) / 16 * 16)

/* Largest K: 128 * 128 * K stays below 2^31. */
#define JAMBA_SSM_I8_MAX_K 131056

/*
 * Rows to 8 bits, each with its own scale:
 *     scale[r] = max_k |x[r, k]| / 127,   q[r, k] = x[r, k] / scale[r]
 * rounded to the nearest integer (ties to even) of the exact quotient by the
 * scale as it is stored, in [-127, 127].  A row of zeros has scale 0 and q 0; a
 * row with an infinity or a NaN has scale NaN and q 0, so that what is made of
 * it is NaN.  Serves the activations of each token and, once, the rows of a
 * weight (one scale for each output channel).
 *   x       [rows, k] x_dtype, row r at x + r * x_stride elements (0: k).
 *   q       [rows, JAMBA_SSM_I8_PITCH(k)] int8, 16-byte aligned; written whole.
 *   scale   [rows] fp32.
 * rows in [0, 2^31 - 2^16], k in [1, JAMBA_SSM_I8_MAX_K].
 */
typedef struct jamba_ssm_i8_quant_params {
    size_t struct_size;              /* = sizeof(jamba_ssm_i8_quant_params) */
    int64_t rows, k;
    int32_t x_dtype;                 /* jamba_ssm_dtype */
    int32_t reserved;                /* 0 */
    const void *x;
    int64_t x_stride;
    int8_t *q;
    float *scale;
} jamba_ssm_i8_quant_params;

jamba_ssm_status jamba_ssm_i8_quant(const jamba_ssm_i8_quant_params *p, void *stream);

/*
 * out[t, o] = (sum_k q[t, k] w[o, k]) * q_scale[t] * w_scale[o] + bias[o]
 * The sum is exact (32-bit integers); the rest is fp32, rounded once to
 * out_dtype.  A token's outputs have the same bits whatever the other tokens of
 * the call and their number are.
 *   q        [ntok, pitch] int8, w [n_out, pitch] int8, pitch =
 *            JAMBA_SSM_I8_PITCH(k); both 16-byte aligned; the columns behind k
 *            must be zero in one of the two at least.
 *   q_scale  [ntok] fp32; w_scale [n_out] fp32; bias [n_out] fp32 or NULL.
 *   out      [ntok, n_out] out_dtype, contiguous; overlaps no input.
 * ntok in [0, 2^31 - 2^16], n_out in [1, 2^24], k in [1, JAMBA_SSM_I8_MAX_K].
 * timeout_cycles: limit of the kernel's waits in SM clock cycles (0 = about
 * 2 s); a wait that ran out is recorded as JAMBA_SSM_ERR_TIMEOUT, and the
 * outputs are not all written then: those that depend on the lost copies stay
 * as they were, and none is written with a part of its sum.  debug_flags: 0 in
 * production; bit 0 withholds every CTA's first copies, so that its waits run
 * out, bit 1 those of the first of the CTAs that share a tile's K (the tests
 * of that path).
 */
typedef struct jamba_ssm_i8_proj_params {
    size_t struct_size;              /* = sizeof(jamba_ssm_i8_proj_params) */
    int64_t ntok, k, n_out;
    int32_t out_dtype;               /* jamba_ssm_dtype */
    int32_t reserved;                /* 0 */
    const int8_t *q;
    const float *q_scale;
    const int8_t *w;
    const float *w_scale;
    const float *bias;
    void *out;
    uint64_t timeout_cycles;
    uint32_t debug_flags;
} jamba_ssm_i8_proj_params;

jamba_ssm_status jamba_ssm_i8_proj(const jamba_ssm_i8_proj_params *p, void *stream);

/*
 * The maps of one step of a continuous batch, from its requests' lengths, in
 * one launch and with nothing read back by the host.  Request b brings
 * new_lens[b] tokens (a negative length counts as 0) behind ctx_lens[b] tokens
 * it had before.
 *   n[b]           the tokens that fit: new_lens cut where the batch reaches
 *                  max_tokens (the requests behind get fewer or none).
 *   cu_seqlens     [requests + 1]: their running sum, for the packed scans.
 *   positions      [max_tokens]: ctx_lens[b] + the token's place in n[b], or
 *                  -1 where that is 2^31 or more (the token has no block then).
 *   token_request  [max_tokens]: b.
 *   block_tables   [requests, max_blocks], read and written: the cache blocks
 *                  of block_size tokens that a request holds, in order.  The
 *                  first ceil(ctx / block_size) entries are taken as they are;
 *                  a request with n > 0 gets its entries up to
 *                  ceil((ctx + n) / block_size) from free_blocks, request by
 *                  request in order; the entries behind are left as they were.
 *   slot_map       [max_tokens] int64: block * block_size + position %
 *                  block_size, or -1 where the table has no block (a negative
 *                  entry, a position past max_blocks, no free block left).
 *   request_slots  [requests], read and written: the state slot a request
 *                  holds.  A request with n > 0 and ctx 0 takes the next of
 *                  free_slots, in order (-1 when none is left).
 *   state_indices  [requests]: request_slots[b] where n > 0, else -1 (the
 *                  scans' state_indices).
 *   initial_indices [requests]: as state_indices, but -1 where ctx is 0 (the
 *                  gated scan's initial_indices: a new request starts from
 *                  zero).  The calls without initial_indices -- jamba_ssm_scan,
 *                  jamba_ssm_state_update, jamba_ssm_gated_state_update -- start
 *                  from row state_indices[b] whatever an earlier request left
 *                  there: for them a slot's row is zeroed when the request that
 *                  held it ends, before the slot is in free_slots again.
 *   counts         [4]: tokens, blocks taken, state slots taken, largest n.
 * Rows of the per-token maps behind the last token hold -1, so a captured step
 * of max_tokens rows can run on fewer.
 * Recorded as JAMBA_SSM_ERR_INVALID_ARG in the status word: tokens past
 * max_tokens, blocks or slots past the free ones, a request longer than
 * max_blocks blocks or with a position past 2^31 - 1.  The maps are then as
 * said above.
 * requests in [0, 2^20], max_tokens in [0, 2^30], max_blocks in [1, 2^24],
 * block_size in [1, 2^20]; requests * max_blocks and the sums of lengths may
 * pass 2^31.
 * free_blocks / free_slots may be NULL when their count is 0; ctx_lens NULL
 * means zeros.  All are device pointers, int32 unless said otherwise, aligned
 * to their element.  Outputs must not overlap one another or an input.
 */
typedef struct jamba_ssm_batch_maps_params {
    size_t struct_size;              /* = sizeof(jamba_ssm_batch_maps_params) */
    int64_t requests, max_tokens, max_blocks, block_size;
    const int32_t *new_lens;
    const int32_t *ctx_lens;
    const int32_t *free_blocks;
    int64_t num_free_blocks;
    const int32_t *free_slots;
    int64_t num_free_slots;
    int32_t *block_tables;
    int32_t *request_slots;
    int32_t *cu_seqlens;
    int32_t *positions;
    int32_t *token_request;
    int64_t *slot_map;
    int32_t *state_indices;
    int32_t *initial_indices;
    int32_t *counts;
} jamba_ssm_batch_maps_params;

jamba_ssm_status jamba_ssm_batch_maps(const jamba_ssm_batch_maps_params *p, void *stream);

/* Waits for `stream`, then reads and clears this library's status word of the
 * current device. */
jamba_ssm_status jamba_ssm_serve_get_status(void *stream);
int jamba_ssm_serve_last_cuda_error(void);
int jamba_ssm_serve_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* JAMBA_SSM_SERVE_H */
