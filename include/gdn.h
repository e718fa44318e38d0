/* gdn.h -- C ABI of the Gated DeltaNet recurrent scan on GB300 (sm_103a).
 *
 * "Optimizing on-device inference for Apple Silicon", section "Qwen creates
 * three distinct workload shapes": a Gated DeltaNet layer keeps a recurrent
 * state of fixed size; a learned gate sets how much of the state survives
 * each token and a delta update writes the token in.  Section "Keep the
 * recurrent state on chip": the state is a matrix, kept (with its gate) in
 * 32-bit float, each column held in registers for the whole scan and written
 * back only at its end; the query and key (and value) activations are
 * bfloat16.  The update (the published gated delta rule), per value head h,
 * value coordinate j and token t, with S[h][j] the d_k-vector of column j:
 *
 *     r     = S[h][j] . k_t            (k_t, q_t of key head h / (H_v / H_k))
 *     u     = beta_t[h] * (v_t[h][j] - alpha_t[h] * r)
 *     S[h][j] = alpha_t[h] * S[h][j] + u * k_t
 *     o_t[h][j] = S[h][j] . q_t
 *
 * Columns are independent, so one call scans any number of heads; a long
 * sequence may be scanned in pieces, passing state_out of one piece as
 * state_in of the next.  Pieces cut at multiples of 8 tokens give results
 * bit-identical to one scan (the kernel takes tokens 8 at a time and passes
 * the state in the float32 it keeps it in); other cuts agree up to float
 * rounding.
 * The caller applies the model's preprocessing (normalising q and k, the
 * query scale, the gate and write-strength activations) before the call.
 */
#ifndef GDN_H
#define GDN_H

#include "moe.h" /* MOE_OK and the error codes */

#ifdef __cplusplus
extern "C" {
#endif

/* One scan over T tokens on `cuda_stream` (asynchronous; all pointers device
 * memory, owned by the caller, not retained after the call returns).
 *   q, k       bf16 [T][n_k_heads][d_k]
 *   v          bf16 [T][n_v_heads][d_v]
 *   alpha      float32 [T][n_v_heads], the gate (state kept), in [0, 1]
 *   beta       float32 [T][n_v_heads], the write strength
 *   state_in   float32 [n_v_heads][d_v][d_k] (column j of head h contiguous),
 *              or NULL for a zero state
 *   state_out  float32, same layout, written after the scan, or NULL; may be
 *              state_in (each column is read before it is written)
 *   o          bf16 [T][n_v_heads][d_v], round-to-nearest of the fp32 result
 * Supported: d_k == 128, d_v a multiple of 16, n_v_heads a multiple of
 * n_k_heads, T >= 0 (T == 0 copies state_in to state_out).
 * Returns MOE_OK; MOE_ERR_INVALID_ARG for NULL required pointers, negative
 * sizes or a head count that does not divide; MOE_ERR_UNSUPPORTED for other
 * dimensions; MOE_ERR_ALIGNMENT unless q, k, v are 16-byte aligned, the
 * state pointers 8-byte, alpha and beta 4-byte and o 2-byte aligned;
 * MOE_ERR_CUDA if a launch fails (nothing is written then).  All checks are
 * made on the host before anything is launched.
 * Device-side faults are not produced by this kernel (it waits on nothing
 * but block barriers). */
int gdn_scan(const void *q, const void *k, const void *v, const float *alpha, const float *beta,
             const float *state_in, float *state_out, void *o, int T, int n_k_heads,
             int n_v_heads, int d_k, int d_v, void *cuda_stream);

/*
 * Linear attention with one decay per value head: the recurrence without the
 * delta, S a head's state [d_v][d_k],
 *
 *     S   <- decay[h] * S + v_t[h] k_t^T     (k_t, q_t of key head h / (H_v / H_k))
 *     o_t[h] = S q_t
 *
 * over n_seq independent sequences in one call: prompts and single tokens.
 *   q, k      bf16 [n_tokens][n_k_heads][d_k], tokens q_stride / k_stride
 *             elements apart (the slices of a fused projection are taken as
 *             they are)
 *   v         bf16 [n_tokens][n_v_heads][d_v], tokens v_stride elements apart
 *   decay     float32 [n_v_heads], in [0, 1] (0: the state holds one token)
 *   state_in  float32 [n_seq][n_v_heads][d_v][d_k], or NULL for zero states
 *   state_out float32, same layout, or NULL; may be state_in.  A sequence
 *             without tokens gets its state_in.
 *   o         bf16 [n_tokens][n_v_heads][d_v], contiguous, round-to-nearest,
 *             overlapping none of the inputs
 *   offsets   int32 [n_seq + 1] in device memory: sequence i is the tokens
 *             offsets[i] .. offsets[i + 1] - 1 (from 0, never decreasing, to
 *             n_tokens; lengths may be 0).  Values outside that are clamped to
 *             it, and tokens of no sequence keep what o held.  NULL: n_seq
 *             sequences of n_tokens / n_seq tokens.
 *   workspace device memory of at least the bytes gdn_decay_workspace gives
 *             for the same sizes, 16-byte aligned, used by the call's kernels
 *             alone; NULL where that is 0.
 * Sequences of up to 16 tokens take the recurrent form (fp32 arithmetic), longer
 * ones the chunked form on the tensor cores: the state is kept and updated in
 * fp32 there too (its error stays that of fp32 arithmetic); for the outputs
 * alone, state and scores are rounded to bf16 before their products (within 2^-8
 * of each term, so that an output whose terms cancel has lost as much).
 * A long sequence may be taken in pieces, passing the state along; pieces
 * agree with one call up to these roundings.  The same inputs give the same
 * bits.  NaN and infinities of one sequence reach no other, nor its earlier
 * tokens; in the chunked form an infinity in k or v may become NaN in the state.
 * The caller applies the model's preprocessing (norms, query scale) before the
 * call.
 * Supported: d_k 64 or 128, d_v a multiple of 16 up to 1024, n_v_heads a
 * multiple of n_k_heads and at most 4096, n_tokens < 2^31, strides < 2^39.
 * Pointers 16-byte aligned (decay and offsets 4-byte), strides multiples of 8.
 * n_seq == 0 is a no-op.  Asynchronous on cuda_stream; all checks are made on
 * the host before anything is launched.  A bounded wait in the kernels that
 * runs out leaves the results unspecified and records MOE_ERR_DEVICE_TIMEOUT
 * in the status word of the calls without a handle (moe_noalloc_status); the
 * first call on a device looks that word up, so make it before any stream
 * capture.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_ALIGNMENT, MOE_ERR_UNSUPPORTED,
 * MOE_ERR_CUDA.
 */
int gdn_decay_scan(const void *q, const void *k, const void *v, const float *decay,
                   const float *state_in, float *state_out, void *o, const int *offsets,
                   long long n_tokens, int n_seq, int n_k_heads, int n_v_heads, int d_k, int d_v,
                   long long q_stride, long long k_stride, long long v_stride, void *workspace,
                   size_t workspace_bytes, void *cuda_stream);

/* Bytes of workspace that gdn_decay_scan wants for these sizes, whatever the
 * number of key heads; ragged: 1 for a call with offsets, 0 for one without
 * (host only).  It holds the states between the segments of cut sequences: with
 * offsets, at most two for each segment's length of the tokens. */
int gdn_decay_workspace(long long n_tokens, int n_seq, int ragged, int n_v_heads, int d_k, int d_v,
                        size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
