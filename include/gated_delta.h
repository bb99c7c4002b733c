/*
 * gated_delta.h — the gated delta rule with one decay and one write strength
 * per head and token, on MI355X (gfx950): whole sequences with their VJP, and
 * single tokens on a pool of states.
 *
 * Operation.  Per sequence and value head h, a state S of shape [K, V] evolves
 * over the tokens from S = initial_state:
 *
 *     S = exp(log_decay_t) S
 *     u = beta_t (value_t - S^T key_t)
 *     S = S + key_t u^T
 *     out_t = scale S^T query_t
 *
 * Queries and keys have Hk heads, values Hv = r Hk; value head h reads key
 * head h / r.  (Gated DeltaNet-2 of gdn2.h is the same recurrence with a decay
 * per latent row and erase and write vectors, in float32.)
 *
 * Layout, token by token as projections leave them: query, key [B, T, Hk, K],
 * value, out [B, T, Hv, V] of one dtype (GDR_F32, GDR_BF16, GDR_F16);
 * log_decay, beta [B, T, Hv] float32; states [.., Hv, K, V] float32.  query,
 * key and value are read through the batch, token and head strides of
 * gdr_dims (elements; their last axis is dense); everything else is dense and
 * row-major.
 *
 * Packed sequences: with `offsets` (N + 1 int32 in device memory, ascending),
 * B is 1 and sequence n is the rows offsets[n] .. offsets[n + 1] - 1; lengths
 * of zero are allowed (the final state is then the initial one).  Without,
 * N = B and a sequence is a batch entry.  Rows of no sequence are neither read
 * nor written, in no tensor, gradients included.  Offsets are device data and
 * not checked by the host: the kernels clamp them into 0 .. T and take a
 * sequence that ends before it begins as empty, so no access leaves the
 * tensors; offsets that do not ascend give unspecified values.
 *
 * Arithmetic: products run on bfloat16 MFMA with every operand split into
 * bfloat16 parts that hold its whole significand (three for float32), and are
 * summed in float32: float32 accuracy for every dtype.  Decays are cumulated
 * in float64.  log_decay of -inf clears a finite state, as exp(-inf) = 0 says.
 * A key, gate (other than -inf) or value that is not finite makes the outputs
 * of its own and all later tokens of its sequence NaN, in the heads that read
 * it (a value: in its column), and the final state; a query its own token's;
 * what comes before is as without it.  The backward pass may return NaN for
 * any token of such a sequence, and so may the forward pass for the tokens
 * before in a chunk of 64 whose products leave the range of float32 (keys of
 * 1e19, say).
 * States and gate gradients are float32; out and the gradients of query, key
 * and value are rounded once to the dtype.  Results do not depend on what else
 * runs, bit for bit.
 *
 * Limits: 1 <= K <= 128, 1 <= V <= 1024, Hv a multiple of Hk and at most 2^20,
 * B, T, N >= 0, T below 2^31, element counts at most 2^40.  gdr_fwd, gdr_bwd:
 * Hv times the chunks of 64 tokens (N ceil(T / 64); with offsets T / 64 + N)
 * below 2^23, and N Hk rounded up to a multiple of 8, times Hv / Hk ceil(V / 16),
 * below 2^23.  gdr_step: N Hv ceil(V / 32) up to 2^25.
 *
 * Conventions: as in gdn2.h.  Device pointers are the caller's; the library
 * never allocates, frees or keeps one.  Validation is on the host, before any
 * HIP call; the return value is 0 or a negative QC_ERR_* code of
 * quat_cumprod.h.  Launches are asynchronous on `stream` (a hipStream_t as
 * void*), on the device that is current.  Workspace and saved buffers are
 * 256-byte aligned internal formats; a workspace may be reused as soon as the
 * work that was enqueued with it on the same stream is ordered before.
 */
#ifndef QC_GATED_DELTA_H
#define QC_GATED_DELTA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { GDR_F32 = 0, GDR_BF16 = 1, GDR_F16 = 2 };

typedef struct {
    int64_t B, T, Hk, Hv, K, V;
    int64_t N;                 /* sequences: B, or those that offsets delimit */
    int64_t q_stride[3];       /* batch, token, head strides in elements      */
    int64_t k_stride[3];
    int64_t v_stride[3];
    int32_t dtype;
    float scale;
    int32_t packed;            /* 1: offsets delimit the sequences, B is 1    */
    int32_t reserved;
} gdr_dims;

/* Bytes of the state a forward saves for its backward, and of the workspace
 * of a forward (backward 0) or a backward (1); 0 if out of range. */
size_t gdr_saved_bytes(const gdr_dims* dims);
size_t gdr_workspace_bytes(const gdr_dims* dims, int32_t backward);

/* initial_state NULL: zeros.  final_state may be NULL, and saved if no
 * backward follows. */
int gdr_fwd(const gdr_dims* dims, const void* query, const void* key, const void* value, const float* log_decay,
            const float* beta, const int32_t* offsets, const float* initial_state, void* out, float* final_state,
            void* saved, void* workspace, size_t workspace_bytes, void* stream);

/* VJP.  `saved` is what gdr_fwd wrote for the same inputs; d_out is dense
 * [B, T, Hv, V], d_final_state may be NULL (zero).  Each of the six gradients,
 * dense, may be NULL; if all are, the call does nothing. */
int gdr_bwd(const gdr_dims* dims, const void* query, const void* key, const void* value, const float* log_decay,
            const float* beta, const int32_t* offsets, const void* saved, const void* d_out, const float* d_final_state,
            void* d_query, void* d_key, void* d_value, float* d_log_decay, float* d_beta, float* d_initial_state,
            void* workspace, size_t workspace_bytes, void* stream);

/* One or a few tokens (dims.T) for each of dims.N = dims.B rows, on states
 * that are updated in place: row n reads and writes state slots[n] of the pool
 * [n_slots, Hv, K, V] float32, whose slots are slot_stride elements apart
 * (slots NULL: row n has slot n).  A row whose slot is outside 0 .. n_slots - 1
 * (a padding row's -1, say), or is already named by an earlier row of the
 * call, is not run: its out is zero and no state changes. */
int gdr_step(const gdr_dims* dims, const void* query, const void* key, const void* value, const float* log_decay,
             const float* beta, float* state, int64_t n_slots, int64_t slot_stride, const int32_t* slots, void* out,
             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QC_GATED_DELTA_H */
