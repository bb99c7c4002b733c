/*
 * decay_attention.h — linear attention with a decay for each head, on MI355X
 * (gfx950): whole sequences with their VJP, and single tokens on a pool of
 * states.
 *
 * Operation.  Per sequence and value head h, a state S of shape [K, V] evolves
 * over the tokens from S = initial_state:
 *
 *     S = exp(log_decay_t) S + key_t value_t^T
 *     out_t = scale S^T query_t
 *
 * Queries and keys have Hk heads, values Hv = r Hk; value head h reads key
 * head h / r.  (The gated delta rule of gated_delta.h is the same recurrence
 * with what the state already holds of a key taken from its value.)
 *
 * Layout, token by token as projections leave them: query, key [B, T, Hk, K],
 * value, out [B, T, Hv, V] of one dtype (DCA_F32, DCA_BF16, DCA_F16); states
 * [.., Hv, K, V] float32; log_decay float32, [B, T, Hv], or with head_decay
 * [Hv], one decay of a head for all its tokens.  query, key and value are read
 * through the batch, token and head strides of dca_dims (elements; their last
 * axis is dense); everything else is dense and row-major.
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
 * Arithmetic: products run on bfloat16 MFMA with operands split into bfloat16
 * parts, summed in float32.  Inputs are held whole (three parts for float32).
 * Computed operands keep three parts, whole significands, so that everything
 * has float32 accuracy before its rounding.  Decays are cumulated in float64;
 * below -10^4 they count as -10^4 (their exponential is zero in float32).
 * log_decay of -inf clears a finite state, as exp(-inf) = 0 says.  A key,
 * decay (other than -inf) or value that is not finite reaches its own and later
 * tokens of its sequence and the final state, in the heads that read it (a
 * value: in its column), as by the recurrence; a query its own token; what
 * comes before is as without it.  The backward pass may return NaN for any
 * token of such a sequence.  States, out and the gradients of query, key and
 * value are rounded once.  float32 above 3.38e38, which bfloat16 cannot hold,
 * counts as infinite.  Results do not depend on what else runs, bit for bit; a
 * long sequence's sums are joined by segments, whose length goes by the sizes of
 * the call.
 *
 * Limits: 1 <= K <= 128, 1 <= V <= 1024, Hv a multiple of Hk and at most 2^20,
 * B, T, N >= 0, T below 2^31, element counts at most 2^40.  dca_fwd, dca_bwd:
 * Hv ceil(V / 64) times the chunks of 32 tokens (N ceil(T / 32); with offsets
 * T / 32 + N) below 2^23, and N Hk rounded up to a multiple of 8, times
 * Hv / Hk ceil(V / 64), too.  dca_step: N Hv ceil(V / 32) up to 2^25, and with
 * slots, N times that up to 2^40 (a row looks through the slots of those before
 * it, once for each head and 32 columns).
 *
 * Conventions: as in gated_delta.h.  Device pointers are the caller's; the
 * library never allocates, frees or keeps one.  Validation is on the host,
 * before any HIP call; the return value is 0 or a negative QC_ERR_* code of
 * quat_cumprod.h.  Launches are asynchronous on `stream` (a hipStream_t as
 * void*), on the device that is current.  Workspace and saved buffers are
 * 256-byte aligned internal formats; a workspace may be reused as soon as the
 * work that was enqueued with it on the same stream is ordered before.
 */
#ifndef QC_DECAY_ATTENTION_H
#define QC_DECAY_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { DCA_F32 = 0, DCA_BF16 = 1, DCA_F16 = 2 };

typedef struct {
    int64_t B, T, Hk, Hv, K, V;
    int64_t N;                 /* sequences: B, or those that offsets delimit */
    int64_t q_stride[3];       /* batch, token, head strides in elements      */
    int64_t k_stride[3];
    int64_t v_stride[3];
    int32_t dtype;
    float scale;
    int32_t packed;            /* 1: offsets delimit the sequences, B is 1    */
    int32_t head_decay;        /* 1: log_decay is [Hv]                        */
} dca_dims;

/* Bytes of the state a forward saves for its backward, and of the workspace
 * of a forward (backward 0) or a backward (1); 0 if out of range. */
size_t dca_saved_bytes(const dca_dims* dims);
size_t dca_workspace_bytes(const dca_dims* dims, int32_t backward);

/* initial_state NULL: zeros.  final_state may be NULL, and saved if no
 * backward follows. */
int dca_fwd(const dca_dims* dims, const void* query, const void* key, const void* value, const float* log_decay,
            const int32_t* offsets, const float* initial_state, void* out, float* final_state, void* saved,
            void* workspace, size_t workspace_bytes, void* stream);

/* VJP.  `saved` is what dca_fwd wrote for the same inputs; d_out is dense
 * [B, T, Hv, V], d_final_state may be NULL (zero).  Each of the five gradients,
 * dense, may be NULL; if all are, the call does nothing.  d_log_decay has
 * log_decay's shape. */
int dca_bwd(const dca_dims* dims, const void* query, const void* key, const void* value, const float* log_decay,
            const int32_t* offsets, const void* saved, const void* d_out, const float* d_final_state, void* d_query,
            void* d_key, void* d_value, float* d_log_decay, float* d_initial_state, void* workspace,
            size_t workspace_bytes, void* stream);

/* One or a few tokens (dims.T) for each of dims.N = dims.B rows, on states
 * that are updated in place: row n reads and writes state slots[n] of the pool
 * [n_slots, Hv, K, V] float32, whose slots are slot_stride elements apart
 * (slots NULL: row n has slot n).  A row whose slot is outside 0 .. n_slots - 1
 * (a padding row's -1, say), or is already named by an earlier row of the
 * call, is not run: its out is zero and no state changes. */
int dca_step(const dca_dims* dims, const void* query, const void* key, const void* value, const float* log_decay,
             float* state, int64_t n_slots, int64_t slot_stride, const int32_t* slots, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QC_DECAY_ATTENTION_H */
