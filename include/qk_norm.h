/*
 * qk_norm.h — norms of query and key heads with the position rotation in the
 * same pass, and their VJP, on MI355X (gfx950).
 *
 * Operation.  Every head x [D] of query [B, T, Hq, D] and key [B, T, Hk, D]:
 *
 *     r = 1 / sqrt(sum x^2 / D + eps)      (QKN_RMS)
 *     r = 1 / sqrt(sum x^2 + eps)          (QKN_L2)
 *     n = x r w                            (w [D]: query's or key's weight, NULL: ones)
 *     y = n with its first R elements turned, pair by pair, by the angles of
 *         the token's table row:  (a, b) -> (a cos - b sin, b cos + a sin)
 *
 * The pairs are (i, i + R/2), or (2i, 2i + 1) with `interleaved`.  cos and sin
 * are tables [P, R/2] float32 (NULL with R = 0: no rotation).  Token (b, t)
 * takes row positions[b, t] (int32 or int64, device memory), or row t without
 * positions.  A position outside 0 .. P - 1 turns the token's heads into NaN
 * (positions are device data, not checked by the host).  Angles per token, as
 * data-dependent rotations have, are a table with one row per token.
 *
 * Layout: query and key are read through their batch, token and head strides
 * (elements; the last axis is dense); outputs, cotangents and gradients are
 * dense [B, T, H, D].  One dtype (QKN_F32, QKN_BF16, QKN_F16) for query, key,
 * weights, outputs and gradients; arithmetic is float32, rounded once.
 * The sum of squares is float32 too: a head whose sum passes its range (elements
 * of 1e19) becomes zeros.
 * Outputs may not overlap inputs.
 *
 * The VJP takes the outputs' cotangents and returns those of query, key and
 * the weights.  A weight's gradient is a sum over all tokens and heads, made
 * of one partial sum per block in a fixed order (bit-reproducible); the
 * partial sums go through `workspace`.
 *
 * Limits: 1 <= D <= 1024, R even, 0 <= R <= D, element counts below 2^40.
 * Conventions and error codes: as in gated_delta.h.
 */
#ifndef QC_QK_NORM_H
#define QC_QK_NORM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { QKN_F32 = 0, QKN_BF16 = 1, QKN_F16 = 2 };
enum { QKN_RMS = 0, QKN_L2 = 1 };

typedef struct {
    int64_t B, T, Hq, Hk, D, R, P;
    int64_t q_stride[3];       /* batch, token, head strides in elements */
    int64_t k_stride[3];
    int32_t dtype, kind, interleaved, positions64;
    float eps;
    int32_t reserved;
} qkn_dims;

int qkn_fwd(const qkn_dims* dims, const void* query, const void* key, const void* query_weight, const void* key_weight,
            const float* cos, const float* sin, const void* positions, void* query_out, void* key_out, void* stream);

/* Bytes of the VJP's workspace (0 if out of range). */
size_t qkn_workspace_bytes(const qkn_dims* dims);

/* d_query_out and d_key_out are the outputs' cotangents; each of the four
 * gradients may be NULL (if all are, the call does nothing).  The workspace is
 * needed for the weights' gradients alone. */
int qkn_bwd(const qkn_dims* dims, const void* query, const void* key, const void* query_weight, const void* key_weight,
            const float* cos, const float* sin, const void* positions, const void* d_query_out, const void* d_key_out,
            void* d_query, void* d_key, void* d_query_weight, void* d_key_weight, void* workspace,
            size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QC_QK_NORM_H */
