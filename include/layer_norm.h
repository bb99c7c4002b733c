/*
 * layer_norm.h — layer norm over the last axis and its VJP, on MI355X (gfx950).
 *
 * Operation.  Every row x [D] of a tensor [B, T, H, D]:
 *
 *     mean = sum x / D,   r = 1 / sqrt(sum (x - mean)^2 / D + eps)
 *     y = (x - mean) r w + b
 *
 * weight and bias are [D], or with by_head [H, D], one row for each index of
 * the third axis (the norm of a layer's heads); NULL: ones, zeros.  A plain
 * tensor of rows has H = 1.
 *
 * Layout: x is read through its batch, token and head strides (elements; the
 * last axis is dense); y, cotangents and gradients are dense.  One dtype
 * (LNM_F32, LNM_BF16, LNM_F16) for x, weight, bias, outputs and gradients;
 * arithmetic is float32, the variance from the differences to the mean, and
 * every result is rounded once.  Sums are float32 too: a row whose sum, or whose
 * sum of squared differences, passes its range does not have these values.
 * y may not overlap x.
 *
 * The forward writes `stats`, [rows][4] float32 on 16 bytes (mean, what rounding
 * left in it, r, 0), where it is given; the VJP takes them.  A weight's or bias' gradient is a sum over all rows, made of
 * one partial sum per block in a fixed order (bit-reproducible); the partial
 * sums go through `workspace`.
 *
 * Limits: 1 <= D <= 16384, H <= 2^20, element counts below 2^40, with by_head
 * H D below 2^31.  A constant row and eps = 0: not finite, as the formula says.  Conventions and error codes: as in gated_delta.h.
 */
#ifndef QC_LAYER_NORM_H
#define QC_LAYER_NORM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { LNM_F32 = 0, LNM_BF16 = 1, LNM_F16 = 2 };

typedef struct {
    int64_t B, T, H, D;
    int64_t x_stride[3];       /* batch, token, head strides in elements */
    int32_t dtype, by_head;
    float eps;
    int32_t reserved;
} lnm_dims;

int lnm_fwd(const lnm_dims* dims, const void* x, const void* weight, const void* bias, void* y, float* stats, void* stream);

/* Bytes of the VJP's workspace (0 if out of range). */
size_t lnm_workspace_bytes(const lnm_dims* dims);

/* d_y is y's cotangent; each of the three gradients may be NULL (if all are,
 * the call does nothing).  The workspace is needed for the weights' gradients
 * alone. */
int lnm_bwd(const lnm_dims* dims, const void* x, const void* weight, const float* stats, const void* d_y, void* d_x,
            void* d_weight, void* d_bias, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QC_LAYER_NORM_H */
