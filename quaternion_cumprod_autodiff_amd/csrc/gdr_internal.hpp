// gdr_internal.hpp -- declarations shared by the gated-delta-rule entry points
// and kernels (include/gated_delta.h).  Not installed.
#pragma once

#include "gated_delta.h"
#include "lm_common.hpp"
#include "qc_internal.hpp"
#include "quat_cumprod.h"

namespace qc {

constexpr int kGdrMaxK = 128;
constexpr int kGdrMaxV = 1024;

// Sizes within the documented limits and a known dtype.
inline int gdr_check(const gdr_dims* d) {
    if (!d) return QC_ERR_NULL;
    if (d->dtype < 0 || d->dtype > 2) return QC_ERR_DTYPE;
    if (d->B < 0 || d->T < 0 || d->N < 0 || d->Hk < 1 || d->Hv < 1 || d->Hv % d->Hk) return QC_ERR_SHAPE;
    if (d->K < 1 || d->K > kGdrMaxK || d->V < 1 || d->V > kGdrMaxV) return QC_ERR_SHAPE;
    if (d->T > (int64_t(1) << 31) - 1 || d->Hv > (1 << 20)) return QC_ERR_SHAPE;
    const int64_t tokens = count(d->B, d->T);
    if (tokens < 0 || count(tokens, count(d->Hk, d->K)) < 0 || count(tokens, count(d->Hv, d->V)) < 0) return QC_ERR_SHAPE;
    if (count(d->N, count(d->Hv, d->K * d->V)) < 0) return QC_ERR_SHAPE;
    const size_t e = dtype_bytes(d->dtype);
    if (strided_bytes(d->B, d->T, d->Hk, d->K, d->q_stride, e) < 0 || strided_bytes(d->B, d->T, d->Hk, d->K, d->k_stride, e) < 0 ||
        strided_bytes(d->B, d->T, d->Hv, d->V, d->v_stride, e) < 0)
        return QC_ERR_SHAPE;
    return QC_OK;
}

}  // namespace qc
