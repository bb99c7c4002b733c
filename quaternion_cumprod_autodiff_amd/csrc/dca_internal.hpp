// dca_internal.hpp -- declarations shared by the entry points and kernels of
// linear attention with decays (include/decay_attention.h).  Not installed.
#pragma once

#include "dca_chunk.hpp"

namespace qc {

constexpr int kDcaMaxK = 128;
constexpr int kDcaMaxV = 1024;

// Sizes within the documented limits and a known dtype.
inline int dca_check(const dca_dims* d) {
    if (!d) return QC_ERR_NULL;
    if (d->dtype < 0 || d->dtype > 2) return QC_ERR_DTYPE;
    if (d->B < 0 || d->T < 0 || d->N < 0 || d->Hk < 1 || d->Hv < 1 || d->Hv % d->Hk) return QC_ERR_SHAPE;
    if (d->K < 1 || d->K > kDcaMaxK || d->V < 1 || d->V > kDcaMaxV) return QC_ERR_SHAPE;
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
