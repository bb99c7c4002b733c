// qk_norm.hip -- norms of query and key heads with the position rotation in
// the same pass, and their VJP (include/qk_norm.h).
//
// Forward, per head x [D] with r = 1 / sqrt(sum x^2 / size + eps) (size D or
// 1): n = x r w, y = turn(n).  VJP, with the cotangent g of y:
//     dn = turn^-1(g),   dh = dn w,   h = x r,   c = sum dh h
//     dx = r (dh - h c / size),       dw = sum over tokens and heads of dn h
// (r^3, in the same gradient's r dh - x r^3 sum(dh x) / size, leaves the range
// of float32 long before dx does.)
// The statistics, the products and the weights' sums are float32.
//
// Bound by memory: every element is read once (twice as x and g in the VJP)
// and written once, so a group of lanes holds a head in registers between the
// sum and the product.  A lane holds W pairs of elements, chosen so that a
// pair that turns together is in one lane: with 16-byte rows (D, R / 2
// multiples of 8 and every row on 16 bytes) W = 8, else W = 1.
#include "lm_common.hpp"
#include "qc_internal.hpp"
#include "qk_norm.h"
#include "quat_cumprod.h"

#include <type_traits>

namespace qc {
namespace {

constexpr int kThreads = 256;
// Blocks that share a weight gradient's sum: enough to fill 256 CUs several
// times, few enough that the second pass over their partial sums is short.
constexpr int kMaxPartials = 1024;

struct QknArgs {
    const void *q, *k, *wq, *wk;
    const float *cos, *sin;
    const void* pos;
    void *yq, *yk;                 // forward: outputs; VJP: dx (may be null)
    const void *gq, *gk;           // VJP: cotangents
    float *pq, *pk;                // VJP: partial sums [blocks][D] (null: no gradient of that weight)
    int64_t qs[3], ks[3];
    int64_t T, tokens, D, R, P;
    int hq, hk, blocks_q, blocks_k;
    int pos64, interleaved, small;
    float eps, inv_size;
};

// Elements of the pair slot p (W pairs) of a head: those that turn, (first,
// first + step * i) and (second, ...), then the others in two runs.
template <int W>
struct Slot {
    int64_t a, b;
    bool turns, has_a, has_b;
};

template <int W>
__device__ __forceinline__ Slot<W> slot_of(int p, int D, int R, bool interleaved) {
    const int turning = R / (2 * W);
    Slot<W> s;
    s.turns = p < turning;
    if (s.turns) {
        s.a = interleaved ? 2 * p * W : p * W;
        s.b = interleaved ? (2 * p + 1) * W : R / 2 + p * W;
    } else {
        s.a = R + 2 * (p - turning) * W;
        s.b = s.a + W;
    }
    s.has_a = s.a < D;
    s.has_b = s.b < D;
    return s;
}

template <int W, bool FULL, class E>
__device__ __forceinline__ void load_pair(const E* row, const Slot<W>& s, float (&a)[W], float (&b)[W]) {
    if constexpr (FULL) {
        load_floats<W>(row + s.a, a);
        load_floats<W>(row + s.b, b);
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) a[i] = b[i] = 0.f;
    if (s.has_a) load_floats<W>(row + s.a, a);
    if (s.has_b) load_floats<W>(row + s.b, b);
}

// (a, b) as pairs that turn together: as loaded for halves, unzipped for
// neighbours (a then b hold 2W consecutive elements).
template <int W>
__device__ __forceinline__ void turn(float (&a)[W], float (&b)[W], const float* c, const float* s, bool interleaved, float sign) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float& x = 2 * i < W ? a[2 * i % W] : b[(2 * i) % W];
            float& y = 2 * i + 1 < W ? a[(2 * i + 1) % W] : b[(2 * i + 1) % W];
            const float u = x * c[i] - sign * (y * s[i]);
            y = y * c[i] + sign * (x * s[i]);
            x = u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float u = a[i] * c[i] - sign * (b[i] * s[i]);
            b[i] = b[i] * c[i] + sign * (a[i] * s[i]);
            a[i] = u;
        }
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int m = 1; m < G; m *= 2) x += __shfl_xor(x, m, 64);
    return x;
}

__device__ __forceinline__ int64_t table_row(const QknArgs& a, int64_t token, int64_t t) {
    if (!a.pos) return t;
    return a.pos64 ? static_cast<const int64_t*>(a.pos)[token] : int64_t(static_cast<const int32_t*>(a.pos)[token]);
}

// n / d: in 32 bits where everything fits, as it nearly always does (a 64-bit
// division is some hundred instructions).
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d, bool small) {
    return small ? int64_t(uint32_t(n) / uint32_t(d)) : n / d;
}

// One head per group of G lanes; S slots of W pairs per lane.  A group takes HC
// heads of one token in a row: they share the token's angles and its place.
// DT: storage type; BWD: the VJP; FULL: every lane has its elements (D = 2 W G S)
// and every group its HC heads, so that nothing is checked.
template <int DT, int W, int G, int S, int HC, bool BWD, bool FULL>
__global__ void __launch_bounds__(kThreads) qkn_kernel(QknArgs a) {
    using E = typename Storage<DT>::type;
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    const bool is_q = int(blockIdx.x) < a.blocks_q;
    const int heads = is_q ? a.hq : a.hk;
    const int block = is_q ? blockIdx.x : blockIdx.x - a.blocks_q, blocks = is_q ? a.blocks_q : a.blocks_k;
    const E* x = static_cast<const E*>(is_q ? a.q : a.k);
    const E* wt = static_cast<const E*>(is_q ? a.wq : a.wk);
    E* y = static_cast<E*>(is_q ? a.yq : a.yk);
    const E* g = static_cast<const E*>(is_q ? a.gq : a.gk);
    float* part = is_q ? a.pq : a.pk;
    const int64_t sb = is_q ? a.qs[0] : a.ks[0], st = is_q ? a.qs[1] : a.ks[1], sh = is_q ? a.qs[2] : a.ks[2];
    const int D = int(a.D), R = int(a.R);
    const bool inter = a.interleaved != 0, small = a.small != 0;
    Slot<W> slot[S];
    float wa[S][W], wb[S][W], sa[S][W], sb_[S][W];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        slot[s] = slot_of<W>(lane + G * s, D, R, inter);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            wa[s][i] = wb[s][i] = 1.f;
            sa[s][i] = sb_[s][i] = 0.f;
        }
        if (wt) load_pair<W, FULL>(wt, slot[s], wa[s], wb[s]);
    }
    constexpr int kGroups = kThreads / G;
    const int per = (heads + HC - 1) / HC;
    const int64_t units = a.tokens * per;
    for (int64_t u = int64_t(block) * kGroups + group; u < units; u += int64_t(blocks) * kGroups) {
        const int64_t token = per == 1 ? u : quotient(u, per, small);
        const int h0 = int(u - token * per) * HC;
        const int64_t b = quotient(token, a.T, small), t = token - b * a.T;
        const E* px = x + b * sb + t * st + h0 * sh;
        const int64_t dense = (token * heads + h0) * D;
        // The position first: its wait then covers nothing else, and the angles are on their way with the heads.
        int64_t row = R ? table_row(a, token, t) : 0;
        constexpr int kHeld = BWD ? 1 : HC;      // heads in registers
        float xa[kHeld][S][W], xb[kHeld][S][W], ga[BWD ? kHeld : 1][S][W], gb[BWD ? kHeld : 1][S][W], c[S][W], sn[S][W];
        auto load_head = [&](int k) {
            if (FULL || HC == 1 || h0 + k < heads)
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    load_pair<W, FULL>(px + k * sh, slot[s], xa[BWD ? 0 : k][s], xb[BWD ? 0 : k][s]);
                    if constexpr (BWD) load_pair<W, FULL>(g + dense + k * D, slot[s], ga[0][s], gb[0][s]);
                }
        };
        if constexpr (!BWD) {
#pragma unroll
            for (int k = 0; k < HC; ++k) load_head(k);
        }
        float poison = 0.f;
        if (R) {
            if (row < 0 || row >= a.P) {
                row = 0;
                poison = __builtin_nanf("");
            }
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (slot[s].turns) {
                    const int64_t at = row * (R / 2) + int64_t(lane + G * s) * W;
                    load_floats<W>(a.cos + at, c[s]);
                    load_floats<W>(a.sin + at, sn[s]);
                }
        }
        if constexpr (!BWD) {
#pragma unroll
            for (int k = 0; k < HC; ++k) {
                if (!FULL && HC > 1 && h0 + k >= heads) break;
                float sum = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int j = 0; j < W; ++j) sum += xa[k][s][j] * xa[k][s][j] + xb[k][s][j] * xb[k][s][j];
                sum = group_sum<G>(sum);
                const float r = 1.f / sqrtf(sum * a.inv_size + a.eps) + poison;
#pragma unroll
                for (int s = 0; s < S; ++s) {
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        xa[k][s][j] = xa[k][s][j] * r * wa[s][j];
                        xb[k][s][j] = xb[k][s][j] * r * wb[s][j];
                    }
                    if (slot[s].turns) turn<W>(xa[k][s], xb[k][s], c[s], sn[s], inter, 1.f);
                    E* py = y + dense + k * D;
                    if (FULL || slot[s].has_a) store_floats<W>(py + slot[s].a, xa[k][s]);
                    if (FULL || slot[s].has_b) store_floats<W>(py + slot[s].b, xb[k][s]);
                }
            }
        } else {
#pragma unroll 1
            for (int k = 0; k < HC; ++k) {
                if (!FULL && HC > 1 && h0 + k >= heads) break;
                load_head(k);
                float (&pa)[S][W] = xa[0], (&pb)[S][W] = xb[0], (&pg)[S][W] = ga[0], (&ph)[S][W] = gb[0];
                float sum = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int j = 0; j < W; ++j) sum += pa[s][j] * pa[s][j] + pb[s][j] * pb[s][j];
                sum = group_sum<G>(sum);
                const float r = 1.f / sqrtf(sum * a.inv_size + a.eps) + poison;
                float dot = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if (slot[s].turns) turn<W>(pg[s], ph[s], c[s], sn[s], inter, -1.f);
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        pa[s][j] *= r;
                        pb[s][j] *= r;
                        sa[s][j] += pg[s][j] * pa[s][j];
                        sb_[s][j] += ph[s][j] * pb[s][j];
                        pg[s][j] *= wa[s][j];
                        ph[s][j] *= wb[s][j];
                        dot += pg[s][j] * pa[s][j] + ph[s][j] * pb[s][j];
                    }
                }
                dot = group_sum<G>(dot);
                const float f = dot * a.inv_size;
                if (y) {
                    E* py = y + dense + k * D;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            pa[s][j] = r * (pg[s][j] - pa[s][j] * f);
                            pb[s][j] = r * (ph[s][j] - pb[s][j] * f);
                        }
                        if (FULL || slot[s].has_a) store_floats<W>(py + slot[s].a, pa[s]);
                        if (FULL || slot[s].has_b) store_floats<W>(py + slot[s].b, pb[s]);
                    }
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!part) return;
        // The block's sum in a fixed order: groups of a wave by shuffles, waves through LDS.
        __shared__ float red[kThreads / 64][G * S * W * 2];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < W; ++j) {
#pragma unroll
                for (int m = G; m < 64; m *= 2) {
                    sa[s][j] += __shfl_xor(sa[s][j], m, 64);
                    sb_[s][j] += __shfl_xor(sb_[s][j], m, 64);
                }
            }
        const int wave = threadIdx.x / 64;
        if (threadIdx.x % 64 < G) {
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    red[wave][(s * W + j) * 2 * G + lane] = sa[s][j];
                    red[wave][((s * W + j) * 2 + 1) * G + lane] = sb_[s][j];
                }
        }
        __syncthreads();
        if (threadIdx.x < G) {
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    float ta = 0.f, tb = 0.f;
                    for (int w = 0; w < kThreads / 64; ++w) {
                        ta += red[w][(s * W + j) * 2 * G + lane];
                        tb += red[w][((s * W + j) * 2 + 1) * G + lane];
                    }
                    if (slot[s].has_a) part[int64_t(block) * D + slot[s].a + j] = ta;
                    if (slot[s].has_b) part[int64_t(block) * D + slot[s].b + j] = tb;
                }
        }
    }
}

// dw[d] = sum of the blocks' partial sums, 16 columns and 64 runs of blocks to
// a block of threads, the runs joined in order.
constexpr int kRuns = 64;

template <int DT>
__global__ void __launch_bounds__(16 * kRuns) qkn_weight_kernel(const float* pq, const float* pk, int nq, int nk, void* dq, void* dk, int D) {
    using E = typename Storage<DT>::type;
    const float* part = blockIdx.y ? pk : pq;
    const int n = blockIdx.y ? nk : nq;
    E* out = static_cast<E*>(blockIdx.y ? dk : dq);
    if (!out) return;
    const int col = blockIdx.x * 16 + threadIdx.x % 16, run = threadIdx.x / 16;
    __shared__ float red[kRuns][17];
    float s = 0.f;
    if (col < D)
#pragma unroll 4
        for (int i = run; i < n; i += kRuns) s += part[int64_t(i) * D + col];
    red[run][threadIdx.x % 16] = s;
    __syncthreads();
    if (threadIdx.x < 16 && col < D) {
        float t = 0.f;
#pragma unroll 8
        for (int i = 0; i < kRuns; ++i) t += red[i][threadIdx.x];
        out[col] = E(t);
    }
}

int pow2_at_least(int64_t n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

struct Shape {
    bool wide;          // W = 8
    int g, s, hc;       // lanes per head, slots per lane, heads in a row
};

// Four heads of a token in a row where that still leaves two waves for each of
// 1024 SIMDs, one otherwise: they share the angles, the position and the
// divisions.  By four and one by one, heads of 128 in bfloat16, forward and
// VJP: 256 tokens of 40 heads 4.5 us (3.5) and 9.7 (8.0), 1024 tokens 6.2
// (5.6) and 12.0 (14.0), 2048 tokens 9.3 (9.5) and 17.4 (19.6), 16384 tokens
// 60 (79) forward; 16384 tokens of 32 heads 48 (61) and 82 (88).
Shape shape_of(const qkn_dims& d, bool wide) {
    Shape sh;
    sh.wide = wide;
    const int64_t slots = (d.D + (wide ? 15 : 1)) / (wide ? 16 : 2);
    sh.g = wide ? pow2_at_least(slots) : 64;
    if (wide && sh.g < 4) sh.g = 4;
    sh.s = wide ? 1 : pow2_at_least((slots + 63) / 64);
    sh.hc = d.B * d.T * (d.Hq + d.Hk) * sh.g >= 4 * 64 * 2 * 1024 ? 4 : 1;
    return sh;
}

// Blocks for so many tokens' heads; past 2^20 blocks the blocks loop.
int64_t blocks_for(int64_t tokens, int64_t heads, const Shape& sh) {
    const int64_t n = (tokens * ((heads + sh.hc - 1) / sh.hc) * sh.g + kThreads - 1) / kThreads;
    return n < (int64_t(1) << 20) ? n : int64_t(1) << 20;
}

template <class F>
hipError_t by_dtype(int dt, F&& f) {
    if (dt == 0) return f(std::integral_constant<int, 0>{});
    if (dt == 1) return f(std::integral_constant<int, 1>{});
    return f(std::integral_constant<int, 2>{});
}

template <int DT, int HC, bool BWD, bool FULL>
const void* wide_kernel(int g) {
    return g == 4    ? reinterpret_cast<const void*>(&qkn_kernel<DT, 8, 4, 1, HC, BWD, FULL>)
           : g == 8  ? reinterpret_cast<const void*>(&qkn_kernel<DT, 8, 8, 1, HC, BWD, FULL>)
           : g == 16 ? reinterpret_cast<const void*>(&qkn_kernel<DT, 8, 16, 1, HC, BWD, FULL>)
           : g == 32 ? reinterpret_cast<const void*>(&qkn_kernel<DT, 8, 32, 1, HC, BWD, FULL>)
                     : reinterpret_cast<const void*>(&qkn_kernel<DT, 8, 64, 1, HC, BWD, FULL>);
}

template <int DT, int HC, bool BWD>
const void* kernel_of(const Shape& sh, bool full) {
    if (sh.wide) return full ? wide_kernel<DT, HC, BWD, true>(sh.g) : wide_kernel<DT, HC, BWD, false>(sh.g);
    return sh.s == 1   ? reinterpret_cast<const void*>(&qkn_kernel<DT, 1, 64, 1, HC, BWD, false>)
           : sh.s == 2 ? reinterpret_cast<const void*>(&qkn_kernel<DT, 1, 64, 2, HC, BWD, false>)
           : sh.s == 4 ? reinterpret_cast<const void*>(&qkn_kernel<DT, 1, 64, 4, HC, BWD, false>)
                       : reinterpret_cast<const void*>(&qkn_kernel<DT, 1, 64, 8, HC, BWD, false>);
}

template <bool BWD>
hipError_t launch(int dt, const Shape& sh, const QknArgs& a, hipStream_t st) {
    return by_dtype(dt, [&](auto t) {
        constexpr int DT = decltype(t)::value;
        const bool full = sh.wide && a.D == 16 * sh.g && a.hq % sh.hc == 0 && a.hk % sh.hc == 0;
        const void* fn = sh.hc == 4 ? kernel_of<DT, 4, BWD>(sh, full) : kernel_of<DT, 1, BWD>(sh, full);
        QknArgs args = a;
        void* params[] = {&args};
        return hipLaunchKernel(fn, dim3(unsigned(a.blocks_q + a.blocks_k)), dim3(kThreads), params, 0, st);
    });
}

int check_dims(const qkn_dims* d) {
    if (!d) return QC_ERR_NULL;
    if (d->B < 0 || d->T < 0 || d->Hq < 0 || d->Hk < 0 || d->P < 0) return QC_ERR_SHAPE;
    if (d->D < 1 || d->D > 1024 || d->R < 0 || d->R > d->D || d->R % 2) return QC_ERR_SHAPE;
    const int64_t tokens = count(d->B, d->T);
    if (tokens < 0 || count(tokens, count(d->Hq, d->D)) < 0 || count(tokens, count(d->Hk, d->D)) < 0) return QC_ERR_SHAPE;
    if (d->Hq > (1 << 20) || d->Hk > (1 << 20) || count(d->P, d->R) < 0) return QC_ERR_SHAPE;
    if (d->dtype < 0 || d->dtype > 2) return QC_ERR_DTYPE;
    if (d->kind < 0 || d->kind > 1 || !(d->eps >= 0.f)) return QC_ERR_OPTION;
    return QC_OK;
}

struct Common {
    int rc;
    QknArgs a;
    Shape sh;
    int64_t q_bytes, k_bytes, q_out, k_out;
};

Common common(const qkn_dims* d, const void* q, const void* k, const void* wq, const void* wk, const float* cos, const float* sin,
              const void* pos) {
    Common c{};
    c.rc = check_dims(d);
    if (c.rc != QC_OK) return c;
    const size_t e = dtype_bytes(d->dtype);
    const int64_t tokens = d->B * d->T;
    c.q_out = tokens * d->Hq * d->D * e;
    c.k_out = tokens * d->Hk * d->D * e;
    c.q_bytes = strided_bytes(d->B, d->T, d->Hq, d->D, d->q_stride, e);
    c.k_bytes = strided_bytes(d->B, d->T, d->Hk, d->D, d->k_stride, e);
    if (c.q_bytes < 0 || c.k_bytes < 0) {
        c.rc = QC_ERR_SHAPE;
        return c;
    }
    if ((c.q_out && !q) || (c.k_out && !k) || (d->R && tokens && (!cos || !sin))) {
        c.rc = QC_ERR_NULL;
        return c;
    }
    if (d->R && tokens && (d->P < 1 || (!pos && d->P < d->T))) {
        c.rc = QC_ERR_SHAPE;
        return c;
    }
    for (const void* p : {q, k, wq, wk})
        if (p && !aligned_to(p, e)) c.rc = QC_ERR_ALIGN;
    for (const void* p : {static_cast<const void*>(cos), static_cast<const void*>(sin)})
        if (p && !aligned_to(p, 4)) c.rc = QC_ERR_ALIGN;
    if (pos && !aligned_to(pos, d->positions64 ? 8 : 4)) c.rc = QC_ERR_ALIGN;
    if (c.rc != QC_OK) return c;
    const bool wide = d->D % 8 == 0 && d->R % 16 == 0 && rows_on_16(q, d->q_stride, e) && rows_on_16(k, d->k_stride, e) &&
                      (!wq || aligned_to(wq, 16)) && (!wk || aligned_to(wk, 16)) &&
                      (!d->R || (aligned_to(cos, 16) && aligned_to(sin, 16)));
    c.sh = shape_of(*d, wide);
    QknArgs& a = c.a;
    a.q = q; a.k = k; a.wq = wq; a.wk = wk; a.cos = cos; a.sin = sin; a.pos = pos;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = d->q_stride[i];
        a.ks[i] = d->k_stride[i];
    }
    a.T = d->T; a.tokens = tokens; a.D = d->D; a.R = d->R; a.P = d->P;
    a.hq = int(d->Hq); a.hk = int(d->Hk);
    a.pos64 = d->positions64; a.interleaved = d->interleaved;
    a.small = tokens * (d->Hq + d->Hk) < (int64_t(1) << 31);
    a.eps = d->eps;
    a.inv_size = d->kind == QKN_RMS ? 1.f / float(d->D) : 1.f;
    return c;
}

int64_t partials(int64_t rows) { return rows < kMaxPartials ? rows : kMaxPartials; }

}  // namespace
}  // namespace qc

extern "C" {

int qkn_fwd(const qkn_dims* dims, const void* query, const void* key, const void* query_weight, const void* key_weight,
            const float* cos, const float* sin, const void* positions, void* query_out, void* key_out, void* stream) {
    qc::Common c = qc::common(dims, query, key, query_weight, key_weight, cos, sin, positions);
    if (c.rc != QC_OK) return c.rc;
    if ((c.q_out && !query_out) || (c.k_out && !key_out)) return QC_ERR_NULL;
    const size_t e = qc::dtype_bytes(dims->dtype), w = size_t(dims->D) * e, table = size_t(dims->P * (dims->R / 2)) * 4;
    if ((query_out && !qc::aligned_to(query_out, c.sh.wide ? 16 : e)) || (key_out && !qc::aligned_to(key_out, c.sh.wide ? 16 : e))) {
        if ((query_out && !qc::aligned_to(query_out, e)) || (key_out && !qc::aligned_to(key_out, e))) return QC_ERR_ALIGN;
        c.sh = qc::shape_of(*dims, false);
    }
    const qc::ByteSpan sp[] = {{query_out, size_t(c.q_out)}, {key_out, size_t(c.k_out)}, {query, size_t(c.q_bytes)},
                               {key, size_t(c.k_bytes)}, {query_weight, w}, {key_weight, w}, {cos, table}, {sin, table},
                               {positions, size_t(dims->B * dims->T) * (dims->positions64 ? 8 : 4)}};
    if (qc::outputs_overlap(sp, 2, 9)) return QC_ERR_ALIAS;
    c.a.yq = query_out;
    c.a.yk = key_out;
    c.a.blocks_q = int(qc::blocks_for(c.a.tokens, c.a.hq, c.sh));
    c.a.blocks_k = int(qc::blocks_for(c.a.tokens, c.a.hk, c.sh));
    if (c.a.blocks_q + c.a.blocks_k == 0) return QC_OK;
    const hipError_t err = qc::launch<false>(dims->dtype, c.sh, c.a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}

size_t qkn_workspace_bytes(const qkn_dims* dims) {
    if (qc::check_dims(dims) != QC_OK) return 0;
    const int64_t tokens = dims->B * dims->T;
    return size_t(qc::partials(tokens * dims->Hq) + qc::partials(tokens * dims->Hk)) * size_t(dims->D) * 4 + 16;
}

int qkn_bwd(const qkn_dims* dims, const void* query, const void* key, const void* query_weight, const void* key_weight,
            const float* cos, const float* sin, const void* positions, const void* d_query_out, const void* d_key_out,
            void* d_query, void* d_key, void* d_query_weight, void* d_key_weight, void* workspace,
            size_t workspace_bytes, void* stream) {
    qc::Common c = qc::common(dims, query, key, query_weight, key_weight, cos, sin, positions);
    if (c.rc != QC_OK) return c.rc;
    if (!d_query && !d_key && !d_query_weight && !d_key_weight) return QC_OK;
    const bool any_q = d_query || d_query_weight, any_k = d_key || d_key_weight;
    if ((c.q_out && any_q && !d_query_out) || (c.k_out && any_k && !d_key_out)) return QC_ERR_NULL;
    if ((d_query_weight && !query_weight) || (d_key_weight && !key_weight)) return QC_ERR_NULL;
    const size_t e = qc::dtype_bytes(dims->dtype), w = size_t(dims->D) * e, table = size_t(dims->P * (dims->R / 2)) * 4;
    const size_t need = qkn_workspace_bytes(dims);
    const bool weights = d_query_weight || d_key_weight;
    if (weights && (!workspace || workspace_bytes < need)) return QC_ERR_WORKSPACE;
    if (weights && !qc::aligned_to(workspace, 16)) return QC_ERR_ALIGN;
    bool wide = c.sh.wide;
    for (const void* p : {d_query_out, d_key_out, static_cast<const void*>(d_query), static_cast<const void*>(d_key)}) {
        if (p && !qc::aligned_to(p, e)) return QC_ERR_ALIGN;
        if (p && !qc::aligned_to(p, 16)) wide = false;
    }
    for (const void* p : {d_query_weight, d_key_weight})
        if (p && !qc::aligned_to(p, e)) return QC_ERR_ALIGN;
    c.sh = qc::shape_of(*dims, wide);
    const qc::ByteSpan sp[] = {{d_query, size_t(c.q_out)}, {d_key, size_t(c.k_out)}, {d_query_weight, w}, {d_key_weight, w},
                               {weights ? workspace : nullptr, need}, {query, size_t(c.q_bytes)}, {key, size_t(c.k_bytes)},
                               {query_weight, w}, {key_weight, w}, {cos, table}, {sin, table},
                               {positions, size_t(dims->B * dims->T) * (dims->positions64 ? 8 : 4)},
                               {d_query_out, size_t(c.q_out)}, {d_key_out, size_t(c.k_out)}};
    if (qc::outputs_overlap(sp, 5, 14)) return QC_ERR_ALIAS;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    auto blocks = [&](bool any, const void* dw, int64_t heads) -> int {
        if (!any) return 0;
        const int64_t n = qc::blocks_for(c.a.tokens, heads, c.sh), most = qc::partials(c.a.tokens * heads);
        return int(dw && n > most ? most : n);
    };
    c.a.blocks_q = blocks(any_q, d_query_weight, c.a.hq);
    c.a.blocks_k = blocks(any_k, d_key_weight, c.a.hk);
    c.a.yq = d_query; c.a.yk = d_key; c.a.gq = d_query_out; c.a.gk = d_key_out;
    c.a.pq = d_query_weight ? static_cast<float*>(workspace) : nullptr;
    c.a.pk = d_key_weight ? static_cast<float*>(workspace) + (d_query_weight ? int64_t(c.a.blocks_q) * dims->D : 0) : nullptr;
    hipError_t err = hipSuccess;
    if (c.a.blocks_q + c.a.blocks_k) err = qc::launch<true>(dims->dtype, c.sh, c.a, st);
    if (err == hipSuccess && weights) {
        err = qc::by_dtype(dims->dtype, [&](auto t) {
            const float *pq = c.a.pq, *pk = c.a.pk;
            int nq = c.a.blocks_q, nk = c.a.blocks_k, D = int(dims->D);
            void *dq = d_query_weight, *dk = d_key_weight;
            void* params[] = {&pq, &pk, &nq, &nk, &dq, &dk, &D};
            return hipLaunchKernel(reinterpret_cast<const void*>(&qc::qkn_weight_kernel<decltype(t)::value>),
                                   dim3(unsigned((D + 15) / 16), 2), dim3(16 * qc::kRuns), params, 0, st);
        });
    }
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}

}  // extern "C"
