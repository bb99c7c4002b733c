// layer_norm.hip -- layer norm over the last axis and its VJP (include/layer_norm.h).
//
// Forward, per row x [D]: mean = sum x / D, d = x - mean, m = sum d / D (what
// rounding left in the mean), v = sum d^2 / D - m^2, r = 1 / sqrt(v + eps),
// h = (d - m) r, y = h w + b.  VJP, with the cotangent g of y: dh = g w,
//     dx = r (dh - sum(dh) / D - h sum(dh h) / D),   dw = sum of g h,   db = sum of g
// over the rows.  Statistics and sums are float32; the mean is kept as (mean, m),
// so that rows far from zero have the forward's differences in the VJP.
//
// Bound by memory: every element is read once (twice as x and g in the VJP) and
// written once, so TR threads hold a row in registers between the sums and the
// result, S runs of W consecutive elements each: W = 8 where rows lie on 16
// bytes, else 1.  Rows of up to 512 elements (W = 8) share a wave with others,
// next to each other in memory: heads of a token, or rows.  What is under way
// counts, so rows stay as they lie, in half the registers of floats, and sums
// are made without LDS.  16384 rows of 4096 in bfloat16: 58 us, 4.6 TB/s (as
// floats, by four waves to a row, 71), and VJP 126 us, 3.2 TB/s: weight and bias of
// long rows stay in no register and are read again for each, from the caches, as
// many bytes as the rows.  4 x 4096 tokens of 32 heads of 128 with weights of each
// head, held by their groups: forward 50 us, 5.5 TB/s (one row at a time, heads
// apart, 64), VJP 82 us, 5.0 TB/s (92), and 4 us for the weights' sums.  Rows that
// are not on 16 bytes go element by element: 16384 of 4100 in bfloat16 292 us, VJP
// 360; the 4096 of a view that begins at the second element 211, 502.  The VJP
// spills above 8192 elements: float32 on 16 bytes 100 bytes of scratch a lane, and
// any type off them 212 to 220 (4096 rows of 16380 in bfloat16: 724 us).
#include "layer_norm.h"
#include "lm_common.hpp"
#include "qc_internal.hpp"
#include "quat_cumprod.h"

#include <type_traits>

namespace qc {
namespace {

constexpr int kLnThreads = 256;                // threads of a block, or TR if that is more
constexpr int kLnMaxD = 16384;
// Blocks that share a weight gradient's sum, for all heads together: enough to
// fill 256 CUs several times, few enough that their partial sums are short.
constexpr int64_t kLnPartials = 1024;

struct LnArgs {
    const void *x, *w, *b, *gy;
    void* y;                       // forward: y; VJP: dx (may be null)
    float* stats;                  // [rows][4]: mean, m, r, 0
    float* part;                   // VJP: partial sums [blocks][heads][2][D] (null: no gradient of weight or bias)
    int64_t xs[3];
    int64_t T, H, rows;            // rows of a head (by_head), or all
    int64_t blocks;                // that share the rows
    int D, heads, flat, small;     // heads: H with by_head, else 1
    int side, sides;               // heads of a token to a block (a power of two), and blocks for all of them
    float eps, inv;
};

__device__ __forceinline__ int64_t ln_quotient(int64_t n, int64_t d, bool small) {
    return small ? int64_t(uint32_t(n) / uint32_t(d)) : n / d;
}

// Sums over a row's TR threads, in each of them.  Every thread of the block calls it.
template <int TR, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*red)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = lanes_sum<(TR < 64 ? TR : 64)>(x[n]);
    if constexpr (TR > 64) {
        __syncthreads();
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) red[threadIdx.x / 64][n] = x[n];
        __syncthreads();
        const int w0 = threadIdx.x / TR * (TR / 64);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            x[n] = 0.f;
#pragma unroll
            for (int w = 0; w < TR / 64; ++w) x[n] += red[w0 + w][n];
        }
    }
}

// R rows of a group of TR threads at once, so that their loads are under way together.
template <int DT, int W, int S, int TR, int R, bool BWD>
__global__ void __launch_bounds__(TR > kLnThreads ? TR : kLnThreads) ln_kernel(LnArgs a) {
    using E = typename Storage<DT>::type;
    constexpr int kBlock = TR > kLnThreads ? TR : kLnThreads, kGroups = kBlock / TR;
    constexpr bool kHeld = S * W <= 16;        // weight and bias in registers, or read again for every row (from L1)
    const int lane = threadIdx.x % TR, group = threadIdx.x / TR;
    // Groups of a block: `side` heads of a token next to each other, then tokens; without heads, rows.
    const int head = int(blockIdx.x % a.sides) * a.side + group % a.side, first = group / a.side, step = kGroups / a.side;
    const bool on_head = head < a.heads;
    const int D = a.D, h = on_head ? head : 0;
    const int64_t block = blockIdx.x / a.sides;
    const bool small = a.small != 0;
    const E *pw = a.w ? static_cast<const E*>(a.w) + int64_t(h) * D : nullptr, *pb = a.b ? static_cast<const E*>(a.b) + int64_t(h) * D : nullptr;
    __shared__ float red1[kBlock / 64][R], red2[kBlock / 64][2 * R];
    float hw[kHeld ? S : 1][W], hb[kHeld && !BWD ? S : 1][W];
    float sw[BWD ? S : 1][W], sb[BWD ? S : 1][W];
    auto get = [&](const E* p, int s, float none, float (&x)[W]) {
        const int at = (s * TR + lane) * W;
#pragma unroll
        for (int j = 0; j < W; ++j) x[j] = none;
        if (p && at < D) load_floats<W>(p + at, x);
    };
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if constexpr (kHeld) {
            get(pw, s, 1.f, hw[s]);
            if constexpr (!BWD) get(pb, s, 0.f, hb[s]);
        }
        if constexpr (BWD)
#pragma unroll
            for (int j = 0; j < W; ++j) sw[s][j] = sb[s][j] = 0.f;
    }
    // (Every group of a block takes as many turns as the first: the sums over more than a wave are the block's.)
    for (int64_t r0 = block * (step * R); r0 < a.rows; r0 += a.blocks * (step * R)) {
        // Rows stay as they lie in memory, half the registers of floats, and are taken apart in each pass over them.
        Held<E, W, (W > 1)> hx[R][S], hg[BWD ? R : 1][S];
        int64_t row[R];
        bool in[R];
        f32x4 st[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            in[k] = on_head && r0 + first + k * step < a.rows;
            const int64_t i = in[k] ? r0 + first + k * step : a.rows - 1;
            // Row i of a head is token i; without heads, row i is head i % H of token i / H.
            int64_t src;
            row[k] = i;
            if (a.heads > 1) {
                row[k] = i * a.H + h;
                if (a.flat) {
                    src = i * a.xs[1] + h * a.xs[2];
                } else {
                    const int64_t bt = ln_quotient(i, a.T, small);
                    src = bt * a.xs[0] + (i - bt * a.T) * a.xs[1] + h * a.xs[2];
                }
            } else if (a.flat) {
                src = i * a.xs[2];
            } else {
                const int64_t token = ln_quotient(i, a.H, small), bt = ln_quotient(token, a.T, small);
                src = bt * a.xs[0] + (token - bt * a.T) * a.xs[1] + (i - token * a.H) * a.xs[2];
            }
            if constexpr (BWD) st[k] = *reinterpret_cast<const f32x4*>(a.stats + row[k] * 4);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int at = (s * TR + lane) * W;
                hx[k][s].load(static_cast<const E*>(a.x) + src + at, D - at);
                if constexpr (BWD) hg[k][s].load(static_cast<const E*>(a.gy) + row[k] * D + at, D - at);
            }
        }
        auto renew = [&] {
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    hx[k][s].renew();
                    if constexpr (BWD) hg[k][s].renew();
                }
        };
        if constexpr (!BWD) {
            float one[R], two[2 * R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                one[k] = two[2 * k] = two[2 * k + 1] = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    float x[W];
                    hx[k][s].get(x);
#pragma unroll
                    for (int j = 0; j < W; ++j) one[k] += x[j];
                }
            }
            row_sums<TR, R>(one, red1);
            renew();
#pragma unroll
            for (int k = 0; k < R; ++k) {
                one[k] *= a.inv;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if ((s * TR + lane) * W >= D) continue;
                    float x[W];
                    hx[k][s].get(x);
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        x[j] -= one[k];
                        two[2 * k] += x[j];
                        two[2 * k + 1] += x[j] * x[j];
                    }
                }
            }
            row_sums<TR, 2 * R>(two, red2);
            renew();
            float r[R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const float m = two[2 * k] * a.inv, v = two[2 * k + 1] * a.inv - m * m;
                two[2 * k] = m;
                r[k] = 1.f / sqrtf((v > 0.f ? v : v == v ? 0.f : v) + a.eps);
                if (in[k] && a.stats && lane == 0) *reinterpret_cast<f32x4*>(a.stats + row[k] * 4) = f32x4{one[k], m, r[k], 0.f};
            }
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int at = (s * TR + lane) * W;
                float w[W], b[W];
                if constexpr (kHeld) {
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        w[j] = hw[s][j];
                        b[j] = hb[s][j];
                    }
                } else {
                    get(pw, s, 1.f, w);
                    get(pb, s, 0.f, b);
                }
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    float x[W];
                    hx[k][s].get(x);
#pragma unroll
                    for (int j = 0; j < W; ++j) x[j] = (x[j] - one[k] - two[2 * k]) * r[k] * w[j] + b[j];
                    if (in[k] && at < D) store_floats<W>(static_cast<E*>(a.y) + row[k] * D + at, x);
                }
            }
        } else {
            float two[2 * R];
#pragma unroll
            for (int k = 0; k < R; ++k) two[2 * k] = two[2 * k + 1] = 0.f;
            // h = (x - mean) r and the cotangent, 0 outside the row and the rows.
            auto pass = [&](int k, int s, float (&h)[W], float (&g)[W]) {
                const bool on = in[k] && (s * TR + lane) * W < D;
                hx[k][s].get(h);
                hg[k][s].get(g);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    h[j] = on ? (h[j] - st[k][0] - st[k][1]) * st[k][2] : 0.f;
                    g[j] = on ? g[j] : 0.f;
                }
            };
            auto weight = [&](int s, float (&w)[W]) {
                if constexpr (kHeld) {
#pragma unroll
                    for (int j = 0; j < W; ++j) w[j] = hw[s][j];
                } else {
                    get(pw, s, 1.f, w);
                }
            };
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float w[W];
                weight(s, w);
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    float h[W], g[W];
                    pass(k, s, h, g);
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        sw[s][j] += g[j] * h[j];
                        sb[s][j] += g[j];
                        g[j] *= w[j];
                        two[2 * k] += g[j];
                        two[2 * k + 1] += g[j] * h[j];
                    }
                }
            }
            if (!a.y) continue;
            row_sums<TR, 2 * R>(two, red2);
            renew();
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int at = (s * TR + lane) * W;
                float w[W];
                weight(s, w);
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    float h[W], g[W];
                    pass(k, s, h, g);
                    const float c0 = two[2 * k] * a.inv, c1 = two[2 * k + 1] * a.inv;
#pragma unroll
                    for (int j = 0; j < W; ++j) h[j] = st[k][2] * (g[j] * w[j] - c0 - h[j] * c1);
                    if (in[k] && at < D) store_floats<W>(static_cast<E*>(a.y) + row[k] * D + at, h);
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        // The sums, in a fixed order.  Heads: a group's own.  Else the block's: groups of a wave by shuffles, waves through LDS.
        if (kGroups == 1 || a.heads > 1) {
            if (!on_head) return;
            float* part = a.part + ((block * step + first) * a.heads + head) * 2 * int64_t(D);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int at = (s * TR + lane) * W;
                if (at < D) {
                    store_floats<W>(part + at, sw[s]);
                    store_floats<W>(part + D + at, sb[s]);
                }
            }
        } else {
            float* part = a.part + block * 2 * int64_t(D);
            constexpr int kSum = TR < 64 ? TR : 64, kWaves = kBlock / 64, kPer = TR < 64 ? kWaves : kBlock / TR;
            __shared__ float red[kWaves][W * 2][kSum];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (s) __syncthreads();
#pragma unroll
                for (int j = 0; j < W; ++j) {
#pragma unroll
                    for (int m = TR; m < 64; m *= 2) {
                        sw[s][j] += __shfl_xor(sw[s][j], m, 64);
                        sb[s][j] += __shfl_xor(sb[s][j], m, 64);
                    }
                    if (threadIdx.x % 64 < kSum) {
                        red[threadIdx.x / 64][j * 2][threadIdx.x % 64] = sw[s][j];
                        red[threadIdx.x / 64][j * 2 + 1][threadIdx.x % 64] = sb[s][j];
                    }
                }
                __syncthreads();
                const int at = (s * TR + lane) * W;
                if (threadIdx.x < TR && at < D) {
                    constexpr int kStep = TR < 64 ? 1 : TR / 64;       // waves that hold the same elements are kStep apart
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        float tw = 0.f, tb = 0.f;
#pragma unroll
                        for (int c = 0; c < kPer; ++c) {
                            tw += red[threadIdx.x / 64 + c * kStep][j * 2][threadIdx.x % 64];
                            tb += red[threadIdx.x / 64 + c * kStep][j * 2 + 1][threadIdx.x % 64];
                        }
                        part[at + j] = tw;
                        part[D + at + j] = tb;
                    }
                }
            }
        }
    }
}

struct LnShape {
    bool wide;          // W = 8
    int tr, s, r;       // threads of a row, runs of a thread, rows at once
};

// A row's threads and runs go by its length alone, so that its result does not depend on the rows it comes with: a wave
// has up to 8 runs to a lane (VJP: 4) before a row gets another, since waves that wait for each other cost more than the
// loads of one.  Where there are rows for two waves on each of 1024 SIMDs and four to spare, short ones come four to a group.
LnShape ln_shape(int64_t D, int64_t all, bool wide, bool bwd) {
    LnShape sh{wide, 4, 1, 1};
    if (wide) {
        const int64_t runs = (D + 7) / 8;
        while (sh.tr < 64 && sh.tr < runs) sh.tr *= 2;
        while (sh.s < (bwd ? 4 : 8) && sh.tr * sh.s < runs) sh.s *= 2;
        while (sh.tr * sh.s < runs) sh.tr *= 2;
        if (sh.s == 1 && all * sh.tr >= int64_t(64) * 2048 * 4) sh.r = 4;
    } else {
        sh.tr = D <= 1024 ? 64 : D <= 4096 ? 256 : 1024;
        while (sh.tr * sh.s < D) sh.s *= 2;
    }
    return sh;
}

// The weights' gradients from the blocks' partial sums: 16 columns and 64 runs
// of blocks to a block of threads, the runs joined in order.  A launch holds
// less than 2^32 threads, so blocks take every kLnColumns-th 16 columns.
constexpr int kLnRuns = 64;
constexpr int64_t kLnColumns = int64_t(1) << 20;

template <int DT>
__global__ void __launch_bounds__(16 * kLnRuns) ln_weight_kernel(const float* part, int64_t n, int heads, int D, void* dw, void* db) {
    using E = typename Storage<DT>::type;
    E* out = static_cast<E*>(blockIdx.y ? db : dw);
    if (!out) return;
    const int64_t all = int64_t(heads) * D;
    const int run = threadIdx.x / 16;
    __shared__ float red[kLnRuns][17];
    for (int64_t first = int64_t(blockIdx.x) * 16; first < all; first += kLnColumns * 16) {
        const int64_t col = first + threadIdx.x % 16;
        float s = 0.f;
        if (col < all) {
            const float* p = part + (col / D * 2 + blockIdx.y) * D + col % D;
#pragma unroll 4
            for (int64_t i = run; i < n; i += kLnRuns) s += p[i * 2 * all];
        }
        red[run][threadIdx.x % 16] = s;
        __syncthreads();
        if (threadIdx.x < 16 && col < all) {
            float t = 0.f;
#pragma unroll 8
            for (int i = 0; i < kLnRuns; ++i) t += red[i][threadIdx.x];
            out[col] = E(t);
        }
        __syncthreads();
    }
}

template <class F>
hipError_t ln_by_dtype(int dt, F&& f) {
    if (dt == 0) return f(std::integral_constant<int, 0>{});
    if (dt == 1) return f(std::integral_constant<int, 1>{});
    return f(std::integral_constant<int, 2>{});
}

template <int DT, bool BWD>
const void* ln_kernel_of(const LnShape& sh) {
#define LN_WIDE(s_, tr_, r_) \
    if (sh.wide && sh.s == s_ && sh.tr == tr_ && sh.r == r_) return reinterpret_cast<const void*>(&ln_kernel<DT, 8, s_, tr_, r_, BWD>);
#define LN_NARROW(s_, tr_) \
    if (!sh.wide && sh.s == s_ && sh.tr == tr_) return reinterpret_cast<const void*>(&ln_kernel<DT, 1, s_, tr_, 1, BWD>);
    LN_WIDE(1, 4, 1) LN_WIDE(1, 8, 1) LN_WIDE(1, 16, 1) LN_WIDE(1, 32, 1) LN_WIDE(1, 64, 1)
    LN_WIDE(1, 4, 4) LN_WIDE(1, 8, 4) LN_WIDE(1, 16, 4) LN_WIDE(1, 32, 4) LN_WIDE(1, 64, 4)
    LN_WIDE(2, 64, 1) LN_WIDE(4, 64, 1)
    if constexpr (BWD) {
        LN_WIDE(4, 128, 1) LN_WIDE(4, 256, 1) LN_WIDE(4, 512, 1)
    } else {
        LN_WIDE(8, 64, 1) LN_WIDE(8, 128, 1) LN_WIDE(8, 256, 1)
    }
    LN_NARROW(1, 64) LN_NARROW(2, 64) LN_NARROW(4, 64) LN_NARROW(8, 64) LN_NARROW(16, 64)
    LN_NARROW(8, 256) LN_NARROW(16, 256) LN_NARROW(8, 1024) LN_NARROW(16, 1024)
#undef LN_WIDE
#undef LN_NARROW
    return nullptr;
}

template <bool BWD>
hipError_t ln_launch(int dt, const LnShape& sh, const LnArgs& a, hipStream_t st) {
    return ln_by_dtype(dt, [&](auto t) {
        const void* fn = ln_kernel_of<decltype(t)::value, BWD>(sh);
        if (!fn) return hipErrorInvalidConfiguration;
        LnArgs args = a;
        void* params[] = {&args};
        return hipLaunchKernel(fn, dim3(unsigned(a.blocks * a.sides)), dim3(unsigned(sh.tr > kLnThreads ? sh.tr : kLnThreads)), params, 0, st);
    });
}

int ln_check(const lnm_dims* d) {
    if (!d) return QC_ERR_NULL;
    if (d->dtype < 0 || d->dtype > 2) return QC_ERR_DTYPE;
    if (d->B < 0 || d->T < 0 || d->H < 0 || d->D < 1 || d->D > kLnMaxD || d->H > (1 << 20)) return QC_ERR_SHAPE;
    if (count(count(d->B, d->T), count(d->H, d->D)) < 0) return QC_ERR_SHAPE;
    if (d->by_head && d->H * d->D >= (int64_t(1) << 31)) return QC_ERR_SHAPE;
    if (strided_bytes(d->B, d->T, d->H, d->D, d->x_stride, dtype_bytes(d->dtype)) < 0) return QC_ERR_SHAPE;
    if (!(d->eps >= 0.f)) return QC_ERR_OPTION;
    return QC_OK;
}

int64_t ln_heads(const lnm_dims& d) { return d.by_head && d.H ? d.H : 1; }
int64_t ln_rows(const lnm_dims& d) { return d.by_head ? d.B * d.T : d.B * d.T * d.H; }

// Partial sums of a head: no more than fill the card.
int64_t ln_partials(const lnm_dims& d) {
    int64_t groups = 1;              // of a block, the most that ln_shape makes of such rows
    if (ln_heads(d) > 1)
        while (groups < 64 && groups * 2 * ((d.D + 7) / 8) <= kLnThreads) groups *= 2;
    const int64_t share = kLnPartials * groups / ln_heads(d);
    return share > 1 ? share : 1;
}

// Grid of a call: heads to a block, blocks for the heads, and blocks that share the rows, at most `most` groups of them
// for a head.  Returns a head's groups, of which each leaves partial sums.
int64_t ln_grid(LnArgs& a, const LnShape& sh, int64_t most) {
    const int groups = sh.tr > kLnThreads ? 1 : kLnThreads / sh.tr;
    a.side = 1;
    if (a.heads > 1)
        while (a.side * 2 <= groups && a.side * 2 <= a.heads) a.side *= 2;
    a.sides = (a.heads + a.side - 1) / a.side;
    const int64_t step = groups / a.side, per = step * sh.r, n = (a.rows + per - 1) / per, cap = a.heads > 1 ? most / step : most;
    a.blocks = n < cap ? n : cap > 1 ? cap : 1;
    if (!a.rows) a.blocks = 0;
    return a.blocks * (a.heads > 1 ? step : 1);
}

LnArgs ln_arguments(const lnm_dims& d, const void* x, const void* w) {
    LnArgs a{};
    a.x = x; a.w = w;
    for (int i = 0; i < 3; ++i) a.xs[i] = d.x_stride[i];
    a.T = d.T; a.H = d.H; a.rows = ln_rows(d);
    a.D = int(d.D); a.heads = int(ln_heads(d));
    const bool tokens = d.B <= 1 || d.x_stride[0] == d.T * d.x_stride[1];
    a.flat = a.heads > 1 ? tokens : (d.H <= 1 && d.T <= 1) ? d.B <= 1 : tokens && (d.H <= 1 || d.x_stride[1] == d.H * d.x_stride[2]);
    // One row to a token: tokens' stride is the rows'.
    if (a.heads == 1 && d.H == 1) a.xs[2] = d.T > 1 ? d.x_stride[1] : d.x_stride[0];
    if (a.heads == 1 && d.H == 1 && d.T <= 1) a.flat = 1;
    a.small = d.B * d.T * d.H < (int64_t(1) << 31);
    a.eps = d.eps;
    a.inv = 1.f / float(d.D);
    return a;
}

}  // namespace
}  // namespace qc

extern "C" {

int lnm_fwd(const lnm_dims* dims, const void* x, const void* weight, const void* bias, void* y, float* stats, void* stream) {
    const int rc = qc::ln_check(dims);
    if (rc != QC_OK) return rc;
    const lnm_dims& d = *dims;
    const int64_t rows = d.B * d.T * d.H;
    if (!rows) return QC_OK;
    if (!x || !y) return QC_ERR_NULL;
    const size_t e = qc::dtype_bytes(d.dtype), w = size_t(qc::ln_heads(d) * d.D) * e;
    for (const void* p : {x, weight, bias, static_cast<const void*>(y)})
        if (!qc::aligned_to(p, e)) return QC_ERR_ALIGN;
    if (!qc::aligned_to(stats, 16)) return QC_ERR_ALIGN;
    const qc::ByteSpan sp[] = {{y, size_t(rows * d.D) * e}, {stats, size_t(rows) * 16},
                               {x, size_t(qc::strided_bytes(d.B, d.T, d.H, d.D, d.x_stride, e))}, {weight, w}, {bias, w}};
    if (qc::outputs_overlap(sp, 2, 5)) return QC_ERR_ALIAS;
    qc::LnArgs a = qc::ln_arguments(d, x, weight);
    a.b = bias; a.y = y; a.stats = stats;
    const bool wide = d.D % 8 == 0 && qc::rows_on_16(x, d.x_stride, e) && qc::aligned_to(y, 16) && qc::aligned_to(weight, 16) && qc::aligned_to(bias, 16);
    const qc::LnShape sh = qc::ln_shape(d.D, rows, wide, false);
    qc::ln_grid(a, sh, (int64_t(1) << 20) / a.heads + 1);
    const hipError_t err = qc::ln_launch<false>(d.dtype, sh, a, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}

size_t lnm_workspace_bytes(const lnm_dims* dims) {
    if (qc::ln_check(dims) != QC_OK) return 0;
    return size_t(qc::ln_partials(*dims) * qc::ln_heads(*dims) * 2 * dims->D) * 4 + 16;
}

int lnm_bwd(const lnm_dims* dims, const void* x, const void* weight, const float* stats, const void* d_y, void* d_x, void* d_weight,
            void* d_bias, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = qc::ln_check(dims);
    if (rc != QC_OK) return rc;
    const lnm_dims& d = *dims;
    if ((!d_x && !d_weight && !d_bias) || (d.by_head && !d.H)) return QC_OK;
    const int64_t rows = d.B * d.T * d.H;
    const bool sums = d_weight || d_bias;
    if (rows && (!x || !stats || !d_y)) return QC_ERR_NULL;
    if (d_weight && !weight) return QC_ERR_NULL;
    const size_t need = lnm_workspace_bytes(dims);
    if (sums && (!workspace || workspace_bytes < need)) return QC_ERR_WORKSPACE;
    if (sums && !qc::aligned_to(workspace, 16)) return QC_ERR_ALIGN;
    const size_t e = qc::dtype_bytes(d.dtype), w = size_t(qc::ln_heads(d) * d.D) * e;
    bool wide = d.D % 8 == 0 && qc::rows_on_16(x, d.x_stride, e) && qc::aligned_to(weight, 16);
    for (const void* p : {d_y, static_cast<const void*>(d_x)}) wide = wide && qc::aligned_to(p, 16);
    for (const void* p : {x, weight, d_y, static_cast<const void*>(d_x), static_cast<const void*>(d_weight), static_cast<const void*>(d_bias)})
        if (!qc::aligned_to(p, e)) return QC_ERR_ALIGN;
    if (!qc::aligned_to(stats, 16)) return QC_ERR_ALIGN;
    const qc::ByteSpan sp[] = {{d_x, size_t(rows * d.D) * e}, {d_weight, w}, {d_bias, w}, {sums ? workspace : nullptr, need},
                               {x, size_t(qc::strided_bytes(d.B, d.T, d.H, d.D, d.x_stride, e))}, {weight, w},
                               {stats, size_t(rows) * 16}, {d_y, size_t(rows * d.D) * e}};
    if (qc::outputs_overlap(sp, 4, 8)) return QC_ERR_ALIAS;
    qc::LnArgs a = qc::ln_arguments(d, x, weight);
    a.gy = d_y; a.y = d_x; a.stats = const_cast<float*>(stats);
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    const qc::LnShape sh = qc::ln_shape(d.D, rows, wide, true);
    const int64_t partials = qc::ln_grid(a, sh, sums ? qc::ln_partials(d) : (int64_t(1) << 20) / a.heads + 1);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t err = hipSuccess;
    if (a.blocks) err = qc::ln_launch<true>(d.dtype, sh, a, st);
    if (err == hipSuccess && sums) {
        err = qc::ln_by_dtype(d.dtype, [&](auto t) {
            const float* part = a.part;
            int64_t blocks = partials;
            int heads = a.heads, D = a.D;
            void *dw = d_weight, *db = d_bias;
            void* params[] = {&part, &blocks, &heads, &D, &dw, &db};
            const int64_t columns = (int64_t(heads) * D + 15) / 16;
            return hipLaunchKernel(reinterpret_cast<const void*>(&qc::ln_weight_kernel<decltype(t)::value>),
                                   dim3(unsigned(columns < qc::kLnColumns ? columns : qc::kLnColumns), 2), dim3(16 * qc::kLnRuns), params, 0, st);
        });
    }
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}

}  // extern "C"
