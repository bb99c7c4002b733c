// dca_state.hip -- states of linear attention with decays from chunk to chunk,
// without outputs (include/decay_attention.h; formulas in dca_chunk.hpp).
#include "dca_chunk.hpp"

namespace qc {
namespace {

// X = gamma_last X + A^T (w B) over a segment's chunks: forward S with A, B, w =
// K, V, eta; REV, from the last chunk to the first, dS with Q, dO, scale gamma.
// SUM: from zero, what a segment adds, stored where the next one takes it.
// Otherwise (REV alone) from the segment's state, which it leaves before each
// chunk as dS1, and at the end of the sequence as the gradient of s0.  A block
// has 64 CT columns of V, a wave 16 CT of them, held as [columns of V, KP] so
// that a lane's accumulators are consecutive in memory, [KP][VP].  Bound, where it
// stores, by memory: 4 x 4096 tokens of 32 heads of 128, bfloat16, 740 MB in 185 us,
// 4.0 TB/s; sums alone of 8192 tokens of 32 heads, 100 MB in 45 us, by a chunk's
// phases (loads two chunks ahead changed nothing: 47 us).
template <int DT, int KB, int CT, bool REV, bool SUM>
__global__ void __launch_bounds__(256, 2) dca_state_kernel(DcaArgs a) {
    using E = typename Storage<DT>::type;
    constexpr int C = dca_chunk(DT), NP = parts_of(DT), JB = C / 32, KP = 32 * KB, VW = 64 * CT, KT = 2 * KB;
    __shared__ __align__(16) char lx[NP * C * KP * 2], ly[NP * C * VW * 2];
    __shared__ __align__(16) Decays<C> dec;
    constexpr bool kTight = DT == 1 && KB == 4 && CT == 2 && !SUM;
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), g = lane / 16, m = lane % 16;
    int64_t u;
    int part;
    if (!dca_unit((SUM && a.offsets ? a.cuts : a.seg_slots) * a.Hk, a.group * a.tiles, u, part)) return;
    int64_t seg_slot = u / a.Hk, n;
    int cut = 0;
    if (SUM && a.offsets) {
        n = cut_owner(a, seg_slot, cut);
        if (n < 0) return;
    } else {
        n = owner<C, true>(a, seg_slot);
    }
    const Span s = span_of<C>(a, n);
    if (SUM && a.offsets) seg_slot = s.seg + cut + REV;       // (from the end, a segment that one is before)
    const int hk = int(u % a.Hk), h = hk * a.group + part / a.tiles, v0 = part % a.tiles * VW;
    const int64_t seg = seg_slot - s.seg;
    const int segs = segments_of(a, s);
    if (seg < 0 || seg >= segs) return;
    if (SUM && seg == (REV ? 0 : segs - 1)) return;
    const int first = int(seg * (a.seg_tokens / C)), all = (s.len + C - 1) / C;
    const int last = seg + 1 == segs ? all : first + int(a.seg_tokens / C);
    const int64_t size = int64_t(KP) * a.VP;
    const int row = wave * 16 * CT + 4 * CT * g;         // first of the lane's 4 CT columns of V, in the block's

    f32x4 X[CT][KT];
    const bool own = !SUM && seg + 1 < segs;
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int r = 0; r < KT; ++r) {
            const int k = 16 * r + m, v = v0 + row + 4 * c;
            X[c][r] = zero4();
            if (own) {
                X[c][r] = *reinterpret_cast<const f32x4*>(a.seg + (cut_slot(a, s, n, seg) * a.Hv + h) * size + int64_t(k) * a.VP + v);
            } else if (!SUM && a.d_fin && k < a.K) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (v + i < a.V) X[c][r][i] = a.d_fin[((n * a.Hv + h) * a.K + k) * a.V + v + i];
            }
        }

    const int64_t* xs = REV ? a.qs : a.ks;
    const int64_t ys = REV ? int64_t(a.Hv) * a.V : a.vs[1];
    const E* x = same_in_all_lanes(static_cast<const E*>(REV ? a.q : a.k) + s.b * xs[0] + s.t0 * xs[1] + hk * xs[2]);
    const E* y = same_in_all_lanes(REV ? static_cast<const E*>(a.d_out) + ((s.b * a.T + s.t0) * a.Hv + h) * int64_t(a.V) + v0
                                       : static_cast<const E*>(a.v) + s.b * a.vs[0] + s.t0 * a.vs[1] + h * a.vs[2] + v0);
    const float* gd = same_in_all_lanes(a.g + s.b * a.gs[0] + s.t0 * a.gs[1] + h * a.gs[2]);
    Rows<DT, C, KP> rx;
    Rows<DT, C, VW> ry;
    float rg = 0.f;
    auto load = [&](int c) {
        const int64_t t = int64_t(c) * C;
        const int rem = int(s.len - t);
        const int id = fresh<kTight>(tid);
        rx.load(x + t * xs[1], xs[1], rem, a.K, a.vec_qk, id);
        ry.load(y + t * ys, ys, rem, a.V - v0, REV ? a.vec_o : a.vec_v, id);
        rg = lane < C && lane < rem ? gd[(t + lane) * a.gs[1]] : 0.f;
    };
    double decay = 0.;
    if (first < last) load(REV ? last - 1 : first);
    for (int step = 0; step < last - first; ++step) {
        const int chunk = REV ? last - 1 - step : first + step;
        __syncthreads();
        const int id = fresh<kTight>(tid), l = id % 64, g = l / 16, m = l % 16;
        rx.store(lx, id);
        ry.store(ly, id);
        if (wave == 0) decay += put_decays<C>(dec, rg, lane);
        if constexpr (!SUM) {
            float* dst = a.ds + ((s.slot + chunk) * a.Hv + h) * size + int64_t(m) * a.VP + v0 + wave * 16 * CT + 4 * CT * g;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int r = 0; r < KT; ++r) *reinterpret_cast<f32x4*>(dst + int64_t(16 * r) * a.VP + 4 * c) = X[c][r];
        }
        __syncthreads();
        if (step + 1 < last - first) load(REV ? chunk - 1 : chunk + 1);
        const float keep = dec.gamma[C - 1];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < KT; ++r) X[c][r] *= keep;
#pragma unroll
        for (int b = 0; b < JB; ++b) {
            float w[8];
            read8((REV ? dec.gamma : dec.eta) + 32 * b + 8 * g, w);
            bf16x8 yf[CT][kParts];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                bf16x8 p[NP];
                col_fragment<C, VW>(ly, b, g, m, wave * 16 * CT + (CT == 2 ? 8 * (m & 3) + 4 * c : 4 * (m & 3)), p);
                float z[8];
                whole(p, z);
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] *= REV ? a.scale * w[j] : w[j];
                split<kParts, 8>(z, yf[c]);
            }
#pragma unroll
            for (int r = 0; r < KT; ++r) {
                bf16x8 xf[NP];
                col_fragment<C, KP>(lx, b, g, m, 16 * r + 4 * (m & 3), xf);
#pragma unroll
                for (int c = 0; c < CT; ++c) mma(X[c][r], yf[c], xf);
            }
        }
    }
    if constexpr (SUM) {
        const int64_t to = cut_slot(a, s, n, REV ? seg - 1 : seg);
        float* dst = a.seg + (to * a.Hv + h) * size + v0 + row;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < KT; ++r) *reinterpret_cast<f32x4*>(dst + int64_t(16 * r + m) * a.VP + 4 * c) = X[c][r];
        if (!v0 && tid == 0) a.seg_decay[to * a.Hv + h] = exp2_of(decay);
    } else if (a.ds0 && seg == 0) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < KT; ++r) {
                const int k = 16 * r + m, v = v0 + row + 4 * c;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (k < a.K && v + i < a.V) a.ds0[((n * a.Hv + h) * a.K + k) * a.V + v + i] = X[c][r][i];
            }
    }
}

// The states at segments' starts (REV: dS at their ends) from what dca_state left there: one after the other, 1024
// elements of a state to a block, eight segments' loads at once (15 segments of 32 heads of 128 x 128: 13 us, 5 TB/s).
template <bool REV>
__global__ void __launch_bounds__(256) dca_join_kernel(DcaArgs a, int KP) {
    const int per = int((int64_t(KP) * a.VP + 1023) / 1024);
    int64_t n = blockIdx.x / (int64_t(per) * a.Hv);
    const int h = int(blockIdx.x / per % a.Hv);
    if (a.offsets) {
        int cut = 0;
        n = cut_owner(a, n, cut);
        if (n < 0 || cut) return;                 // (the sequence's first cut stands for it)
    }
    const Span s = span_of<64>(a, n);         // (its chunks do not matter here)
    const int segs = segments_of(a, s);
    if (segs < 2) return;
    const int64_t size = int64_t(KP) * a.VP;
    const int at = int(blockIdx.x % per * 256 + threadIdx.x) * 4;
    if (at >= size) return;
    const int k = at / a.VP, v = at % a.VP;
    const float* start = REV ? a.d_fin : a.s0;
    f32x4 run = zero4();
    if (start && k < a.K) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (v + i < a.V) run[i] = start[((n * a.Hv + h) * a.K + k) * a.V + v + i];
    }
    // Step i = 1 .. segs - 1 takes the state over segment i - 1 (REV: counted from the end), to where it meets the next.
    auto slot = [&](int i) { return cut_slot(a, s, n, REV ? segs - 1 - i : i - 1); };
    constexpr int kAhead = 8;
    for (int i0 = 1; i0 < segs; i0 += kAhead) {
        f32x4 x[kAhead];
        float d[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j < segs ? i0 + j : segs - 1;
            x[j] = *reinterpret_cast<const f32x4*>(a.seg + (slot(i) * a.Hv + h) * size + at);
            d[j] = a.seg_decay[slot(i) * a.Hv + h];
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j < segs) {
                run = run * d[j] + x[j];
                *reinterpret_cast<f32x4*>(a.seg + (slot(i0 + j) * a.Hv + h) * size + at) = run;
            }
    }
}

}  // namespace

hipError_t launch_dca_state(int dt, int kb, int ct, bool rev, bool sum, const DcaArgs& a, hipStream_t st) {
    return by_dca_shape(dt, kb, ct, [&](auto d, auto k, auto c) {
        constexpr int DT = decltype(d)::value, KB = decltype(k)::value, CT = decltype(c)::value;
        const void* fn = !rev  ? reinterpret_cast<const void*>(&dca_state_kernel<DT, KB, CT, false, true>)
                         : sum ? reinterpret_cast<const void*>(&dca_state_kernel<DT, KB, CT, true, true>)
                               : reinterpret_cast<const void*>(&dca_state_kernel<DT, KB, CT, true, false>);
        DcaArgs args = a;
        void* params[] = {&args};
        const int64_t blocks = ((sum && a.offsets ? a.cuts : a.seg_slots) * a.Hk + 7) / 8 * 8 * (a.group * a.tiles);
        return hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(256), params, 0, st);
    });
}

hipError_t launch_dca_join(int kb, bool rev, const DcaArgs& a, hipStream_t st) {
    const void* fn = rev ? reinterpret_cast<const void*>(&dca_join_kernel<true>) : reinterpret_cast<const void*>(&dca_join_kernel<false>);
    DcaArgs args = a;
    int KP = 32 * kb;
    void* params[] = {&args, &KP};
    return hipLaunchKernel(fn, dim3(unsigned((int64_t(KP) * a.VP + 1023) / 1024 * (a.offsets ? a.cuts : a.N) * a.Hv)), dim3(256), params, 0, st);
}

}  // namespace qc
