// dca_fwd.hip -- linear attention with decays, forward (include/decay_attention.h;
// formulas and layouts in dca_chunk.hpp).
#include "dca_chunk.hpp"

namespace qc {
namespace {

// A block passes over one segment of one sequence for one value head and 64 CT
// columns of V; each of its four waves holds S of 16 CT columns in registers,
// [KP rows, 16 CT columns] as accumulators, which are in place the operands of
// the products with Q.  A chunk: its rows to LDS (loaded during the chunk
// before), P by tiles of 16 rows to a wave and shared through LDS, out^T = S^T
// Q^T gamma + V^T P^T, S = gamma_last S + K^T (eta V).
//
// Bound by instructions: a wave's chunk of 64 x 128 x 128 in bfloat16 is 240 MFMA
// (3840 cycles) and 1570 vector instructions (6280; splits, decays, scaling) in
// five phases.  Two waves to a SIMD, as many as the registers allow, spend 22500
// cycles on a chunk each, 20200 of them in the two kinds of instructions, which
// so hardly run beside each other.  8192 tokens of 32 heads of 128: 110 us, 22
// GFLOP of the recurrence and 200 MB; with S0 saved, 4 x 4096 tokens, 257 us, 940
// MB, 3.7 TB/s.
template <int DT, int KB, int CT, bool SAVE>
__global__ void __launch_bounds__(256, 2) dca_fwd_kernel(DcaArgs a) {
    using E = typename Storage<DT>::type;
    constexpr int C = dca_chunk(DT), NP = parts_of(DT), TT = C / 16, JB = C / 32, KP = 32 * KB, VW = 64 * CT, KT = 2 * KB;
    // Rows of Q, K and V; between chunks, a wave's columns of S on their way to memory.
    __shared__ __align__(16) char rows[NP * C * (2 * KP + VW) * 2];
    char *lq = rows, *lk = lq + NP * C * KP * 2, *lv = lk + NP * C * KP * 2;
    __shared__ __align__(16) bf16x8 lp[dca_tri(C)][kParts][64];
    __shared__ __align__(16) Decays<C> dec;
    // (64 x 128 with S0 saved: 9 registers spilled and 248 us for 4 x 4096 tokens of 32 heads, 224 so; not saved, 4 of them and
    // 118 us for 8192 tokens, 122 so; 128 x 64, saved or not: 2 to 4% slower so.)
    constexpr bool kTight = KB * CT == 8 || (DT == 1 && KB == 2 && CT == 2 && SAVE);
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), g = lane / 16, m = lane % 16;
    int64_t u;
    int part;
    if (!dca_unit(a.seg_slots * a.Hk, a.group * a.tiles, u, part)) return;
    const int64_t seg_slot = u / a.Hk, n = owner<C, true>(a, seg_slot);
    const Span s = span_of<C>(a, n);
    const int hk = int(u % a.Hk), h = hk * a.group + part / a.tiles, v0 = part % a.tiles * VW;
    const int64_t seg = seg_slot - s.seg;
    const int segs = segments_of(a, s);
    if (seg < 0 || seg >= segs) return;
    const int first = int(seg * (a.seg_tokens / C)), all = (s.len + C - 1) / C;
    const int last = seg + 1 == segs ? all : first + int(a.seg_tokens / C);

    // The wave's columns: of column tile c, lane m's.
    const int vw = v0 + wave * 16 * CT;
    auto column = [&](int c) { return vw + (CT == 2 ? 8 * (m >> 2) + 4 * c + (m & 3) : m); };
    f32x4 S[KT][CT];
    {
        // As S0 is saved, the other way round: rows of memory through LDS to columns of lanes.
        constexpr int kStep = 36, kLanes = 4 * CT, kPasses = 32 * kLanes / 64;
        static_assert(4 * 16 * CT * kStep * 4 <= sizeof(rows), "the columns' place");
        const bool own = seg > 0;
        const float* src = own ? a.seg + (cut_slot(a, s, n, seg - 1) * a.Hv + h) * int64_t(KP) * a.VP : a.s0 ? a.s0 + (n * a.Hv + h) * int64_t(a.K) * a.V : nullptr;
        const int nk = own ? KP : a.K, nv = own ? a.VP : a.V, row = lane / kLanes, col = vw + lane % kLanes * 4;
        const bool vec = own || (a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.s0) % 16 == 0);
        float* t = reinterpret_cast<float*>(rows) + wave * (16 * CT * kStep);
        f32x4 x[KB][kPasses];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                const int k = 32 * kb + p * (64 / kLanes) + row;
                const float* at = src + int64_t(k) * nv + col;
                x[kb][p] = zero4();
                if (src && k < nk) {
                    if (vec) {
                        if (col < nv) x[kb][p] = *reinterpret_cast<const f32x4*>(at);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (col + i < nv) x[kb][p][i] = at[i];
                    }
                }
            }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) t[(lane % kLanes * 4 + i) * kStep + p * (64 / kLanes) + row] = x[kb][p][i];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < CT; ++c) S[2 * kb + e][c] = *reinterpret_cast<const f32x4*>(t + (column(c) - vw) * kStep + 8 * g + 4 * e);
            __builtin_amdgcn_wave_barrier();
        }
    }

    const E* q = same_in_all_lanes(static_cast<const E*>(a.q) + s.b * a.qs[0] + s.t0 * a.qs[1] + hk * a.qs[2]);
    const E* k = same_in_all_lanes(static_cast<const E*>(a.k) + s.b * a.ks[0] + s.t0 * a.ks[1] + hk * a.ks[2]);
    const E* v = same_in_all_lanes(static_cast<const E*>(a.v) + s.b * a.vs[0] + s.t0 * a.vs[1] + h * a.vs[2] + v0);
    const float* gd = same_in_all_lanes(a.g + s.b * a.gs[0] + s.t0 * a.gs[1] + h * a.gs[2]);
    E* out = static_cast<E*>(a.out) + ((s.b * a.T + s.t0) * a.Hv + h) * int64_t(a.V);
    Rows<DT, C, KP> rq, rk;
    Rows<DT, C, VW> rv;
    float rg = 0.f;
    auto load = [&](int c) {
        const int64_t t = int64_t(c) * C;
        const int rem = int(s.len - t);
        const int id = fresh<kTight>(tid);
        rq.load(q + t * a.qs[1], a.qs[1], rem, a.K, a.vec_qk, id);
        rk.load(k + t * a.ks[1], a.ks[1], rem, a.K, a.vec_qk, id);
        rv.load(v + t * a.vs[1], a.vs[1], rem, a.V - v0, a.vec_v, id);
        rg = lane < C && lane < rem ? gd[(t + lane) * a.gs[1]] : 0.f;
    };
    if (first < last) load(first);
    for (int chunk = first; chunk < last; ++chunk) {
        const int rem = s.len - chunk * C;
        __syncthreads();
        if constexpr (SAVE) {
            // S0, 32 rows at a time: lanes hold a column's, memory wants a row's.  (Stored as they are, four bytes a lane,
            // 4 x 4096 tokens of 32 heads of 128 took 563 us instead of 240.)
            constexpr int kStep = 36, kLanes = 4 * CT;
            static_assert(4 * 16 * CT * kStep * 4 <= sizeof(rows), "the columns' place");
            const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
            float* t = reinterpret_cast<float*>(rows) + wave * (16 * CT * kStep);
            float* dst = a.save + ((s.slot + chunk) * a.Hv + h) * int64_t(KP) * a.VP + int64_t(l / kLanes) * a.VP + vw + l % kLanes * 4;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        *reinterpret_cast<f32x4*>(t + (CT == 2 ? 8 * (m >> 2) + 4 * c + (m & 3) : m) * kStep + 8 * g + 4 * e) = S[2 * kb + e][c];
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int p = 0; p < 32 * kLanes / 64; ++p) {
                    f32x4 x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = t[(l % kLanes * 4 + j) * kStep + p * (64 / kLanes) + l / kLanes];
                    *reinterpret_cast<f32x4*>(dst + int64_t(32 * kb + p * (64 / kLanes)) * a.VP) = x;
                }
                __builtin_amdgcn_wave_barrier();
            }
            __syncthreads();
        }
        {
            const int id = fresh<kTight>(tid);
            rq.store(lq, id);
            rk.store(lk, id);
            rv.store(lv, id);
        }
        if (wave == 0) put_decays<C>(dec, rg, lane);
        __syncthreads();
        if (chunk + 1 < last) load(chunk + 1);

        if (wave < TT) {
            const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
#pragma unroll
            for (int b = 0; b < JB; ++b) {
                if (b > (wave >> 1)) continue;
                f32x4 pt[2] = {zero4(), zero4()};
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    bf16x8 qf[NP];
                    row_fragment<C, KP>(lq, 16 * wave + m, kb, g, qf);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        bf16x8 kf[NP];
                        row_fragment<C, KP>(lk, tile_index(2 * b + e, m), kb, g, kf);
                        mma(pt[e], kf, qf);
                    }
                }
                float x[8];
                decayed_pairs(dec, pt, wave, b, g, m, 1.f, x);
                bf16x8 p[kParts];
                split<kParts, 8>(x, p);
#pragma unroll
                for (int j = 0; j < kParts; ++j) lp[tri_of(wave, b)][j][lane] = p[j];
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        f32x4 o[CT][TT];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int t = 0; t < TT; ++t) o[c][t] = zero4();
        const int l1 = fresh<kTight>(lane), g1 = l1 / 16, m1 = l1 % 16;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            bf16x8 sf[CT][kParts];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const float x[8] = {S[2 * kb][c][0], S[2 * kb][c][1], S[2 * kb][c][2], S[2 * kb][c][3],
                                    S[2 * kb + 1][c][0], S[2 * kb + 1][c][1], S[2 * kb + 1][c][2], S[2 * kb + 1][c][3]};
                split<kParts, 8>(x, sf[c]);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                bf16x8 qf[NP];
                row_fragment<C, KP>(lq, 16 * t + m1, kb, g1, qf);
#pragma unroll
                for (int c = 0; c < CT; ++c) mma(o[c][t], sf[c], qf);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float gamma = dec.gamma[16 * t + m];
#pragma unroll
            for (int c = 0; c < CT; ++c) o[c][t] *= gamma;
        }

        bf16x8 vf[CT][JB][NP];
        auto values = [&] {
            const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int b = 0; b < JB; ++b) col_fragment<C, VW>(lv, b, g, m, wave * 16 * CT + (CT == 2 ? 8 * (m & 3) + 4 * c : 4 * (m & 3)), vf[c][b]);
        };
        values();
        // A value that is not finite would meet the zeros of P above the diagonal and reach the tokens before it: it enters
        // as zero there, and its column is NaN from its own token on.
        bool bad = false;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int b = 0; b < JB; ++b) bad |= not_finite(vf[c][b][0]);
        const bool any = __any(bad);
        int from[CT];
        if (any) {
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                from[c] = C;
#pragma unroll
                for (int b = JB - 1; b >= 0; --b)
#pragma unroll
                    for (int j = 7; j >= 0; --j)
                        if (!__builtin_isfinite(float(vf[c][b][0][j]))) {
                            from[c] = 32 * b + 8 * g + j;
#pragma unroll
                            for (int p = 0; p < NP; ++p) vf[c][b][p][j] = __bf16(0.f);
                        }
                int x = __shfl_xor(from[c], 16, 64);
                from[c] = x < from[c] ? x : from[c];
                x = __shfl_xor(from[c], 32, 64);
                from[c] = x < from[c] ? x : from[c];
            }
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int b = 0; b < JB; ++b) {
                if (b > (t >> 1)) continue;
                bf16x8 pf[kParts];
#pragma unroll
                for (int j = 0; j < kParts; ++j) pf[j] = lp[tri_of(t, b)][j][lane];
#pragma unroll
                for (int c = 0; c < CT; ++c) mma(o[c][t], vf[c][b], pf);
            }
        if (any) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = __shfl(from[c], 4 * g + i, 64);
#pragma unroll
                    for (int t = 0; t < TT; ++t)
                        if (16 * t + m >= f) o[c][t][i] = __builtin_nanf("");
                }
            values();
        }
        const int l2 = fresh<kTight>(lane), g2 = l2 / 16, m2 = l2 % 16, col = vw + 4 * CT * g2;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (16 * t + m2 >= rem) continue;
            E* p = out + (int64_t(chunk) * C + 16 * t + m2) * a.Hv * a.V + col;
            float x[4 * CT];
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * c + i] = a.scale * o[c][t][i];
            if (a.vec_o) {
                if (col < a.V) store_floats<4 * CT>(p, x);
            } else {
#pragma unroll
                for (int i = 0; i < 4 * CT; ++i)
                    if (col + i < a.V) p[i] = E(x[i]);
            }
        }

        __builtin_amdgcn_sched_barrier(0);
        const float keep = dec.gamma[C - 1];
        const int l3 = fresh<kTight>(lane), g3 = l3 / 16, m3 = l3 % 16;
#pragma unroll
        for (int r = 0; r < KT; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c) S[r][c] *= keep;
#pragma unroll
        for (int b = 0; b < JB; ++b) {
            float eta[8];
            read8(dec.eta + 32 * b + 8 * g3, eta);
            bf16x8 yf[CT][kParts];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                float x[8];
                whole(vf[c][b], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= eta[j];
                split<kParts, 8>(x, yf[c]);
            }
#pragma unroll
            for (int r = 0; r < KT; ++r) {
                bf16x8 kf[NP];
                col_fragment<C, KP>(lk, b, g3, m3, 32 * (r >> 1) + 8 * (m3 & 3) + 4 * (r & 1), kf);
#pragma unroll
                for (int c = 0; c < CT; ++c) mma(S[r][c], kf, yf[c]);
                if (r % 2) __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if (a.fin && seg + 1 == segs) {
        float* dst = a.fin + (n * a.Hv + h) * int64_t(a.K) * a.V;
#pragma unroll
        for (int r = 0; r < KT; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const int k = acc_index(r, g) + i, v = column(c);
                    if (k < a.K && v < a.V) dst[int64_t(k) * a.V + v] = S[r][c][i];
                }
    }
}

}  // namespace

hipError_t launch_dca_fwd(int dt, int kb, int ct, const DcaArgs& a, hipStream_t st) {
    return by_dca_shape(dt, kb, ct, [&](auto d, auto k, auto c) {
        constexpr int DT = decltype(d)::value, KB = decltype(k)::value, CT = decltype(c)::value;
        const void* fn = a.save ? reinterpret_cast<const void*>(&dca_fwd_kernel<DT, KB, CT, true>) : reinterpret_cast<const void*>(&dca_fwd_kernel<DT, KB, CT, false>);
        DcaArgs args = a;
        void* params[] = {&args};
        const int64_t blocks = (a.seg_slots * a.Hk + 7) / 8 * 8 * (a.group * a.tiles);
        return hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(256), params, 0, st);
    });
}

}  // namespace qc
