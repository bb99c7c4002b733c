// dca_grad.hip -- gradients of linear attention with decays, chunk by chunk
// (include/decay_attention.h; formulas and layouts in dca_chunk.hpp).
#include "dca_chunk.hpp"

namespace qc {
namespace {

// Sum over the 16 lanes that share lane / 16, in each of them.
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int i = 1; i < 16; i *= 2) x += __shfl_xor(x, i, 64);
    return x;
}

// One chunk and key head to a block, its value heads one after the other, so
// that a shared head's gradients are summed in registers in one order.  Four
// waves.  P and Phi: a wave makes the 16 rows of its own tile.  dQ^T and dK^T
// [KP, tokens]: a wave has a quarter of the rows (of 32 in all: half, and half
// of the tokens); dV^T [64 CT, tokens]: a quarter.  S0 and dS1 come from memory
// as rows, and as columns for dV.
template <int DT, int KB, int CT>
__global__ void __launch_bounds__(256, DT == 0 ? 1 : 2) dca_grad_kernel(DcaArgs a) {
    using E = typename Storage<DT>::type;
    constexpr int C = dca_chunk(DT), NP = parts_of(DT), PP = dca_parts(DT), TT = C / 16, JB = C / 32, KP = 32 * KB, VW = 64 * CT;
    constexpr int KW = KB == 4 ? 2 : 1, TW = KB == 1 ? TT / 2 : TT;       // a wave's tiles of K rows and of tokens
    __shared__ __align__(16) char lq[NP * C * KP * 2], lk[NP * C * KP * 2], lv[NP * C * VW * 2], lo[NP * C * VW * 2];
    __shared__ __align__(16) bf16x8 lp[dca_tri(C)][PP][64];
    __shared__ __align__(16) Decays<C> dec;
    struct Sums {
        float reads[4][C], writes[4][C], pairs[4][C], dot[4];
    };
    static_assert(sizeof(Sums) <= sizeof(lo), "the sums take the cotangents' place");
    Sums& sum = *reinterpret_cast<Sums*>(lo);
    constexpr bool kTight = true;
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), g = lane / 16, m = lane % 16;
    const int64_t slot = blockIdx.x / a.Hk;
    const int hk = int(blockIdx.x % a.Hk);
    const int64_t n = owner<C, false>(a, slot);
    const Span s = span_of<C>(a, n);
    const int64_t chunk = slot - s.slot;
    if (chunk < 0 || chunk * C >= s.len) {
        if (a.dg_part)
            for (int j = tid; j < a.group; j += 256) a.dg_part[slot * a.Hv + hk * a.group + j] = 0.f;
        return;
    }
    const int rem = int(s.len - chunk * C);
    const int64_t t0 = s.t0 + chunk * C, size = int64_t(KP) * a.VP;
    const bool want_dg = a.dg || a.dg_part;

    // The wave's first K row and first tile of tokens.
    const int k0 = KB == 4 ? 32 * wave : KB == 2 ? 16 * wave : 16 * (wave & 1), tt0 = KB == 1 ? (wave >> 1) * TW : 0;
    const int kacc = k0 + 4 * KW * g;                     // the 4 KW rows of a lane's accumulators
    {
        Rows<DT, C, KP> rq, rk;
        rq.load(static_cast<const E*>(a.q) + s.b * a.qs[0] + t0 * a.qs[1] + hk * a.qs[2], a.qs[1], rem, a.K, a.vec_qk, tid);
        rk.load(static_cast<const E*>(a.k) + s.b * a.ks[0] + t0 * a.ks[1] + hk * a.ks[2], a.ks[1], rem, a.K, a.vec_qk, tid);
        rq.store(lq, tid);
        rk.store(lk, tid);
    }
    __syncthreads();
    f32x4 qk[JB][2];                                      // q_i.k_j of the wave's row tile, as its pairs lie in P
#pragma unroll
    for (int b = 0; b < JB; ++b) {
        qk[b][0] = qk[b][1] = zero4();
        if (wave >= TT || b > (wave >> 1)) continue;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            bf16x8 qf[NP];
            row_fragment<C, KP>(lq, 16 * wave + m, kb, g, qf);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                bf16x8 kf[NP];
                row_fragment<C, KP>(lk, tile_index(2 * b + e, m), kb, g, kf);
                mma(qk[b][e], kf, qf);
            }
        }
    }
    f32x4 dq[KW][TW], dk[KW][TW];
#pragma unroll
    for (int e = 0; e < KW; ++e)
#pragma unroll
        for (int t = 0; t < TW; ++t) dq[e][t] = dk[e][t] = zero4();

    for (int j = 0; j < a.group; ++j) {
        const int h = hk * a.group + j;
        const float* S0 = a.save + (slot * a.Hv + h) * size;
        const float* D1 = a.ds + (slot * a.Hv + h) * size;
        f32x4 ov[JB][2];
#pragma unroll
        for (int b = 0; b < JB; ++b) ov[b][0] = ov[b][1] = zero4();
        float reads[TW], writes[TW], dot = 0.f;
#pragma unroll
        for (int t = 0; t < TW; ++t) reads[t] = writes[t] = 0.f;
        for (int tile = 0; tile < a.tiles; ++tile) {
            const int v0 = tile * VW;
            {
                Rows<DT, C, VW> rv, ro;
                const int id = fresh<kTight>(tid);
                rv.load(static_cast<const E*>(a.v) + s.b * a.vs[0] + t0 * a.vs[1] + h * a.vs[2] + v0, a.vs[1], rem, a.V - v0, a.vec_v, id);
                ro.load(static_cast<const E*>(a.d_out) + ((s.b * a.T + t0) * a.Hv + h) * int64_t(a.V) + v0, int64_t(a.Hv) * a.V, rem, a.V - v0, a.vec_o, id);
                __syncthreads();                          // what read the rows before is done
                rv.store(lv, id);
                ro.store(lo, id);
            }
            if (tile == 0 && wave == 0)
                put_decays<C>(dec, lane < C && lane < rem ? a.g[s.b * a.gs[0] + (t0 + lane) * a.gs[1] + h * a.gs[2]] : 0.f, lane);
            __syncthreads();
            if (tile == 0 && wave < TT) {
                const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
#pragma unroll
                for (int b = 0; b < JB; ++b) {
                    if (b > (wave >> 1)) continue;
                    float x[8];
                    decayed_pairs(dec, qk[b], wave, b, g, m, a.scale, x);
                    bf16x8 p[PP];
                    split<PP, 8>(x, p);
#pragma unroll
                    for (int i = 0; i < PP; ++i) lp[tri_of(wave, b)][i][lane] = p[i];
                }
            }
            if (wave < TT) {
                const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
#pragma unroll
                for (int b = 0; b < JB; ++b) {
                    if (b > (wave >> 1)) continue;
#pragma unroll
                    for (int x = 0; x < 2 * CT; ++x) {
                        bf16x8 of[NP];
                        row_fragment<C, VW>(lo, 16 * wave + m, x, g, of);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            bf16x8 vf[NP];
                            row_fragment<C, VW>(lv, tile_index(2 * b + e, m), x, g, vf);
                            mma(ov[b][e], vf, of);
                        }
                    }
                }
            }
            // O S0^T, then V dS1^T, over this block's columns of V: gamma and eta of them, and what dg needs.
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
                const char* rows = side ? lv : lo;
                f32x4 acc[KW][TW];
#pragma unroll
                for (int e = 0; e < KW; ++e)
#pragma unroll
                    for (int t = 0; t < TW; ++t) acc[e][t] = zero4();
                const int64_t place = int64_t(KW == 2 ? k0 + 8 * (m >> 2) + (m & 3) : k0 + m) * a.VP + v0 + 8 * g;
                const float *p0 = (side ? D1 : S0) + place, *p1 = S0 + place;
#pragma unroll
                for (int x = 0; x < 2 * CT; ++x) {
                    bf16x8 sf[KW][kParts];
#pragma unroll
                    for (int e = 0; e < KW; ++e) {
                        float y[8];
                        read8(p0 + int64_t(4 * e) * a.VP + 32 * x, y);
                        if (side && want_dg) {
                            float z[8];
                            read8(p1 + int64_t(4 * e) * a.VP + 32 * x, z);
#pragma unroll
                            for (int i = 0; i < 8; ++i) dot += y[i] * z[i];
                        }
                        split<kParts, 8>(y, sf[e]);
                    }
#pragma unroll
                    for (int t = 0; t < TW; ++t) {
                        bf16x8 rf[NP];
                        row_fragment<C, VW>(rows, 16 * (tt0 + t) + m, x, g, rf);
#pragma unroll
                        for (int e = 0; e < KW; ++e) mma(acc[e][t], sf[e], rf);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                const int kacc = k0 + 4 * KW * g;
#pragma unroll
                for (int t = 0; t < TW; ++t) {
                    const int token = 16 * (tt0 + t) + m;
                    const float w = side ? dec.eta[token] : dec.gamma[token] * a.scale;
                    const char* at = (side ? lk : lq) + lds_piece<KP>(token, kacc >> 3) + (kacc & 7) * 2;
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < KW; ++e) {
                        acc[e][t] *= w;
                        if (side) dk[e][t] += acc[e][t];
                        else dq[e][t] += acc[e][t];
                        if (want_dg) {
                            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int p = NP - 1; p >= 0; --p) {
                                const bf16x4 part = *reinterpret_cast<const bf16x4*>(at + p * (C * KP * 2) + 8 * e);
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[i] += float(part[i]);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum += x[i] * acc[e][t][i];
                        }
                    }
                    if (side) writes[t] += sum;
                    else reads[t] += sum;
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (a.dv) {
                const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
                f32x4 dv[CT][TT];
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int t = 0; t < TT; ++t) dv[c][t] = zero4();
                const int vw = wave * 16 * CT;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    bf16x8 df[CT][PP];
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const float* p = D1 + int64_t(32 * kb + 8 * g) * a.VP + v0 + vw + (CT == 2 ? 8 * (m >> 2) + 4 * c + (m & 3) : m);
                        float z[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[i] = p[int64_t(i) * a.VP];
                        split<PP, 8>(z, df[c]);
                    }
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        bf16x8 kf[NP];
                        row_fragment<C, KP>(lk, 16 * t + m, kb, g, kf);
#pragma unroll
                        for (int c = 0; c < CT; ++c) mma(dv[c][t], df[c], kf);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const float eta = dec.eta[16 * t + m];
#pragma unroll
                    for (int c = 0; c < CT; ++c) dv[c][t] *= eta;
                }
                if (tile == 0) __syncthreads();           // P is there
#pragma unroll
                for (int b = 0; b < JB; ++b) {
                    bf16x8 of[CT][NP];
#pragma unroll
                    for (int c = 0; c < CT; ++c) col_fragment<C, VW>(lo, b, g, m, vw + (CT == 2 ? 8 * (m & 3) + 4 * c : 4 * (m & 3)), of[c]);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        if (b < (t >> 1)) continue;
                        bf16x8 pf[PP];
                        tri_cols(lp, b, g, m, t, pf);
#pragma unroll
                        for (int c = 0; c < CT; ++c) mma(dv[c][t], of[c], pf);
                    }
                }
                const int col = v0 + vw + 4 * CT * g;
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (16 * t + m >= rem) continue;
                    E* p = static_cast<E*>(a.dv) + ((s.b * a.T + t0 + 16 * t + m) * a.Hv + h) * int64_t(a.V) + col;
                    float x[4 * CT];
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[4 * c + i] = dv[c][t][i];
                    if (a.vec_o) {
                        if (col < a.V) store_floats<4 * CT>(p, x);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4 * CT; ++i)
                            if (col + i < a.V) p[i] = E(x[i]);
                    }
                }
            }
        }
        __syncthreads();                                  // P and the cotangents are done with
        if (wave < TT) {
            const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
            f32x4 before[TT];                             // [t][i]: sum over j < t of M_ij
#pragma unroll
            for (int t = 0; t < TT; ++t) before[t] = zero4();
#pragma unroll
            for (int b = 0; b < JB; ++b) {
                if (b > (wave >> 1)) continue;
                float x[8];
                decayed_pairs(dec, ov[b], wave, b, g, m, a.scale, x);
                bf16x8 p[PP];
                split<PP, 8>(x, p);
#pragma unroll
                for (int i = 0; i < PP; ++i) lp[tri_of(wave, b)][i][lane] = p[i];
                if (want_dg) {
                    bf16x8 mf[kParts];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] *= 32 * b + 8 * g + i < 16 * wave + m ? qk[b][i >> 2][i & 3] : 0.f;
                    split<kParts, 8>(x, mf);
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        if (t > wave) continue;
                        bf16x8 one[1];
#pragma unroll
                        for (int i = 0; i < 8; ++i) one[0][i] = __bf16(32 * b + 8 * g + i < 16 * t + m ? 1.f : 0.f);
                        mma(before[t], one, mf);
                    }
                }
            }
            if (want_dg) {
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int token = 16 * t + 4 * g + i;
                        const float x = sum16(16 * wave + m >= token ? before[t][i] : 0.f);
                        if (m == 0) sum.pairs[wave][token] = x;
                    }
            }
        }
        if (want_dg) {
            if constexpr (TW < TT) {
                for (int i = lane; i < C; i += 64) sum.reads[wave][i] = sum.writes[wave][i] = 0.f;
                __builtin_amdgcn_wave_barrier();
            }
#pragma unroll
            for (int t = 0; t < TW; ++t) {
                float x = reads[t], y = writes[t];
                x += __shfl_xor(x, 16, 64);
                y += __shfl_xor(y, 16, 64);
                x += __shfl_xor(x, 32, 64);
                y += __shfl_xor(y, 32, 64);
                if (g == 0) {
                    sum.reads[wave][16 * (tt0 + t) + m] = x;
                    sum.writes[wave][16 * (tt0 + t) + m] = y;
                }
            }
            float x = tt0 == 0 ? dot : 0.f;               // (each row of S0 once)
#pragma unroll
            for (int i = 1; i < 64; i *= 2) x += __shfl_xor(x, i, 64);
            if (lane == 0) sum.dot[wave] = x;
        }
        __syncthreads();
        if (a.dq || a.dk) {
            const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
#pragma unroll
            for (int b = 0; b < JB; ++b) {
                bf16x8 kf[KW][NP], qf[KW][NP];
#pragma unroll
                for (int e = 0; e < KW; ++e) {
                    const int col = KW == 2 ? k0 + 8 * (m & 3) + 4 * e : k0 + 4 * (m & 3);
                    col_fragment<C, KP>(lk, b, g, m, col, kf[e]);
                    col_fragment<C, KP>(lq, b, g, m, col, qf[e]);
                }
#pragma unroll
                for (int t = 0; t < TW; ++t) {
                    const int tile = tt0 + t;
                    bf16x8 pf[PP];
                    if (b <= (tile >> 1)) {
#pragma unroll
                        for (int i = 0; i < PP; ++i) pf[i] = lp[tri_of(tile, b)][i][lane];
#pragma unroll
                        for (int e = 0; e < KW; ++e) mma(dq[e][t], kf[e], pf);
                    }
                    if (b >= (tile >> 1)) {
                        tri_cols(lp, b, g, m, tile, pf);
#pragma unroll
                        for (int e = 0; e < KW; ++e) mma(dk[e][t], qf[e], pf);
                    }
                }
            }
        }
        if (want_dg && wave == 0) {
            // A lane's token t: what it and later tokens read of S0, what earlier ones leave in S1, and the pairs across it.
            float d = 0.f, z = 0.f, pairs = 0.f, x = 0.f;
            if (lane < C) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    d += sum.reads[c][lane];
                    z += sum.writes[c][lane];
                    if (c < TT) pairs += sum.pairs[c][lane];
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) x += sum.dot[c];
#pragma unroll
            for (int i = 1; i < C; i *= 2) {
                const float y = __shfl_down(d, i, 64), w = __shfl_up(z, i, 64);
                d += lane + i < C ? y : 0.f;
                z += lane >= i ? w : 0.f;
            }
            z = __shfl_up(z, 1, 64);
            float dg = dec.gamma[C - 1] * x + d + (lane ? z : 0.f) + pairs;
            if (a.dg && lane < C && lane < rem) a.dg[(s.b * a.T + t0 + lane) * a.Hv + h] = dg;
            if (a.dg_part) {
                dg = lane < C && lane < rem ? dg : 0.f;
#pragma unroll
                for (int i = 1; i < 64; i *= 2) dg += __shfl_xor(dg, i, 64);
                if (lane == 0) a.dg_part[slot * a.Hv + h] = dg;
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TW; ++t) {
        const int token = 16 * (tt0 + t) + m;
        if (token >= rem) continue;
        const int64_t at = ((s.b * a.T + t0 + token) * a.Hk + hk) * a.K + kacc;
        float x[4 * KW], y[4 * KW];
#pragma unroll
        for (int e = 0; e < KW; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[4 * e + i] = dq[e][t][i];
                y[4 * e + i] = dk[e][t][i];
            }
        E* pq = static_cast<E*>(a.dq) + at;
        E* pk = static_cast<E*>(a.dk) + at;
        if (a.vec_qk) {
            if (kacc >= a.K) continue;
            if (a.dq) store_floats<4 * KW>(pq, x);
            if (a.dk) store_floats<4 * KW>(pk, y);
        } else {
#pragma unroll
            for (int i = 0; i < 4 * KW; ++i) {
                if (kacc + i >= a.K) continue;
                if (a.dq) pq[i] = E(x[i]);
                if (a.dk) pk[i] = E(y[i]);
            }
        }
    }
}

// The gradient of a head's one decay: the chunks' sums, joined in order.
__global__ void __launch_bounds__(256) dca_heads_kernel(const float* part, int64_t slots, int Hv, float* out) {
    __shared__ double run[256];
    const int h = blockIdx.x;
    double x = 0.;
    for (int64_t i = threadIdx.x; i < slots; i += 256) x += double(part[i * Hv + h]);
    run[threadIdx.x] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        double y = 0.;
        for (int i = 0; i < 256; ++i) y += run[i];
        out[h] = float(y);
    }
}

}  // namespace

hipError_t launch_dca_grad(int dt, int kb, int ct, const DcaArgs& a, hipStream_t st) {
    if (!a.slots) return hipSuccess;
    return by_dca_shape(dt, kb, ct, [&](auto d, auto k, auto c) {
        const void* fn = reinterpret_cast<const void*>(&dca_grad_kernel<decltype(d)::value, decltype(k)::value, decltype(c)::value>);
        DcaArgs args = a;
        void* params[] = {&args};
        return hipLaunchKernel(fn, dim3(unsigned(a.slots * a.Hk)), dim3(256), params, 0, st);
    });
}

hipError_t launch_dca_heads(const DcaArgs& a, float* out, hipStream_t st) {
    const float* part = a.dg_part;
    int64_t slots = a.slots;
    int Hv = a.Hv;
    void* params[] = {&part, &slots, &Hv, &out};
    return hipLaunchKernel(reinterpret_cast<const void*>(&dca_heads_kernel), dim3(unsigned(Hv)), dim3(256), params, 0, st);
}

}  // namespace qc
