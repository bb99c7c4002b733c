// dca_grad.hip -- gradients of linear attention with decays, chunk by chunk
// (include/decay_attention.h; formulas and layouts in dca_chunk.hpp).
#include "dca_chunk.hpp"

namespace qc {
namespace {

// One chunk and one key head to a block, its value heads one after the other, so
// that a shared head's gradients are summed in registers in one order, and 32
// columns of V at a time.  P and Phi: pairs of a 16-token tile of rows and a
// 32-token block of columns, each wave every fourth.  dQ^T and dK^T [KP, tokens]:
// a wave has a quarter of the rows (of 32 in all: half, and half of the tokens).
// dV^T [32, tokens]: 16 columns of V and half of the tokens.  S0 and dS1 come from
// memory as rows, the next 32 columns' while these are worked on; dV takes dS1's
// columns from LDS.
//
// 4 x 4096 tokens of 32 heads of 128, bfloat16: 629 us, 1.75 GB of inputs, states
// and gradients (340 us at the rate of a copy), 47% of the time in vector
// instructions and 15% in MFMA, one wave's hardly beside another's.  With two
// parts of what is computed it took 566 us, of which 35 were the states' way from
// memory (out of cache 531) and no phase between barriers more than 90; then were
// tried 128 tokens to a block of eight waves, which halves the states' way (1205
// us: one block to a CU, every phase's wait in full), 64 tokens and eight waves,
// everything a phase ahead (629), columns of dS1 read from memory as such (643).
// Two registers spill at K > 64 in bfloat16, once for a value head.  One key
// head's value heads follow each other in a block: 2048 tokens of one key head and
// 64 value heads of 128 x 64 are 32 blocks, and 1.19 ms with the states' pass,
// where 64 key heads take 0.21.
template <int DT, int KB>
__global__ void __launch_bounds__(256, DT == 0 && KB == 4 ? 1 : 2) dca_grad_kernel(DcaArgs a) {
    using E = typename Storage<DT>::type;
    constexpr int C = dca_chunk(DT), NP = parts_of(DT), TT = C / 16, JB = C / 32, KP = 32 * KB, VW = 32, KT = 2 * KB;
    constexpr int NW = 4, NT = 64 * NW;
    constexpr bool kTight = DT == 1 ? KB > 1 : DT == 2 && KB == 4;
    constexpr int KW = KT / 4 > 0 ? KT / 4 : 1;                // a wave's tiles of K rows
    constexpr int TW = KT / 4 > 0 ? TT : TT / 2, TV = TT / 2;  // and of tokens, of dQ and dK, and of dV
    // dS1 in LDS as halves of floats, split where it is read, where its three parts would leave room for one block to a CU
    // alone (89 KB of 80).  The third part later, in the place of V's rows and of the sums, after a barrier of its own: 674 us
    // where halves took 668; elsewhere parts cost less (float32 64 x 128, whole step: 667 us, halves 675).
    constexpr bool kHalves = DT == 1 && KB == 4;
    constexpr int kPairs = dca_tri(C), PW = (kPairs + NW - 1) / NW;
    struct Sums {
        float reads[NW][C], writes[NW][C], pairs[NW][C], dot[NW], last;
    };
    __shared__ __align__(16) char lq[NP * C * KP * 2], lk[NP * C * KP * 2], lv[NP * C * VW * 2], lo[NP * C * VW * 2], ld[(kHalves ? 2 : kParts) * KP * VW * 2];
    __shared__ __align__(16) bf16x8 lp[kPairs][kParts][64];
    __shared__ __align__(16) Decays<C> decays[2];              // of this value head and the next
    __shared__ Sums sum;
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), g = lane / 16, m = lane % 16;
    const int64_t slot = blockIdx.x / a.Hk;
    const int hk = int(blockIdx.x % a.Hk);
    const int64_t n = owner<C, false>(a, slot);
    const Span s = span_of<C>(a, n);
    const int64_t chunk = slot - s.slot;
    if (chunk < 0 || chunk * C >= s.len) {
        if (a.dg_part)
            for (int j = tid; j < a.group; j += NT) a.dg_part[slot * a.Hv + hk * a.group + j] = 0.f;
        return;
    }
    const int rem = int(s.len - chunk * C);
    const int64_t t0 = s.t0 + chunk * C, size = int64_t(KP) * a.VP;
    const bool want_dg = a.dg || a.dg_part;
    const int vtiles = a.VP / VW;

    const int k0 = wave % KT * 16 * KW, tt0 = wave / KT * TW;  // the wave's rows of K, and first tile of tokens
    const int v_col = wave % 2 * 16, tv0 = wave / 2 * TV;
    // The wave's pair number j: row tile i, block b.
    auto pair = [&](int j, int& i, int& b) {
        static_assert(kPairs <= 6, "six places");
        const int p = wave + NW * j;
        i = p < 2 ? p : p < 4 ? 2 : 3;
        b = p < 2 ? 0 : p & 1;
        return p < kPairs;
    };
    auto products = [&](const char* x, const char* y, int i, int b, int l, f32x4 (&pt)[2], auto width) {      // x_i.y_j
        constexpr int W = decltype(width)::value;
        const int g = l / 16, m = l % 16;
#pragma unroll
        for (int kb = 0; kb < W / 32; ++kb) {
            bf16x8 xf[NP];
            row_fragment<C, W>(x, 16 * i + m, kb, g, xf);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                bf16x8 yf[NP];
                row_fragment<C, W>(y, tile_index(2 * b + e, m), kb, g, yf);
                mma(pt[e], yf, xf);
            }
        }
    };
    // Rows of value head j and V's columns from v0 on, and the wave's rows of its S0 and dS1.
    Rows<DT, C, VW, NT> rv, ro;
    f32x4 sr[KW][2], dr[KW][2];
    auto load_rows = [&](int j, int v0) {
        const int h = hk * a.group + j, id = fresh<kTight>(tid);
        rv.load(same_in_all_lanes(static_cast<const E*>(a.v) + s.b * a.vs[0] + t0 * a.vs[1] + h * a.vs[2] + v0), a.vs[1], rem, a.V - v0, a.vec_v, id);
        ro.load(same_in_all_lanes(static_cast<const E*>(a.d_out) + ((s.b * a.T + t0) * a.Hv + h) * int64_t(a.V) + v0), int64_t(a.Hv) * a.V, rem, a.V - v0, a.vec_o, id);
    };
    auto load_states = [&](int j, int v0) {
        const int l = fresh<kTight>(lane);
        const int64_t at = (slot * a.Hv + hk * a.group + j) * size + int64_t(k0 + l % 16) * a.VP + v0 + 8 * (l / 16);
#pragma unroll
        for (int e = 0; e < KW; ++e)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                sr[e][x] = *reinterpret_cast<const f32x4*>(a.save + at + int64_t(16 * e) * a.VP + 4 * x);
                dr[e][x] = *reinterpret_cast<const f32x4*>(a.ds + at + int64_t(16 * e) * a.VP + 4 * x);
            }
    };
    auto make_decays = [&](int j) {
        const int h = hk * a.group + j;
        put_decays<C>(decays[j & 1], lane < C && lane < rem ? a.g[s.b * a.gs[0] + (t0 + lane) * a.gs[1] + h * a.gs[2]] : 0.f, lane);
    };
    // dg of value head j from its sums: what a token and later ones read of S0, what earlier ones leave in S1, and the
    // pairs across it; a lane has a token.
    auto finish = [&](int j) {
        float d = 0.f, z = 0.f, pairs = 0.f, x = 0.f;
#pragma unroll
        for (int c = 0; c < NW; ++c) x += sum.dot[c];
        if (lane < C)
#pragma unroll
            for (int c = 0; c < NW; ++c) {
                d += sum.reads[c][lane];
                z += sum.writes[c][lane];
                pairs += sum.pairs[c][lane];
            }
#pragma unroll
        for (int k = 1; k < C; k *= 2) {
            const float y = __shfl_down(d, k, 64), w = __shfl_up(z, k, 64);
            d += lane + k < C ? y : 0.f;
            z += lane >= k ? w : 0.f;
        }
        z = __shfl_up(z, 1, 64);
        const bool in = lane < C && lane < rem;
        const float dg = sum.last * x + d + (lane ? z : 0.f) + pairs;
        const int h = hk * a.group + j;
        if (a.dg && in) a.dg[(s.b * a.T + t0 + lane) * a.Hv + h] = dg;
        if (a.dg_part) {
            const float all = lanes_sum<64>(in ? dg : 0.f);
            if (lane == 0) a.dg_part[slot * a.Hv + h] = all;
        }
    };

    {
        Rows<DT, C, KP, NT> rq, rk;
        rq.load(same_in_all_lanes(static_cast<const E*>(a.q) + s.b * a.qs[0] + t0 * a.qs[1] + hk * a.qs[2]), a.qs[1], rem, a.K, a.vec_qk, tid);
        rk.load(same_in_all_lanes(static_cast<const E*>(a.k) + s.b * a.ks[0] + t0 * a.ks[1] + hk * a.ks[2]), a.ks[1], rem, a.K, a.vec_qk, tid);
        load_rows(0, 0);
        load_states(0, 0);
        if (wave == 0) make_decays(0);
        rq.store(lq, tid);
        rk.store(lk, tid);
    }
    f32x4 dq[KW][TW], dk[KW][TW];
#pragma unroll
    for (int e = 0; e < KW; ++e)
#pragma unroll
        for (int t = 0; t < TW; ++t) dq[e][t] = dk[e][t] = zero4();
    for (int j = 0; j < a.group; ++j) {
        const int h = hk * a.group + j;
        const Decays<C>& dec = decays[j & 1];
        f32x4 ov[PW][2], rd[KW][TW], wr[KW][TW];              // O V^T; O S0^T and V dS1^T
#pragma unroll
        for (int p = 0; p < PW; ++p) ov[p][0] = ov[p][1] = zero4();
#pragma unroll
        for (int e = 0; e < KW; ++e)
#pragma unroll
            for (int t = 0; t < TW; ++t) rd[e][t] = wr[e][t] = zero4();
        float dot = 0.f;
        for (int tile = 0; tile < vtiles; ++tile) {
            const int v0 = tile * VW;
            __syncthreads();                                  // what read the rows before is done
            {
                const int id = fresh<kTight>(tid);
                rv.store(lv, id);
                ro.store(lo, id);
            }
            __syncthreads();
            const bool more = tile + 1 < vtiles || j + 1 < a.group;
            const int next_j = tile + 1 < vtiles ? j : j + 1, next_v = tile + 1 < vtiles ? v0 + VW : 0;
            if (more) load_rows(next_j, next_v);
            if (tile == 0) {                                  // (these waves have a pair less)
                if (wave == NW - 1 && j && want_dg) finish(j - 1);
                if (wave == NW - 2 && j + 1 < a.group) make_decays(j + 1);
            }
#pragma unroll
            for (int p = 0; p < PW; ++p) {
                int i, b;
                if (!pair(p, i, b)) continue;
                const int l = fresh<kTight>(lane);
                if (tile == 0) {
                    f32x4 pt[2] = {zero4(), zero4()};
                    products(lq, lk, i, b, l, pt, std::integral_constant<int, KP>{});
                    float x[8];
                    decayed_pairs(dec, pt, i, b, l / 16, l % 16, a.scale, x);
                    bf16x8 f[kParts];
                    split<kParts, 8>(x, f);
#pragma unroll
                    for (int q = 0; q < kParts; ++q) lp[tri_of(i, b)][q][l] = f[q];
                }
                products(lo, lv, i, b, l, ov[p], std::integral_constant<int, VW>{});
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int e = 0; e < KW; ++e)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) dot += sr[e][x][i] * dr[e][x][i];
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
                bf16x8 sf[KW][kParts];
#pragma unroll
                for (int e = 0; e < KW; ++e) {
                    const f32x4 &lo4 = side ? dr[e][0] : sr[e][0], &hi4 = side ? dr[e][1] : sr[e][1];
                    const float y[8] = {lo4[0], lo4[1], lo4[2], lo4[3], hi4[0], hi4[1], hi4[2], hi4[3]};
                    split<kParts, 8>(y, sf[e]);
                    if (side && tt0 == 0) {
                        char* to = ld + lds_piece<VW>(k0 + 16 * e + m, g);
                        if constexpr (kHalves) {
                            bf16x8 f[2];
                            halves(y, f);
#pragma unroll
                            for (int p = 0; p < 2; ++p) *reinterpret_cast<bf16x8*>(to + p * (KP * VW * 2)) = f[p];
                        } else {
#pragma unroll
                            for (int p = 0; p < kParts; ++p) *reinterpret_cast<bf16x8*>(to + p * (KP * VW * 2)) = sf[e][p];
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < TW; ++t) {
                    bf16x8 rf[NP];
                    row_fragment<C, VW>(side ? lv : lo, 16 * (tt0 + t) + m, 0, g, rf);
#pragma unroll
                    for (int e = 0; e < KW; ++e) mma(side ? wr[e][t] : rd[e][t], sf[e], rf);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            // (Beside them what the halves take would spill accumulators, 360 MB written for 290 of results: 664 us, 629 so.)
            if (more && !kHalves) load_states(next_j, next_v);
            __syncthreads();                                  // P and dS1 are there
            if (a.dv) {
                const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
                f32x4 dv[TV];
#pragma unroll
                for (int t = 0; t < TV; ++t) dv[t] = zero4();
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    bf16x8 df[kParts];
                    if constexpr (kHalves) {
                        bf16x8 f[2];
                        col_fragment<KP, VW>(ld, kb, g, m, v_col + 4 * (m & 3), f);
                        float x[8];
                        of_halves(f, x);
                        split<kParts, 8>(x, df);
                    } else {
                        col_fragment<KP, VW>(ld, kb, g, m, v_col + 4 * (m & 3), df);
                    }
#pragma unroll
                    for (int t = 0; t < TV; ++t) {
                        bf16x8 kf[NP];
                        row_fragment<C, KP>(lk, 16 * (tv0 + t) + m, kb, g, kf);
                        mma(dv[t], df, kf);
                    }
                }
#pragma unroll
                for (int t = 0; t < TV; ++t) dv[t] *= dec.eta[16 * (tv0 + t) + m];
#pragma unroll
                for (int b = 0; b < JB; ++b) {
                    bf16x8 of[NP];
                    col_fragment<C, VW>(lo, b, g, m, v_col + 4 * (m & 3), of);
#pragma unroll
                    for (int t = 0; t < TV; ++t) {
                        if (b < ((tv0 + t) >> 1)) continue;
                        bf16x8 pf[kParts];
                        tri_cols(lp, b, g, m, tv0 + t, pf);
                        mma(dv[t], of, pf);
                    }
                }
                const int col = v0 + v_col + 4 * g;
#pragma unroll
                for (int t = 0; t < TV; ++t) {
                    const int token = 16 * (tv0 + t) + m;
                    if (token >= rem) continue;
                    E* p = static_cast<E*>(a.dv) + ((s.b * a.T + t0 + token) * a.Hv + h) * int64_t(a.V) + col;
                    const float x[4] = {dv[t][0], dv[t][1], dv[t][2], dv[t][3]};
                    if (a.vec_o) {
                        if (col < a.V) store_floats<4>(p, x);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (col + i < a.V) p[i] = E(x[i]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (more && kHalves) load_states(next_j, next_v);
        }
        // gamma and eta of them, and what dg needs: q and k with their shares of dQ and dK.
        float reads[TW], writes[TW];
        {
            const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
#pragma unroll
            for (int t = 0; t < TW; ++t) {
                const int token = 16 * (tt0 + t) + m;
                const float gamma = dec.gamma[token] * a.scale, eta = dec.eta[token];
                reads[t] = writes[t] = 0.f;
#pragma unroll
                for (int e = 0; e < KW; ++e) {
                    const int kacc = k0 + 16 * e + 4 * g, at = lds_piece<KP>(token, kacc >> 3) + (kacc & 7) * 2;
                    rd[e][t] *= gamma;
                    wr[e][t] *= eta;
                    dq[e][t] += rd[e][t];
                    dk[e][t] += wr[e][t];
                    if (want_dg) {
                        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int p = NP - 1; p >= 0; --p) {
                            const bf16x4 qp = *reinterpret_cast<const bf16x4*>(lq + at + p * (C * KP * 2));
                            const bf16x4 kp = *reinterpret_cast<const bf16x4*>(lk + at + p * (C * KP * 2));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                x[i] += float(qp[i]);
                                y[i] += float(kp[i]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            reads[t] += x[i] * rd[e][t][i];
                            writes[t] += y[i] * wr[e][t][i];
                        }
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();                                      // P is done with
        if (want_dg && lane < C) sum.pairs[wave][lane] = 0.f;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int p = 0; p < PW; ++p) {
            int i, b;
            if (!pair(p, i, b)) continue;
            const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
            float x[8];
            decayed_pairs(dec, ov[p], i, b, g, m, a.scale, x);
            bf16x8 f[kParts];
            split<kParts, 8>(x, f);
#pragma unroll
            for (int q = 0; q < kParts; ++q) lp[tri_of(i, b)][q][l] = f[q];
            if (want_dg) {
                // M_ij of this pair, i > j, and its sums over j < t <= i, for each t.
                f32x4 qk[2] = {zero4(), zero4()};
                products(lq, lk, i, b, l, qk, std::integral_constant<int, KP>{});
                const int row = 16 * i + m, col = 32 * b + 8 * g;
                float all = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) all += x[c] *= col + c < row ? qk[c >> 2][c & 3] : 0.f;
                // t in the block's 32 tokens, col + c here: what is left of it in its row, then over the rows from it on.
                float left = all, y = __shfl_up(left, 16, 64);
                left += g >= 1 ? y : 0.f;
                y = __shfl_up(left, 32, 64);
                left += g >= 2 ? y : 0.f;
                left = __shfl_up(left, 16, 64);
                left = g >= 1 ? left : 0.f;
                float* to = sum.pairs[wave] + col;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float z = lanes_sum<16>(row >= col + c ? left : 0.f);
                    if (m == c) to[c] += z;
                    left += x[c];
                }
                // t behind them, in the rows' tile or (two blocks of 32) between: whole rows.
                if (2 * b + 2 <= i) {
                    const float total = rows_of_lanes_sum(all);
                    float from = total + moved<0x101>(total);
                    from += moved<0x102>(from);
                    from += moved<0x104>(from);
                    from += moved<0x108>(from);
                    if (g == 0) sum.pairs[wave][16 * i + m] += from;
                    if (i == 2 * b + 3) {
                        const float z = lanes_sum<16>(total);
                        if (g == 0) sum.pairs[wave][16 * i - 16 + m] += z;
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (want_dg) {
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (TW < TT && (t < tt0 || t >= tt0 + TW) && g == 0) sum.reads[wave][16 * t + m] = sum.writes[wave][16 * t + m] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < TW; ++t) {
                const float x = rows_of_lanes_sum(reads[t]), y = rows_of_lanes_sum(writes[t]);
                if (g == 0) {
                    sum.reads[wave][16 * (tt0 + t) + m] = x;
                    sum.writes[wave][16 * (tt0 + t) + m] = y;
                }
            }
            const float x = lanes_sum<64>(tt0 == 0 ? dot : 0.f);      // (each row of S0 once)
            if (lane == 0) {
                sum.dot[wave] = x;
                if (wave == 0) sum.last = dec.gamma[C - 1];
            }
        }
        __syncthreads();                                      // Phi and the sums are there
        if (a.dq || a.dk) {
            const int l = fresh<kTight>(lane), g = l / 16, m = l % 16;
#pragma unroll
            for (int b = 0; b < JB; ++b) {
                bf16x8 kf[KW][NP], qf[KW][NP];
#pragma unroll
                for (int e = 0; e < KW; ++e) {
                    col_fragment<C, KP>(lk, b, g, m, k0 + 16 * e + 4 * (m & 3), kf[e]);
                    col_fragment<C, KP>(lq, b, g, m, k0 + 16 * e + 4 * (m & 3), qf[e]);
                }
#pragma unroll
                for (int t = 0; t < TW; ++t) {
                    const int tile = tt0 + t;
                    bf16x8 pf[kParts];
                    if (b <= (tile >> 1)) {
#pragma unroll
                        for (int i = 0; i < kParts; ++i) pf[i] = lp[tri_of(tile, b)][i][l];
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
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (want_dg && wave == NW - 1) finish(a.group - 1);
#pragma unroll
    for (int t = 0; t < TW; ++t) {
        const int token = 16 * (tt0 + t) + m;
        if (token >= rem) continue;
#pragma unroll
        for (int e = 0; e < KW; ++e) {
            const int kacc = k0 + 16 * e + 4 * g;
            const int64_t at = ((s.b * a.T + t0 + token) * a.Hk + hk) * a.K + kacc;
            const float x[4] = {dq[e][t][0], dq[e][t][1], dq[e][t][2], dq[e][t][3]}, y[4] = {dk[e][t][0], dk[e][t][1], dk[e][t][2], dk[e][t][3]};
            E* pq = static_cast<E*>(a.dq) + at;
            E* pk = static_cast<E*>(a.dk) + at;
            if (a.vec_qk) {
                if (kacc >= a.K) continue;
                if (a.dq) store_floats<4>(pq, x);
                if (a.dk) store_floats<4>(pk, y);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (kacc + i >= a.K) continue;
                    if (a.dq) pq[i] = E(x[i]);
                    if (a.dk) pk[i] = E(y[i]);
                }
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

hipError_t launch_dca_grad(int dt, int kb, const DcaArgs& a, hipStream_t st) {
    if (!a.slots) return hipSuccess;
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        const void* fn = reinterpret_cast<const void*>(&dca_grad_kernel<decltype(d)::value, decltype(k)::value>);
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
