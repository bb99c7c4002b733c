// gdr_grad.hip -- the chunked gated delta rule's gradients of q, k and the
// gates (gdr_chunk.hpp), every chunk at once.
//
// One block of 8 waves per chunk and key head, walking the value heads that
// share it, so that the sums of a shared head's gradients are made in
// registers and in one order.  V is taken in pieces of up to 128 columns:
// X, U and dO go to LDS as operand parts; S0 and dS1 are read once, straight
// into operands.  Wave (cg, rh) owns columns of K (group cg of the tiles) and
// half rh of the tokens; the 64 x 64 products X U^T, dO U^T are dealt by row
// tiles.
//
// One block to a CU: its operand parts fill LDS, and a wave takes up to all 256
// registers (K = 128 spills: bfloat16 2, float16 22, float32 76).  It reads what
// the two passes left, S0, dS1, U and X in float32: at 4 x 4096 tokens of 32
// heads of 128 that is 1.6 GB, 290 us at the rate of a copy, and the kernel takes
// 825 us (8 x 2048 tokens of 16 heads of 64 by 128, float32: 459): bound by the
// phases of a block, loads and splits, products, row sums, which one block to a
// CU does not overlap (matrix units 22% in use, LDS 18%, waves at a wait or a
// barrier half of the time).  With operands staged as plain rows and gathered,
// and row sums through LDS, it took twice that.
#include "gdr_chunk.hpp"

namespace qc {
namespace {

constexpr int kPiece = 128;     // columns of V at a time
constexpr int kPairRow = 68;    // LDS row of a 64 x 64 float matrix

// Sum over the 16 lanes of a row, in every one of them.
template <int CTRL>
__device__ __forceinline__ float rotated(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum16(float x) {
    x += rotated<0x128>(x);      // by 8, 4, 2, 1 lanes within the row
    x += rotated<0x124>(x);
    x += rotated<0x122>(x);
    x += rotated<0x121>(x);
    return x;
}

// x, as a value of its own: places in LDS that depend on the lane alone are
// formed where they are used, for each head.  Kept through the loops over V
// they take registers that these loops spill for: at K = 128 in bfloat16 33
// registers without this, 2 with it, and a training step of 4 x 4096 tokens of
// 32 heads 2364 us and 2167 (float32 K = 128: 108 registers and 76).
__device__ __forceinline__ int formed_here(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

template <int DT, int KB>
__global__ void __launch_bounds__(512) gdr_grad_kernel(GdrArgs a) {
    using E = typename Storage<DT>::type;
    constexpr int NPI = parts_of(DT);
    constexpr int TW = KB == 4 ? 2 : 1;                 // tiles of K of a wave
    constexpr int VB = kPiece / 32;
    // First X, U, dO as rows of V, then Phi, Phi^T, Psi, Psi^T.
    struct Rows {
        bf16x8 x[4][VB][kParts][64], u[4][VB][kParts][64], o[4][VB][NPI][64];
    };
    struct Tri {
        bf16x8 phi[4][2][kParts][64], phit[4][2][kParts][64], psi[4][2][kParts][64], psit[4][2][kParts][64];
        float pairs[64 * kPairRow];      // M
    };
    union Shared {
        __device__ Shared() {}
        Rows rows;
        Tri tri;
    };
    __shared__ __align__(16) Shared sh;
    __shared__ double cum[64];
    __shared__ __align__(16) float gamma[64], eta[64], beta[64], xv[VB][64], rowsum[2][64], red[3][4][64], across[8][64], dots[8];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int cg = wave >> 1, rh = wave & 1;
    const int rt = wave >> 1, ch = wave & 1;             // 64 x 64 products: row tile, half of the columns
    const bool tri_on = ch == 0 || rt >= 2;
    const bool k_on = cg * TW < 2 * KB;
    const int hk = int(blockIdx.x % a.Hk);
    const int64_t slot = blockIdx.x / a.Hk;
    Sequence s;
    int chunk;
    if (slot_sequence(a, slot, s, chunk) < 0) return;
    const int rem = s.len - chunk * kChunk;
    const int64_t token0 = s.b * a.T + s.t0 + int64_t(chunk) * kChunk;      // dense index of the chunk's first token
    const bf16x8* kr = reinterpret_cast<const bf16x8*>(a.krec + (hk * a.slots + slot) * krec_bytes(KB, NPI));
    const bf16x8* qt_set = kr + set_frags(KB, NPI) * 64;
    const bf16x8* kt_set = qt_set + set_frags(KB, NPI) * 64;

    // K K^T, row tile rt against the column tiles 2 ch + 0, 1.
    f32x4 kk[2] = {zero4(), zero4()};
    if (tri_on) {
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            bf16x8 ka[NPI], kb[NPI];
#pragma unroll
            for (int p = 0; p < NPI; ++p) ka[p] = kr[((rt * KB + b) * NPI + p) * 64 + lane];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int p = 0; p < NPI; ++p) kb[p] = kr[(((2 * ch + c) * KB + b) * NPI + p) * 64 + lane];
                mma(kk[c], ka, kb);
            }
        }
    }
    f32x4 dq_all[TW][2], dk_all[TW][2];
#pragma unroll
    for (int x = 0; x < TW; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r) dq_all[x][r] = dk_all[x][r] = zero4();

#pragma unroll 1
    for (int hv = hk * a.group; hv < (hk + 1) * a.group; ++hv) {
        const char* hr = a.hrec + (hv * a.slots + slot) * kHrecBytes;
        const Gates* ga = reinterpret_cast<const Gates*>(hr + kGateOffset);
        const bf16x8* pf = reinterpret_cast<const bf16x8*>(hr) + kTriFrags * 64;      // P transposed
        // P's lines on their way to L2, beside the gates: they are needed where nothing hides how far away they are.
        int line = 0;
        if (tid < int(kTriFrags * kFrag * 2 / 128)) line = reinterpret_cast<const int*>(pf)[tid * 32];
        __syncthreads();                                  // the head before is done with what is in LDS
        if (tid < 64) {
            gamma[tid] = ga->gamma[tid];
            eta[tid] = ga->eta[tid];
            beta[tid] = ga->beta[tid];
            cum[tid] = ga->cum[tid];
        }
        asm volatile("" ::"v"(line));
        f32x4 aq[TW][2], ar[TW][2], aw[TW][2], op[2] = {zero4(), zero4()}, xp[2] = {zero4(), zero4()};
#pragma unroll
        for (int x = 0; x < TW; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) aq[x][r] = ar[x][r] = aw[x][r] = zero4();
        float sds = 0.f;
        const int64_t piece = (hv * a.slots + slot) * int64_t(a.VP / 16) * 256;
        const float *s0 = a.save_s + piece * (2 * KB), *s1 = a.ds + piece * (2 * KB);
        const float *us = a.save_u + piece * 4, *xs = a.x + piece * 4;
#pragma unroll 1
        for (int v0 = 0; v0 < a.V; v0 += kPiece) {
            if (v0) __syncthreads();                      // the piece before is done
            // A wave takes two (row tile, block of V) pairs: what a lane loads is what it holds of the fragment.  X . v on
            // the way.
            const int here = formed_here(lane);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int lane = here, m = lane & 15, g = lane >> 4;
                const int tile = wave >> 1, b = 2 * (wave & 1) + i, t = tile_index(tile, m), v = v0 + 32 * b + 8 * g;
                const bool in = t < rem, have = v < a.VP;
                const E* op_ = static_cast<const E*>(a.d_out) + ((token0 + (in ? t : 0)) * a.Hv + hv) * a.V;
                const E* vp = static_cast<const E*>(a.v) + s.b * a.vs[0] + (s.t0 + int64_t(chunk) * kChunk + (in ? t : 0)) * a.vs[1] + int64_t(hv) * a.vs[2];
                const int at = have ? (v >> 4) * 1024 + tile * 256 + m * 16 + (v & 15) : 0;
                float x8[8], u8[8];
                load_floats<8>(xs + at, x8);
                load_floats<8>(us + at, u8);
                const int left = in ? a.V - v : 0;
                bf16x8 p3[kParts], o8[NPI], v8[NPI];
                load_parts<DT>(op_ + v, left, a.vec_o, o8);
                load_parts<DT>(vp + v, left, a.vec_v, v8);
                float dot = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x8[e] = have ? x8[e] : 0.f;
                    u8[e] = have ? u8[e] : 0.f;
                    float ve = 0.f;
#pragma unroll
                    for (int p = NPI - 1; p >= 0; --p) ve += float(v8[p][e]);
                    dot += x8[e] * ve;
                }
                split<kParts, 8>(x8, p3);
#pragma unroll
                for (int p = 0; p < kParts; ++p) sh.rows.x[tile][b][p][lane] = p3[p];
                split<kParts, 8>(u8, p3);
#pragma unroll
                for (int p = 0; p < kParts; ++p) sh.rows.u[tile][b][p][lane] = p3[p];
#pragma unroll
                for (int p = 0; p < NPI; ++p) sh.rows.o[tile][b][p][lane] = o8[p];
                dot += __shfl_xor(dot, 16, 64);
                dot += __shfl_xor(dot, 32, 64);
                if (g == 0) xv[b][t] = (v0 ? xv[b][t] : 0.f) + dot;
            }
            // The states' operands are loaded one block of V ahead.
            float s8[TW][8], d8[TW][8];
            auto load_states = [&](int b) {
                const int v = v0 + 32 * b + 8 * g;
                const bool have = v < a.VP && k_on;
#pragma unroll
                for (int y = 0; y < TW; ++y) {
                    const int at = have ? (v >> 4) * (2 * KB * 256) + (cg * TW + y) * 256 + m * 16 + (v & 15) : 0;
                    load_floats<8>(s0 + at, s8[y]);
                    load_floats<8>(s1 + at, d8[y]);
                }
            };
            load_states(0);
            __syncthreads();
            const int blocks = a.V - v0 >= kPiece ? VB : (a.V - v0 + 31) / 32;
            if (k_on) {
#pragma unroll 1
                for (int b = 0; b < blocks; ++b) {
                    const bool have = v0 + 32 * b + 8 * g < a.VP;
                    // One state at a time: both states' parts together do not fit the registers.
                    auto take = [&](float (&x)[TW][8], bf16x8 (&p)[TW][kParts]) {
#pragma unroll
                        for (int y = 0; y < TW; ++y) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[y][e] = have ? x[y][e] : 0.f;
                            split<kParts, 8>(x[y], p[y]);
                        }
                    };
                    {
                        bf16x8 sp[TW][kParts];
                        take(s8, sp);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            bf16x8 f[kParts], o[NPI];
#pragma unroll
                            for (int p = 0; p < kParts; ++p) f[p] = sh.rows.x[2 * rh + r][b][p][lane];
#pragma unroll
                            for (int p = 0; p < NPI; ++p) o[p] = sh.rows.o[2 * rh + r][b][p][lane];
#pragma unroll
                            for (int y = 0; y < TW; ++y) mma(ar[y][r], f, sp[y]);
#pragma unroll
                            for (int y = 0; y < TW; ++y) mma(aq[y][r], o, sp[y]);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    {
                        bf16x8 dp[TW][kParts];
                        take(d8, dp);
#pragma unroll
                        for (int y = 0; y < TW; ++y)
#pragma unroll
                            for (int e = 0; e < 8; ++e) sds += s8[y][e] * d8[y][e];
                        load_states(b + 1 < blocks ? b + 1 : b);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            bf16x8 f[kParts];
#pragma unroll
                            for (int p = 0; p < kParts; ++p) f[p] = sh.rows.u[2 * rh + r][b][p][lane];
#pragma unroll
                            for (int y = 0; y < TW; ++y) mma(aw[y][r], f, dp[y]);
                        }
                    }
                }
            }
            if (tri_on) {
#pragma unroll 1
                for (int b = 0; b < blocks; ++b) {
                    bf16x8 xa[kParts], oa[NPI];
#pragma unroll
                    for (int p = 0; p < kParts; ++p) xa[p] = sh.rows.x[rt][b][p][lane];
#pragma unroll
                    for (int p = 0; p < NPI; ++p) oa[p] = sh.rows.o[rt][b][p][lane];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        bf16x8 ub[kParts];
#pragma unroll
                        for (int p = 0; p < kParts; ++p) ub[p] = sh.rows.u[2 * ch + c][b][p][lane];
                        mma(op[c], oa, ub);
                        mma(xp[c], xa, ub);
                    }
                }
            }
        }
        // The wave's columns of K and Q, transposed: [tile][block of tokens].
        bf16x8 kt[TW][2][NPI], qt[TW][2][NPI];
#pragma unroll
        for (int x = 0; x < TW; ++x)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int p = 0; p < NPI; ++p) {
                    const int f = (((k_on ? cg * TW + x : 0) * 2 + b) * NPI + p) * 64 + lane;
                    kt[x][b][p] = kt_set[f];
                    qt[x][b][p] = qt_set[f];
                }
        // P of the wave's products, which the factors hold transposed: a lane's accumulators are half of its fragment.
        bf16x4 pt[2][kParts];
        if (tri_on) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int p = 0; p < kParts; ++p)
                    pt[c][p] = reinterpret_cast<const bf16x4*>(pf + (tri_index<true>(2 * ch + c, rt >> 1) * kParts + p) * 64 + lane)[rt & 1];
        }
        __syncthreads();                                  // X, U, dO are done; Phi and Psi take their place
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sds += __shfl_xor(sds, d, 64);
        if (lane == 0) dots[wave] = rh == 0 ? sds : 0.f;
        {
            const int here = formed_here(lane), m = here & 15, g = here >> 4, i0 = acc_index(rt, g);
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            if (tri_on) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int ct = 2 * ch + c, j = tile_index(ct, m);
                    f32x4 phi, psi;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = i0 + r;
                        const float d = i >= j ? expf(float(cum[i] - cum[j])) : 0.f;
                        phi[r] = i >= j ? a.scale * d * op[c][r] : 0.f;
                        psi[r] = i > j ? -beta[i] * d * xp[c][r] : 0.f;
                        const float xl = i > j ? xp[c][r] * (d * kk[c][r]) : 0.f;
                        part[r] += xl;
                        const float p = float(pt[c][2][r]) + float(pt[c][1][r]) + float(pt[c][0][r]);
                        sh.tri.pairs[i * kPairRow + j] = i > j ? a.scale * op[c][r] * p - beta[i] * xl : 0.f;
                    }
                    bf16x4 pp[kParts], ps[kParts];
                    split4(phi, pp);
                    split4(psi, ps);
                    put_parts(&sh.tri.phit[ct][rt >> 1][0][0], 64, 16 * g + m, rt & 1, pp);
                    put_parts(&sh.tri.psit[ct][rt >> 1][0][0], 64, 16 * g + m, rt & 1, ps);
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            // Row 4 g + r; column j: lane group m / 4, element 4 (ct % 2) + m % 4.
                            const int at = 16 * (m >> 2) + 4 * g + r, e = 4 * (ct & 1) + (m & 3);
                            reinterpret_cast<__bf16*>(&sh.tri.phi[rt][ct >> 1][p][at])[e] = pp[p][r];
                            reinterpret_cast<__bf16*>(&sh.tri.psi[rt][ct >> 1][p][at])[e] = ps[p][r];
                        }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float t = sum16(part[r]);
                if (m == 0) rowsum[ch][i0 + r] = t;
            }
        }
        // The products with the states: their shares of the gates' gradients, then their scales.
        float kd[TW][2][4], qd[TW][2][4];                 // the wave's columns of K and Q at its own tokens
#pragma unroll
        for (int x = 0; x < TW; ++x)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float k = 0.f, q = 0.f;
#pragma unroll
                for (int p = NPI - 1; p >= 0; --p) {
                    k += float(rh ? kt[x][1][p][e] : kt[x][0][p][e]);
                    q += float(rh ? qt[x][1][p][e] : qt[x][0][p][e]);
                }
                kd[x][e >> 2][e & 3] = k;
                qd[x][e >> 2][e & 3] = q;
            }
        // Sums over the wave's columns of K, per token.
        const int here = formed_here(lane);
        auto reduce = [&](int which, int r, f32x4 v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = sum16(v[i]);
            if ((here & 15) == 0) *reinterpret_cast<f32x4*>(&red[which][cg][acc_index(2 * rh + r, here >> 4)]) = v;
        };
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t0 = acc_index(2 * rh + r, here >> 4);
            const f32x4 ga4 = *reinterpret_cast<const f32x4*>(&gamma[t0]), be4 = *reinterpret_cast<const f32x4*>(&beta[t0]),
                        et4 = *reinterpret_cast<const f32x4*>(&eta[t0]);
            f32x4 d0 = zero4(), b0 = zero4(), z = zero4();
#pragma unroll
            for (int x = 0; x < TW; ++x) {
                const f32x4 k = {kd[x][r][0], kd[x][r][1], kd[x][r][2], kd[x][r][3]}, q = {qd[x][r][0], qd[x][r][1], qd[x][r][2], qd[x][r][3]};
                d0 += q * aq[x][r];
                b0 += k * ar[x][r];
                z += k * aw[x][r];
                aq[x][r] *= a.scale * ga4;
                ar[x][r] *= -ga4 * be4;
                aw[x][r] *= et4;
            }
            reduce(0, r, a.scale * d0 - be4 * b0);
            reduce(1, r, b0);
            reduce(2, r, et4 * z);
        }
        __syncthreads();                                  // Phi, Psi and M are in LDS
        // The sums of M over i >= t > j: a thread has eight columns of a row, whose sums over j < t a row's eight threads join;
        // then a wave's eight rows meet, each thread left with one t.  Adding alone, so that no larger term is ever taken away
        // again.
        {
            const int own = formed_here(lane), i = 8 * wave + (own >> 3), t0 = 8 * (own & 7);
            float x[8], sum = 0.f;
            load_floats<8>(&sh.tri.pairs[i * kPairRow + t0], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = t0 + e < i ? x[e] : 0.f;      // what lies across the diagonal was not written
                x[e] = sum;
                sum += y;
            }
#pragma unroll
            for (int n = 1; n < 8; n *= 2) {
                const float y = __shfl_up(sum, n, 8);
                sum += (own & 7) >= n ? y : 0.f;
            }
            const float y = __shfl_up(sum, 1, 8), before = own & 7 ? y : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = t0 + e <= i ? before + x[e] : 0.f;
#pragma unroll
            for (int n = 4; n >= 1; n /= 2) {
                const bool upper = own & (8 * n);
#pragma unroll
                for (int e = 0; e < n; ++e) {
                    const float other = __shfl_xor(upper ? x[e] : x[e + n], 8 * n, 64);
                    x[e] = (upper ? x[e + n] : x[e]) + other;
                }
            }
            across[wave][t0 + (own >> 3 & 1) + 2 * (own >> 4 & 1) + 4 * (own >> 5)] = x[0];
        }
        if (k_on) {
            auto times = [&](const bf16x8 (&f)[4][2][kParts][64], int b, f32x4 (&acc)[TW][2], const bf16x8 (&k)[TW][2][NPI]) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    bf16x8 v[kParts];
#pragma unroll
                    for (int p = 0; p < kParts; ++p) v[p] = f[2 * rh + r][b][p][lane];
#pragma unroll
                    for (int x = 0; x < TW; ++x) mma(acc[x][r], v, k[x][b]);
                }
            };
            times(sh.tri.phi, 0, aq, kt);                 // blocks of tokens at or before the wave's
            times(sh.tri.psi, 0, ar, kt);
            times(sh.tri.phit, 1, aw, qt);                // at or behind them
            times(sh.tri.psit, 1, aw, kt);
            if (rh) {
                times(sh.tri.phi, 1, aq, kt);
                times(sh.tri.psi, 1, ar, kt);
            } else {
                times(sh.tri.phit, 0, aw, qt);
                times(sh.tri.psit, 0, aw, kt);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int x = 0; x < TW; ++x) {
                dq_all[x][r] += aq[x][r];
                dk_all[x][r] += ar[x][r] + aw[x][r];
            }
        __syncthreads();
        if (wave == 0) {
            float d = 0.f, b0 = 0.f, z = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                d += red[0][c][lane];
                b0 += red[1][c][lane];
                z += red[2][c][lane];
            }
            // A lane's token t: what it and later tokens read of S0, what earlier ones leave in S1, and the pairs across it.
            d *= gamma[lane];
#pragma unroll
            for (int i = 1; i < 64; i *= 2) {
                const float x = __shfl_down(d, i, 64), y = __shfl_up(z, i, 64);
                d += lane + i < 64 ? x : 0.f;
                z += lane >= i ? y : 0.f;
            }
            z = __shfl_up(z, 1, 64);
            float dot = 0.f, pairs = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dot += dots[i];
                pairs += across[i][lane];
            }
            if (lane < rem) {
                const int64_t at = (token0 + lane) * a.Hv + hv;
                if (a.dg) a.dg[at] = gamma[63] * dot + d + (lane ? z : 0.f) + pairs;
                if (a.db) a.db[at] = (xv[0][lane] + xv[1][lane] + xv[2][lane] + xv[3][lane]) - gamma[lane] * b0 - (rowsum[0][lane] + rowsum[1][lane]);
            }
        }
    }
    if (k_on) {
#pragma unroll
        for (int x = 0; x < TW; ++x) {
            const int c = tile_index(cg * TW + x, m);
            if (c >= a.K) continue;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = acc_index(2 * rh + r, g) + i;
                    if (t >= rem) continue;
                    const int64_t at = ((token0 + t) * a.Hk + hk) * a.K + c;
                    if (a.dq) static_cast<E*>(a.dq)[at] = E(dq_all[x][r][i]);
                    if (a.dk) static_cast<E*>(a.dk)[at] = E(dk_all[x][r][i]);
                }
        }
    }
}

}  // namespace

hipError_t launch_gdr_grad(int dt, int kb, const GdrArgs& a, hipStream_t st) {
    if (!a.slots) return hipSuccess;
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        const void* fn = reinterpret_cast<const void*>(&gdr_grad_kernel<decltype(d)::value, decltype(k)::value>);
        GdrArgs args = a;
        void* params[] = {&args};
        return hipLaunchKernel(fn, dim3(unsigned(a.slots * a.Hk)), dim3(512), params, 0, st);
    });
}

}  // namespace qc
