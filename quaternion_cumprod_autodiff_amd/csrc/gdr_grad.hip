// gdr_grad.hip -- the chunked gated delta rule's gradients of q, k and the
// gates (gdr_chunk.hpp), every chunk at once.
//
// One block of 8 waves per chunk and key head, walking the value heads that
// share it, so that the sums of a shared head's gradients are made in
// registers and in one order.  V is taken in pieces of up to 128 columns:
// X, U and dO go to LDS as operand parts; S0 and dS1 are read once, straight
// into operands.  Wave (cg, rh) owns columns of K (group cg of the tiles) and
// half rh of the tokens; the 64 x 64 products X U^T, dO U^T are dealt by row
// tiles.  Bound by its MFMAs (3 to 6 per product for float32 accuracy).
#include "gdr_chunk.hpp"

namespace qc {
namespace {

constexpr int kPiece = 128;     // columns of V at a time

__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) x += __shfl_xor(x, d, 64);
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
    };
    union Shared {
        __device__ Shared() {}
        Rows rows;
        Tri tri;
    };
    __shared__ __align__(16) Shared sh;
    __shared__ double cum[64];
    __shared__ __align__(16) float gamma[64], eta[64], beta[64], xv[64], rowsum[2][64], red[3][4][64], dots[8];
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

    f32x4 dq_all[TW][2], dk_all[TW][2];
#pragma unroll
    for (int x = 0; x < TW; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r) dq_all[x][r] = dk_all[x][r] = zero4();

#pragma unroll 1
    for (int hv = hk * a.group; hv < (hk + 1) * a.group; ++hv) {
        const Gates* ga = reinterpret_cast<const Gates*>(a.hrec + (hv * a.slots + slot) * kHrecBytes + kGateOffset);
        __syncthreads();                                  // the head before is done with what is in LDS
        if (tid < 64) {
            gamma[tid] = ga->gamma[tid];
            eta[tid] = ga->eta[tid];
            beta[tid] = ga->beta[tid];
            cum[tid] = ga->cum[tid];
        }
        f32x4 aq[TW][2], ar[TW][2], aw[TW][2], op[2] = {zero4(), zero4()}, xp[2] = {zero4(), zero4()};
#pragma unroll
        for (int x = 0; x < TW; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) aq[x][r] = ar[x][r] = aw[x][r] = zero4();
        float sds = 0.f, xdotv = 0.f;
        const int64_t piece = (hv * a.slots + slot) * int64_t(a.VP / 16) * 256;
        const float *s0 = a.save_s + piece * (2 * KB), *s1 = a.ds + piece * (2 * KB);
        const float *us = a.save_u + piece * 4, *xs = a.x + piece * 4;
#pragma unroll 1
        for (int v0 = 0; v0 < a.V; v0 += kPiece) {
            if (v0) __syncthreads();                      // the piece before is done
            // Thread (token, group of 16 columns): X, U, dO as fragments; X . v.
            {
                const int t = tid >> 3, c0 = (tid & 7) * 16;
                const bool in = t < rem;
                // Token t: tile 2 (t / 32) + (t / 4) % 2, row 4 ((t % 32) / 8) + t % 4.
                const int tile = 2 * (t >> 5) + ((t >> 2) & 1), row = 4 * ((t & 31) >> 3) + (t & 3);
                const E* op_ = static_cast<const E*>(a.d_out) + ((token0 + (in ? t : 0)) * a.Hv + hv) * a.V;
                const E* vp = static_cast<const E*>(a.v) + s.b * a.vs[0] + (s.t0 + int64_t(chunk) * kChunk + (in ? t : 0)) * a.vs[1] + int64_t(hv) * a.vs[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = c0 + 8 * i, v = v0 + c;
                    float x8[8], u8[8];
                    const bool have = v < a.VP;
                    if (have) {
                        const int at = (v >> 4) * 1024 + tile * 256 + row * 16 + (v & 15);
                        load_floats<8>(xs + at, x8);
                        load_floats<8>(us + at, u8);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x8[e] = u8[e] = 0.f;
                    }
                    bf16x8 xp8[kParts], up8[kParts], o8[NPI], v8[NPI];
                    split<kParts, 8>(x8, xp8);
                    split<kParts, 8>(u8, up8);
                    const int left = in ? a.V - v : 0;
                    load_parts<DT>(op_ + v, left, a.vec_o, o8);
                    load_parts<DT>(vp + v, left, a.vec_v, v8);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float ve = 0.f;
#pragma unroll
                        for (int p = NPI - 1; p >= 0; --p) ve += float(v8[p][e]);
                        xdotv += x8[e] * ve;
                    }
                    const int at = 16 * ((c & 31) >> 3) + row;
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        sh.rows.x[tile][c >> 5][p][at] = xp8[p];
                        sh.rows.u[tile][c >> 5][p][at] = up8[p];
                    }
#pragma unroll
                    for (int p = 0; p < NPI; ++p) sh.rows.o[tile][c >> 5][p][at] = o8[p];
                }
            }
            __syncthreads();
            const int blocks = a.V - v0 >= kPiece ? VB : (a.V - v0 + 31) / 32;
            if (k_on) {
                // The states' operands are loaded one block of V ahead.
                float s8[TW][8], d8[TW][8];
                auto load_states = [&](int b) {
                    const int v = v0 + 32 * b + 8 * g;
                    const bool have = v < a.VP;
#pragma unroll
                    for (int y = 0; y < TW; ++y) {
                        const int at = have ? (v >> 4) * (2 * KB * 256) + (cg * TW + y) * 256 + m * 16 + (v & 15) : 0;
                        load_floats<8>(s0 + at, s8[y]);
                        load_floats<8>(s1 + at, d8[y]);
                    }
                };
                load_states(0);
#pragma unroll 1
                for (int b = 0; b < blocks; ++b) {
                    bf16x8 sp[TW][kParts], dp[TW][kParts];
                    const bool have = v0 + 32 * b + 8 * g < a.VP;
#pragma unroll
                    for (int y = 0; y < TW; ++y) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            s8[y][e] = have ? s8[y][e] : 0.f;
                            d8[y][e] = have ? d8[y][e] : 0.f;
                            sds += s8[y][e] * d8[y][e];
                        }
                        split<kParts, 8>(s8[y], sp[y]);
                        split<kParts, 8>(d8[y], dp[y]);
                    }
                    load_states(b + 1 < blocks ? b + 1 : b);
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
#pragma unroll
                        for (int p = 0; p < kParts; ++p) f[p] = sh.rows.u[2 * rh + r][b][p][lane];
#pragma unroll
                        for (int y = 0; y < TW; ++y) mma(aw[y][r], f, dp[y]);
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
        // K K^T, row tile rt against the column tiles 2 ch + 0, 1.
        f32x4 kk[2] = {zero4(), zero4()};
        if (tri_on) {
#pragma unroll 1
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
        __syncthreads();                                  // X, U, dO are done; Phi and Psi take their place
#pragma unroll
        for (int d = 1; d < 8; d *= 2) xdotv += __shfl_xor(xdotv, d, 64);
        if ((tid & 7) == 0) xv[tid >> 3] = xdotv;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sds += __shfl_xor(sds, d, 64);
        if (lane == 0) dots[wave] = rh == 0 ? sds : 0.f;
        {
            const int i0 = acc_index(rt, g);
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
                        if (i > j) part[r] += xp[c][r] * (d * kk[c][r]);
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
        // The wave's columns of K and Q at its own tokens, as its accumulators have them.
        float kd[TW][2][4], qd[TW][2][4];
#pragma unroll
        for (int x = 0; x < TW; ++x) {
#pragma unroll
            for (int e = 0; e < 8; ++e) kd[x][e >> 2][e & 3] = qd[x][e >> 2][e & 3] = 0.f;
            if (k_on)
#pragma unroll
                for (int p = NPI - 1; p >= 0; --p) {
                    const int f = (((cg * TW + x) * 2 + rh) * NPI + p) * 64 + lane;
                    const bf16x8 kv = kt_set[f], qv = qt_set[f];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        kd[x][e >> 2][e & 3] += float(kv[e]);
                        qd[x][e >> 2][e & 3] += float(qv[e]);
                    }
                }
        }
        // The products with the states: their shares of the gates' gradients, then their scales.
        auto reduce = [&](int which, int r, int i, float v) {
            v = sum16(v);
            if (m == 0) red[which][cg][acc_index(2 * rh + r, g) + i] = v;
        };
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t0 = acc_index(2 * rh + r, g);
            const f32x4 ga4 = *reinterpret_cast<const f32x4*>(&gamma[t0]), be4 = *reinterpret_cast<const f32x4*>(&beta[t0]),
                        et4 = *reinterpret_cast<const f32x4*>(&eta[t0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float b0 = 0.f, z = 0.f;
#pragma unroll
                for (int x = 0; x < TW; ++x) {
                    b0 += kd[x][r][i] * ar[x][r][i];
                    z += kd[x][r][i] * aw[x][r][i];
                }
                reduce(1, r, i, b0);
                reduce(2, r, i, et4[i] * z);
            }
#pragma unroll
            for (int x = 0; x < TW; ++x) {
                aq[x][r] *= a.scale * ga4;
                ar[x][r] *= -ga4 * be4;
                aw[x][r] *= et4;
            }
        }
        __syncthreads();                                  // Phi and Psi are in LDS
        if (k_on) {
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                bf16x8 kt[TW][NPI], qt[TW][NPI];
#pragma unroll
                for (int x = 0; x < TW; ++x)
#pragma unroll
                    for (int p = 0; p < NPI; ++p) {
                        kt[x][p] = kt_set[(((cg * TW + x) * 2 + b) * NPI + p) * 64 + lane];
                        qt[x][p] = qt_set[(((cg * TW + x) * 2 + b) * NPI + p) * 64 + lane];
                    }
                auto times = [&](const bf16x8 (&f)[4][2][kParts][64], f32x4 (&acc)[TW][2], const bf16x8 (&k)[TW][NPI]) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        bf16x8 v[kParts];
#pragma unroll
                        for (int p = 0; p < kParts; ++p) v[p] = f[2 * rh + r][b][p][lane];
#pragma unroll
                        for (int x = 0; x < TW; ++x) mma(acc[x][r], v, k[x]);
                    }
                };
                if (b <= rh) {
                    times(sh.tri.phi, aq, kt);
                    times(sh.tri.psi, ar, kt);
                }
                if (b >= rh) {
                    times(sh.tri.phit, aw, qt);
                    times(sh.tri.psit, aw, kt);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float d = 0.f;
#pragma unroll
                for (int x = 0; x < TW; ++x) {
                    d += qd[x][r][i] * aq[x][r][i] + kd[x][r][i] * (ar[x][r][i] - aw[x][r][i]);
                    dq_all[x][r][i] += aq[x][r][i];
                    dk_all[x][r][i] += ar[x][r][i] + aw[x][r][i];
                }
                reduce(0, r, i, d);
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
#pragma unroll
            for (int i = 1; i < 64; i *= 2) z += __shfl_xor(z, i, 64);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) dot += dots[i];
            double sum = d;
            if (lane == 63) sum += double(gamma[63]) * dot + z;
#pragma unroll
            for (int i = 1; i < 64; i *= 2) {
                const double y = __shfl_down(sum, i, 64);
                if (lane + i < 64) sum += y;
            }
            if (lane < rem) {
                const int64_t at = (token0 + lane) * a.Hv + hv;
                // dg is a multiple of exp(g): nothing where that is 0, whatever rounding leaves of the sum.
                const float decay = expf(float(cum[lane] - (lane ? cum[lane - 1] : 0.0)));
                if (a.dg) a.dg[at] = decay > 0.f || decay != decay ? float(sum) : 0.f;
                if (a.db) a.db[at] = xv[lane] - gamma[lane] * b0 - (rowsum[0][lane] + rowsum[1][lane]);
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
