// gdr_factor.hip -- the per-chunk factors of the chunked gated delta rule
// (gdr_chunk.hpp): T = (I + diag(b) L)^-1, P, the gates' exponentials, and the
// chunk's q and k rows as operand fragments.
//
// One block of 4 waves per chunk and value head, all chunks at once.  Wave w
// holds row tile w of K and Q; K K^T and Q K^T go to LDS with the decays.  The
// inverse: each wave solves one diagonal 16 x 16 block by substitution (a lane
// per column), then owns that block column and extends it downwards,
//     X_ij = -X_ii sum_{j <= k < i} A_ik X_kj,
// on the float32 MFMA, the X_kj staying in accumulators.  Forward
// substitution by blocks, so no power of A is formed: alike keys do not cost
// accuracy.
//
// Bound by the latency of its steps in a row (loads, product, substitution of
// 16 rows, three block rows), which the blocks of a CU hide in part: three, by
// LDS; two for float32 K = 64 and float16 K = 128, one for float32 K = 128.
// Matrix units 9% in use, waves at a wait or a barrier half of the time.  8192
// tokens of 32 heads of 128, bfloat16, 77 us; 4 x 4096, 143 us before the
// forward pass and 152 before the backward one; 8 x 2048 tokens of 16 heads of
// 64, float32, 129 and 137.
#include "gdr_chunk.hpp"

namespace qc {
namespace {

constexpr int kRow = 68;    // LDS row of a 64 x 64 float matrix

template <int DT, int KB, bool BWD>
__global__ void __launch_bounds__(256) gdr_factor_kernel(GdrArgs a) {
    using E = typename Storage<DT>::type;
    constexpr int NPI = parts_of(DT);
    // The inverse takes K's place once K K^T and the transposed fragments are made.
    struct Rows {
        bf16x8 k[4][KB][NPI][64];
    };
    union Shared {
        __device__ Shared() {}
        Rows rows;
        float inverse[64 * kRow];
    };
    __shared__ __align__(16) Shared sh;
    // Q's rows, for its transposed fragments (backward), then A and P.
    union Matrices {
        __device__ Matrices() {}
        bf16x8 q[BWD ? 4 : 1][BWD ? KB : 1][BWD ? NPI : 1][64];
        float ap[2][64 * kRow];
    };
    __shared__ __align__(16) Matrices mat;
    auto& qf = mat.q;
    float *ma = mat.ap[0], *mp = mat.ap[1];
    auto& kf = sh.rows.k;
    float* mx = sh.inverse;
    __shared__ double cum[64];
    __shared__ __align__(16) float beta[64];
    __shared__ int first_bad[5];      // of a row tile's keys and of the gates: the first token that is not finite
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), m = lane & 15, g = lane >> 4;
    const int hv = int(blockIdx.x % a.Hv);
    const int64_t slot = blockIdx.x / a.Hv;
    Sequence s;
    int chunk;
    if (slot_sequence(a, slot, s, chunk) < 0) return;
    const int hk = hv / a.group;
    const bool lead = hv % a.group == 0;
    const int rem = s.len - chunk * kChunk;          // rows of this chunk, and of the ones behind it
    const int64_t t0 = s.t0 + int64_t(chunk) * kChunk;
    char* kr = a.krec + (hk * a.slots + slot) * krec_bytes(KB, NPI);
    char* hr = a.hrec + (hv * a.slots + slot) * kHrecBytes;
    bf16x8* k_rows = reinterpret_cast<bf16x8*>(kr);
    bf16x8* q_set = k_rows + set_frags(KB, NPI) * 64;
    bf16x8* k_cols = q_set + set_frags(KB, NPI) * 64;

    // Everything that comes from far away first: the gates (wave 0), row tile w of K and Q.
    const int64_t gate_at = (s.b * a.T + t0 + (lane < rem ? lane : 0)) * a.Hv + hv;
    float g_raw = 0.f, b_raw = 0.f;
    if (w == 0) {
        g_raw = a.g[gate_at];
        b_raw = a.b[gate_at];
    }
    bf16x8 qa[KB][NPI], ka[KB][NPI];
    {
        const int t = tile_index(w, m);
        const bool in = t < rem;
        const E* kp = static_cast<const E*>(a.k) + s.b * a.ks[0] + (t0 + (in ? t : 0)) * a.ks[1] + int64_t(hk) * a.ks[2];
        const E* qp = static_cast<const E*>(a.q) + s.b * a.qs[0] + (t0 + (in ? t : 0)) * a.qs[1] + int64_t(hk) * a.qs[2];
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            const int c = 32 * b + 8 * g, left = in ? a.K - c : 0;
            load_parts<DT>(kp + c, left, a.vec_qk, ka[b]);
            load_parts<DT>(qp + c, left, a.vec_qk, qa[b]);
        }
    }
    if constexpr (!BWD) {
        bool bad = false;
#pragma unroll
        for (int b = 0; b < KB; ++b) bad |= not_finite(ka[b][0]);
        const uint64_t mask = __ballot(bad);
        int first = kChunk;
        if (mask) {
            const uint32_t rows = uint32_t(mask | mask >> 16 | mask >> 32 | mask >> 48) & 0xffffu;
            first = tile_index(w, __builtin_ctz(rows));
            if (rows >> m & 1)
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int p = 0; p < NPI; ++p)
#pragma unroll
                        for (int j = 0; j < 8; ++j) ka[b][p][j] = __bf16(0.f);
        }
        if (lane == 0) first_bad[w] = first;
    }
    // Gates: decays cumulated in 64 bits.  -2000 stands for every decay below it: exp() of it is 0, and sums with it
    // leave the differences behind it exact to 1e-11.
    if (w == 0) {
        const bool in = lane < rem;
        float gt = in ? g_raw : 0.f, bt = in ? b_raw : 0.f;
        if constexpr (!BWD) {
            const bool bad = !(gt < __builtin_inff()) || !(fabsf(bt) < __builtin_inff());
            const uint64_t mask = __ballot(bad);
            gt = bad ? 0.f : gt;
            bt = bad ? 0.f : bt;
            if (lane == 0) first_bad[4] = mask ? __builtin_ctzll(mask) : kChunk;
        }
        double c = gt < -2000.f ? -2000.0 : double(gt);
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const double x = __shfl_up(c, d, 64);
            if (lane >= d) c += x;
        }
        const double last = __shfl(c, 63, 64);
        cum[lane] = c;
        beta[lane] = bt;
        Gates* ga = reinterpret_cast<Gates*>(hr + kGateOffset);
        ga->gamma[lane] = expf(float(c));
        ga->eta[lane] = expf(float(last - c));
        ga->beta[lane] = bt;
        ga->cum[lane] = c;
    }
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int p = 0; p < NPI; ++p) {
            kf[w][b][p][lane] = ka[b][p];
            if constexpr (BWD) qf[w][b][p][lane] = qa[b][p];
        }
    __syncthreads();
    if (!BWD && w == 0) {
        int first = first_bad[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) first = first_bad[i] < first ? first_bad[i] : first;
        reinterpret_cast<Gates*>(hr + kGateOffset)->poison[lane] = lane >= first ? __builtin_nanf("") : 0.f;
    }
    // K (backward: Q too) transposed: tiles of K, blocks of tokens.
    if (lead) {
        const __bf16* ks = reinterpret_cast<const __bf16*>(&kf);
        const __bf16* qs = reinterpret_cast<const __bf16*>(&qf);
        for (int f = w; f < 4 * KB; f += 4) {
            const int tile = f >> 1, b = f & 1;
            const int c = tile_index(tile, m);
#pragma unroll
            for (int p = 0; p < NPI; ++p) {
                bf16x8 kx, qx;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // Token 32 b + 8 g + e: row tile 2 b + e / 4, row 4 g + e % 4; element c: block c / 32, lane group (c % 32) / 8.
                    const int at = (((2 * b + (e >> 2)) * KB + (c >> 5)) * NPI + p) * 512 + (16 * ((c & 31) >> 3) + 4 * g + (e & 3)) * 8 + (c & 7);
                    kx[e] = ks[at];
                    if constexpr (BWD) qx[e] = qs[at];
                }
                k_cols[(f * NPI + p) * 64 + lane] = kx;
                if constexpr (BWD) q_set[(f * NPI + p) * 64 + lane] = qx;
            }
        }
    }
    if constexpr (BWD) __syncthreads();      // A and P take Q's place
    if (lead) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int p = 0; p < NPI; ++p) {
                k_rows[((w * KB + b) * NPI + p) * 64 + lane] = ka[b][p];
                if constexpr (!BWD) q_set[((w * KB + b) * NPI + p) * 64 + lane] = qa[b][p];
            }
    }
    // K K^T and Q K^T, the rows of tile w, against the tokens of no later block of 32, two tiles at a time.
    {
        const int i0 = acc_index(w, g);
        for (int c = 0; c < 2 * (w >> 1) + 2; c += 2) {
            f32x4 kk[2] = {zero4(), zero4()}, qk[2] = {zero4(), zero4()};
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    bf16x8 kb[NPI];
#pragma unroll
                    for (int p = 0; p < NPI; ++p) kb[p] = kf[c + y][b][p][lane];
                    mma(kk[y], ka[b], kb);
                    mma(qk[y], qa[b], kb);
                }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int j = tile_index(c + y, m);
                const double cj = cum[j];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = i0 + r;
                    const float d = expf(float(cum[i] - cj));
                    ma[i * kRow + j] = i > j ? beta[i] * d * kk[y][r] : 0.f;
                    mp[i * kRow + j] = i >= j ? d * qk[y][r] : 0.f;
                }
            }
        }
    }
    __syncthreads();
    // Diagonal blocks: column `lane` of (I + A_ww)^-1.
    if (lane < 16) {
        const float* blk = ma + (16 * w) * kRow + 16 * w;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) v -= blk[i * kRow + j] * x[j];
            x[i] = v;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) mx[(16 * w + i) * kRow + 16 * w + lane] = x[i];
    }
    __syncthreads();
    // Block column w, downwards.
    {
        f32x4 x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[0][r] = mx[(16 * w + 4 * g + r) * kRow + 16 * w + m];
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            const int i = w + d;
            if (i < 4) {
                f32x4 y = zero4();
#pragma unroll
                for (int e = 0; e < d; ++e) {
                    const f32x4 ak = *reinterpret_cast<const f32x4*>(&ma[(16 * i + m) * kRow + 16 * (w + e) + 4 * g]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y = __builtin_amdgcn_mfma_f32_16x16x4f32(ak[r], x[e][r], y, 0, 0, 0);
                }
                const f32x4 xi = *reinterpret_cast<const f32x4*>(&mx[(16 * i + m) * kRow + 16 * i + 4 * g]);
                f32x4 z = zero4();
#pragma unroll
                for (int r = 0; r < 4; ++r) z = __builtin_amdgcn_mfma_f32_16x16x4f32(-xi[r], y[r], z, 0, 0, 0);
                x[d] = z;
#pragma unroll
                for (int r = 0; r < 4; ++r) mx[(16 * i + 4 * g + r) * kRow + 16 * w + m] = z[r];
            }
        }
    }
    __syncthreads();
    // T and P as fragments, row tile w: forward T diag(b) and P, backward T^T and P^T.
    {
        const int row = tile_index(w, m);
        bf16x8* tf = reinterpret_cast<bf16x8*>(hr);
        bf16x8* pf = tf + kTriFrags * 64;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            if (!tri_has<BWD>(w, b)) continue;
            float t[8], p[8];
            const int c0 = 32 * b + 8 * g;
            if constexpr (BWD) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    t[e] = mx[(c0 + e) * kRow + row];
                    p[e] = mp[(c0 + e) * kRow + row];
                }
            } else {
                float bt[8];
                load_floats<8>(&mx[row * kRow + c0], t);
                load_floats<8>(&mp[row * kRow + c0], p);
                load_floats<8>(&beta[c0], bt);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] *= bt[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {      // what lies across the diagonal was never written
                const bool in = BWD ? c0 + e >= row : row >= c0 + e;
                t[e] = in ? t[e] : 0.f;
                p[e] = in ? p[e] : 0.f;
            }
            bf16x8 ts[kParts], ps[kParts];
            split<kParts, 8>(t, ts);
            split<kParts, 8>(p, ps);
            const int f = tri_index<BWD>(w, b) * kParts;
#pragma unroll
            for (int n = 0; n < kParts; ++n) {
                tf[(f + n) * 64 + lane] = ts[n];
                pf[(f + n) * 64 + lane] = ps[n];
            }
        }
    }
}

}  // namespace

hipError_t launch_gdr_factor(int dt, int kb, bool bwd, const GdrArgs& a, hipStream_t st) {
    if (!a.slots) return hipSuccess;
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        constexpr int DT = decltype(d)::value, KB = decltype(k)::value;
        const void* fn = bwd ? reinterpret_cast<const void*>(&gdr_factor_kernel<DT, KB, true>)
                             : reinterpret_cast<const void*>(&gdr_factor_kernel<DT, KB, false>);
        GdrArgs args = a;
        void* params[] = {&args};
        return hipLaunchKernel(fn, dim3(unsigned(a.slots * a.Hv)), dim3(256), params, 0, st);
    });
}

}  // namespace qc
