// gdr_fwd.hip -- the chunked gated delta rule's forward pass over the chunks
// of a sequence (gdr_chunk.hpp).
//
// One block of 8 waves per sequence, value head and 16 NT columns of V; the
// state's columns never meet, so blocks are independent.  Per chunk:
//     phase 1   chain wave w: rows of tile w of V - gamma (K S0);    output wave w: gamma (Q S0)
//     phase 2   chain wave w: rows of tile w of U = T b (..)
//     phase 3   chain wave w: its tiles of S1 = gamma_last S0 + K^T (eta U);    output wave w: + P U, stored
// with a barrier after each; S0, the bracket and U pass between waves as
// fragments in LDS.  What a wave multiplies from the left it alone needs, and
// loads straight into registers, one chunk ahead.  A sequence's time is the
// chain of these phases (36 MFMA, three splits and three barriers per chunk),
// not their sum: the output waves fill the chain's gaps.
#include "gdr_chunk.hpp"

namespace qc {
namespace {

template <int DT, int KB, int NT, bool SAVE>
__global__ void __launch_bounds__(512) gdr_fwd_kernel(GdrArgs a, int strips) {
    using E = typename Storage<DT>::type;
    constexpr int NPI = parts_of(DT);
    // Parts of S0 and U that the output takes: two leave 2^-17 of them, below the half step of 16-bit outputs.
    constexpr int NPO = DT == 0 ? 3 : 2;
    constexpr int ST = (2 * KB + 3) / 4;             // tiles of S of a chain wave
    __shared__ __align__(16) bf16x8 sf[KB][NT][kParts][64], rf[2][NT][kParts][64], ef[2][NT][kParts][64], uf[2][NT][NPO][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
    const int m = lane & 15, g = lane >> 4;
    int64_t n;
    int hv, strip;
    if (!unit_of(a, strips, n, hv, strip)) return;
    const int hk = hv / a.group;
    const Sequence s = sequence(a, n);
    const int chunks = (s.len + kChunk - 1) / kChunk;
    const int col = strip * 16 * NT + m;
    const int i0 = acc_index(w, g);
    const int64_t krec = krec_bytes(KB, NPI);
    const char* kr = a.krec + (s.slot * a.Hk + hk) * krec;
    const char* hr = a.hrec + (s.slot * a.Hv + hv) * kHrecBytes;
    const int64_t kstep = a.Hk * krec, hstep = a.Hv * kHrecBytes;

    if (wave < 4) {
        f32x4 st[ST][NT];
        const int64_t state0 = (n * a.Hv + hv) * int64_t(a.K) * a.V;
        auto put_state = [&] {
#pragma unroll
            for (int x = 0; x < ST; ++x) {
                const int tile = w + 4 * x;
                if (tile < 2 * KB)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        bf16x4 p[kParts];
                        split4(st[x][t], p);
                        put_parts(&sf[tile >> 1][t][0][0], 64, lane, tile & 1, p);
                    }
            }
        };
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = acc_index(w + 4 * x, g) + r, c = col + 16 * t;
                    st[x][t][r] = a.s0 && row < a.K && c < a.V ? a.s0[state0 + int64_t(row) * a.V + c] : 0.f;
                }
        put_state();
        bf16x8 ka[KB][NPI], kt[ST][2][NPI], ta[2][kParts];
        float vr[NT][4];
        f32x4 gamma, eta;
        float last;
        auto load_k = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(kr + c * kstep) + int64_t(w) * KB * NPI * 64 + lane;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < NPI; ++i) ka[b][i] = p[(b * NPI + i) * 64];
        };
        auto load_v = [&](int c) {
            const E* v = static_cast<const E*>(a.v) + s.b * a.vs[0] + int64_t(hv) * a.vs[2] + col;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = c * kChunk + i0 + r;
                    vr[t][r] = i < s.len && col + 16 * t < a.V ? float(v[(s.t0 + i) * a.vs[1] + 16 * t]) : 0.f;
                }
        };
        auto load_gates = [&](int c) {
            const Gates* p = reinterpret_cast<const Gates*>(hr + c * hstep + kGateOffset);
            gamma = *reinterpret_cast<const f32x4*>(&p->gamma[i0]);
            eta = *reinterpret_cast<const f32x4*>(&p->eta[i0]);
            last = p->gamma[kChunk - 1];
        };
        auto load_t = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(hr + c * hstep) + lane;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<false>(w, b))
#pragma unroll
                    for (int i = 0; i < kParts; ++i) ta[b][i] = p[(tri_index<false>(w, b) * kParts + i) * 64];
        };
        auto load_kt = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(kr + c * kstep) + 2 * set_frags(KB, NPI) * 64 + lane;
#pragma unroll
            for (int x = 0; x < ST; ++x)
                if (w + 4 * x < 2 * KB)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < NPI; ++i) kt[x][b][i] = p[(((w + 4 * x) * 2 + b) * NPI + i) * 64];
        };
        if (chunks) {
            load_k(0);
            load_v(0);
            load_gates(0);
            load_t(0);
            load_kt(0);
        }
        __syncthreads();
        for (int c = 0; c < chunks; ++c) {
            const int next = c + 1 < chunks ? c + 1 : c;
            if constexpr (SAVE) {
                float* p = a.save_s + ((s.slot + c) * a.Hv + hv) * int64_t(32 * KB) * a.VP;
#pragma unroll
                for (int x = 0; x < ST; ++x)
                    if (w + 4 * x < 2 * KB)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (col + 16 * t < a.VP) p[int64_t(acc_index(w + 4 * x, g) + r) * a.VP + col + 16 * t] = st[x][t][r];
            }
            f32x4 acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = zero4();
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    bf16x8 x[kParts];
#pragma unroll
                    for (int i = 0; i < kParts; ++i) x[i] = sf[b][t][i][lane];
                    mma(acc[t], ka[b], x);
                }
            load_k(next);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = vr[t][r] - gamma[r] * acc[t][r];
                bf16x4 p[kParts];
                split4(x, p);
                put_parts(&rf[w >> 1][t][0][0], 64, lane, w & 1, p);
            }
            load_v(next);
            __syncthreads();
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = zero4();
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<false>(w, b))
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        bf16x8 x[kParts];
#pragma unroll
                        for (int i = 0; i < kParts; ++i) x[i] = rf[b][t][i][lane];
                        mma(acc[t], ta[b], x);
                    }
            load_t(next);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                bf16x4 p[kParts], o[NPO];
                f32x4 e;
#pragma unroll
                for (int r = 0; r < 4; ++r) e[r] = eta[r] * acc[t][r];
                split4(e, p);
                put_parts(&ef[w >> 1][t][0][0], 64, lane, w & 1, p);
                split4(acc[t], o);
                put_parts(&uf[w >> 1][t][0][0], 64, lane, w & 1, o);
                if constexpr (SAVE) {
                    float* u = a.save_u + ((s.slot + c) * a.Hv + hv) * int64_t(kChunk) * a.VP;
                    if (col + 16 * t < a.VP)
#pragma unroll
                        for (int r = 0; r < 4; ++r) u[int64_t(i0 + r) * a.VP + col + 16 * t] = acc[t][r];
                }
            }
            __syncthreads();
#pragma unroll
            for (int x = 0; x < ST; ++x)
                if (w + 4 * x < 2 * KB)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        f32x4 z;
#pragma unroll
                        for (int r = 0; r < 4; ++r) z[r] = last * st[x][t][r];
                        st[x][t] = z;
                    }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    bf16x8 y[kParts];
#pragma unroll
                    for (int i = 0; i < kParts; ++i) y[i] = ef[b][t][i][lane];
#pragma unroll
                    for (int x = 0; x < ST; ++x)
                        if (w + 4 * x < 2 * KB) mma(st[x][t], kt[x][b], y);
                }
            load_kt(next);
            load_gates(next);
            put_state();
            __syncthreads();
        }
        if (a.fin) {
#pragma unroll
            for (int x = 0; x < ST; ++x)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = acc_index(w + 4 * x, g) + r, c = col + 16 * t;
                        if (row < a.K && c < a.V) a.fin[state0 + int64_t(row) * a.V + c] = st[x][t][r];
                    }
        }
    } else {
        bf16x8 qa[KB][NPI], pa[2][kParts];
        f32x4 gamma;
        auto load = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(kr + c * kstep) + (set_frags(KB, NPI) + int64_t(w) * KB * NPI) * 64 + lane;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < NPI; ++i) qa[b][i] = p[(b * NPI + i) * 64];
            gamma = *reinterpret_cast<const f32x4*>(&reinterpret_cast<const Gates*>(hr + c * hstep + kGateOffset)->gamma[i0]);
        };
        auto load_p = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(hr + c * hstep) + kTriFrags * 64 + lane;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<false>(w, b))
#pragma unroll
                    for (int i = 0; i < kParts; ++i) pa[b][i] = p[(tri_index<false>(w, b) * kParts + i) * 64];
        };
        if (chunks) {
            load(0);
            load_p(0);
        }
        __syncthreads();
        for (int c = 0; c < chunks; ++c) {
            const int next = c + 1 < chunks ? c + 1 : c;
            f32x4 acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = zero4();
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    bf16x8 x[NPO];
#pragma unroll
                    for (int i = 0; i < NPO; ++i) x[i] = sf[b][t][i][lane];
                    mma(acc[t], qa[b], x);
                }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[t][r] *= gamma[r];
            load(next);
            __syncthreads();
            __syncthreads();
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<false>(w, b))
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        bf16x8 x[NPO];
#pragma unroll
                        for (int i = 0; i < NPO; ++i) x[i] = uf[b][t][i][lane];
                        mma(acc[t], pa[b], x);
                    }
            load_p(next);
            E* o = static_cast<E*>(a.out) + (s.b * a.T + s.t0) * int64_t(a.Hv) * a.V + int64_t(hv) * a.V + col;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = c * kChunk + i0 + r;
                    if (i < s.len && col + 16 * t < a.V) o[int64_t(i) * a.Hv * a.V + 16 * t] = E(a.scale * acc[t][r]);
                }
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_gdr_fwd(int dt, int kb, bool save, const GdrArgs& a, hipStream_t st) {
    if (!a.N) return hipSuccess;
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        constexpr int DT = decltype(d)::value, KB = decltype(k)::value;
        const int nt = 1;
        int strips = (a.V + 16 * nt - 1) / (16 * nt);
        const int64_t blocks = (a.N * a.Hk + 7) / 8 * 8 * strips * a.group;
        const void* fn = save ? reinterpret_cast<const void*>(&gdr_fwd_kernel<DT, KB, 1, true>)
                              : reinterpret_cast<const void*>(&gdr_fwd_kernel<DT, KB, 1, false>);
        GdrArgs args = a;
        void* params[] = {&args, &strips};
        return hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(512), params, 0, st);
    });
}

}  // namespace qc
