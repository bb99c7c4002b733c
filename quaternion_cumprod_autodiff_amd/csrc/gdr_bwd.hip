// gdr_bwd.hip -- the chunked gated delta rule's backward pass over the chunks
// of a sequence, last to first (gdr_chunk.hpp): the state's cotangent, X, dV.
//
// One block of 8 waves per sequence, value head and 16 columns of V, as the
// forward pass.  Per chunk:
//     phase 1   chain wave w: rows of tile w of dU = P^T O + eta (K dS1)
//     phase 2   chain wave w: rows of tile w of X = T^T dU;  dV = b X, stored with X
//     phase 3   chain wave w: its tiles of dS0 = gamma_last dS1 + Q^T (gamma O) - K^T (gamma b X)
// with a barrier after each.  What does not depend on dS1 (P^T O, Q^T (gamma O))
// the helper waves prepare one chunk ahead:
//     phase 1   helper wave w: rows of tile w of the next chunk's dO into LDS, as the operands dO and scale gamma dO
//     phase 2   its P^T O;    phase 3   its Q^T (gamma O), the tiles of chain wave w
#include "gdr_chunk.hpp"

namespace qc {
namespace {

template <int DT, int KB>
__global__ void __launch_bounds__(512) gdr_bwd_kernel(GdrArgs a, int strips) {
    using E = typename Storage<DT>::type;
    constexpr int NPI = parts_of(DT);
    constexpr int ST = (2 * KB + 3) / 4;
    __shared__ __align__(16) bf16x8 sf[KB][kParts][64], uf[2][kParts][64], xf[2][kParts][64];
    __shared__ __align__(16) bf16x8 of[2][NPI][64], gf[2][kParts][64];
    __shared__ __align__(16) f32x4 po[4][64], qo[2 * KB][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
    const int m = lane & 15, g = lane >> 4;
    int64_t n;
    int hv, strip;
    if (!unit_of(a, strips, n, hv, strip)) return;
    const int hk = hv / a.group;
    const Sequence s = sequence(a, n);
    const int chunks = (s.len + kChunk - 1) / kChunk;
    const int col = strip * 16 + m;
    const int i0 = acc_index(w, g);
    const int64_t krec = krec_bytes(KB, NPI);
    const char* kr = a.krec + (hk * a.slots + s.slot) * krec;
    const char* hr = a.hrec + (hv * a.slots + s.slot) * kHrecBytes;
    const int64_t kstep = krec, hstep = kHrecBytes;
    const int64_t row0 = (s.b * a.T + s.t0) * a.Hv + hv;      // this head's row of the sequence's first token

    if (wave < 4) {
        f32x4 st[ST];
        const int64_t state0 = (n * a.Hv + hv) * int64_t(a.K) * a.V;
        auto put_state = [&] {
#pragma unroll
            for (int x = 0; x < ST; ++x) {
                const int tile = w + 4 * x;
                if (tile < 2 * KB) {
                    bf16x4 p[kParts];
                    split4(st[x], p);
                    put_parts(&sf[tile >> 1][0][0], 64, lane, tile & 1, p);
                }
            }
        };
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = acc_index(w + 4 * x, g) + r;
                st[x][r] = a.d_fin && row < a.K && col < a.V ? a.d_fin[state0 + int64_t(row) * a.V + col] : 0.f;
            }
        put_state();
        bf16x8 ka[KB][NPI], kt[ST][2][NPI], ta[2][kParts];
        // The gates of the next chunk are loaded a whole chunk ahead: the first of them is needed at the end of phase 1.
        f32x4 gamma, eta, beta, gamma_next, eta_next, beta_next;
        float last, last_next;
        const int zero = lane_zero();
        auto load_k = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(kr + c * kstep) + int64_t(w) * KB * NPI * 64 + lane;
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < NPI; ++i) ka[b][i] = p[(b * NPI + i) * 64];
        };
        auto load_gates = [&](int c) {
            const Gates* p = reinterpret_cast<const Gates*>(hr + c * hstep + kGateOffset);
            gamma_next = *reinterpret_cast<const f32x4*>(&p->gamma[i0]);
            eta_next = *reinterpret_cast<const f32x4*>(&p->eta[i0]);
            beta_next = *reinterpret_cast<const f32x4*>(&p->beta[i0]);
            last_next = p->gamma[kChunk - 1 + zero];
        };
        auto load_t = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(hr + c * hstep) + lane;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<true>(w, b))
#pragma unroll
                    for (int i = 0; i < kParts; ++i) ta[b][i] = p[(tri_index<true>(w, b) * kParts + i) * 64];
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
            load_k(chunks - 1);
            load_gates(chunks - 1);
            load_t(chunks - 1);
            load_kt(chunks - 1);
        }
        __syncthreads();      // the last chunk's dO
        __syncthreads();      // its P^T O
        __syncthreads();      // its Q^T (gamma O)
        for (int c = chunks - 1; c >= 0; --c) {
            const int next = c > 0 ? c - 1 : 0;
            gamma = gamma_next;
            eta = eta_next;
            beta = beta_next;
            last = last_next;
            load_gates(next);
            {
                float* p = a.ds + (hv * a.slots + s.slot + c) * int64_t(32 * KB) * a.VP + col;
#pragma unroll
                for (int x = 0; x < ST; ++x)
                    if (w + 4 * x < 2 * KB)
#pragma unroll
                        for (int r = 0; r < 4; ++r) p[int64_t(acc_index(w + 4 * x, g) + r) * a.VP] = st[x][r];
            }
            f32x4 acc = zero4(), odd = zero4();       // two sums, so that products need not wait for each other
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                bf16x8 x[kParts];
#pragma unroll
                for (int i = 0; i < kParts; ++i) x[i] = sf[b][i][lane];
                mma(b & 1 ? odd : acc, ka[b], x);
            }
            load_k(next);
            acc += odd;
            {
                const f32x4 y = po[w][lane];
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = y[r] + eta[r] * acc[r];
                bf16x4 p[kParts];
                split4(x, p);
                put_parts(&uf[w >> 1][0][0], 64, lane, w & 1, p);
            }
            __syncthreads();
            acc = zero4();
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<true>(w, b)) {
                    bf16x8 x[kParts];
#pragma unroll
                    for (int i = 0; i < kParts; ++i) x[i] = uf[b][i][lane];
                    mma(acc, ta[b], x);
                }
            load_t(next);
            {
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = -(gamma[r] * beta[r]) * acc[r];
                bf16x4 p[kParts];
                split4(x, p);
                put_parts(&xf[w >> 1][0][0], 64, lane, w & 1, p);
            }
            float* xs = a.x + (hv * a.slots + s.slot + c) * int64_t(kChunk) * a.VP + col;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = c * kChunk + i0 + r;
                xs[int64_t(i0 + r) * a.VP] = acc[r];
                if (a.dv && i < s.len && col < a.V) static_cast<E*>(a.dv)[(row0 + int64_t(i) * a.Hv) * a.V + col] = E(beta[r] * acc[r]);
            }
#pragma unroll
            for (int x = 0; x < ST; ++x)
                if (w + 4 * x < 2 * KB) {
                    const f32x4 y = qo[w + 4 * x][lane];
#pragma unroll
                    for (int r = 0; r < 4; ++r) st[x][r] = last * st[x][r] + y[r];
                }
            __syncthreads();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                bf16x8 y[kParts];
#pragma unroll
                for (int i = 0; i < kParts; ++i) y[i] = xf[b][i][lane];
#pragma unroll
                for (int x = 0; x < ST; ++x)
                    if (w + 4 * x < 2 * KB) mma(st[x], kt[x][b], y);
            }
            load_kt(next);
            put_state();
            __syncthreads();
        }
        if (a.ds0) {
#pragma unroll
            for (int x = 0; x < ST; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = acc_index(w + 4 * x, g) + r;
                    if (row < a.K && col < a.V) a.ds0[state0 + int64_t(row) * a.V + col] = st[x][r];
                }
        }
    } else {
        bf16x8 pa[2][kParts], qt[ST][2][NPI];
        E dr[4];          // as loaded
        f32x4 gamma;
        auto load_do = [&](int c) {
            // Rows behind the end and columns past V read the nearest one inside, and are dropped where used: no branches.
            const E* p = static_cast<const E*>(a.d_out) + row0 * a.V + (col < a.V ? col : 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = c * kChunk + i0 + r < s.len ? c * kChunk + i0 + r : s.len - 1;
                dr[r] = p[int64_t(i) * a.Hv * a.V];
            }
            gamma = *reinterpret_cast<const f32x4*>(&reinterpret_cast<const Gates*>(hr + c * hstep + kGateOffset)->gamma[i0]);
        };
        auto load_p = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(hr + c * hstep) + kTriFrags * 64 + lane;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<true>(w, b))
#pragma unroll
                    for (int i = 0; i < kParts; ++i) pa[b][i] = p[(tri_index<true>(w, b) * kParts + i) * 64];
        };
        auto load_qt = [&](int c) {
            const bf16x8* p = reinterpret_cast<const bf16x8*>(kr + c * kstep) + set_frags(KB, NPI) * 64 + lane;
#pragma unroll
            for (int x = 0; x < ST; ++x)
                if (w + 4 * x < 2 * KB)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < NPI; ++i) qt[x][b][i] = p[(((w + 4 * x) * 2 + b) * NPI + i) * 64];
        };
        if (chunks) {
            load_do(chunks - 1);
            load_p(chunks - 1);
            load_qt(chunks - 1);
        }
        // Round c prepares chunk c while the chain waves work on chunk c + 1; the first round is the chain's prologue.
        // The last chunk's round (c = 0) is followed by one more that only keeps the barriers.
        for (int c = chunks - 1; c >= -1; --c) {
            const int next = c > 0 ? c - 1 : 0;
            if (c >= 0) {
                f32x4 x;
                bf16x4 o[NPI], p[kParts];
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = c * kChunk + i0 + r < s.len && col < a.V ? float(dr[r]) : 0.f;
                split4(x, o);
                put_parts(&of[w >> 1][0][0], 64, lane, w & 1, o);
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] *= a.scale * gamma[r];
                split4(x, p);
                put_parts(&gf[w >> 1][0][0], 64, lane, w & 1, p);
                load_do(next);
            }
            __syncthreads();
            if (c >= 0) {
                f32x4 acc = zero4();
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (tri_has<true>(w, b)) {
                        bf16x8 x[NPI];
#pragma unroll
                        for (int i = 0; i < NPI; ++i) x[i] = of[b][i][lane];
                        mma(acc, pa[b], x);
                    }
                load_p(next);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] *= a.scale;
                po[w][lane] = acc;
            }
            __syncthreads();
            if (c >= 0) {
                f32x4 acc[ST];
#pragma unroll
                for (int x = 0; x < ST; ++x) acc[x] = zero4();
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    bf16x8 y[kParts];
#pragma unroll
                    for (int i = 0; i < kParts; ++i) y[i] = gf[b][i][lane];
#pragma unroll
                    for (int x = 0; x < ST; ++x)
                        if (w + 4 * x < 2 * KB) mma(acc[x], qt[x][b], y);
                }
                load_qt(next);
#pragma unroll
                for (int x = 0; x < ST; ++x)
                    if (w + 4 * x < 2 * KB) qo[w + 4 * x][lane] = acc[x];
            }
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_gdr_bwd_state(int dt, int kb, const GdrArgs& a, hipStream_t st) {
    if (!a.N) return hipSuccess;
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        int strips = (a.V + 15) / 16;
        const int64_t blocks = (a.N * a.Hk + 7) / 8 * 8 * strips * a.group;
        const void* fn = reinterpret_cast<const void*>(&gdr_bwd_kernel<decltype(d)::value, decltype(k)::value>);
        GdrArgs args = a;
        void* params[] = {&args, &strips};
        return hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(512), params, 0, st);
    });
}

}  // namespace qc
