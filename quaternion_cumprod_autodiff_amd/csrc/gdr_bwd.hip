// gdr_bwd.hip -- the chunked gated delta rule's backward pass over the chunks
// of a sequence, last to first (gdr_chunk.hpp): the state's cotangent, X, dV.
//
// One block of 4 waves per sequence, value head and 16 columns of V, as the
// forward pass.  Per chunk, wave w:
//     phase 1   rows of tile w of dU = P^T O + eta (K dS1)
//     phase 2   rows of tile w of X = T^T dU;  dV = b X, stored with X;  the next chunk's dO into LDS, as the operands
//               dO and scale gamma dO
//     phase 3   its tiles of dS0 = gamma_last dS1 + Q^T (gamma O) - K^T (gamma b X)
// with a barrier after each.
#include "gdr_chunk.hpp"

namespace qc {
namespace {

template <int DT, int KB>
__global__ void __launch_bounds__(256, DT == 1 ? 2 : 1) gdr_bwd_kernel(GdrArgs a, int strips) {
    using E = typename Storage<DT>::type;
    constexpr int NPI = parts_of(DT);
    constexpr int ST = (2 * KB + 3) / 4;
    __shared__ __align__(16) bf16x8 sf[KB][kParts][64], uf[2][kParts][64], xf[2][kParts][64];
    __shared__ __align__(16) bf16x8 of[2][2][NPI][64], gf[2][2][kParts][64];      // this chunk's and the next one's
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    int64_t n;
    int hv, strip;
    if (!unit_of(a, strips, n, hv, strip)) return;
    const int hk = hv / a.group;
    const Sequence s = sequence(a, n);
    const int chunks = (s.len + kChunk - 1) / kChunk;
    const int col = strip * 16 + m;
    const bool col_in = col < a.V;
    const int i0 = acc_index(w, g);
    const int64_t krec = krec_bytes(KB, NPI);
    const char* kr = a.krec + (hk * a.slots + s.slot) * krec;
    const char* hr = a.hrec + (hv * a.slots + s.slot) * kHrecBytes;

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
            st[x][r] = a.d_fin && row < a.K && col_in ? a.d_fin[state0 + int64_t(row) * a.V + col] : 0.f;
        }
    put_state();

    bf16x8 ka[KB][NPI], kt[ST][2][NPI], qt[ST][2][NPI], ta[2][kParts], pa[2][kParts];
    E dr[4];          // as loaded
    // The gates of the next chunk are loaded a whole chunk ahead: the first of them is needed at the end of phase 1.
    f32x4 gamma, eta, beta, gamma_next, eta_next, beta_next;
    float last, last_next;
    const int zero = lane_zero();
    auto load_rows = [&](int c) {
        const char* p = kr + c * krec;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < NPI; ++i) ka[b][i] = fragment(p, (w * KB + b) * NPI + i, lane);
    };
    auto load_gates = [&](int c) {
        const Gates* p = reinterpret_cast<const Gates*>(hr + c * kHrecBytes + kGateOffset);
        gamma_next = *reinterpret_cast<const f32x4*>(&p->gamma[i0]);
        eta_next = *reinterpret_cast<const f32x4*>(&p->eta[i0]);
        beta_next = *reinterpret_cast<const f32x4*>(&p->beta[i0]);
        last_next = p->gamma[kChunk - 1 + zero];
    };
    auto load_tri = [&](int c, int64_t first, bf16x8 (&x)[2][kParts]) {
        const char* p = hr + c * kHrecBytes;
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (tri_has<true>(w, b))
#pragma unroll
                for (int i = 0; i < kParts; ++i) x[b][i] = fragment(p, first + tri_index<true>(w, b) * kParts + i, lane);
    };
    auto load_cols = [&](int c, int set, bf16x8 (&x)[ST][2][NPI]) {
        const char* p = kr + c * krec;
#pragma unroll
        for (int y = 0; y < ST; ++y)
            if (w + 4 * y < 2 * KB)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < NPI; ++i) x[y][b][i] = fragment(p, set * set_frags(KB, NPI) + ((w + 4 * y) * 2 + b) * NPI + i, lane);
    };
    // Columns past V read column 0 and rows behind the end the last one, and are dropped where used: no branches between
    // the loads.
    const int64_t o_step = int64_t(a.Hv) * a.V;
    const int64_t o_at = (s.b * a.T + s.t0 + i0) * o_step + int64_t(hv) * a.V;
    const E* o_lane = static_cast<const E*>(a.d_out) + o_at + (col_in ? col : 0);
    E* dv_lane = static_cast<E*>(a.dv) + o_at + col;
    auto load_do = [&](int c) {
        const E* p = o_lane + c * kChunk * o_step;
        if (c * kChunk + kChunk <= s.len) {
#pragma unroll
            for (int r = 0; r < 4; ++r) dr[r] = p[r * o_step];
        } else {
            const int left = s.len - c * kChunk - 1 - i0;
#pragma unroll
            for (int r = 0; r < 4; ++r) dr[r] = p[(r < left ? r : left) * o_step];
        }
    };
    // Chunk c's dO (in dr) as operands; ga: its gamma.
    auto put_do = [&](int c, const f32x4& ga) {
        f32x4 x;
        bf16x4 o[NPI], p[kParts];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = c * kChunk + i0 + r < s.len && col_in ? float(dr[r]) : 0.f;
        split4(x, o);
        put_parts(&of[c & 1][w >> 1][0][0], 64, lane, w & 1, o);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] *= a.scale * ga[r];
        split4(x, p);
        put_parts(&gf[c & 1][w >> 1][0][0], 64, lane, w & 1, p);
    };
    if (chunks) {
        const int c = chunks - 1;
        load_gates(c);
        load_do(c);
        load_rows(c);
        load_tri(c, kTriFrags, pa);
        load_tri(c, 0, ta);
        load_cols(c, 1, qt);
        load_cols(c, 2, kt);
        put_do(c, gamma_next);
        load_do(c > 0 ? c - 1 : 0);
    }
    __syncthreads();
    for (int c = chunks - 1; c >= 0; --c) {
        const int next = c > 0 ? c - 1 : 0;
        gamma = gamma_next;
        eta = eta_next;
        beta = beta_next;
        last = last_next;
        const int64_t piece = ((hv * a.slots + s.slot + c) * strips + strip) * 256;
        // Phase 1.
        f32x4 acc = zero4(), odd = zero4();       // two sums, so that products need not wait for each other
        {
            bf16x8 x[KB][kParts], o[2][NPI];
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int i = 0; i < kParts; ++i) x[b][i] = sf[b][i][lane];
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<true>(w, b))
#pragma unroll
                    for (int i = 0; i < NPI; ++i) o[b][i] = of[c & 1][b][i][lane];
            load_gates(next);
            float* p = a.ds + piece * (2 * KB) + w * 256 + (4 * g) * 16 + m;
#pragma unroll
            for (int y = 0; y < ST; ++y)
                if (w + 4 * y < 2 * KB)
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[1024 * y + 16 * r] = st[y][r];
#pragma unroll
            for (int b = 0; b < KB; ++b) mma(b & 1 ? odd : acc, ka[b], x[b]);
            acc += odd;
            odd = zero4();
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<true>(w, b)) mma(odd, pa[b], o[b]);
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = a.scale * odd[r] + eta[r] * acc[r];
            bf16x4 q[kParts];
            split4(y, q);
            put_parts(&uf[w >> 1][0][0], 64, lane, w & 1, q);
        }
        load_rows(next);
        load_tri(next, kTriFrags, pa);
        __syncthreads();
        // Phase 2.
        acc = odd = zero4();
        {
            bf16x8 x[2][kParts];
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<true>(w, b))
#pragma unroll
                    for (int i = 0; i < kParts; ++i) x[b][i] = uf[b][i][lane];
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<true>(w, b)) mma(b ? odd : acc, ta[b], x[b]);
            acc += odd;
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = -(gamma[r] * beta[r]) * acc[r];
            bf16x4 q[kParts];
            split4(y, q);
            put_parts(&xf[w >> 1][0][0], 64, lane, w & 1, q);
        }
        load_tri(next, 0, ta);
        {
            float* p = a.x + piece * 4 + w * 256 + (4 * g) * 16 + m;
#pragma unroll
            for (int r = 0; r < 4; ++r) p[16 * r] = acc[r];
        }
        if (a.dv && col_in) {
            E* p = dv_lane + c * kChunk * o_step;
            const int left = s.len - c * kChunk - i0;
            if (left >= 4) {
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r * o_step] = E(beta[r] * acc[r]);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r < left) p[r * o_step] = E(beta[r] * acc[r]);
            }
        }
        if (c > 0) {
            put_do(c - 1, gamma_next);
            load_do(c > 1 ? c - 2 : 0);
        }
        __syncthreads();
        // Phase 3.
#pragma unroll
        for (int y = 0; y < ST; ++y) st[y] *= last;
        {
            bf16x8 x[2][kParts], o[2][kParts];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    o[b][i] = gf[c & 1][b][i][lane];
                    x[b][i] = xf[b][i][lane];
                }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int y = 0; y < ST; ++y)
                    if (w + 4 * y < 2 * KB) mma(st[y], qt[y][b], o[b]);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int y = 0; y < ST; ++y)
                    if (w + 4 * y < 2 * KB) mma(st[y], kt[y][b], x[b]);
        }
        load_cols(next, 1, qt);
        load_cols(next, 2, kt);
        put_state();
        __syncthreads();
    }
    if (a.ds0) {
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = acc_index(w + 4 * x, g) + r;
                if (row < a.K && col_in) a.ds0[state0 + int64_t(row) * a.V + col] = st[x][r];
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
        return hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(256), params, 0, st);
    });
}

}  // namespace qc
