// gdr_fwd.hip -- the chunked gated delta rule's forward pass over the chunks
// of a sequence (gdr_chunk.hpp).
//
// One block of 4 waves per sequence, value head and 16 columns of V; the
// state's columns never meet, so blocks are independent.  Per chunk, wave w:
//     phase 1   rows of tile w of V - gamma (K S0)
//     phase 2   rows of tile w of U = T b (..), and of gamma (Q S0)
//     phase 3   its tiles of S1 = gamma_last S0 + K^T (eta U), then its rows of out
// with a barrier after each; S0, the bracket and U pass between waves as
// fragments in LDS, where one read of S0 serves both of its products.  What a
// wave multiplies from the left it alone needs, and loads straight into
// registers, ahead of its phase.  A sequence's time is the chain of these
// phases; blocks that share a CU fill each other's gaps.
#include "gdr_chunk.hpp"

namespace qc {
namespace {

template <int DT, int KB, bool SAVE>
__global__ void __launch_bounds__(256, DT == 1 ? 2 : 1) gdr_fwd_kernel(GdrArgs a, int strips) {
    using E = typename Storage<DT>::type;
    constexpr int NPI = parts_of(DT);
    // Parts of S0, P and U that the output takes: two leave 2^-18 of them, far below the half step of bfloat16, 2^-9.
    constexpr int NPO = DT == 1 ? 2 : 3;
    constexpr int ST = (2 * KB + 3) / 4;             // tiles of S of a wave
    __shared__ __align__(16) bf16x8 sf[KB][kParts][64], rf[2][kParts][64], ef[2][kParts][64], uf[2][NPO][64];
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
            st[x][r] = a.s0 && row < a.K && col_in ? a.s0[state0 + int64_t(row) * a.V + col] : 0.f;
        }
    put_state();

    bf16x8 ka[KB][NPI], qa[KB][NPI], kt[ST][2][NPI], ta[2][kParts], pa[2][NPO];
    E vr[4];          // as loaded: a conversion there would wait for the load
    // The gates of the next chunk are loaded a whole chunk ahead: the first of them is needed at the end of phase 1.
    f32x4 gamma, eta, gamma_next, eta_next;
    float last, last_next;
    const int zero = lane_zero();
    auto load_rows = [&](int c, int set, bf16x8 (&x)[KB][NPI]) {
        const char* p = kr + c * krec;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < NPI; ++i) x[b][i] = fragment(p, set * set_frags(KB, NPI) + (w * KB + b) * NPI + i, lane);
    };
    // Columns past V read column 0 and rows behind the end the last one, and are dropped where used: no branches between
    // the loads.
    const int64_t v_step = a.vs[1];
    const E* v_lane = static_cast<const E*>(a.v) + s.b * a.vs[0] + int64_t(hv) * a.vs[2] + (s.t0 + i0) * v_step + (col_in ? col : 0);
    auto load_v = [&](int c) {
        const E* p = v_lane + c * kChunk * v_step;
        if (c * kChunk + kChunk <= s.len) {
#pragma unroll
            for (int r = 0; r < 4; ++r) vr[r] = p[r * v_step];
        } else {
            const int left = s.len - c * kChunk - 1 - i0;
#pragma unroll
            for (int r = 0; r < 4; ++r) vr[r] = p[(r < left ? r : left) * v_step];
        }
    };
    auto load_gates = [&](int c) {
        const Gates* p = reinterpret_cast<const Gates*>(hr + c * kHrecBytes + kGateOffset);
        gamma_next = *reinterpret_cast<const f32x4*>(&p->gamma[i0]);
        eta_next = *reinterpret_cast<const f32x4*>(&p->eta[i0]);
        last_next = p->gamma[kChunk - 1 + zero];
    };
    auto load_t = [&](int c) {
        const char* p = hr + c * kHrecBytes;
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (tri_has<false>(w, b))
#pragma unroll
                for (int i = 0; i < kParts; ++i) ta[b][i] = fragment(p, tri_index<false>(w, b) * kParts + i, lane);
    };
    auto load_p = [&](int c) {
        const char* p = hr + c * kHrecBytes;
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (tri_has<false>(w, b))
#pragma unroll
                for (int i = 0; i < NPO; ++i) pa[b][i] = fragment(p, kTriFrags + tri_index<false>(w, b) * kParts + i, lane);
    };
    auto load_kt = [&](int c) {
        const char* p = kr + c * krec;
#pragma unroll
        for (int x = 0; x < ST; ++x)
            if (w + 4 * x < 2 * KB)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < NPI; ++i) kt[x][b][i] = fragment(p, 2 * set_frags(KB, NPI) + ((w + 4 * x) * 2 + b) * NPI + i, lane);
    };
    const int64_t o_step = int64_t(a.Hv) * a.V;
    E* o_lane = static_cast<E*>(a.out) + (s.b * a.T + s.t0 + i0) * o_step + int64_t(hv) * a.V + col;
    float *save_s = nullptr, *save_u = nullptr;
    if constexpr (SAVE) {
        const int64_t piece = ((hv * a.slots + s.slot) * strips + strip) * 256;
        save_s = a.save_s + piece * (2 * KB) + w * 256 + (4 * g) * 16 + m;
        save_u = a.save_u + piece * 4 + w * 256 + (4 * g) * 16 + m;
    }
    if (chunks) {
        load_rows(0, 0, ka);
        load_v(0);
        load_gates(0);
        load_rows(0, 1, qa);
        load_t(0);
        load_kt(0);
    }
    __syncthreads();
    for (int c = 0; c < chunks; ++c) {
        const int next = c + 1 < chunks ? c + 1 : c;
        gamma = gamma_next;
        eta = eta_next;
        last = last_next;
        // Phase 1.
        bf16x8 x[KB][kParts];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < kParts; ++i) x[b][i] = sf[b][i][lane];
        load_gates(next);
        if constexpr (SAVE) {
#pragma unroll
            for (int y = 0; y < ST; ++y)
                if (w + 4 * y < 2 * KB)
#pragma unroll
                    for (int r = 0; r < 4; ++r) save_s[1024 * y + 16 * r] = st[y][r];
            save_s += int64_t(strips) * (2 * KB) * 256;
        }
        f32x4 acc = zero4(), odd = zero4();       // two sums, so that products need not wait for each other
#pragma unroll
        for (int b = 0; b < KB; ++b) mma(b & 1 ? odd : acc, ka[b], x[b]);
        acc += odd;
        {
            f32x4 y;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool in = c * kChunk + i0 + r < s.len && col_in;
                y[r] = (in ? float(vr[r]) : 0.f) - gamma[r] * acc[r];
            }
            bf16x4 p[kParts];
            split4(y, p);
            put_parts(&rf[w >> 1][0][0], 64, lane, w & 1, p);
        }
        load_rows(next, 0, ka);
        load_v(next);
        __syncthreads();
        // Phase 2.
        f32x4 o = zero4();
        {
            bf16x8 y[2][kParts];
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<false>(w, b))
#pragma unroll
                    for (int i = 0; i < kParts; ++i) y[b][i] = rf[b][i][lane];
            odd = zero4();
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                bf16x8 z[NPO];
#pragma unroll
                for (int i = 0; i < NPO; ++i) z[i] = x[b][i];
                mma(b & 1 ? odd : o, qa[b], z);
            }
            o += odd;
            load_p(c);
            acc = odd = zero4();
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (tri_has<false>(w, b)) mma(b ? odd : acc, ta[b], y[b]);
            acc += odd;
            f32x4 e;
#pragma unroll
            for (int r = 0; r < 4; ++r) e[r] = eta[r] * acc[r];
            bf16x4 p[kParts], q[NPO];
            split4(e, p);
            put_parts(&ef[w >> 1][0][0], 64, lane, w & 1, p);
            split4(acc, q);
            put_parts(&uf[w >> 1][0][0], 64, lane, w & 1, q);
        }
        load_rows(next, 1, qa);
        load_t(next);
        if constexpr (SAVE) {
#pragma unroll
            for (int r = 0; r < 4; ++r) save_u[16 * r] = acc[r];
            save_u += int64_t(strips) * 4 * 256;
        }
        __syncthreads();
        // Phase 3.
#pragma unroll
        for (int y = 0; y < ST; ++y) st[y] *= last;
        {
            bf16x8 y[2][kParts];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < kParts; ++i) y[b][i] = ef[b][i][lane];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int z = 0; z < ST; ++z)
                    if (w + 4 * z < 2 * KB) mma(st[z], kt[z][b], y[b]);
        }
        load_kt(next);
        put_state();
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] *= gamma[r];
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (tri_has<false>(w, b)) {
                bf16x8 y[NPO];
#pragma unroll
                for (int i = 0; i < NPO; ++i) y[i] = uf[b][i][lane];
                mma(o, pa[b], y);
            }
        if (col_in) {
            E* p = o_lane + c * kChunk * o_step;
            const int left = s.len - c * kChunk - i0;
            if (left >= 4) {
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r * o_step] = E(a.scale * o[r]);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r < left) p[r * o_step] = E(a.scale * o[r]);
            }
        }
        __syncthreads();
    }
    if (a.fin) {
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = acc_index(w + 4 * x, g) + r;
                if (row < a.K && col_in) a.fin[state0 + int64_t(row) * a.V + col] = st[x][r];
            }
    }
}

}  // namespace

hipError_t launch_gdr_fwd(int dt, int kb, bool save, const GdrArgs& a, hipStream_t st) {
    if (!a.N) return hipSuccess;
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        constexpr int DT = decltype(d)::value, KB = decltype(k)::value;
        int strips = (a.V + 15) / 16;
        const int64_t blocks = (a.N * a.Hk + 7) / 8 * 8 * strips * a.group;
        const void* fn = save ? reinterpret_cast<const void*>(&gdr_fwd_kernel<DT, KB, true>)
                              : reinterpret_cast<const void*>(&gdr_fwd_kernel<DT, KB, false>);
        GdrArgs args = a;
        void* params[] = {&args, &strips};
        return hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(256), params, 0, st);
    });
}

}  // namespace qc
