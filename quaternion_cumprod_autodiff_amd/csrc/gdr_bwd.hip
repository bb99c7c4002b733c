// gdr_bwd.hip -- the chunked gated delta rule's backward pass over the chunks
// of a sequence, last to first (gdr_chunk.hpp): the state's cotangent, X, dV.
//
// One block per sequence, value head and 16 columns of V; four waves and the
// memory wave, as in the forward pass.  Per chunk, wave w:
//     phase 1   rows of tile w of dU = P^T O + eta (K dS1)
//     phase 2   rows of tile w of X = T^T dU
//     phase 3   its tiles of dS0 = gamma_last dS1 + Q^T (gamma O) - K^T (gamma b X)
// with a barrier after each.  The memory wave brings dO, as the operands dO and
// scale gamma dO, and takes dS1, X and dV = b X away.  Bound by the chain of
// chunks as the forward pass is: 4 x 4096 tokens of 32 heads of 128, bfloat16,
// 507 us, matrix units 19% in use, LDS 33%, waves at a wait or a barrier 58% of
// the time; 8 x 2048 tokens of 16 heads of 64 by 128, float32, 303.
#include "gdr_chunk.hpp"

namespace qc {
namespace {

template <int DT, int KB, bool VEC, int NS>
__global__ void __launch_bounds__(320 * NS, NS == 2 ? 3 : 1) gdr_bwd_kernel(GdrArgs a, int strips) {
    using E = typename Storage<DT>::type;
    constexpr int NPI = parts_of(DT);
    constexpr int ST = (2 * KB + 3) / 4;
    __shared__ __align__(16) bf16x8 sf_[NS][KB][kParts][64], uf_[NS][2][kParts][64], xf_[NS][2][kParts][64];
    __shared__ __align__(16) bf16x8 of_[NS][2][2][NPI][64], gf_[NS][2][2][kParts][64];      // of this chunk and the next
    __shared__ __align__(16) float db_[NS][16 * kColRow], sb_[NS][2 * KB * kTile], xb_[NS][4 * kTile];
    __shared__ __align__(16) float gates_[NS][2][3][64];                                // gamma, eta and beta of this chunk and the next
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
    const int sub = NS == 1 ? 0 : wave < 4 * NS ? wave >> 2 : wave - 4 * NS;      // which of the block's strips
    auto& sf = sf_[sub];
    auto& uf = uf_[sub];
    auto& xf = xf_[sub];
    auto& of = of_[sub];
    auto& gf = gf_[sub];
    auto& db = db_[sub];
    auto& sb = sb_[sub];
    auto& xb = xb_[sub];
    auto& gates = gates_[sub];
    const int m = lane & 15, g = lane >> 4;
    int64_t n;
    int hv, strip;
    if (!unit_of(a, strips / NS, n, hv, strip)) return;
    strip = strip * NS + sub;
    const Sequence s = sequence(a, n);
    const int chunks = (s.len + kChunk - 1) / kChunk;
    const int hk = hv / a.group;
    constexpr int64_t krec = krec_bytes(KB, NPI);
    const char* kr = a.krec + (hk * a.slots + s.slot) * krec;
    const char* hr = a.hrec + (hv * a.slots + s.slot) * kHrecBytes;

    if (wave >= 4 * NS) {
        const int64_t o_step = int64_t(a.Hv) * a.V, o_at = ((s.b * a.T + s.t0) * a.Hv + hv) * int64_t(a.V);
        const E* d_out = static_cast<const E*>(a.d_out) + o_at;
        E* dv = a.dv ? static_cast<E*>(a.dv) + o_at : nullptr;
        Columns<E, VEC> x;
        float gamma, eta, beta, beta_now = 0.f;
        auto load = [&](int c) {      // rows behind the end read the last one, and are dropped where used
            const int i = c * kChunk + lane;
            x.load(d_out + (i < s.len ? i : s.len - 1) * o_step, strip * 16, a.V);
            const Gates* p = reinterpret_cast<const Gates*>(hr + c * kHrecBytes + kGateOffset);
            gamma = p->gamma[lane];
            eta = p->eta[lane];
            beta = p->beta[lane];
        };
        // What load brought, as the operands dO and scale gamma dO: by token into LDS, by column out of it.
        auto put = [&](int c) {
            gates[c & 1][0][lane] = gamma;
            gates[c & 1][1][lane] = eta;
            gates[c & 1][2][lane] = beta;
            const bool in = c * kChunk + lane < s.len;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float f = x.at(j);
                db[j * kColRow + lane] = in && (VEC || strip * 16 + j < a.V) ? f : 0.f;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float y[8], z[8];
                load_floats<8>(&db[m * kColRow + 32 * b + 8 * g], y);
                load_floats<8>(&gates[c & 1][0][32 * b + 8 * g], z);
                bf16x8 o[NPI], p[kParts];
                split<NPI, 8>(y, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= a.scale * z[e];
                split<kParts, 8>(y, p);
#pragma unroll
                for (int i = 0; i < NPI; ++i) of[c & 1][b][i][lane] = o[i];
#pragma unroll
                for (int i = 0; i < kParts; ++i) gf[c & 1][b][i][lane] = p[i];
            }
        };
        Touch<int(krec)> ahead;
        Tiles<2 * KB> states;
        Tiles<4> xs;
        float y[16];
        const int64_t piece = ((hv * a.slots + s.slot) * strips + strip) * 256;
        float *to_s = a.ds + piece * (2 * KB), *to_x = a.x + piece * 4;
        const float* row = &xb[(2 * (lane >> 5) + ((lane >> 2) & 1)) * kTile + 4 * ((lane & 31) >> 3) + (lane & 3)];      // token `lane`
        auto read_x = [&] {
            xs.read(xb, lane);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = beta_now * row[j * kTileRow];
        };
        auto store_x = [&](int c) {
            xs.store(to_x + int64_t(c) * strips * 1024, lane);
            const int i = c * kChunk + lane;
            if (dv && i < s.len) store_columns<E, VEC>(dv + i * o_step, strip * 16, a.V, y);
        };
        if (chunks) {
            const int c = chunks - 1, then = c > 0 ? c - 1 : 0;
            load(c);
            put(c);
            beta_now = beta;
            load(then);
            ahead.load(kr + then * krec, hr + then * kHrecBytes, strip, strips, lane);
        }
        __syncthreads();
        // Every store follows the loads in its phase: the wait for them, a chunk later, then waits for nothing younger.
        for (int c = chunks - 1; c >= 0; --c) {
            states.read(sb, lane);
            __syncthreads();
            ahead.done();
            const float beta_next = beta;
            if (c > 0) {
                put(c - 1);
                const int then = c > 1 ? c - 2 : 0;
                load(then);
                ahead.load(kr + then * krec, hr + then * kHrecBytes, strip, strips, lane);
            }
            states.store(to_s + int64_t(c) * strips * (2 * KB * 256), lane);
            if (c + 1 < chunks) store_x(c + 1);
            __syncthreads();
            read_x();
            beta_now = beta_next;
            __syncthreads();
        }
        if (chunks) store_x(0);
        return;
    }

    const int i0 = acc_index(w, g);
    const int col = strip * 16 + m;
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
                *reinterpret_cast<f32x4*>(&sb[tile * kTile + m * kTileRow + 4 * g]) = st[x];
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

    bf16x8 ka[KB][NPI], kt[ST][2][NPI], qt[ST][2][NPI], ta[2][kParts], pa[2][kParts];
    auto load_rows = [&](int c) {
        const char* p = kr + c * krec;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < NPI; ++i) ka[b][i] = fragment(p, (w * KB + b) * NPI + i, lane);
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
    // Rows of the chunk's first half need two blocks of T^T and P^T, those of its second half one.
    auto run = [&](auto half) {
        constexpr int B0 = decltype(half)::value ? 1 : 0;
        auto load_tri = [&](int c, int64_t first, bf16x8 (&x)[2][kParts]) {
            const char* p = hr + c * kHrecBytes;
#pragma unroll
            for (int b = B0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < kParts; ++i) x[b][i] = fragment(p, first + tri_index<true>(w, b) * kParts + i, lane);
        };
        if (chunks) {
            load_rows(chunks - 1);
            load_tri(chunks - 1, kTriFrags, pa);
        }
        __syncthreads();
        for (int c = chunks - 1; c >= 0; --c) {
            const int next = c > 0 ? c - 1 : 0;
            const float* gc = &gates[c & 1][0][0];
            // Phase 1.
            load_tri(c, 0, ta);
            f32x4 acc = zero4(), odd = zero4(), po = zero4();       // more than one sum, so that products need not wait for each other
            {
                bf16x8 x[KB][kParts], o[2][NPI];
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < kParts; ++i) x[b][i] = sf[b][i][lane];
#pragma unroll
                for (int b = B0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < NPI; ++i) o[b][i] = of[c & 1][b][i][lane];
#pragma unroll
                for (int b = 0; b < KB; ++b) mma(b & 1 ? odd : acc, ka[b], x[b]);
#pragma unroll
                for (int b = B0; b < 2; ++b) mma(po, pa[b], o[b]);
                acc += odd;
                bf16x4 q[kParts];
                split4(a.scale * po + *reinterpret_cast<const f32x4*>(gc + 64 + i0) * acc, q);
                put_parts(&uf[w >> 1][0][0], 64, lane, w & 1, q);
            }
            __syncthreads();
            // Phase 2.
            load_cols(c, 1, qt);
            load_cols(c, 2, kt);
            acc = odd = zero4();
            {
                bf16x8 x[2][kParts];
#pragma unroll
                for (int b = B0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < kParts; ++i) x[b][i] = uf[b][i][lane];
#pragma unroll
                for (int b = B0; b < 2; ++b) mma(b ? odd : acc, ta[b], x[b]);
                acc += odd;
                *reinterpret_cast<f32x4*>(&xb[w * kTile + m * kTileRow + 4 * g]) = acc;
                bf16x4 q[kParts];
                split4(*reinterpret_cast<const f32x4*>(gc + i0) * *reinterpret_cast<const f32x4*>(gc + 128 + i0) * -acc, q);
                put_parts(&xf[w >> 1][0][0], 64, lane, w & 1, q);
            }
            __syncthreads();
            // Phase 3.
            load_rows(next);
            load_tri(next, kTriFrags, pa);
#pragma unroll
            for (int y = 0; y < ST; ++y) st[y] *= gc[kChunk - 1];
            {
                f32x4 other[ST];
#pragma unroll
                for (int y = 0; y < ST; ++y) other[y] = zero4();
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    bf16x8 x[kParts], o[kParts];
#pragma unroll
                    for (int i = 0; i < kParts; ++i) {
                        o[i] = gf[c & 1][b][i][lane];
                        x[i] = xf[b][i][lane];
                    }
#pragma unroll
                    for (int y = 0; y < ST; ++y)
                        if (w + 4 * y < 2 * KB) {
                            mma(other[y], qt[y][b], o);
                            mma(st[y], kt[y][b], x);
                        }
                }
#pragma unroll
                for (int y = 0; y < ST; ++y) st[y] += other[y];
            }
            put_state();
            __syncthreads();
        }
    };
    if (w >> 1) run(std::true_type{});
    else run(std::false_type{});
    if (a.ds0) {
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = acc_index(w + 4 * x, g) + r;
                if (row < a.K && col < a.V) a.ds0[state0 + int64_t(row) * a.V + col] = st[x][r];
            }
    }
}

}  // namespace

hipError_t launch_gdr_bwd_state(int dt, int kb, const GdrArgs& a, hipStream_t st) {
    if (!a.N) return hipSuccess;
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        constexpr int DT = decltype(d)::value, KB = decltype(k)::value;
        int strips = (a.V + 15) / 16;
        const int ns = strips_per_block(a, strips, DT != 0 || KB <= 2);
        const int64_t blocks = (a.N * a.Hk + 7) / 8 * 8 * (strips / ns) * a.group;
        const bool vec = a.vec_o && a.V % 16 == 0;
        auto pick = [&](auto vc) -> const void* {
            constexpr bool VEC = decltype(vc)::value;
            if constexpr (DT != 0 || KB <= 2)
                if (ns == 2) return reinterpret_cast<const void*>(&gdr_bwd_kernel<DT, KB, VEC, 2>);
            return reinterpret_cast<const void*>(&gdr_bwd_kernel<DT, KB, VEC, 1>);
        };
        const void* fn = vec ? pick(std::true_type{}) : pick(std::false_type{});
        GdrArgs args = a;
        void* params[] = {&args, &strips};
        return hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(320u * ns), params, 0, st);
    });
}

}  // namespace qc
