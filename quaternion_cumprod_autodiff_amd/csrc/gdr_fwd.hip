// gdr_fwd.hip -- the chunked gated delta rule's forward pass over the chunks
// of a sequence (gdr_chunk.hpp).
//
// One block per sequence, value head and 16 columns of V; the state's columns
// never meet, so blocks are independent.  Four waves and the memory wave; per
// chunk, wave w:
//     phase 1   rows of tile w of V - gamma (K S0)
//     phase 2   rows of tile w of U = T b (..), and of gamma (Q S0)
//     phase 3   its tiles of S1 = gamma_last S0 + K^T (eta U), then its rows of out
// with a barrier after each; S0, the bracket and U pass between waves as
// fragments in LDS, where one read of S0 serves both of its products.  What a
// wave multiplies from the left it alone needs, and loads straight into
// registers, ahead of its phase, out of an L2 that the memory wave's touches
// fill two chunks before; V, out and what is saved go through the memory wave.
//
// Bound by the chain of a sequence's chunks, not by bytes: a chunk is three
// barriers with reads of LDS, MFMAs and splits of their results between them,
// about 2 us for heads of 128 in bfloat16.  Counters: matrix units 21% in use,
// LDS 26%, waves at a wait or a barrier 43% of the time (two strips to a block:
// 20, 31 and 60%).  8192 tokens of 32 heads, 128 chunks in line, 255 us; 12001
// tokens of 16 heads in 29 packed sequences 216; 4 x 4096 of 32 heads, saving
// states, 526, two rounds of blocks.  Registers: K = 128 in float32 spills 19 to
// 27.  Set aside, measured on earlier forms of this kernel: eight waves of half
// the columns' rows (more reads of LDS for the same products, slower); no
// touches (431 us became 480 with the factors); 128 registers, for two blocks
// to a CU (spills: 515 became 780).
#include "gdr_chunk.hpp"

namespace qc {
namespace {

template <int DT, int KB, bool SAVE, bool VEC, int NS>
__global__ void __launch_bounds__(320 * NS, NS == 2 ? 3 : 1) gdr_fwd_kernel(GdrArgs a, int strips) {
    using E = typename Storage<DT>::type;
    constexpr int NPI = parts_of(DT);
    constexpr int ST = (2 * KB + 3) / 4;             // tiles of S of a wave
    __shared__ __align__(16) bf16x8 sf_[NS][KB][kParts][64], rf_[NS][2][kParts][64], ef_[NS][2][kParts][64], uf_[NS][2][kParts][64];
    __shared__ __align__(16) float vb_[NS][16 * kColRow], ob_[NS][16 * kColRow], sb_[NS][SAVE ? 2 * KB * kTile : 4], ub_[NS][SAVE ? 4 * kTile : 4];
    __shared__ __align__(16) float gates_[NS][2][2][64];      // gamma and eta of this chunk and the next
    __shared__ float last_[NS][2][16];                        // gamma_last by column: NaN where an input is not finite
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
    const int sub = NS == 1 ? 0 : wave < 4 * NS ? wave >> 2 : wave - 4 * NS;      // which of the block's strips
    auto& sf = sf_[sub];
    auto& rf = rf_[sub];
    auto& ef = ef_[sub];
    auto& uf = uf_[sub];
    auto& vb = vb_[sub];
    auto& ob = ob_[sub];
    auto& sb = sb_[sub];
    auto& ub = ub_[sub];
    auto& gates = gates_[sub];
    auto& last = last_[sub];
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
        const E* v = static_cast<const E*>(a.v) + s.b * a.vs[0] + s.t0 * a.vs[1] + int64_t(hv) * a.vs[2];
        E* out = static_cast<E*>(a.out) + ((s.b * a.T + s.t0) * a.Hv + hv) * int64_t(a.V);
        const int64_t v_step = a.vs[1], o_step = int64_t(a.Hv) * a.V;
        Columns<E, VEC> x;
        auto load_v = [&](int c) {      // rows behind the end read the last one, and are dropped where used
            const int i = c * kChunk + lane;
            x.load(v + (i < s.len ? i : s.len - 1) * v_step, strip * 16, a.V);
        };
        float gamma, eta, key_poison;
        // Columns (bits) in which this lane's token comes at or behind an input that is not finite: of the chunk whose
        // outputs are stored next, of the one in work, of the one to come.
        uint32_t gone_out = 0, gone = 0, gone_next = 0;
        // V as it enters, columns and tokens that are none as zero.  With one strip to a block this is done in phase 1, where
        // the memory wave is early, with two in phase 2, where the strips' waves hide it and phase 1 would wait for V:
        // 8192 tokens of 32 heads 255 us so and 272 the other way, 12001 packed tokens of 16 heads 216 and 220, 4 x 4096 of
        // 32 heads, saving states, 542 and 552.
        float f[16], of_column;
        auto take_v = [&](int c) {
            const bool in = c * kChunk + lane < s.len;
            float sum[4] = {key_poison, 0.f, 0.f, 0.f};
            of_column = __shfl(gamma, kChunk - 1, 64);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float z = x.at(j);
                f[j] = in && (VEC || strip * 16 + j < a.V) ? z : 0.f;
                sum[j % 4] = fmaf(f[j], 0.f, sum[j % 4]);
            }
            gone_next = 0;
            if (__any(sum[0] + sum[1] + (sum[2] + sum[3]) != 0.f)) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const bool bad = fmaf(f[j], 0.f, key_poison) != 0.f;      // NaN too
                    const uint64_t mask = __ballot(bad);
                    if (mask) {
                        gone_next |= uint32_t(lane >= __builtin_ctzll(mask)) << j;
                        f[j] = f[j] * 0.f == 0.f ? f[j] : 0.f;
                        if (lane == j) of_column = __builtin_nanf("");
                    }
                }
            }
        };
        auto put_v = [&](int c) {
#pragma unroll
            for (int j = 0; j < 16; ++j) vb[j * kColRow + lane] = f[j];
            if (lane < 16) last[c & 1][lane] = of_column;
        };
        float y[16];
        auto read_out = [&] {
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = a.scale * ob[j * kColRow + lane];
        };
        auto store_out = [&](int c) {
            const int i = c * kChunk + lane;
            if (__any(gone_out))
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = gone_out >> j & 1 ? __builtin_nanf("") : y[j];
            if (i < s.len) store_columns<E, VEC>(out + i * o_step, strip * 16, a.V, y);
        };
        auto load_gates = [&](int c) {
            const Gates* p = reinterpret_cast<const Gates*>(hr + c * kHrecBytes + kGateOffset);
            gamma = p->gamma[lane];
            eta = p->eta[lane];
            key_poison = p->poison[lane];
        };
        auto put_gates = [&](int c) {
            gates[c & 1][0][lane] = gamma;
            gates[c & 1][1][lane] = eta;
        };
        Touch<int(krec)> ahead;
        if (chunks) {
            load_v(0);
            load_gates(0);
            take_v(0);
            put_v(0);
            gone = gone_next;
            put_gates(0);
            load_v(chunks > 1 ? 1 : 0);
            load_gates(chunks > 1 ? 1 : 0);
            if (chunks > 1) ahead.load(kr + krec, hr + kHrecBytes, strip, strips, lane);
        }
        __syncthreads();
        // Every store follows the loads of V in its phase: the wait for V, a chunk later, then waits for nothing younger.
        Tiles<SAVE ? 2 * KB : 1> states;
        Tiles<SAVE ? 4 : 1> updates;
        float *to_s = nullptr, *to_u = nullptr;
        if constexpr (SAVE) {
            const int64_t piece = ((hv * a.slots + s.slot) * strips + strip) * 256;
            to_s = a.save_s + piece * (2 * KB);
            to_u = a.save_u + piece * 4;
        }
        for (int c = 0; c < chunks; ++c) {
            if (c) read_out();
            if (NS == 1 && c + 1 < chunks) take_v(c + 1);
            if constexpr (SAVE) states.read(sb, lane);
            __syncthreads();
            ahead.done();
            if (c + 1 < chunks) {
                if (NS == 2) take_v(c + 1);
                put_v(c + 1);
                put_gates(c + 1);
                const int then = c + 2 < chunks ? c + 2 : c + 1;
                load_v(then);
                load_gates(then);
                ahead.load(kr + then * krec, hr + then * kHrecBytes, strip, strips, lane);
            }
            if (c) store_out(c - 1);
            if constexpr (SAVE) {
                states.store(to_s + int64_t(c) * strips * (2 * KB * 256), lane);
                if (c) updates.store(to_u + int64_t(c - 1) * strips * 1024, lane);
            }
            __syncthreads();
            if constexpr (SAVE) {
                if (__any(gone)) {      // U as the backward pass has to find it
                    float* row = &ub[(2 * (lane >> 5) + ((lane >> 2) & 1)) * kTile + 4 * ((lane & 31) >> 3) + (lane & 3)];      // token `lane`
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (gone >> j & 1) row[j * kTileRow] = __builtin_nanf("");
                }
                updates.read(ub, lane);
            }
            gone_out = gone;
            gone = gone_next;
            __syncthreads();
        }
        if (chunks) {
            read_out();
            store_out(chunks - 1);
            if constexpr (SAVE) updates.store(to_u + int64_t(chunks - 1) * strips * 1024, lane);
        }
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
                if constexpr (SAVE) *reinterpret_cast<f32x4*>(&sb[tile * kTile + m * kTileRow + 4 * g]) = st[x];
            }
        }
    };
#pragma unroll
    for (int x = 0; x < ST; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = acc_index(w + 4 * x, g) + r;
            st[x][r] = a.s0 && row < a.K && col < a.V ? a.s0[state0 + int64_t(row) * a.V + col] : 0.f;
        }
    put_state();

    bf16x8 ka[KB][NPI], qa[KB][NPI], kt[ST][2][NPI], ta[2][kParts], pa[2][kParts];
    auto load_rows = [&](int c, int set, bf16x8 (&x)[KB][NPI]) {
        const char* p = kr + c * krec;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < NPI; ++i) x[b][i] = fragment(p, set * set_frags(KB, NPI) + (w * KB + b) * NPI + i, lane);
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
    if (chunks) {
        load_rows(0, 0, ka);
        load_rows(0, 1, qa);
    }
    __syncthreads();
    // Rows of the chunk's first half need one block of T and P, those of its second half two.
    auto run = [&](auto half) {
        constexpr bool HI = decltype(half)::value;
        auto load_t = [&](int c) {
            const char* p = hr + c * kHrecBytes;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if ((b == 0 || HI))
#pragma unroll
                    for (int i = 0; i < kParts; ++i) ta[b][i] = fragment(p, tri_index<false>(w, b) * kParts + i, lane);
        };
        auto load_p = [&](int c) {
            const char* p = hr + c * kHrecBytes;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if ((b == 0 || HI))
#pragma unroll
                    for (int i = 0; i < kParts; ++i) pa[b][i] = fragment(p, kTriFrags + tri_index<false>(w, b) * kParts + i, lane);
        };
        for (int c = 0; c < chunks; ++c) {
            const int next = c + 1 < chunks ? c + 1 : c;
            // Phase 1.  The two products share the reads of S0, and fill each other's waits.
            f32x4 acc = zero4(), odd = zero4(), o = zero4(), o_odd = zero4();
            load_t(c);
            const float* gc = &gates[c & 1][0][0];
            const f32x4 gamma = *reinterpret_cast<const f32x4*>(gc + i0);
            {
                bf16x8 x[KB][kParts];
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int i = 0; i < kParts; ++i) x[b][i] = sf[b][i][lane];
                const f32x4 v = *reinterpret_cast<const f32x4*>(&vb[m * kColRow + i0]);
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    mma(b & 1 ? odd : acc, ka[b], x[b]);
                    mma(b & 1 ? o_odd : o, qa[b], x[b]);
                }
                acc += odd;
                bf16x4 p[kParts];
                split4(v - gamma * acc, p);
                put_parts(&rf[w >> 1][0][0], 64, lane, w & 1, p);
            }
            __syncthreads();
            // Phase 2.
            const float gamma_last = last[c & 1][m];
            load_kt(c);
            load_p(c);
            {
                bf16x8 y[2][kParts];
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if ((b == 0 || HI))
#pragma unroll
                        for (int i = 0; i < kParts; ++i) y[b][i] = rf[b][i][lane];
                o = (o + o_odd) * gamma;
                acc = odd = zero4();
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if ((b == 0 || HI)) mma(b ? odd : acc, ta[b], y[b]);
                acc += odd;
                bf16x4 p[kParts], q[kParts];
                split4(*reinterpret_cast<const f32x4*>(gc + 64 + i0) * acc, p);
                put_parts(&ef[w >> 1][0][0], 64, lane, w & 1, p);
                split4(acc, q);
                put_parts(&uf[w >> 1][0][0], 64, lane, w & 1, q);
                if constexpr (SAVE) *reinterpret_cast<f32x4*>(&ub[w * kTile + m * kTileRow + 4 * g]) = acc;
            }
            __syncthreads();
            // Phase 3.
            load_rows(next, 0, ka);
            load_rows(next, 1, qa);
#pragma unroll
            for (int y = 0; y < ST; ++y) st[y] *= gamma_last;
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
            put_state();
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if ((b == 0 || HI)) {
                    bf16x8 y[kParts];
#pragma unroll
                    for (int i = 0; i < kParts; ++i) y[i] = uf[b][i][lane];
                    mma(o, pa[b], y);
                }
            *reinterpret_cast<f32x4*>(&ob[m * kColRow + i0]) = o;
            __syncthreads();
        }
    };
    if (w >> 1) run(std::true_type{});
    else run(std::false_type{});
    if (a.fin) {
#pragma unroll
        for (int x = 0; x < ST; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = acc_index(w + 4 * x, g) + r;
                if (row < a.K && col < a.V) a.fin[state0 + int64_t(row) * a.V + col] = st[x][r];
            }
    }
}

}  // namespace

hipError_t launch_gdr_fwd(int dt, int kb, bool save, const GdrArgs& a, hipStream_t st) {
    if (!a.N) return hipSuccess;
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        constexpr int DT = decltype(d)::value, KB = decltype(k)::value;
        int strips = (a.V + 15) / 16;
        const int ns = strips_per_block(a, strips, DT == 1 || KB <= 2);
        const int64_t blocks = (a.N * a.Hk + 7) / 8 * 8 * (strips / ns) * a.group;
        const bool vec = a.vec_v && a.vec_o && a.V % 16 == 0;
        auto pick = [&](auto sv, auto vc) -> const void* {
            constexpr bool SAVE = decltype(sv)::value, VEC = decltype(vc)::value;
            if constexpr (DT == 1 || KB <= 2)
                if (ns == 2) return reinterpret_cast<const void*>(&gdr_fwd_kernel<DT, KB, SAVE, VEC, 2>);
            return reinterpret_cast<const void*>(&gdr_fwd_kernel<DT, KB, SAVE, VEC, 1>);
        };
        const std::true_type yes;
        const std::false_type no;
        const void* fn = save ? (vec ? pick(yes, yes) : pick(yes, no)) : (vec ? pick(no, yes) : pick(no, no));
        GdrArgs args = a;
        void* params[] = {&args, &strips};
        return hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(320u * ns), params, 0, st);
    });
}

}  // namespace qc
