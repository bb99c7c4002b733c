// gdr_chunk.hpp -- the chunked form of the gated delta rule
// (include/gated_delta.h): its mathematics, its internal formats and the
// device helpers that its kernels share.  Not installed.
//
// Chunks of C = 64 tokens.  With G_i the log decays cumulated from the chunk's
// start, gamma_i = exp(G_i), Gam_ij = exp(G_i - G_j), S0 the state before the
// chunk, and q, k, v, b the chunk's rows, the updates u_i = b_i (v_i - ...) of
// the recurrence solve a unit lower triangular system, so that
//     L_ij = Gam_ij k_i.k_j (i > j),   T = (I + diag(b) L)^-1,   P_ij = Gam_ij q_i.k_j (i >= j)
//     U   = T diag(b) (V - gamma (K S0))                       the updates u, [C, V]
//     out = scale (gamma (Q S0) + P U)
//     S1  = gamma_last S0 + K^T (eta U),   eta_i = exp(G_last - G_i)
// and, for cotangents dO of out (O = scale dO) and dS1 of S1,
//     dU  = P^T O + eta (K dS1),   X = T^T dU,   dV = b X
//     dS0 = gamma_last dS1 + Q^T (gamma O) - K^T (gamma b X)
//     Phi_ij = Gam_ij O_i.U_j (i >= j),   Psi_ij = -b_i Gam_ij X_i.U_j (i > j)
//     dQ  = gamma (O S0^T) + Phi K
//     dKr = -gamma b (X S0^T) + Psi K         (k as the reader of the state)
//     dKw = eta (U dS1^T) + Phi^T Q + Psi^T K   (k as its writer),   dK = dKr + dKw
//     db_i = X_i.v_i - gamma_i k_i.(X S0^T)_i - sum_j (X_i.U_j) L_ij
//     dg_t = gamma_last <S0, dS1> + sum_{i >= t} gamma_i (scale q_i.(dO S0^T)_i - b_i k_i.(X S0^T)_i)
//            + sum_{j < t} eta_j k_j.(U dS1^T)_j + sum_{i >= t > j} M_ij,
//     M_ij = scale (dO_i.U_j) P_ij - b_i (X_i.U_j) L_ij
// Non-finite inputs, forward.  In these products a token's NaN or infinity
// would meet the zeros across the diagonal and reach the tokens before it.  So
// a key, gate or value that is not finite enters as zero, and the places it
// reaches by the recurrence, its own token and all later ones (a value: in its
// column), become NaN at the end: poison in Gates, and the forward pass'
// memory wave.  Queries reach their own token alone as it is.
// All exponents are of differences that decays keep at or below zero.  Every
// term of dg_t carries exp(g_t): with q_i.dQ_i + k_i.dKr_i - k_i.dKw_i summed
// over i >= t, terms of order 1 would have to cancel, and a strong decay's
// gradient would be their rounding.
//
// Kernels: gdr_factor (T, P and the operands' layouts, every chunk at once),
// gdr_fwd and gdr_bwd_state (the states pass from chunk to chunk: one block per
// 16 or 32 columns of V, everything else of a chunk in the same pass),
// gdr_grad (the gradients of q, k, gates, every chunk at once).
//
// Arithmetic.  All products are v_mfma_f32_16x16x32_bf16 on operands split
// into bfloat16 parts: bfloat16 inputs are one part, float16 two, float32 and
// every computed operand three, all exact to 24 bits; of two operands' parts
// i and j the products with i + j < 3 are summed, in float32.  So float32
// accuracy costs 3 to 6 of these instructions, against 16 times one for the
// float32 MFMA.
//
// Layouts.  A lane l = 16 g + m holds of an operand fragment (64 lanes x 8
// bfloat16, 1 KiB, stored lane by lane): row m (A) or column m (B), and the 8
// consecutive indices 32 b + 8 g + .. of the contracted axis' block b.  A
// product's accumulators hold column m and rows 4 g + 0..3.  Rows of tile r of
// an axis stand for the indices 32 (r / 2) + 8 (m / 4) + 4 (r % 2) + m % 4 of
// it, so that the accumulators of tiles 2b and 2b + 1 are, in place, the 8
// consecutive indices of a B fragment's block b: results become operands
// without a transpose.  S0, U, X and dS1 go through memory as pieces of 16
// columns of V, [Hv][slots][VP / 16][tiles][16 rows][16 columns] float32: what
// one block writes of a chunk is whole lines, and 8 columns of a row are 32
// bytes of one.
#pragma once

#include "gdr_internal.hpp"

#include <type_traits>

namespace qc {

constexpr int kChunk = 64;
constexpr int kParts = 3;

constexpr int parts_of(int dt) { return dt == 0 ? 3 : dt == 1 ? 1 : 2; }

// Fragments of one operand set of a chunk: 4 row tiles x KB blocks of K (or
// 2 KB tiles of K x 2 blocks of tokens) x parts.
constexpr int64_t kFrag = 512;                                        // bfloat16 of a fragment
constexpr int64_t set_frags(int kb, int npi) { return int64_t(4) * kb * npi; }
// Per chunk and key head: three sets (forward K rows, Q rows, K transposed;
// backward K rows, Q transposed, K transposed).
constexpr int64_t krec_bytes(int kb, int npi) { return 3 * set_frags(kb, npi) * kFrag * 2; }
// Per chunk and value head: T and P (backward: transposed), 6 fragments of
// non-zero 16 x 32 blocks x 3 parts each; gates.
constexpr int64_t kTriFrags = 6 * kParts;
struct Gates {
    float gamma[kChunk], eta[kChunk], beta[kChunk];
    float poison[kChunk];        // forward: NaN from the first token on whose key or gates are not finite, else 0
    double cum[kChunk];
};
constexpr int64_t kGateOffset = 2 * kTriFrags * kFrag * 2;
constexpr int64_t kHrecBytes = (kGateOffset + int64_t(sizeof(Gates)) + 4095) / 4096 * 4096;

struct GdrArgs {
    const void *q, *k, *v;
    const float *g, *b, *s0;
    const int32_t* offsets;
    void* out;
    float* fin;
    // By head, then by chunk: a block of the passes over a sequence walks through memory, not across it.
    char *krec, *hrec;                 // workspace: [Hk][slots] and [Hv][slots] records
    float *save_s, *save_u;            // saved: S0 and U, pieces (below) of 2 KB and 4 tiles (or null)
    const void* d_out;
    const float* d_fin;
    void *dq, *dk, *dv;
    float *dg, *db, *ds0;
    float *x, *ds;                     // workspace: X and dS1, as U and S0
    int64_t qs[3], ks[3], vs[3];
    int64_t T, slots, N, chunks;       // chunks: per sequence, without offsets
    int Hk, Hv, group, K, V, VP;
    int vec_qk, vec_v, vec_o;          // query and key, value, and out (d_out, dv) rows: on 16 bytes, sizes multiples of 8 (16 for V in the passes)
    float scale;
};

hipError_t launch_gdr_factor(int dt, int kb, bool bwd, const GdrArgs& a, hipStream_t st);
hipError_t launch_gdr_fwd(int dt, int kb, bool save, const GdrArgs& a, hipStream_t st);
hipError_t launch_gdr_bwd_state(int dt, int kb, const GdrArgs& a, hipStream_t st);
hipError_t launch_gdr_grad(int dt, int kb, const GdrArgs& a, hipStream_t st);

// Calls f(dtype, blocks of K) with both as constants.
template <class F>
hipError_t by_dtype_kb(int dt, int kb, F&& f) {
    auto with = [&](auto d) {
        if (kb == 1) return f(d, std::integral_constant<int, 1>{});
        if (kb == 2) return f(d, std::integral_constant<int, 2>{});
        return f(d, std::integral_constant<int, 4>{});
    };
    if (dt == 0) return with(std::integral_constant<int, 0>{});
    if (dt == 1) return with(std::integral_constant<int, 1>{});
    return with(std::integral_constant<int, 2>{});
}

// Device helpers ----------------------------------------------------------------

// Index within an axis of row m of tile r (see Layouts).
__device__ __forceinline__ int tile_index(int r, int m) { return 32 * (r >> 1) + 8 * (m >> 2) + 4 * (r & 1) + (m & 3); }
// First of the four consecutive indices that a lane's accumulators of tile r hold.
__device__ __forceinline__ int acc_index(int r, int g) { return 32 * (r >> 1) + 8 * g + 4 * (r & 1); }

struct Sequence {
    int64_t b, t0, slot;
    int len;
};

__device__ __forceinline__ Sequence sequence(const GdrArgs& a, int64_t n) {
    if (!a.offsets) return {n, 0, n * a.chunks, int(a.T)};
    int64_t lo = a.offsets[n], hi = a.offsets[n + 1];
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    hi = hi < lo ? lo : hi > a.T ? a.T : hi;
    // Sequence n's chunks take the slots from lo / 64 + n: consecutive sequences cannot meet, since
    // floor((lo + len) / 64) + 1 >= floor(lo / 64) + ceil(len / 64); the last slot is below T / 64 + N.
    return {0, lo, lo / kChunk + n, int(hi - lo)};
}

// The sequence a chunk slot belongs to (-1: none), and its chunk there.
__device__ __forceinline__ int64_t slot_sequence(const GdrArgs& a, int64_t slot, Sequence& s, int& chunk) {
    int64_t n;
    if (!a.offsets) {
        n = slot / a.chunks;
    } else {
        int64_t lo = 0, hi = a.N - 1;       // the last n whose first slot is at or before this one
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (sequence(a, mid).slot <= slot) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
    }
    s = sequence(a, n);
    if (slot < s.slot || (slot - s.slot) * kChunk >= s.len) return -1;
    chunk = int(slot - s.slot);
    return n;
}

// x as NP bfloat16 parts, each the rounding of what the ones before leave: one
// leaves 2^-9 of x, two 2^-18, three nothing of its 24 bits.
template <int NP, int W, class Vec>
__device__ __forceinline__ void split(const float (&x)[W], Vec (&p)[NP]) {
    static_assert(W % 2 == 0, "pairs");
    typedef uint32_t Words __attribute__((ext_vector_type(W / 2)));
    typedef __bf16 Pair __attribute__((ext_vector_type(2)));
    Words out[NP];
#pragma unroll
    for (int j = 0; j < W; j += 2) {
        float a = x[j], b = x[j + 1];
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const Pair h = {__bf16(a), __bf16(b)};
            uint32_t u = __builtin_bit_cast(uint32_t, h);
            asm("" : "+v"(u));      // one conversion for both, taken apart by a shift and a mask: left alone, the compiler converts twice
            out[n][j / 2] = u;
            if (n + 1 < NP) {
                a -= __uint_as_float(u << 16);
                b -= __uint_as_float(u & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) p[n] = __builtin_bit_cast(Vec, out[n]);
}

template <int NP>
__device__ __forceinline__ void split4(const f32x4& x, bf16x4 (&p)[NP]) {
    const float v[4] = {x[0], x[1], x[2], x[3]};
    split<NP, 4>(v, p);
}

// acc += A B over one block of 32, the smallest products first.
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const bf16x8 (&a)[NA], const bf16x8 (&b)[NB]) {
#pragma unroll
    for (int s = NA + NB - 2; s >= 0; --s) {
        if (s >= kParts) continue;
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < NB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc, 0, 0, 0);
        }
    }
}

// A lane's share of fragment f of a record (base and f the wave's: one address
// register per lane serves all).
__device__ __forceinline__ bf16x8 fragment(const char* base, int64_t f, int lane) {
    return reinterpret_cast<const bf16x8*>(base + f * (kFrag * 2))[uint32_t(lane)];
}

// Whether any of eight bfloat16 is infinite or NaN: 0x7f80, their exponent bits, plus 0x80 is 0x8000.
__device__ __forceinline__ bool not_finite(const bf16x8& x) {
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    const Words u = __builtin_bit_cast(Words, x);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top |= (u[i] & 0x7f807f80u) + 0x00800080u;
    return top & 0x80008000u;
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// Eight elements from p on, those past `left` as zero, as exact parts.
template <int DT>
__device__ __forceinline__ void load_parts(const typename Storage<DT>::type* p, int left, bool vec, bf16x8 (&x)[parts_of(DT)]) {
    if constexpr (DT == 1) {
        bf16x8 v;
        if (vec) {
            if (left >= 8) v = *reinterpret_cast<const bf16x8*>(p);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __bf16(0.f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : __bf16(0.f);
        }
        x[0] = v;
    } else {
        float v[8];
        if (vec && left >= 8) {
            load_floats<8>(p, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = !vec && j < left ? float(p[j]) : 0.f;
        }
        split<parts_of(DT), 8>(v, x);
    }
}

// Fragments of T or P before row tile r in its record, and its blocks of
// tokens: those at or before the rows (forward), at or behind them (backward).
template <bool BWD> __device__ __forceinline__ int tri_first(int r) {
    return BWD ? (r < 2 ? 2 * r : r + 2) : (r < 2 ? r : 2 * r - 2);
}
template <bool BWD> __device__ __forceinline__ bool tri_has(int r, int b) { return BWD ? b >= (r >> 1) : b <= (r >> 1); }
template <bool BWD> __device__ __forceinline__ int tri_index(int r, int b) { return tri_first<BWD>(r) + (BWD ? b - (r >> 1) : b); }

// The passes over a sequence: blocks of all the columns and heads that share a
// key head run on one XCD (block % 8), where they share its fragments in L2.
__device__ __forceinline__ bool unit_of(const GdrArgs& a, int strips, int64_t& n, int& hv, int& strip) {      // strip: of `strips` blocks
    const int per = strips * a.group;
    const int64_t u = blockIdx.x / (8 * int64_t(per)) * 8 + blockIdx.x % 8;
    const int s = int(blockIdx.x / 8 % per);
    if (u >= a.N * a.Hk) return false;
    n = u / a.Hk;
    hv = int(u % a.Hk) * a.group + s / strips;
    strip = s % strips;
    return true;
}

// Four indices' parts into one half of a lane's place in a fragment (stride: between the parts' fragments, in lanes).
template <int NP>
__device__ __forceinline__ void put_parts(bf16x8* frag, int stride, int lane, int half, const bf16x4 (&p)[NP]) {
#pragma unroll
    for (int n = 0; n < NP; ++n) reinterpret_cast<bf16x4*>(frag + n * stride + lane)[half] = p[n];
}

// Strips of 16 columns to a block of the passes over a sequence.  With one, five
// waves are all that a busy CU was measured to hold (forward, K = 128: registers
// for two waves to a SIMD; backward: a second block's registers and LDS would
// fit), and they wait for each other three times a chunk.  So where strips are
// more than CUs and pair up, a block takes two, ten waves in step, and the
// second strip finds operands in L1: of 4 x 4096 tokens of 32 heads of 128,
// bfloat16, saving states, 56 million reads go on to L2 with one strip, 31 with
// two.  Kernels, one strip and two: that forward pass 606 us and 526, its
// backward 663 and 507; 12001 tokens of 16 heads in 29 packed sequences 255 and
// 216; 8 x 2048 tokens of 16 heads, V = 128, forward and backward, float32
// K = 32: 281 and 246, 338 and 276; K = 64: 321 and 310, 347 and 303; float16
// K = 64: 287 and 258, 321 and 265; K = 128 backward 415 and 359.  Up to 256
// strips each has a CU to itself, and two to a block would leave CUs idle.
// fits: three waves to a SIMD have the registers they need, 168 (float32 K = 64
// spills 3 where no states are saved); more parts of longer keys take up to 256.
inline int strips_per_block(const GdrArgs& a, int strips, bool fits) {
    return fits && strips % 2 == 0 && a.N * a.Hv * strips > 256 ? 2 : 1;
}

// The memory wave of the passes over a sequence -----------------------------------
//
// A fifth wave moves a block's 16 columns between memory and LDS.  Stores wait
// in the same queue as loads, so that a wave which stores would wait for its
// stores at its next operand; and the columns' addresses, ends and conversions
// stay out of the chain.  Between it and the others, columns lie in LDS by
// column: [16][kColRow] floats of 64 tokens, where lane (g, m) finds 4 tokens
// of column m in 16 bytes and the memory wave's lane t token t of each column.
constexpr int kColRow = 68;
// A 16 x 16 tile there: column m's rows 4 g .. in 16 bytes.
constexpr int kTileRow = 20, kTile = 16 * kTileRow;

// Token row p's 16 columns from `first` on, as they lie in memory (elements
// are taken apart where they are used, so that nothing waits here).  VEC: whole
// 16-byte pieces, all columns there; else columns past `size` read column 0.
template <class E, bool VEC>
struct Columns {
    static constexpr int kWords = 16 * sizeof(E) / 4, kPer = 4 / sizeof(E);
    typedef uint32_t Piece __attribute__((ext_vector_type(4)));
    Piece x[kWords / 4];

    __device__ __forceinline__ void load(const E* p, int first, int size) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) x[i] = reinterpret_cast<const Piece*>(p + first)[i];
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                uint32_t u = 0;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int c = first + i * kPer + j;
                    const E e = p[c < size ? c : 0];
                    if constexpr (kPer == 1) u = __builtin_bit_cast(uint32_t, e);
                    else u |= uint32_t(__builtin_bit_cast(uint16_t, e)) << (16 * j);
                }
                x[i / 4][i % 4] = u;
            }
        }
    }

    __device__ __forceinline__ float at(int j) const {
        const uint32_t u = x[j / kPer / 4][j / kPer % 4];
        if constexpr (kPer == 1) return __builtin_bit_cast(float, u);
        else return float(__builtin_bit_cast(E, uint16_t(u >> (16 * (j % kPer)))));
    }
};

template <class E, bool VEC>
__device__ __forceinline__ void store_columns(E* p, int first, int size, const float (&x)[16]) {
    if constexpr (VEC) {
        store_floats<16>(p + first, x);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (first + j < size) p[first + j] = E(x[j]);
    }
}

// The other waves load their operands one phase ahead, from L2: the memory
// wave has them there by then, touching the lines of the records two chunks on
// (4 KiB at a time, the strips of a head in turn; with few strips the last of
// them come from further away).
template <int K_BYTES>
struct Touch {
    static constexpr int kTurns = 4, kUnits = K_BYTES / 4096 + int(kHrecBytes / 4096);
    int x[kTurns] = {};

    __device__ __forceinline__ void load(const char* krec, const char* hrec, int strip, int strips, int lane) {
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            int u = strip + j * strips;
            u = u < kUnits ? u : kUnits - 1;
            const char* p = u < K_BYTES / 4096 ? krec + u * 4096 : hrec + (u - K_BYTES / 4096) * 4096;
            x[j] = reinterpret_cast<const int*>(p)[uint32_t(lane) * 16];
        }
    }
    __device__ __forceinline__ void done() const {      // keeps the loads; waits for them
#pragma unroll
        for (int j = 0; j < kTurns; ++j) asm volatile("" ::"v"(x[j]));
    }
};

// N tiles from LDS (each column by column) as a piece in memory has them (row by
// row): read in one phase, stored in a later one.
template <int N>
struct Tiles {
    f32x4 v[N];

    __device__ __forceinline__ void read(const float* tiles, int lane) {
        const int row = lane >> 2, c = (lane & 3) * 4;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = tiles[i * kTile + (c + j) * kTileRow + row];
    }

    __device__ __forceinline__ void store(float* piece, int lane) const {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<f32x4*>(piece + i * 256 + lane * 4) = v[i];
    }
};

}  // namespace qc
