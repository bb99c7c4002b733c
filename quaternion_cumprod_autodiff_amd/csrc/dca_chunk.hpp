// dca_chunk.hpp -- the chunked form of linear attention with decays
// (include/decay_attention.h): its mathematics, its internal formats and the
// device helpers that its kernels share.  Not installed.
//
// Chunks of C tokens, 64 for bfloat16 and 32 for the types of several parts.
// With G_i the log decays cumulated from the chunk's start, gamma_i = exp(G_i),
// eta_i = exp(G_last - G_i), Gam_ij = exp(G_i - G_j), and S0 the state before
// the chunk,
//     P_ij = Gam_ij q_i.k_j (i >= j)
//     out = scale (gamma (Q S0) + P V)
//     S1  = gamma_last S0 + K^T (eta V)
// and, for cotangents dO of out (O = scale dO) and dS1 of S1,
//     Phi_ij = Gam_ij O_i.V_j (i >= j)
//     dQ  = gamma (O S0^T) + Phi K
//     dK  = eta (V dS1^T) + Phi^T Q
//     dV  = eta (K dS1) + P^T O
//     dS0 = gamma_last dS1 + Q^T (gamma O)
//     dg_t = gamma_last <S0, dS1> + sum_{i >= t} gamma_i q_i.(O S0^T)_i
//            + sum_{j < t} eta_j k_j.(V dS1^T)_j + sum_{i >= t > j} Phi_ij q_i.k_j
// All exponents are of differences that decays keep at or below zero, and every
// term of dg_t carries exp(g_t): by additions alone a strong decay's gradient
// is not the rounding of larger terms that cancel.
//
// Nothing in a chunk but S0 depends on the chunk before, and S0 linearly.  So
// where sequences and heads alone leave CUs idle, a sequence is cut into
// segments of whole chunks: dca_state sums what each segment adds to a state
// that starts from zero, dca_join carries the states over the segments, and
// then every segment runs from its own.  dca_fwd passes over a segment with S
// in registers (and leaves S0 of every chunk for a backward pass), dca_state
// likewise with dS from its end, dca_grad takes every chunk at once.
//
// Arithmetic.  All products are v_mfma_f32_16x16x32_bf16 on operands split into
// bfloat16 parts: inputs whole (one part for bfloat16, two for float16, three
// for float32), computed operands in three, which hold a float32 whole.  Two on
// the way to an output of 16 bits were 3 to 7% faster (prompt of 8192 tokens of
// 32 heads of 128: 144 us, three 154; training step of 4 x 4096: 1036, 1099), but
// put it 15 times as far from the value as float32 does before its rounding, and
// lost the last bits of differences.
//
// Layouts.  A lane l = 16 g + m holds of an operand fragment row m (A) or column
// m (B) and the 8 consecutive indices 32 b + 8 g + .. of the contracted axis'
// block b; of a product column m and rows 4 g + 0..3.  Rows of tiles 2b and
// 2b + 1 stand for the indices 8 (m / 4) + 4 (tile % 2) + m % 4 of block b, so
// that a lane's accumulators of both are 8 consecutive indices: results become
// operands without a transpose.  In LDS lie the chunk's rows as they come, token
// by token, each part for itself, 16-byte pieces swapped within a row so that
// 16 rows' pieces lie in all banks; fragments along a row are 16-byte reads,
// those across tokens two transposing reads of 4 tokens each.
#pragma once

#include "decay_attention.h"
#include "gdr_chunk.hpp"

namespace qc {

constexpr int dca_chunk(int dt) { return dt == 1 ? 64 : 32; }

struct DcaArgs {
    const void *q, *k, *v;
    const float *g, *s0;
    const int32_t* offsets;
    void* out;
    float* fin;
    float* save;                        // S0 of every chunk: [slots][Hv][KP][VP] (or null)
    float* seg;                         // workspace: states where two segments meet (backward: dS), [cuts][Hv][KP][VP]
    float* seg_decay;                   // workspace: of the segment that the state passes to get there, [cuts][Hv]
    const void* d_out;
    const float* d_fin;
    void *dq, *dk, *dv;
    float *dg, *ds0;
    float* ds;                          // workspace: dS1 of every chunk
    float* dg_part;                     // workspace: sums of dg over chunks [slots][Hv], for decays of the head alone
    int64_t qs[3], ks[3], vs[3], gs[3]; // gs: of log_decay, zeros for batch and token where it is of the head alone
    int64_t T, N, chunks, segs;         // chunks, segs: per sequence, without offsets
    int64_t slots, seg_slots, seg_tokens;
    int64_t cuts;                       // packed: multiples of seg_tokens in T; else N segs
    int Hk, Hv, group, K, V, VP, tiles; // tiles: blocks of 64 CT columns of V
    int vec_qk, vec_v, vec_o;           // rows on 16 bytes and sizes multiples of 8
    float scale;
};

hipError_t launch_dca_fwd(int dt, int kb, int ct, const DcaArgs& a, hipStream_t st);
hipError_t launch_dca_state(int dt, int kb, int ct, bool rev, bool sum, const DcaArgs& a, hipStream_t st);
hipError_t launch_dca_join(int kb, bool rev, const DcaArgs& a, hipStream_t st);
hipError_t launch_dca_grad(int dt, int kb, const DcaArgs& a, hipStream_t st);
hipError_t launch_dca_heads(const DcaArgs& a, float* out, hipStream_t st);

// Whether 64 tokens of this stride lie within 2^31 bytes.
inline bool rows_near(int64_t stride, size_t e) { return stride < (int64_t(1) << 24) / int64_t(e); }

// Calls f(dtype, blocks of K, column tiles of a wave) with all as constants.
template <class F>
hipError_t by_dca_shape(int dt, int kb, int ct, F&& f) {
    return by_dtype_kb(dt, kb, [&](auto d, auto k) {
        return ct == 1 ? f(d, k, std::integral_constant<int, 1>{}) : f(d, k, std::integral_constant<int, 2>{});
    });
}

// Device helpers ----------------------------------------------------------------

struct Span {
    int64_t b, t0, slot, seg;          // first token, first chunk's slot, first segment's slot
    int len;
};

template <int C>
__device__ __forceinline__ Span span_of(const DcaArgs& a, int64_t n) {
    if (!a.offsets) return {n, 0, n * a.chunks, n * a.segs, int(a.T)};
    int64_t lo = a.offsets[n], hi = a.offsets[n + 1];
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    hi = hi < lo ? lo : hi > a.T ? a.T : hi;
    // Consecutive sequences' slots cannot meet: floor((lo + len) / s) + 1 >= floor(lo / s) + max(1, ceil(len / s)).
    return {0, lo, lo / C + n, lo / a.seg_tokens + n, int(hi - lo)};
}

__device__ __forceinline__ int segments_of(const DcaArgs& a, const Span& s) {
    const int n = int((s.len + a.seg_tokens - 1) / a.seg_tokens);
    return n > 1 ? n : 1;
}

// The last sequence whose first slot (of chunks, or of segments) is at or before this one.
template <int C, bool SEG>
__device__ __forceinline__ int64_t owner(const DcaArgs& a, int64_t slot) {
    if (!a.offsets) return slot / (SEG ? a.segs : a.chunks);
    int64_t lo = 0, hi = a.N - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        const Span s = span_of<C>(a, mid);
        if ((SEG ? s.seg : s.slot) <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Of packed sequences: a whole segment holds one multiple of seg_tokens, the cut, so that as many blocks as there are
// multiples find every segment that another follows, however many sequences there are.  The one that holds multiple j:
// its sequence, or -1 if no other follows it.
__device__ __forceinline__ int64_t cut_owner(const DcaArgs& a, int64_t j, int& seg) {
    const int64_t token = j * a.seg_tokens;
    int64_t lo = -1, hi = a.N - 1;                   // the last sequence that starts at or before the token
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (a.offsets[mid] <= token) lo = mid;
        else hi = mid - 1;
    }
    if (lo < 0) return -1;
    const Span s = span_of<64>(a, lo);               // (its chunks do not matter here)
    if (token < s.t0 || token >= s.t0 + s.len) return -1;
    seg = int((token - s.t0) / a.seg_tokens);
    return seg + 1 < segments_of(a, s) ? lo : -1;
}

// The slot of the state between segments `seg` and seg + 1 of a sequence; of packed ones, the multiple in the first of
// them.  (Within the cuts: ceil(lo / s) + ceil(len / s) - 2 <= ceil((lo + len) / s) - 1.)
__device__ __forceinline__ int64_t cut_slot(const DcaArgs& a, const Span& s, int64_t n, int64_t seg) {
    return a.offsets ? (s.t0 + a.seg_tokens - 1) / a.seg_tokens + seg : n * a.segs + seg;
}

// Blocks that share a key head's rows run on one XCD (block % 8), next to each other in time.
__device__ __forceinline__ bool dca_unit(int64_t units, int per, int64_t& u, int& s) {
    u = blockIdx.x / (8 * int64_t(per)) * 8 + blockIdx.x % 8;
    s = int(blockIdx.x / 8 % per);
    return u < units;
}

// W columns of C tokens in LDS: the byte of piece `p` (8 columns) of a token.
template <int W>
__device__ __forceinline__ int lds_piece(int token, int p) {
    constexpr int kPieces = W / 8, kRows = kPieces >= 16 ? 1 : 16 / kPieces;
    return token * (W * 2) + ((p ^ ((token / kRows) & (kPieces - 1))) << 4);
}

// A fragment along a row: pieces 4 b + g of a token, every part.
template <int C, int W, int NP>
__device__ __forceinline__ void row_fragment(const char* t, int token, int b, int g, bf16x8 (&x)[NP]) {
    const int at = lds_piece<W>(token, 4 * b + g);
#pragma unroll
    for (int n = 0; n < NP; ++n) x[n] = *reinterpret_cast<const bf16x8*>(t + n * (C * W * 2) + at);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

// TIGHT: a lane's number that the compiler takes for a new one.  Addresses made of it are made again in each phase of a
// chunk, a few instructions, instead of being held over all of them, in registers that the state needs (bfloat16, 128 x
// 128, forward, with two parts of the state: 272 bytes a lane spilled and 160 us, none and 97; but where nothing spills
// 142 us become 160, float32 64 x 128).
template <bool TIGHT>
__device__ __forceinline__ int fresh(int x) {
    if constexpr (TIGHT) asm volatile("" : "+v"(x));
    return x;
}

// Four rows' element of column m, from pieces of 4 columns: lane 4 r + q names piece q of row r.
__device__ __forceinline__ s16x4 read_transposed(const char* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
}

__device__ __forceinline__ bf16x8 joined(s16x4 lo, s16x4 hi) {
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}

// A fragment across tokens 32 b + 8 g + ..: `col` is the first of the four columns of the piece that this
// lane names, m % 4; it gets column m % 4 of piece m / 4.
template <int C, int W, int NP>
__device__ __forceinline__ void col_fragment(const char* t, int b, int g, int m, int col, bf16x8 (&x)[NP]) {
    const int t0 = 32 * b + 8 * g + (m >> 2);
    const int lo = lds_piece<W>(t0, col >> 3) + (col & 7) * 2, hi = lds_piece<W>(t0 + 4, col >> 3) + (col & 7) * 2;
#pragma unroll
    for (int n = 0; n < NP; ++n) x[n] = joined(read_transposed(t + n * (C * W * 2) + lo), read_transposed(t + n * (C * W * 2) + hi));
}

// Fragments of P and Phi in LDS: row tile i (16 tokens) and block b (32 tokens) at or before it.
constexpr int dca_tri(int c) { return (c / 32) * (c / 32 + 1); }
__host__ __device__ constexpr int tri_of(int i, int b) { return ((i >> 1) + (i & 1)) * ((i >> 1) + 1) + b; }

// The same across rows: column tile j's tokens 16 j + m, rows 32 b + 8 g + .. .
template <int NP>
__device__ __forceinline__ void tri_cols(const bf16x8 (*p)[NP][64], int b, int g, int m, int j, bf16x8 (&x)[NP]) {
    const int i = 32 * b + 8 * g + (m >> 2), col = 16 * j + 4 * (m & 3);
    const bf16x8(*f)[64] = p[tri_of(i >> 4, j >> 1)];
    const int at = (((col >> 3) & 3) * 16 + (i & 15)) * 16 + (col & 4) * 2;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const char* s = reinterpret_cast<const char*>(f[n]) + at;
        x[n] = joined(read_transposed(s), read_transposed(s + 64));
    }
}

// C tokens of W columns on their way from memory to LDS, by NT threads: loaded
// in one place, taken apart and stored in a later one.  Tokens from `rem` on and
// columns from `width` on are zero.  p is the same in all lanes.  vec: rows on 16
// bytes, width a multiple of 8, and C tokens within 2^31 bytes (rows_near).
template <int DT, int C, int W, int NT = 256>
struct Rows {
    using E = typename Storage<DT>::type;
    static constexpr int kAll = C * W / 8, kMine = (kAll + NT - 1) / NT, kWords = 8 * sizeof(E) / 16, kPer = 16 / sizeof(E);
    typedef E Piece __attribute__((ext_vector_type(16 / sizeof(E))));
    Piece x[kMine][kWords];

    __device__ __forceinline__ void load(const E* p, int64_t stride, int rem, int width, bool vec, int tid) {
        constexpr int kStep = NT / (W / 8);      // tokens from one of a thread's pieces to the next
        if (vec) {
            const int t0 = tid / (W / 8), c = tid % (W / 8) * 8;
            const uint32_t off = (uint32_t(t0) * uint32_t(stride) + uint32_t(c)) * uint32_t(sizeof(E));
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const bool in = (kAll % NT == 0 || tid + i * NT < kAll) && t0 + i * kStep < rem && c < width;
                const char* s = reinterpret_cast<const char*>(p + i * kStep * stride);
#pragma unroll
                for (int w = 0; w < kWords; ++w) x[i][w] = in ? *reinterpret_cast<const Piece*>(s + off + 16 * w) : Piece(E(0.f));
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int at = tid + i * NT, token = at / (W / 8), c = at % (W / 8) * 8;
            const bool in = (kAll % NT == 0 || at < kAll) && token < rem;
            const E* s = p + token * stride + c;
#pragma unroll
            for (int w = 0; w < kWords; ++w)
#pragma unroll
                for (int j = 0; j < kPer; ++j) x[i][w][j] = in && c + w * kPer + j < width ? s[w * kPer + j] : E(0.f);
        }
    }

    __device__ __forceinline__ void store(char* t, int tid) const {
        constexpr int NP = parts_of(DT);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int at = tid + i * NT, token = at / (W / 8), c = at % (W / 8);
            if (kAll % NT && at >= kAll) continue;
            bf16x8 y[NP];
            if constexpr (DT == 1) {
                y[0] = x[i][0];
            } else {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = float(x[i][j / kPer][j % kPer]);
                split<NP, 8>(f, y);
            }
#pragma unroll
            for (int n = 0; n < NP; ++n) *reinterpret_cast<bf16x8*>(t + n * (C * W * 2) + lds_piece<W>(token, c)) = y[n];
        }
    }
};

template <class T>
__device__ __forceinline__ const T* same_in_all_lanes(const T* p) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(u)), hi = __builtin_amdgcn_readfirstlane(uint32_t(u >> 32));
    return reinterpret_cast<const T*>(uint64_t(hi) << 32 | lo);
}

// A chunk's decays, in LDS.  cum is in units of log 2, for exp2.
template <int C>
struct Decays {
    double cum[C];
    float gamma[C], eta[C];
};

__device__ __forceinline__ float exp2_of(double x) { return __builtin_amdgcn_exp2f(float(x)); }

template <int CTRL>
__device__ __forceinline__ double moved64(double x) {      // by a DPP control, zero where there is no lane
    typedef int Pair __attribute__((ext_vector_type(2)));
    const Pair p = __builtin_bit_cast(Pair, x);
    return __builtin_bit_cast(double, Pair{__builtin_amdgcn_update_dpp(0, p[0], CTRL, 0xf, 0xf, true), __builtin_amdgcn_update_dpp(0, p[1], CTRL, 0xf, 0xf, true)});
}
__device__ __forceinline__ double lane64(double x, int l) {
    typedef int Pair __attribute__((ext_vector_type(2)));
    const Pair p = __builtin_bit_cast(Pair, x);
    return __builtin_bit_cast(double, Pair{__builtin_amdgcn_readlane(p[0], l), __builtin_amdgcn_readlane(p[1], l)});
}

// One wave: lane l has the log decay of token l (from C on, and where there is no token: zero).  Returns the chunk's
// whole log2 decay.  The sums run within 16 lanes, then over their totals, in registers alone.
template <int C>
__device__ __forceinline__ double put_decays(Decays<C>& d, float g, int lane) {
    double x = double(g < -1e4f ? -1e4f : g) * 1.4426950408889634;
    x += moved64<0x111>(x);
    x += moved64<0x112>(x);
    x += moved64<0x114>(x);
    x += moved64<0x118>(x);
    const double a = lane64(x, 15), b = lane64(x, 31), c = lane64(x, 47);
    double before = 0.;
    if (lane >= 16) before = a;
    if (lane >= 32) before += b;
    if (lane >= 48) before += c;
    x += before;
    const double last = lane64(x, C - 1);
    if (lane < C) {
        d.cum[lane] = x;
        d.gamma[lane] = exp2_of(x);
        d.eta[lane] = exp2_of(last - x);
    }
    return last;
}

// Eight consecutive floats of LDS.
__device__ __forceinline__ void read8(const float* p, float (&x)[8]) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = a[j];
        x[4 + j] = b[j];
    }
}

// The sum of an operand's parts, element by element: exact.
template <int NP>
__device__ __forceinline__ void whole(const bf16x8 (&p)[NP], float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[j] = float(p[NP - 1][j]);
#pragma unroll
        for (int n = NP - 2; n >= 0; --n) x[j] += float(p[n][j]);
    }
}

// Eight floats as their upper and their lower 16 bits: whole in two planes of LDS that are read transposed like bfloat16,
// where three parts take three planes.
__device__ __forceinline__ void halves(const float (&x)[8], bf16x8 (&h)[2]) {
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    Words hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = __float_as_uint(x[2 * j]), b = __float_as_uint(x[2 * j + 1]);
        hi[j] = __builtin_amdgcn_perm(b, a, 0x07060302);
        lo[j] = __builtin_amdgcn_perm(b, a, 0x05040100);
    }
    h[0] = __builtin_bit_cast(bf16x8, hi);
    h[1] = __builtin_bit_cast(bf16x8, lo);
}
__device__ __forceinline__ void of_halves(const bf16x8 (&h)[2], float (&x)[8]) {
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    const Words hi = __builtin_bit_cast(Words, h[0]), lo = __builtin_bit_cast(Words, h[1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(__builtin_amdgcn_perm(hi[j], lo[j], 0x05040100));
        x[2 * j + 1] = __uint_as_float(__builtin_amdgcn_perm(hi[j], lo[j], 0x07060302));
    }
}

// gamma-weighted pairs of row tile i and block b from their products (pt: tiles 2 b and 2 b + 1, tokens 32 b + 8 g
// + .. by row, 16 i + m by column): what lies above the diagonal is zero, whatever the product.
template <int C>
__device__ __forceinline__ void decayed_pairs(const Decays<C>& d, const f32x4 (&pt)[2], int i, int b, int g, int m, float factor, float (&x)[8]) {
    const int row = 16 * i + m, first = 32 * b + 8 * g;
    const double at = d.cum[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = first + j <= row ? exp2_of(at - d.cum[first + j]) * (pt[j >> 2][j & 3] * factor) : 0.f;
}

}  // namespace qc
