// gdr_step.hip -- the gated delta rule for one or a few tokens, on a pool of
// states (include/gated_delta.h, gdr_step).
//
// With a = exp(g), both products of the old state are taken in one pass,
//     p = S^T k,   r = S^T q,   kq = k . q
//     u = b (v - a p),   out = scale (a r + kq u),   S = a S + k u^T,
// so a token costs one reduction over the rows.  Bound by memory: a state is
// read once and written once whatever the tokens, and everything else is
// small.  A wave owns 32 columns of one state, in registers: lane l holds
// rows (l / 8) NR .. of columns 4 (l % 8) .. + 3 (NR = K / 8 rounded up to 4,
// 8 or 16), so a row's piece is one 128-byte line, all of a state's loads are
// in flight at once, and the reduction stays inside the wave.  810 MB of states
// (read and written): 156 us, 5.2 TB/s, a copy's rate; one row of 32 heads of
// 128 x 128: 7 us, the loads, the reductions and the stores in a row.
#include "gdr_internal.hpp"

#include <type_traits>

namespace qc {
namespace {

constexpr int kCols = 32;

struct StepArgs {
    const void *q, *k, *v;
    const float *g, *b;
    float* state;
    const int32_t* slots;
    void* out;
    int64_t qs[3], ks[3], vs[3];
    int64_t N, T, n_slots, slot_stride;
    int Hv, group, K, V, tiles;
    float scale;
};

// N consecutive elements as they lie in memory: taken apart where they are used,
// so that the next token's are on their way during this one's work.  VEC: pieces
// of up to 16 bytes, each inside or outside `left` as a whole.
template <class E, int N, bool VEC>
struct Held {
    static constexpr int kPer = N * sizeof(E) >= 16 ? 16 / sizeof(E) : N;
    typedef E Vec __attribute__((ext_vector_type(kPer)));
    Vec x[N / kPer];

    __device__ __forceinline__ void load(const E* p, int left) {
#pragma unroll
        for (int i = 0; i < N / kPer; ++i) {
            if constexpr (VEC) {
                x[i] = i * kPer < left ? reinterpret_cast<const Vec*>(p)[i] : Vec(E(0.f));
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j) x[i][j] = i * kPer + j < left ? p[i * kPer + j] : E(0.f);
            }
        }
    }
    __device__ __forceinline__ void get(float (&y)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = float(x[i / kPer][i % kPer]);
    }
};

// Sum over the eight row groups: lanes l, l ^ 8, l ^ 16, l ^ 32.
__device__ __forceinline__ float rows_sum(float x) {
    x += __shfl_xor(x, 8, 64);
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
    return x;
}

// NR: rows per lane.  VEC: K a multiple of 8, V of 4 and every row on 16 bytes;
// otherwise elements are read one by one.  MANY: more than one token, the next
// one's q, k, v loaded ahead.  STREAM: the states pass by the caches.
template <int DT, int NR, bool VEC, bool MANY, bool STREAM>
__global__ void __launch_bounds__(64) gdr_step_kernel(StepArgs a) {
    using E = typename Storage<DT>::type;
    const int lane = threadIdx.x, c0 = lane % 8 * 4, r0 = lane / 8 * NR;
    // The tiles of a state on one XCD (block % 8), next to each other in time.
    const int tile = int(blockIdx.x / 8 % a.tiles);
    const int64_t rest = blockIdx.x / (8 * a.tiles) * 8 + blockIdx.x % 8;
    if (rest >= a.N * a.Hv) return;
    const int h = int(rest % a.Hv);
    const int64_t n = rest / a.Hv;
    const int col = tile * kCols + c0;
    const int64_t slot = a.slots ? a.slots[n] : n;
    bool run = slot >= 0 && slot < a.n_slots;
    E* out = static_cast<E*>(a.out) + (n * a.T * a.Hv + h) * int64_t(a.V) + col;
    const int64_t out_step = int64_t(a.Hv) * a.V;
    // The state is on its way while the earlier rows' slots are looked through.
    float* st = a.state + (run ? slot : 0) * a.slot_stride + int64_t(h) * a.K * a.V;
    float s[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        if constexpr (VEC) {
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
            if (run && col < a.V && r0 + i < a.K) {
                const f32x4* p = reinterpret_cast<const f32x4*>(st + int64_t(r0 + i) * a.V + col);
                if constexpr (STREAM) x = __builtin_nontemporal_load(p);
                else x = *p;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = x[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = run && r0 + i < a.K && col + j < a.V ? st[int64_t(r0 + i) * a.V + col + j] : 0.f;
        }
    }
    if (a.slots && run) {
        bool twin = false;
        for (int64_t m = lane; m < n; m += 64) twin |= a.slots[m] == slot;
        run = __ballot(twin) == 0;
    }
    if (!run) {
        if (lane < 8)
            for (int64_t t = 0; t < a.T; ++t)
                for (int j = 0; j < 4; ++j)
                    if (col + j < a.V) out[t * out_step + j] = E(0.f);
        return;
    }
    const E* q = static_cast<const E*>(a.q) + n * a.qs[0] + (h / a.group) * a.qs[2] + r0;
    const E* k = static_cast<const E*>(a.k) + n * a.ks[0] + (h / a.group) * a.ks[2] + r0;
    const E* v = static_cast<const E*>(a.v) + n * a.vs[0] + h * a.vs[2] + col;
    const float* g = a.g + n * a.T * a.Hv + h;
    const float* b = a.b + n * a.T * a.Hv + h;
    Held<E, NR, VEC> k_next, q_next;
    Held<E, 4, false> v_next;
    float g_next, b_next;
    auto load = [&] {
        k_next.load(k, a.K - r0);
        q_next.load(q, a.K - r0);
        v_next.load(v, a.V - col);
        g_next = *g;
        b_next = *b;
        q += a.qs[1];
        k += a.ks[1];
        v += a.vs[1];
        g += a.Hv;
        b += a.Hv;
    };
    load();
    for (int64_t t = 0; t < a.T; ++t) {
        float kr[NR], qr[NR], vr[4];
        k_next.get(kr);
        q_next.get(qr);
        v_next.get(vr);
        const float decay = expf(g_next), beta = b_next;
        if (MANY && t + 1 < a.T) load();
        float p[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f}, kq = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            kq += kr[i] * qr[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[j] += s[i][j] * kr[i];
                r[j] += s[i][j] * qr[i];
            }
        }
        kq = rows_sum(kq);
        float u[4], o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[j] = beta * (vr[j] - decay * rows_sum(p[j]));
            o[j] = a.scale * (decay * rows_sum(r[j]) + kq * u[j]);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = decay * s[i][j] + kr[i] * u[j];
        if (lane < 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col + j < a.V) out[j] = E(o[j]);
        }
        out += out_step;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        if constexpr (VEC) {
            if (col < a.V && r0 + i < a.K) {
                f32x4* p = reinterpret_cast<f32x4*>(st + int64_t(r0 + i) * a.V + col);
                const f32x4 x = {s[i][0], s[i][1], s[i][2], s[i][3]};
                if constexpr (STREAM) __builtin_nontemporal_store(x, p);
                else *p = x;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r0 + i < a.K && col + j < a.V) st[int64_t(r0 + i) * a.V + col + j] = s[i][j];
        }
    }
}

template <int DT, bool VEC, bool MANY, bool STREAM>
const void* step_kernel(int nr) {
    return nr == 4   ? reinterpret_cast<const void*>(&gdr_step_kernel<DT, 4, VEC, MANY, STREAM>)
           : nr == 8 ? reinterpret_cast<const void*>(&gdr_step_kernel<DT, 8, VEC, MANY, STREAM>)
                     : reinterpret_cast<const void*>(&gdr_step_kernel<DT, 16, VEC, MANY, STREAM>);
}

template <int DT>
const void* step_kernel(int nr, bool vec, bool many, bool stream) {
    if (!vec) return many ? step_kernel<DT, false, true, false>(nr) : step_kernel<DT, false, false, false>(nr);
    if (stream) return many ? step_kernel<DT, true, true, true>(nr) : step_kernel<DT, true, false, true>(nr);
    return many ? step_kernel<DT, true, true, false>(nr) : step_kernel<DT, true, false, false>(nr);
}

// From how many bytes of states on a call streams them.  A model calls for one
// layer after another, so that a layer's states are gone from the 256 MB cache
// when its turn comes again; three pools in turn: 48 MB 20.3 us (19.4 streamed),
// 134 MB 60.7 (53.6), 268 MB 112 (104), 805 MB 168 (156).  One pool alone stays
// there up to its size: 100 MB 37 us (42), 268 MB 92 (103).
constexpr int64_t kStreamBytes = int64_t(128) << 20;

}  // namespace
}  // namespace qc

extern "C" int gdr_step(const gdr_dims* dims, const void* query, const void* key, const void* value, const float* log_decay,
                        const float* beta, float* state, int64_t n_slots, int64_t slot_stride, const int32_t* slots, void* out,
                        void* stream) {
    const int rc = qc::gdr_check(dims);
    if (rc != QC_OK) return rc;
    const gdr_dims& d = *dims;
    if (d.N != d.B || n_slots < 0 || slot_stride < 0) return QC_ERR_SHAPE;
    if (!d.N || !d.T) return QC_OK;
    if (!query || !key || !value || !log_decay || !beta || (n_slots && !state) || !out) return QC_ERR_NULL;
    if (n_slots > 1 && slot_stride < d.Hv * d.K * d.V) return QC_ERR_SHAPE;
    const int64_t extent = n_slots ? qc::count(n_slots - 1, slot_stride) : 0;
    if (extent < 0 || (!slots && n_slots < d.N)) return QC_ERR_SHAPE;
    const int tiles = int((d.V + qc::kCols - 1) / qc::kCols);
    const int64_t heads = qc::count(d.N, d.Hv), used = heads < 0 ? -1 : qc::count(heads, tiles);
    if (used < 0 || used > (int64_t(1) << 25)) return QC_ERR_SHAPE;
    const int64_t blocks = (heads + 7) / 8 * 8 * tiles;      // 64 threads each: below 2^32 in all
    const size_t e = qc::dtype_bytes(d.dtype);
    for (const void* p : {query, key, value, static_cast<const void*>(out)})
        if (!qc::aligned_to(p, e)) return QC_ERR_ALIGN;
    for (const void* p : {static_cast<const void*>(log_decay), static_cast<const void*>(beta), static_cast<const void*>(state),
                          static_cast<const void*>(slots)})
        if (p && !qc::aligned_to(p, 4)) return QC_ERR_ALIGN;
    const size_t gates = size_t(d.N * d.T * d.Hv) * 4;
    const qc::ByteSpan sp[] = {{out, size_t(d.N * d.T * d.Hv * d.V) * e},
                               {state, n_slots ? size_t(extent + d.Hv * d.K * d.V) * 4 : 0},
                               {query, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.q_stride, e))},
                               {key, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.k_stride, e))},
                               {value, size_t(qc::strided_bytes(d.B, d.T, d.Hv, d.V, d.v_stride, e))},
                               {log_decay, gates}, {beta, gates}, {slots, size_t(d.N) * 4}};
    if (qc::outputs_overlap(sp, 2, 8)) return QC_ERR_ALIAS;
    qc::StepArgs a{};
    a.q = query; a.k = key; a.v = value; a.g = log_decay; a.b = beta; a.state = state; a.slots = slots; a.out = out;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = d.q_stride[i];
        a.ks[i] = d.k_stride[i];
        a.vs[i] = d.v_stride[i];
    }
    a.N = d.N; a.T = d.T; a.n_slots = n_slots; a.slot_stride = slot_stride;
    a.Hv = int(d.Hv); a.group = int(d.Hv / d.Hk); a.K = int(d.K); a.V = int(d.V); a.tiles = tiles;
    a.scale = d.scale;
    const int nr = d.K <= 32 ? 4 : d.K <= 64 ? 8 : 16;
    const bool vec = d.K % 8 == 0 && d.V % 4 == 0 && qc::aligned_to(state, 16) && slot_stride % 4 == 0 &&
                     qc::rows_on_16(query, d.q_stride, e) && qc::rows_on_16(key, d.k_stride, e);
    const bool far = heads * d.K * d.V * 4 >= qc::kStreamBytes;
    const void* fn = d.dtype == GDR_F32 ? qc::step_kernel<0>(nr, vec, d.T > 1, far) : d.dtype == GDR_BF16 ? qc::step_kernel<1>(nr, vec, d.T > 1, far) : qc::step_kernel<2>(nr, vec, d.T > 1, far);
    void* params[] = {&a};
    const hipError_t err = hipLaunchKernel(fn, dim3(unsigned(blocks)), dim3(64), params, 0, static_cast<hipStream_t>(stream));
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}
