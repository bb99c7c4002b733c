// dca_api.cpp -- the entry points of whole-sequence linear attention with decays
// (include/decay_attention.h): host checks, buffer layouts, launches.
#include "dca_internal.hpp"

namespace qc {
namespace {

struct DcaPlan {
    int rc;
    int kb, ct, chunk;
    int64_t slots, seg_slots, segs, seg_tokens, cuts, tokens, vp;
    int64_t states, seg, decays, part;         // bytes of S0 (or dS1) of every chunk, and of the workspace's parts
    int64_t q_bytes, out, gates, fin;
};

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Blocks that a pass over a sequence wants: two to each of 256 CUs (bfloat16, heads of 128, calls: 8192 tokens of 32 heads
// 162 us with 512, 203 with 256, 194 with 1024, whose states pass through memory for more than they gain; 4096 of 32 heads
// 96, 114, 111; 2048 of 32 heads 69, 74, 66; 8 x 2048 of 16 heads of 64 x 128 in float32 168, 218, 191).  (dca_plan's
// division leaves segments a chunk longer than an even cut has them, 9 for 8 at the first of these.)
constexpr int64_t kBlocks = 512;
// The backward states' pass does without segments from these blocks of 64 columns on: it is bound by the states that it
// stores, and a block to each CU stores as fast (4 x 4096 tokens of 32 heads of 128: 179 us, and 283 with segments of
// 128 columns, their sums and joins among them; the forward pass 398, and 332).
constexpr int64_t kNarrow = 256;
// Packed sequences may be of unlike length, so they are always cut, at a length that none has where equal ones fill the
// card: one of 8192 tokens and 63 of 64, 16 heads of 128, without: 822 us, and 144 with; 64 of 192: 87 us, and 115.
// Tokens to a segment, at least (bfloat16, heads of 128, calls with 128, 64 and 256: 1024 tokens of one head 39, 31 and 57
// us, of 16 heads 45, 39 and 60; 4096 of 4 heads 50, 49 and 62, of 16 heads 71, 70 and 70; 30 packed sequences of 64, 8
// heads, 30.7, 32.8 and 29.5: shorter ones gain where heads are few, and cost states through memory).
constexpr int64_t kLeast = 128;

DcaPlan dca_plan(const dca_dims* dims) {
    DcaPlan p{};
    p.rc = dca_check(dims);
    if (p.rc != QC_OK) return p;
    const dca_dims& d = *dims;
    p.rc = QC_ERR_SHAPE;
    if (d.packed ? d.B != 1 : d.N != d.B) return p;
    const int64_t narrow = d.packed ? d.T / 32 + d.N : count(d.N, (d.T + 31) / 32), strips = (d.V + 63) / 64;
    if (narrow < 0 || count(narrow, d.Hv * strips) < 0 || narrow * d.Hv * strips >= (int64_t(1) << 23)) return p;
    const int64_t units = count(d.N, d.Hk);
    const int64_t blocks = units < 0 ? -1 : count((units + 7) / 8 * 8, d.Hv / d.Hk * strips);
    if (blocks < 0 || blocks >= (int64_t(1) << 23)) return p;
    p.kb = d.K <= 32 ? 1 : d.K <= 64 ? 2 : 4;
    p.ct = d.V <= 64 ? 1 : 2;
    p.chunk = dca_chunk(d.dtype);
    p.vp = (d.V + 64 * p.ct - 1) / (64 * p.ct) * (64 * p.ct);
    const int64_t per = (d.T + p.chunk - 1) / p.chunk;
    p.slots = !d.T || !d.N ? 0 : d.packed ? d.T / p.chunk + d.N : d.N * per;
    // Segments: as many as fill the card where sequences, heads and columns do not.
    const int64_t wide = d.Hv * (p.vp / (64 * p.ct));
    int64_t len = per > 0 ? per : 1;
    if (d.N && (d.packed || d.N * wide < kBlocks)) {
        const int64_t share = (d.packed ? per : d.N * per) * wide / kBlocks + 1;
        len = share * p.chunk > kLeast ? share : kLeast / p.chunk;
        if (len > per) len = per > 0 ? per : 1;
    }
    p.seg_tokens = len * p.chunk;
    p.segs = per > len ? (per + len - 1) / len : 1;
    p.seg_slots = d.packed ? d.T / p.seg_tokens + d.N : d.N * p.segs;
    p.cuts = d.packed ? (d.T + p.seg_tokens - 1) / p.seg_tokens : d.N * p.segs;
    p.tokens = d.B * d.T;
    const int64_t state = int64_t(32) * p.kb * p.vp * 4;
    p.states = up256(p.slots * d.Hv * state);
    p.seg = p.segs > 1 ? up256(p.cuts * d.Hv * state) : 0;
    p.decays = p.segs > 1 ? up256(p.cuts * d.Hv * 4) : 0;
    p.part = d.head_decay ? up256(p.slots * d.Hv * 4) : 0;
    const size_t e = dtype_bytes(d.dtype);
    p.q_bytes = p.tokens * d.Hk * d.K * e;
    p.out = p.tokens * d.Hv * d.V * e;
    p.gates = (d.head_decay ? 1 : p.tokens) * d.Hv * 4;
    p.fin = d.N * d.Hv * d.K * d.V * 4;
    p.rc = QC_OK;
    return p;
}

DcaArgs arguments(const dca_dims& d, const DcaPlan& p, const void* q, const void* k, const void* v, const float* g, const int32_t* offsets) {
    DcaArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.offsets = d.packed ? offsets : nullptr;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = d.q_stride[i];
        a.ks[i] = d.k_stride[i];
        a.vs[i] = d.v_stride[i];
    }
    a.gs[0] = d.head_decay ? 0 : d.T * d.Hv;
    a.gs[1] = d.head_decay ? 0 : d.Hv;
    a.gs[2] = 1;
    a.T = d.T; a.N = d.N; a.chunks = (d.T + p.chunk - 1) / p.chunk; a.segs = p.segs;
    a.slots = p.slots; a.seg_slots = p.seg_slots; a.seg_tokens = p.seg_tokens;
    a.cuts = p.cuts;
    a.Hk = int(d.Hk); a.Hv = int(d.Hv); a.group = int(d.Hv / d.Hk); a.K = int(d.K); a.V = int(d.V); a.VP = int(p.vp);
    a.tiles = int(p.vp / (64 * p.ct));
    a.scale = d.scale;
    const size_t e = dtype_bytes(d.dtype);
    a.vec_v = d.V % 8 == 0 && rows_on_16(v, d.v_stride, e) && rows_near(d.v_stride[1], e);
    a.vec_qk = d.K % 8 == 0 && rows_on_16(q, d.q_stride, e) && rows_on_16(k, d.k_stride, e) && rows_near(d.q_stride[1], e) && rows_near(d.k_stride[1], e);
    return a;
}

int check_inputs(const dca_dims& d, const DcaPlan& p, const void* q, const void* k, const void* v, const float* g, const int32_t* offsets) {
    if (p.tokens && (!q || !k || !v || !g)) return QC_ERR_NULL;
    if (d.packed && d.N && !offsets) return QC_ERR_NULL;
    const size_t e = dtype_bytes(d.dtype);
    for (const void* x : {q, k, v})
        if (!aligned_to(x, e)) return QC_ERR_ALIGN;
    for (const void* x : {static_cast<const void*>(g), static_cast<const void*>(offsets)})
        if (!aligned_to(x, 4)) return QC_ERR_ALIGN;
    return QC_OK;
}

}  // namespace
}  // namespace qc

extern "C" {

size_t dca_saved_bytes(const dca_dims* dims) {
    const qc::DcaPlan p = qc::dca_plan(dims);
    return p.rc == QC_OK ? size_t(p.states) + 256 : 0;
}

size_t dca_workspace_bytes(const dca_dims* dims, int32_t backward) {
    const qc::DcaPlan p = qc::dca_plan(dims);
    return p.rc == QC_OK ? size_t(p.seg + p.decays + (backward ? p.states + p.part : 0)) + 256 : 0;
}

int dca_fwd(const dca_dims* dims, const void* query, const void* key, const void* value, const float* log_decay, const int32_t* offsets,
            const float* initial_state, void* out, float* final_state, void* saved, void* workspace, size_t workspace_bytes, void* stream) {
    const qc::DcaPlan p = qc::dca_plan(dims);
    if (p.rc != QC_OK) return p.rc;
    const dca_dims& d = *dims;
    const int rc = qc::check_inputs(d, p, query, key, value, log_decay, offsets);
    if (rc != QC_OK) return rc;
    if (p.out && !out) return QC_ERR_NULL;
    const size_t e = qc::dtype_bytes(d.dtype);
    if (!qc::aligned_to(out, e) || !qc::aligned_to(final_state, 4) || !qc::aligned_to(initial_state, 4) || !qc::aligned_to(saved, 256) ||
        !qc::aligned_to(workspace, 256))
        return QC_ERR_ALIGN;
    const size_t need = dca_workspace_bytes(dims, 0);
    if (!workspace || workspace_bytes < need) return QC_ERR_WORKSPACE;
    const qc::ByteSpan sp[] = {{out, size_t(p.out)}, {final_state, size_t(p.fin)}, {saved, size_t(p.states)}, {workspace, need},
                               {query, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.q_stride, e))},
                               {key, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.k_stride, e))},
                               {value, size_t(qc::strided_bytes(d.B, d.T, d.Hv, d.V, d.v_stride, e))},
                               {log_decay, size_t(p.gates)}, {offsets, d.packed ? size_t(d.N + 1) * 4 : 0}, {initial_state, size_t(p.fin)}};
    if (qc::outputs_overlap(sp, 4, 10)) return QC_ERR_ALIAS;
    if (!d.N) return QC_OK;
    qc::DcaArgs a = qc::arguments(d, p, query, key, value, log_decay, offsets);
    a.vec_o = d.V % 8 == 0 && qc::aligned_to(out, 16);
    a.s0 = initial_state; a.out = out; a.fin = final_state;
    a.save = static_cast<float*>(saved);
    a.seg = static_cast<float*>(workspace);
    a.seg_decay = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.seg);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t err = hipSuccess;
    if (p.segs > 1) {
        err = qc::launch_dca_state(d.dtype, p.kb, p.ct, false, true, a, st);
        if (err == hipSuccess) err = qc::launch_dca_join(p.kb, false, a, st);
    }
    if (err == hipSuccess) err = qc::launch_dca_fwd(d.dtype, p.kb, p.ct, a, st);
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}

int dca_bwd(const dca_dims* dims, const void* query, const void* key, const void* value, const float* log_decay, const int32_t* offsets,
            const void* saved, const void* d_out, const float* d_final_state, void* d_query, void* d_key, void* d_value,
            float* d_log_decay, float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
    const qc::DcaPlan p = qc::dca_plan(dims);
    if (p.rc != QC_OK) return p.rc;
    const dca_dims& d = *dims;
    const int rc = qc::check_inputs(d, p, query, key, value, log_decay, offsets);
    if (rc != QC_OK) return rc;
    if (!d_query && !d_key && !d_value && !d_log_decay && !d_initial_state) return QC_OK;
    if ((p.out && !d_out) || !saved) return QC_ERR_NULL;
    const size_t e = qc::dtype_bytes(d.dtype);
    for (const void* x : {d_out, static_cast<const void*>(d_query), static_cast<const void*>(d_key), static_cast<const void*>(d_value)})
        if (!qc::aligned_to(x, e)) return QC_ERR_ALIGN;
    for (const float* x : {d_final_state, static_cast<const float*>(d_log_decay), static_cast<const float*>(d_initial_state)})
        if (!qc::aligned_to(x, 4)) return QC_ERR_ALIGN;
    if (!qc::aligned_to(saved, 256) || !qc::aligned_to(workspace, 256)) return QC_ERR_ALIGN;
    const size_t need = dca_workspace_bytes(dims, 1);
    if (!workspace || workspace_bytes < need) return QC_ERR_WORKSPACE;
    const qc::ByteSpan sp[] = {{d_query, size_t(p.q_bytes)}, {d_key, size_t(p.q_bytes)}, {d_value, size_t(p.out)},
                               {d_log_decay, size_t(p.gates)}, {d_initial_state, size_t(p.fin)}, {workspace, need},
                               {query, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.q_stride, e))},
                               {key, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.k_stride, e))},
                               {value, size_t(qc::strided_bytes(d.B, d.T, d.Hv, d.V, d.v_stride, e))},
                               {log_decay, size_t(p.gates)}, {offsets, d.packed ? size_t(d.N + 1) * 4 : 0}, {saved, size_t(p.states)},
                               {d_out, size_t(p.out)}, {d_final_state, size_t(p.fin)}};
    if (qc::outputs_overlap(sp, 6, 14)) return QC_ERR_ALIAS;
    const bool heads = d.head_decay && d_log_decay;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    qc::DcaArgs a = qc::arguments(d, p, query, key, value, log_decay, offsets);
    a.vec_o = d.V % 8 == 0 && qc::aligned_to(d_out, 16) && qc::aligned_to(d_value, 16) && qc::rows_near(d.Hv * d.V, e);
    a.vec_qk = a.vec_qk && qc::aligned_to(d_query, 16) && qc::aligned_to(d_key, 16);
    char* ws = static_cast<char*>(workspace);
    a.ds = reinterpret_cast<float*>(ws);
    a.seg = reinterpret_cast<float*>(ws + p.states);
    a.seg_decay = reinterpret_cast<float*>(ws + p.states + p.seg);
    a.dg_part = heads ? reinterpret_cast<float*>(ws + p.states + p.seg + p.decays) : nullptr;
    a.save = const_cast<float*>(static_cast<const float*>(saved));
    a.d_out = d_out; a.d_fin = d_final_state;
    a.dq = d_query; a.dk = d_key; a.dv = d_value; a.dg = heads ? nullptr : d_log_decay; a.ds0 = d_initial_state;
    hipError_t err = hipSuccess;
    if (d.N) {
        int ct = p.ct;
        if (p.segs > 1 && !d.packed && d.N * d.Hv * (p.vp / 64) >= qc::kNarrow) {
            ct = 1;
            a.tiles = int(p.vp / 64);
            a.segs = 1;
            a.seg_slots = d.N;
            a.seg_tokens = a.chunks * p.chunk;
        } else if (p.segs > 1) {
            err = qc::launch_dca_state(d.dtype, p.kb, ct, true, true, a, st);
            if (err == hipSuccess) err = qc::launch_dca_join(p.kb, true, a, st);
        }
        if (err == hipSuccess) err = qc::launch_dca_state(d.dtype, p.kb, ct, true, false, a, st);
        if (err == hipSuccess && (d_query || d_key || d_value || d_log_decay)) err = qc::launch_dca_grad(d.dtype, p.kb, a, st);
    }
    // (Without tokens there are no sums, and a head's decay has a gradient of zero.)
    if (err == hipSuccess && heads) err = qc::launch_dca_heads(a, d_log_decay, st);
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}

}  // extern "C"
