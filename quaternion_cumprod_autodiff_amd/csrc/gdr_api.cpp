// gdr_api.cpp -- the entry points of the whole-sequence gated delta rule
// (include/gated_delta.h): host checks, buffer layouts, launches.
#include "gdr_chunk.hpp"

namespace qc {
namespace {

struct Plan {
    int rc;
    int kb, npi;
    int64_t slots, tokens, vp;
    int64_t saved_s, saved_u;                  // bytes of the two parts of the saved buffer
    int64_t krec, hrec, x, ds;                 // bytes of the workspace's parts
    int64_t q_bytes, gates, states, out;
};

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

Plan plan(const gdr_dims* dims) {
    Plan p{};
    p.rc = gdr_check(dims);
    if (p.rc != QC_OK) return p;
    const gdr_dims& d = *dims;
    p.rc = QC_ERR_SHAPE;
    if (d.packed ? d.B != 1 : d.N != d.B) return p;
    p.kb = d.K <= 32 ? 1 : d.K <= 64 ? 2 : 4;
    p.npi = parts_of(d.dtype);
    p.vp = (d.V + 15) / 16 * 16;
    const int64_t per = (d.T + kChunk - 1) / kChunk;
    p.slots = d.packed ? d.T / kChunk + d.N : count(d.N, per);
    // Grids stay below 2^32 threads: 512 to a block.
    if (p.slots < 0 || count(p.slots, d.Hv) < 0 || p.slots * d.Hv >= (int64_t(1) << 23)) return p;
    const int64_t units = count(d.N, d.Hk);
    const int64_t blocks = units < 0 ? -1 : count((units + 7) / 8 * 8, d.Hv / d.Hk * (p.vp / 16));
    if (blocks < 0 || blocks >= (int64_t(1) << 23)) return p;
    if (!d.T) p.slots = 0;
    p.tokens = d.B * d.T;
    const int64_t heads = p.slots * d.Hv;
    p.saved_s = up256(heads * 32 * p.kb * p.vp * 4);
    p.saved_u = up256(heads * kChunk * p.vp * 4);
    p.krec = up256(p.slots * d.Hk * krec_bytes(p.kb, p.npi));
    p.hrec = up256(heads * kHrecBytes);
    p.x = p.saved_u;
    p.ds = p.saved_s;
    const size_t e = dtype_bytes(d.dtype);
    p.q_bytes = p.tokens * d.Hk * d.K * e;
    p.out = p.tokens * d.Hv * d.V * e;
    p.gates = p.tokens * d.Hv * 4;
    p.states = d.N * d.Hv * d.K * d.V * 4;
    p.rc = QC_OK;
    return p;
}

GdrArgs arguments(const gdr_dims& d, const Plan& p, const void* q, const void* k, const void* v, const float* g, const float* b,
                  const int32_t* offsets) {
    GdrArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.b = b; a.offsets = d.packed ? offsets : nullptr;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = d.q_stride[i];
        a.ks[i] = d.k_stride[i];
        a.vs[i] = d.v_stride[i];
    }
    a.T = d.T; a.slots = p.slots; a.N = d.N; a.chunks = (d.T + kChunk - 1) / kChunk;
    a.Hk = int(d.Hk); a.Hv = int(d.Hv); a.group = int(d.Hv / d.Hk); a.K = int(d.K); a.V = int(d.V); a.VP = int(p.vp);
    a.scale = d.scale;
    const size_t e = dtype_bytes(d.dtype);
    a.vec_v = d.V % 8 == 0 && rows_on_16(v, d.v_stride, e);
    a.vec_qk = d.K % 8 == 0 && rows_on_16(q, d.q_stride, e) && rows_on_16(k, d.k_stride, e);
    return a;
}

int check_inputs(const gdr_dims& d, const Plan& p, const void* q, const void* k, const void* v, const float* g, const float* b,
                 const int32_t* offsets) {
    if (p.tokens && (!q || !k || !v || !g || !b)) return QC_ERR_NULL;
    if (d.packed && d.N && !offsets) return QC_ERR_NULL;
    const size_t e = dtype_bytes(d.dtype);
    for (const void* x : {q, k, v})
        if (!aligned_to(x, e)) return QC_ERR_ALIGN;
    for (const void* x : {static_cast<const void*>(g), static_cast<const void*>(b), static_cast<const void*>(offsets)})
        if (!aligned_to(x, 4)) return QC_ERR_ALIGN;
    return QC_OK;
}

}  // namespace
}  // namespace qc

extern "C" {

size_t gdr_saved_bytes(const gdr_dims* dims) {
    const qc::Plan p = qc::plan(dims);
    return p.rc == QC_OK ? size_t(p.saved_s + p.saved_u) + 256 : 0;
}

size_t gdr_workspace_bytes(const gdr_dims* dims, int32_t backward) {
    const qc::Plan p = qc::plan(dims);
    return p.rc == QC_OK ? size_t(p.krec + p.hrec + (backward ? p.x + p.ds : 0)) + 256 : 0;
}

int gdr_fwd(const gdr_dims* dims, const void* query, const void* key, const void* value, const float* log_decay, const float* beta,
            const int32_t* offsets, const float* initial_state, void* out, float* final_state, void* saved, void* workspace,
            size_t workspace_bytes, void* stream) {
    const qc::Plan p = qc::plan(dims);
    if (p.rc != QC_OK) return p.rc;
    const gdr_dims& d = *dims;
    const int rc = qc::check_inputs(d, p, query, key, value, log_decay, beta, offsets);
    if (rc != QC_OK) return rc;
    if (p.out && !out) return QC_ERR_NULL;
    const size_t e = qc::dtype_bytes(d.dtype);
    if (!qc::aligned_to(out, e) || !qc::aligned_to(final_state, 4) || !qc::aligned_to(initial_state, 4) || !qc::aligned_to(saved, 256) ||
        !qc::aligned_to(workspace, 256))
        return QC_ERR_ALIGN;
    const size_t need = gdr_workspace_bytes(dims, 0);
    if (!workspace || workspace_bytes < need) return QC_ERR_WORKSPACE;
    const qc::ByteSpan sp[] = {{out, size_t(p.out)}, {final_state, size_t(p.states)}, {saved, size_t(p.saved_s + p.saved_u)},
                               {workspace, need},
                               {query, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.q_stride, e))},
                               {key, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.k_stride, e))},
                               {value, size_t(qc::strided_bytes(d.B, d.T, d.Hv, d.V, d.v_stride, e))},
                               {log_decay, size_t(p.gates)}, {beta, size_t(p.gates)},
                               {offsets, d.packed ? size_t(d.N + 1) * 4 : 0}, {initial_state, size_t(p.states)}};
    if (qc::outputs_overlap(sp, 4, 11)) return QC_ERR_ALIAS;
    if (!d.N) return QC_OK;
    qc::GdrArgs a = qc::arguments(d, p, query, key, value, log_decay, beta, offsets);
    a.vec_o = d.V % 8 == 0 && qc::aligned_to(out, 16);
    a.s0 = initial_state; a.out = out; a.fin = final_state;
    a.krec = static_cast<char*>(workspace);
    a.hrec = a.krec + p.krec;
    a.save_s = static_cast<float*>(saved);
    a.save_u = saved ? reinterpret_cast<float*>(static_cast<char*>(saved) + p.saved_s) : nullptr;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t err = qc::launch_gdr_factor(d.dtype, p.kb, false, a, st);
    if (err == hipSuccess) err = qc::launch_gdr_fwd(d.dtype, p.kb, saved != nullptr, a, st);
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}

int gdr_bwd(const gdr_dims* dims, const void* query, const void* key, const void* value, const float* log_decay, const float* beta,
            const int32_t* offsets, const void* saved, const void* d_out, const float* d_final_state, void* d_query, void* d_key,
            void* d_value, float* d_log_decay, float* d_beta, float* d_initial_state, void* workspace, size_t workspace_bytes,
            void* stream) {
    const qc::Plan p = qc::plan(dims);
    if (p.rc != QC_OK) return p.rc;
    const gdr_dims& d = *dims;
    const int rc = qc::check_inputs(d, p, query, key, value, log_decay, beta, offsets);
    if (rc != QC_OK) return rc;
    if (!d_query && !d_key && !d_value && !d_log_decay && !d_beta && !d_initial_state) return QC_OK;
    if ((p.out && !d_out) || !saved) return QC_ERR_NULL;
    const size_t e = qc::dtype_bytes(d.dtype);
    for (const void* x : {d_out, static_cast<const void*>(d_query), static_cast<const void*>(d_key), static_cast<const void*>(d_value)})
        if (!qc::aligned_to(x, e)) return QC_ERR_ALIGN;
    for (const float* x : {d_final_state, static_cast<const float*>(d_log_decay), static_cast<const float*>(d_beta),
                           static_cast<const float*>(d_initial_state)})
        if (!qc::aligned_to(x, 4)) return QC_ERR_ALIGN;
    if (!qc::aligned_to(saved, 256) || !qc::aligned_to(workspace, 256)) return QC_ERR_ALIGN;
    const size_t need = gdr_workspace_bytes(dims, 1);
    if (!workspace || workspace_bytes < need) return QC_ERR_WORKSPACE;
    const qc::ByteSpan sp[] = {{d_query, size_t(p.q_bytes)}, {d_key, size_t(p.q_bytes)}, {d_value, size_t(p.out)},
                               {d_log_decay, size_t(p.gates)}, {d_beta, size_t(p.gates)}, {d_initial_state, size_t(p.states)},
                               {workspace, need},
                               {query, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.q_stride, e))},
                               {key, size_t(qc::strided_bytes(d.B, d.T, d.Hk, d.K, d.k_stride, e))},
                               {value, size_t(qc::strided_bytes(d.B, d.T, d.Hv, d.V, d.v_stride, e))},
                               {log_decay, size_t(p.gates)}, {beta, size_t(p.gates)},
                               {offsets, d.packed ? size_t(d.N + 1) * 4 : 0}, {saved, size_t(p.saved_s + p.saved_u)},
                               {d_out, size_t(p.out)}, {d_final_state, size_t(p.states)}};
    if (qc::outputs_overlap(sp, 7, 16)) return QC_ERR_ALIAS;
    if (!d.N) return QC_OK;
    qc::GdrArgs a = qc::arguments(d, p, query, key, value, log_decay, beta, offsets);
    a.vec_o = d.V % 8 == 0 && qc::aligned_to(d_out, 16) && qc::aligned_to(d_value, 16);
    a.krec = static_cast<char*>(workspace);
    a.hrec = a.krec + p.krec;
    a.x = reinterpret_cast<float*>(a.hrec + p.hrec);
    a.ds = reinterpret_cast<float*>(a.hrec + p.hrec + p.x);
    a.save_s = const_cast<float*>(static_cast<const float*>(saved));
    a.save_u = const_cast<float*>(reinterpret_cast<const float*>(static_cast<const char*>(saved) + p.saved_s));
    a.d_out = d_out; a.d_fin = d_final_state;
    a.dq = d_query; a.dk = d_key; a.dv = d_value; a.dg = d_log_decay; a.db = d_beta; a.ds0 = d_initial_state;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t err = qc::launch_gdr_factor(d.dtype, p.kb, true, a, st);
    if (err == hipSuccess) err = qc::launch_gdr_bwd_state(d.dtype, p.kb, a, st);
    if (err == hipSuccess && (d_query || d_key || d_log_decay || d_beta)) err = qc::launch_gdr_grad(d.dtype, p.kb, a, st);
    return err == hipSuccess ? QC_OK : qc::record_hip_error(err);
}

}  // extern "C"
