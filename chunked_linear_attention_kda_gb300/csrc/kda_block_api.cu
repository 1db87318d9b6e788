// kda_block_api.cu -- the C ABI of the operators around and beside the bounded recurrence:
// the gated delta rule and linear attention with one decay per head, the norms before and after a
// block and the norm of queries and keys with the position rotation.
// Argument validation and launch; no arithmetic.
#include <cuda_runtime.h>

#include <cfloat>

#include "kda_api.h"
#include "kda_internal.h"

namespace {

using kda::api_fail;
using kda::api_ok;

kda_status launched(cudaError_t e, const char *what) {
    if (e != cudaSuccess) return api_fail(KDA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
    return api_ok();
}
bool misaligned(const void *p, size_t a) { return (uintptr_t)p % a != 0; }

struct Range { const void *p; size_t bytes; };
// `n` rows of `width` elements, `stride` elements apart
Range rows(const void *p, int64_t n, int64_t stride, int64_t width, size_t es) {
    return {p, p && n > 0 ? (size_t)((n - 1) * stride + width) * es : 0};
}
bool overlap(const Range &x, const Range &y) {
    if (!x.p || !y.p || !x.bytes || !y.bytes) return false;
    const uintptr_t a = (uintptr_t)x.p, b = (uintptr_t)y.p;
    return a < b + y.bytes && b < a + x.bytes;
}
// no output may overlap an input or another output
template <int NI, int NO>
bool clash(const Range (&ins)[NI], const Range (&outs)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (const Range &r : ins)
            if (overlap(outs[i], r)) return true;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

constexpr const char *kOverlap = "an output or the workspace overlaps an input or another output";

kda_status check_heads(int32_t n_k_heads, int32_t n_heads, int32_t d_k, int32_t d_v, int dtype) {
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return api_fail(KDA_ERR_UNSUPPORTED, "dtype must be KDA_F32 or KDA_BF16");
    if (n_k_heads <= 0 || n_heads <= 0 || n_heads % n_k_heads != 0)
        return api_fail(KDA_ERR_INVALID_ARG, "n_heads must be a positive multiple of n_k_heads > 0");
    if (d_k <= 0 || d_v <= 0) return api_fail(KDA_ERR_INVALID_ARG, "d_k and d_v must be positive");
    if (d_k > 128 || d_v > 128) return api_fail(KDA_ERR_UNSUPPORTED, "d_k and d_v above 128 are not built");
    if (n_k_heads > 65535) return api_fail(KDA_ERR_UNSUPPORTED, "n_k_heads above 65535");
    return KDA_OK;
}

kda_status check_gdr(const kda::GdrArgs &p, int dtype) {
    kda_status s = check_heads(p.n_k_heads, p.n_heads, p.d_k, p.d_v, dtype);
    if (s != KDA_OK) return s;
    if (p.n_tok < 0 || p.n_seq < 0) return api_fail(KDA_ERR_INVALID_ARG, "n_tok and n_seq must be >= 0");
    if (p.n_tok > 0x7fffffffLL) return api_fail(KDA_ERR_UNSUPPORTED, "n_tok above 2^31 - 1");
    if (p.n_tok > 0 && p.n_seq == 0) return api_fail(KDA_ERR_INVALID_ARG, "n_tok > 0 needs at least one sequence");
    if ((int64_t)p.n_seq * p.n_heads > 0x7fffffffLL / 8)
        return api_fail(KDA_ERR_INVALID_ARG, "n_seq * n_heads exceeds 2^28");
    if (p.n_seq > 0 && !p.cu_seqlens) return api_fail(KDA_ERR_INVALID_ARG, "cu_seqlens is NULL");
    if (p.n_tok > 0 && (!p.q || !p.k || !p.v || !p.g || !p.beta))
        return api_fail(KDA_ERR_INVALID_ARG, "q, k, v, g and beta are required");
    const int64_t wk = (int64_t)p.n_k_heads * p.d_k, wv = (int64_t)p.n_heads * p.d_v;
    if (p.q_stride < wk || p.k_stride < wk || p.v_stride < wv)
        return api_fail(KDA_ERR_INVALID_ARG, "a token stride is smaller than a token's row");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    const void *elems[] = {p.q, p.k, p.v, p.out, p.dout, p.dq, p.dk, p.dv};
    for (const void *x : elems)
        if (misaligned(x, es)) return api_fail(KDA_ERR_INVALID_ARG, "q, k, v, out and their gradients must be aligned to their element size");
    const void *f32[] = {p.g, p.beta, p.h0, p.cu_seqlens, p.h_final, p.dh_final, p.dg, p.dbeta, p.dh0};
    for (const void *x : f32)
        if (misaligned(x, 4)) return api_fail(KDA_ERR_INVALID_ARG, "g, beta, cu_seqlens, the states and their gradients must be 4-byte aligned");
    return KDA_OK;
}

kda_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need > 0 && (!ws || have < need || misaligned(ws, 16)))
        return api_fail(KDA_ERR_INVALID_ARG, "the workspace must be 16-byte aligned and hold the bytes its size function gives");
    return KDA_OK;
}

kda::GdrArgs gdr_args(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, const float *g, const float *beta, const float *h0,
                      const int32_t *cu, void *workspace, int64_t n_tok, int32_t n_seq, int32_t n_k_heads,
                      int32_t n_heads, int32_t d_k, int32_t d_v, kda_dtype dtype) {
    kda::GdrArgs p{};
    p.q = q; p.k = k; p.v = v;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.g = g; p.beta = beta; p.h0 = h0; p.cu_seqlens = cu; p.workspace = workspace;
    p.n_tok = n_tok; p.n_seq = n_seq; p.n_k_heads = n_k_heads; p.n_heads = n_heads;
    p.d_k = d_k; p.d_v = d_v; p.bf16 = dtype == KDA_BF16;
    return p;
}

}  // namespace

extern "C" {

static bool gdr_sizes(int64_t n_tok, int32_t n_seq, int32_t n_k_heads, int32_t n_heads, int32_t d_k, int32_t d_v) {
    return n_tok >= 0 && n_seq >= 0 && n_k_heads > 0 && n_heads > 0 && d_k > 0 && d_v > 0 && d_k <= 128 && d_v <= 128;
}

size_t kda_gdr_chunk_fwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_k_heads, int32_t n_heads,
                                         int32_t d_k, int32_t d_v, kda_dtype dtype) {
    if (!gdr_sizes(n_tok, n_seq, n_k_heads, n_heads, d_k, d_v)) return 0;
    return kda::gdr_fwd_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, dtype == KDA_BF16);
}

kda_status kda_gdr_chunk_fwd(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, const float *g, const float *beta, const float *h0,
                             const int32_t *cu_seqlens, void *out, float *h_final, void *workspace,
                             size_t workspace_bytes, int64_t n_tok, int32_t n_seq, int32_t n_k_heads,
                             int32_t n_heads, int32_t d_k, int32_t d_v, kda_dtype dtype, void *stream) {
    kda::GdrArgs p = gdr_args(q, k, v, q_stride, k_stride, v_stride, g, beta, h0, cu_seqlens, workspace, n_tok,
                              n_seq, n_k_heads, n_heads, d_k, d_v, dtype);
    p.out = out;
    p.h_final = h_final;
    kda_status s = check_gdr(p, dtype);
    if (s != KDA_OK) return s;
    if (n_tok > 0 && !out) return api_fail(KDA_ERR_INVALID_ARG, "out is required");
    if (n_seq == 0) return api_ok();
    const size_t need = n_tok ? kda::gdr_fwd_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, p.bf16) : 0;
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != KDA_OK) return s;
    const size_t es = p.bf16 ? 2 : 4, st = (size_t)n_seq * n_heads * d_k * d_v * 4;
    const int64_t wk = (int64_t)n_k_heads * d_k, wv = (int64_t)n_heads * d_v;
    const Range ins[] = {rows(q, n_tok, q_stride, wk, es), rows(k, n_tok, k_stride, wk, es),
                         rows(v, n_tok, v_stride, wv, es), rows(g, n_tok, n_heads, n_heads, 4),
                         rows(beta, n_tok, n_heads, n_heads, 4), {h0, st}, {cu_seqlens, (size_t)(n_seq + 1) * 4}};
    const Range outs[] = {rows(out, n_tok, wv, wv, es), {h_final, st}, {workspace, need}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    return launched(kda::launch_gdr_fwd(p, (cudaStream_t)stream), "gated delta rule forward launch");
}

size_t kda_gdr_chunk_bwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_k_heads, int32_t n_heads,
                                         int32_t d_k, int32_t d_v, kda_dtype dtype) {
    if (!gdr_sizes(n_tok, n_seq, n_k_heads, n_heads, d_k, d_v)) return 0;
    return kda::gdr_bwd_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, dtype == KDA_BF16);
}

kda_status kda_gdr_chunk_bwd(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, const float *g, const float *beta, const float *h0,
                             const int32_t *cu_seqlens, const void *dout, const float *dh_final, void *dq,
                             void *dk, void *dv, float *dg, float *dbeta, float *dh0, void *workspace,
                             size_t workspace_bytes, int64_t n_tok, int32_t n_seq, int32_t n_k_heads,
                             int32_t n_heads, int32_t d_k, int32_t d_v, kda_dtype dtype, void *stream) {
    kda::GdrArgs p = gdr_args(q, k, v, q_stride, k_stride, v_stride, g, beta, h0, cu_seqlens, workspace, n_tok,
                              n_seq, n_k_heads, n_heads, d_k, d_v, dtype);
    p.dout = dout; p.dh_final = dh_final;
    p.dq = dq; p.dk = dk; p.dv = dv; p.dg = dg; p.dbeta = dbeta; p.dh0 = dh0;
    kda_status s = check_gdr(p, dtype);
    if (s != KDA_OK) return s;
    if (n_tok > 0 && (!dout || !dq || !dk || !dv || !dg || !dbeta))
        return api_fail(KDA_ERR_INVALID_ARG, "dout, dq, dk, dv, dg and dbeta are required");
    if (n_seq == 0) return api_ok();
    const size_t need = n_tok ? kda::gdr_bwd_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, p.bf16) : 0;
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != KDA_OK) return s;
    const size_t es = p.bf16 ? 2 : 4, st = (size_t)n_seq * n_heads * d_k * d_v * 4;
    const int64_t wk = (int64_t)n_k_heads * d_k, wv = (int64_t)n_heads * d_v;
    const Range ins[] = {rows(q, n_tok, q_stride, wk, es), rows(k, n_tok, k_stride, wk, es),
                         rows(v, n_tok, v_stride, wv, es), rows(g, n_tok, n_heads, n_heads, 4),
                         rows(beta, n_tok, n_heads, n_heads, 4), {h0, st}, {cu_seqlens, (size_t)(n_seq + 1) * 4},
                         rows(dout, n_tok, wv, wv, es), {dh_final, st}};
    const Range outs[] = {rows(dq, n_tok, wk, wk, es), rows(dk, n_tok, wk, wk, es), rows(dv, n_tok, wv, wv, es),
                          rows(dg, n_tok, n_heads, n_heads, 4), rows(dbeta, n_tok, n_heads, n_heads, 4), {dh0, st},
                          {workspace, need}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    return launched(kda::launch_gdr_bwd(p, (cudaStream_t)stream), "gated delta rule backward launch");
}

kda_status kda_gdr_step(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                        int64_t v_stride, const float *g, const float *beta, float *state,
                        const int32_t *slots, void *out, int32_t n_rows, int32_t n_slots,
                        int32_t n_k_heads, int32_t n_heads, int32_t d_k, int32_t d_v, kda_dtype dtype,
                        void *stream) {
    kda_status s = check_heads(n_k_heads, n_heads, d_k, d_v, dtype);
    if (s != KDA_OK) return s;
    if (n_rows < 0 || n_slots < 0) return api_fail(KDA_ERR_INVALID_ARG, "n_rows and n_slots must be >= 0");
    if (!slots && n_rows > n_slots) return api_fail(KDA_ERR_INVALID_ARG, "without slots every row needs its state");
    if ((int64_t)n_rows * n_heads > 0x7fffffffLL / 4)
        return api_fail(KDA_ERR_INVALID_ARG, "n_rows * n_heads exceeds 2^29");
    if (n_rows == 0) return api_ok();
    if (!q || !k || !v || !g || !beta || !out || (!state && n_slots > 0))
        return api_fail(KDA_ERR_INVALID_ARG, "every pointer but slots is required");
    const int64_t wk = (int64_t)n_k_heads * d_k, wv = (int64_t)n_heads * d_v;
    if (q_stride < wk || k_stride < wk || v_stride < wv)
        return api_fail(KDA_ERR_INVALID_ARG, "a token stride is smaller than a token's row");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    if (misaligned(q, es) || misaligned(k, es) || misaligned(v, es) || misaligned(out, es))
        return api_fail(KDA_ERR_INVALID_ARG, "q, k, v and out must be aligned to their element size");
    if (misaligned(g, 4) || misaligned(beta, 4) || misaligned(state, 4) || misaligned(slots, 4))
        return api_fail(KDA_ERR_INVALID_ARG, "g, beta, state and slots must be 4-byte aligned");
    const Range ins[] = {rows(q, n_rows, q_stride, wk, es), rows(k, n_rows, k_stride, wk, es),
                         rows(v, n_rows, v_stride, wv, es), rows(g, n_rows, n_heads, n_heads, 4),
                         rows(beta, n_rows, n_heads, n_heads, 4), {slots, (size_t)n_rows * 4}};
    const Range outs[] = {rows(out, n_rows, wv, wv, es), {state, (size_t)n_slots * n_heads * d_k * d_v * 4}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    kda::GdrStepArgs p{q, k, v, q_stride, k_stride, v_stride, g, beta, state, slots, out, n_rows, n_slots,
                       n_k_heads, n_heads, d_k, d_v, dtype == KDA_BF16};
    return launched(kda::launch_gdr_step(p, (cudaStream_t)stream), "gated delta rule step launch");
}

// ---------------------------------------------------------------- linear attention, one decay per head

static kda_status check_dla(const kda::DlaArgs &p, int dtype) {
    kda_status s = check_heads(p.n_k_heads, p.n_heads, p.d_k, p.d_v, dtype);
    if (s != KDA_OK) return s;
    if (p.n_heads > 65535) return api_fail(KDA_ERR_UNSUPPORTED, "n_heads above 65535");
    if (p.n_tok < 0 || p.n_seq < 0) return api_fail(KDA_ERR_INVALID_ARG, "n_tok and n_seq must be >= 0");
    if (p.n_tok > 0x7fffffffLL) return api_fail(KDA_ERR_UNSUPPORTED, "n_tok above 2^31 - 1");
    if (p.n_tok > 0 && p.n_seq == 0) return api_fail(KDA_ERR_INVALID_ARG, "n_tok > 0 needs at least one sequence");
    if ((int64_t)p.n_seq * p.n_heads > 0x7fffffffLL / 8)
        return api_fail(KDA_ERR_INVALID_ARG, "n_seq * n_heads exceeds 2^28");
    // a grid of a CTA for every chunk or segment and head
    if ((p.n_tok / 64 + p.n_seq) * (int64_t)p.n_heads > 0x7fffffffLL)
        return api_fail(KDA_ERR_UNSUPPORTED, "(n_tok / 64 + n_seq) * n_heads above 2^31 - 1");
    if (p.n_seq > 0 && !p.cu_seqlens) return api_fail(KDA_ERR_INVALID_ARG, "cu_seqlens is NULL");
    if (p.n_tok > 0 && (!p.q || !p.k || !p.v || !p.g))
        return api_fail(KDA_ERR_INVALID_ARG, "q, k, v and g are required");
    if (p.g_stride != 0 && p.g_stride != p.n_heads)
        return api_fail(KDA_ERR_INVALID_ARG, "g_stride must be n_heads (a decay per token) or 0 (one per head)");
    if (!(p.scale == p.scale) || p.scale > FLT_MAX || p.scale < -FLT_MAX)
        return api_fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    const int64_t wk = (int64_t)p.n_k_heads * p.d_k, wv = (int64_t)p.n_heads * p.d_v;
    if (p.q_stride < wk || p.k_stride < wk || p.v_stride < wv)
        return api_fail(KDA_ERR_INVALID_ARG, "a token stride is smaller than a token's row");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    const void *elems[] = {p.q, p.k, p.v, p.out, p.dout, p.dq, p.dk, p.dv};
    for (const void *x : elems)
        if (misaligned(x, es)) return api_fail(KDA_ERR_INVALID_ARG, "q, k, v, out and their gradients must be aligned to their element size");
    const void *f32[] = {p.g, p.h0, p.cu_seqlens, p.h_final, p.dh_final, p.dg, p.dh0};
    for (const void *x : f32)
        if (misaligned(x, 4)) return api_fail(KDA_ERR_INVALID_ARG, "g, cu_seqlens, the states and their gradients must be 4-byte aligned");
    return KDA_OK;
}

static kda::DlaArgs dla_args(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, const float *g, int64_t g_stride, const float *h0, const int32_t *cu,
                             float scale, void *workspace, int64_t n_tok, int32_t n_seq, int32_t n_k_heads,
                             int32_t n_heads, int32_t d_k, int32_t d_v, kda_dtype dtype) {
    kda::DlaArgs p{};
    p.q = q; p.k = k; p.v = v;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.g = g; p.g_stride = g_stride; p.h0 = h0; p.cu_seqlens = cu; p.scale = scale; p.workspace = workspace;
    p.n_tok = n_tok; p.n_seq = n_seq; p.n_k_heads = n_k_heads; p.n_heads = n_heads;
    p.d_k = p.in_k = d_k; p.d_v = p.in_v = d_v; p.bf16 = dtype == KDA_BF16;
    return p;
}
static Range dla_decays(const float *g, const kda::DlaArgs &p) {
    return {g, (size_t)(p.g_stride ? p.n_tok : 1) * p.n_heads * 4};
}

size_t kda_dla_chunk_fwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_k_heads, int32_t n_heads,
                                         int32_t d_k, int32_t d_v, kda_dtype dtype) {
    if (!gdr_sizes(n_tok, n_seq, n_k_heads, n_heads, d_k, d_v)) return 0;
    return kda::dla_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, dtype == KDA_BF16, false);
}

kda_status kda_dla_chunk_fwd(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, const float *g, int64_t g_stride, const float *h0,
                             const int32_t *cu_seqlens, float scale, void *out, float *h_final, void *workspace,
                             size_t workspace_bytes, int64_t n_tok, int32_t n_seq, int32_t n_k_heads,
                             int32_t n_heads, int32_t d_k, int32_t d_v, kda_dtype dtype, void *stream) {
    kda::DlaArgs p = dla_args(q, k, v, q_stride, k_stride, v_stride, g, g_stride, h0, cu_seqlens, scale, workspace,
                              n_tok, n_seq, n_k_heads, n_heads, d_k, d_v, dtype);
    p.out = out;
    p.h_final = h_final;
    kda_status s = check_dla(p, dtype);
    if (s != KDA_OK) return s;
    if (n_tok > 0 && !out) return api_fail(KDA_ERR_INVALID_ARG, "out is required");
    if (n_seq == 0) return api_ok();
    const size_t need = n_tok ? kda::dla_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, p.bf16, false) : 0;
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != KDA_OK) return s;
    const size_t es = p.bf16 ? 2 : 4, st = (size_t)n_seq * n_heads * d_k * d_v * 4;
    const int64_t wk = (int64_t)n_k_heads * d_k, wv = (int64_t)n_heads * d_v;
    const Range ins[] = {rows(q, n_tok, q_stride, wk, es), rows(k, n_tok, k_stride, wk, es),
                         rows(v, n_tok, v_stride, wv, es), dla_decays(g, p), {h0, st},
                         {cu_seqlens, (size_t)(n_seq + 1) * 4}};
    const Range outs[] = {rows(out, n_tok, wv, wv, es), {h_final, st}, {workspace, need}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    return launched(kda::launch_dla_fwd(p, (cudaStream_t)stream), "linear attention forward launch");
}

size_t kda_dla_chunk_bwd_workspace_bytes(int64_t n_tok, int32_t n_seq, int32_t n_k_heads, int32_t n_heads,
                                         int32_t d_k, int32_t d_v, kda_dtype dtype) {
    if (!gdr_sizes(n_tok, n_seq, n_k_heads, n_heads, d_k, d_v)) return 0;
    return kda::dla_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, dtype == KDA_BF16, true);
}

kda_status kda_dla_chunk_bwd(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, const float *g, int64_t g_stride, const float *h0,
                             const int32_t *cu_seqlens, float scale, const void *dout, const float *dh_final,
                             void *dq, void *dk, void *dv, float *dg, float *dh0, void *workspace,
                             size_t workspace_bytes, int64_t n_tok, int32_t n_seq, int32_t n_k_heads,
                             int32_t n_heads, int32_t d_k, int32_t d_v, kda_dtype dtype, void *stream) {
    kda::DlaArgs p = dla_args(q, k, v, q_stride, k_stride, v_stride, g, g_stride, h0, cu_seqlens, scale, workspace,
                              n_tok, n_seq, n_k_heads, n_heads, d_k, d_v, dtype);
    p.dout = dout; p.dh_final = dh_final;
    p.dq = dq; p.dk = dk; p.dv = dv; p.dg = dg; p.dh0 = dh0;
    kda_status s = check_dla(p, dtype);
    if (s != KDA_OK) return s;
    if (n_tok > 0 && (!dout || !dq || !dk || !dv))
        return api_fail(KDA_ERR_INVALID_ARG, "dout, dq, dk and dv are required");
    if (n_seq == 0 && !(dg && g_stride == 0)) return api_ok();  // one sum per head is 0 even so
    const size_t need = n_tok ? kda::dla_workspace_bytes(n_tok, n_seq, n_heads, n_k_heads, d_k, d_v, p.bf16, true) : 0;
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != KDA_OK) return s;
    const size_t es = p.bf16 ? 2 : 4, st = (size_t)n_seq * n_heads * d_k * d_v * 4;
    const int64_t wk = (int64_t)n_k_heads * d_k, wv = (int64_t)n_heads * d_v;
    const Range ins[] = {rows(q, n_tok, q_stride, wk, es), rows(k, n_tok, k_stride, wk, es),
                         rows(v, n_tok, v_stride, wv, es), dla_decays(g, p), {h0, st},
                         {cu_seqlens, (size_t)(n_seq + 1) * 4}, rows(dout, n_tok, wv, wv, es), {dh_final, st}};
    const Range outs[] = {rows(dq, n_tok, wk, wk, es), rows(dk, n_tok, wk, wk, es), rows(dv, n_tok, wv, wv, es),
                          dla_decays(dg, p), {dh0, st}, {workspace, need}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    return launched(kda::launch_dla_bwd(p, (cudaStream_t)stream), "linear attention backward launch");
}

kda_status kda_dla_step(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                        int64_t v_stride, const float *g, int64_t g_stride, float *state, const int32_t *slots,
                        float scale, void *out, int32_t n_rows, int32_t n_slots, int32_t n_k_heads, int32_t n_heads,
                        int32_t d_k, int32_t d_v, kda_dtype dtype, void *stream) {
    kda_status s = check_heads(n_k_heads, n_heads, d_k, d_v, dtype);
    if (s != KDA_OK) return s;
    if (n_rows < 0 || n_slots < 0) return api_fail(KDA_ERR_INVALID_ARG, "n_rows and n_slots must be >= 0");
    if (!slots && n_rows > n_slots) return api_fail(KDA_ERR_INVALID_ARG, "without slots every row needs its state");
    if ((int64_t)n_rows * n_heads > 0x7fffffffLL / 4)
        return api_fail(KDA_ERR_INVALID_ARG, "n_rows * n_heads exceeds 2^29");
    if (g_stride != 0 && g_stride != n_heads)
        return api_fail(KDA_ERR_INVALID_ARG, "g_stride must be n_heads (a decay per row) or 0 (one per head)");
    if (!(scale == scale) || scale > FLT_MAX || scale < -FLT_MAX)
        return api_fail(KDA_ERR_INVALID_ARG, "scale must be finite");
    if (n_rows == 0) return api_ok();
    if (!q || !k || !v || !g || !out || (!state && n_slots > 0))
        return api_fail(KDA_ERR_INVALID_ARG, "every pointer but slots is required");
    const int64_t wk = (int64_t)n_k_heads * d_k, wv = (int64_t)n_heads * d_v;
    if (q_stride < wk || k_stride < wk || v_stride < wv)
        return api_fail(KDA_ERR_INVALID_ARG, "a token stride is smaller than a token's row");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    if (misaligned(q, es) || misaligned(k, es) || misaligned(v, es) || misaligned(out, es))
        return api_fail(KDA_ERR_INVALID_ARG, "q, k, v and out must be aligned to their element size");
    if (misaligned(g, 4) || misaligned(state, 4) || misaligned(slots, 4))
        return api_fail(KDA_ERR_INVALID_ARG, "g, state and slots must be 4-byte aligned");
    const Range ins[] = {rows(q, n_rows, q_stride, wk, es), rows(k, n_rows, k_stride, wk, es),
                         rows(v, n_rows, v_stride, wv, es), {g, (size_t)(g_stride ? n_rows : 1) * n_heads * 4},
                         {slots, (size_t)n_rows * 4}};
    const Range outs[] = {rows(out, n_rows, wv, wv, es), {state, (size_t)n_slots * n_heads * d_k * d_v * 4}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    kda::DlaStepArgs p{q, k, v, q_stride, k_stride, v_stride, g, g_stride, state, slots, scale, out, n_rows, n_slots,
                       n_k_heads, n_heads, d_k, d_v, dtype == KDA_BF16};
    return launched(kda::launch_dla_step(p, (cudaStream_t)stream), "linear attention step launch");
}

// ---------------------------------------------------------------- queries and keys

static kda_status check_qk_norm(const kda::QkNormArgs &p, int dtype) {
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return api_fail(KDA_ERR_UNSUPPORTED, "dtype must be KDA_F32 or KDA_BF16");
    if (p.n_tok < 0 || p.heads[0] <= 0 || p.heads[1] <= 0 || p.d <= 0)
        return api_fail(KDA_ERR_INVALID_ARG, "n_tok must be >= 0, the head counts and d positive");
    if (p.d > 256) return api_fail(KDA_ERR_UNSUPPORTED, "d above 256 is not built");
    if (p.heads[0] > 32768 || p.heads[1] > 32768) return api_fail(KDA_ERR_UNSUPPORTED, "more than 32768 heads");
    if (p.n_tok > 0x7fffffffLL) return api_fail(KDA_ERR_UNSUPPORTED, "n_tok above 2^31 - 1");
    if (p.n_freqs < 0 || 2 * (int64_t)p.n_freqs > p.d)
        return api_fail(KDA_ERR_INVALID_ARG, "n_freqs must be from 0 to d / 2");
    if (!(p.eps > 0.f)) return api_fail(KDA_ERR_INVALID_ARG, "eps must be positive");
    if (!p.weight[0] || !p.weight[1]) return api_fail(KDA_ERR_INVALID_ARG, "the weights are required");
    if (p.n_tok > 0 && (!p.x[0] || !p.x[1] || !p.y[0] || !p.y[1]))
        return api_fail(KDA_ERR_INVALID_ARG, "q, k and their results are required");
    if (p.n_tok > 0 && p.n_freqs > 0 && (!p.positions || !p.freqs))
        return api_fail(KDA_ERR_INVALID_ARG, "positions and freqs are required with n_freqs > 0");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    for (int i = 0; i < 2; ++i) {
        if (p.stride[i] < (int64_t)p.heads[i] * p.d || p.dy_stride[i] < (int64_t)p.heads[i] * p.d)
            return api_fail(KDA_ERR_INVALID_ARG, "a token stride is smaller than a token's row");
        if (misaligned(p.x[i], es) || misaligned(p.dy[i], es) || misaligned(p.y[i], es) ||
            misaligned(p.weight[i], 4) || misaligned(p.dw[i], 4))
            return api_fail(KDA_ERR_INVALID_ARG, "every tensor must be aligned to its element size");
    }
    if (misaligned(p.positions, p.wide_positions ? 8 : 4) || misaligned(p.freqs, 8))
        return api_fail(KDA_ERR_INVALID_ARG, "positions and freqs must be aligned to their element size");
    return KDA_OK;
}

kda_status kda_qk_norm_rope_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                const float *q_weight, const float *k_weight, const void *positions,
                                int32_t position_bytes, const double *freqs, int32_t n_freqs, void *q_out,
                                void *k_out, int64_t n_tok, int32_t n_q_heads, int32_t n_k_heads, int32_t d,
                                float eps, int32_t interleaved, kda_dtype dtype, void *stream) {
    if (position_bytes != 4 && position_bytes != 8)
        return api_fail(KDA_ERR_INVALID_ARG, "position_bytes must be 4 or 8");
    kda::QkNormArgs p{};
    p.x[0] = q; p.x[1] = k; p.stride[0] = p.dy_stride[0] = q_stride; p.stride[1] = p.dy_stride[1] = k_stride;
    p.weight[0] = q_weight; p.weight[1] = k_weight; p.y[0] = q_out; p.y[1] = k_out;
    p.positions = positions; p.freqs = freqs; p.n_freqs = n_freqs; p.wide_positions = position_bytes == 8;
    p.n_tok = n_tok; p.heads[0] = n_q_heads; p.heads[1] = n_k_heads; p.d = d; p.eps = eps;
    p.interleaved = interleaved != 0; p.bf16 = dtype == KDA_BF16;
    kda_status s = check_qk_norm(p, dtype);
    if (s != KDA_OK) return s;
    if (n_tok == 0) return api_ok();
    const size_t es = p.bf16 ? 2 : 4;
    const int64_t wq = (int64_t)n_q_heads * d, wk = (int64_t)n_k_heads * d;
    const Range ins[] = {rows(q, n_tok, q_stride, wq, es), rows(k, n_tok, k_stride, wk, es), {q_weight, (size_t)d * 4},
                         {k_weight, (size_t)d * 4}, {positions, (size_t)n_tok * position_bytes}, {freqs, (size_t)n_freqs * 8}};
    const Range outs[] = {rows(q_out, n_tok, wq, wq, es), rows(k_out, n_tok, wk, wk, es)};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    return launched(kda::launch_qk_norm(p, false, (cudaStream_t)stream), "query and key norm launch");
}

size_t kda_qk_norm_rope_bwd_workspace_bytes(int64_t n_tok, int32_t d) {
    if (n_tok < 0 || d <= 0 || d > 256) return 0;
    return kda::qk_norm_workspace_bytes(n_tok, d);
}

kda_status kda_qk_norm_rope_bwd(const void *dq_out, int64_t dq_out_stride, const void *dk_out, int64_t dk_out_stride,
                                const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                const float *q_weight, const float *k_weight, const void *positions,
                                int32_t position_bytes, const double *freqs, int32_t n_freqs, void *dq, void *dk,
                                float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                                int64_t n_tok, int32_t n_q_heads, int32_t n_k_heads, int32_t d, float eps,
                                int32_t interleaved, kda_dtype dtype, void *stream) {
    if (position_bytes != 4 && position_bytes != 8)
        return api_fail(KDA_ERR_INVALID_ARG, "position_bytes must be 4 or 8");
    kda::QkNormArgs p{};
    p.x[0] = q; p.x[1] = k; p.stride[0] = q_stride; p.stride[1] = k_stride;
    p.dy[0] = dq_out; p.dy[1] = dk_out; p.dy_stride[0] = dq_out_stride; p.dy_stride[1] = dk_out_stride;
    p.weight[0] = q_weight; p.weight[1] = k_weight; p.y[0] = dq; p.y[1] = dk; p.dw[0] = dq_weight; p.dw[1] = dk_weight;
    p.partial = static_cast<float *>(workspace);
    p.positions = positions; p.freqs = freqs; p.n_freqs = n_freqs; p.wide_positions = position_bytes == 8;
    p.n_tok = n_tok; p.heads[0] = n_q_heads; p.heads[1] = n_k_heads; p.d = d; p.eps = eps;
    p.interleaved = interleaved != 0; p.bf16 = dtype == KDA_BF16;
    kda_status s = check_qk_norm(p, dtype);
    if (s != KDA_OK) return s;
    if (!dq_weight || !dk_weight) return api_fail(KDA_ERR_INVALID_ARG, "the weights' gradients are required");
    if (n_tok > 0 && (!dq_out || !dk_out)) return api_fail(KDA_ERR_INVALID_ARG, "dq_out and dk_out are required");
    const size_t need = kda::qk_norm_workspace_bytes(n_tok, d);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != KDA_OK) return s;
    const size_t es = p.bf16 ? 2 : 4;
    const int64_t wq = (int64_t)n_q_heads * d, wk = (int64_t)n_k_heads * d;
    const Range ins[] = {rows(q, n_tok, q_stride, wq, es), rows(k, n_tok, k_stride, wk, es),
                         rows(dq_out, n_tok, dq_out_stride, wq, es), rows(dk_out, n_tok, dk_out_stride, wk, es),
                         {q_weight, (size_t)d * 4}, {k_weight, (size_t)d * 4},
                         {positions, (size_t)n_tok * position_bytes}, {freqs, (size_t)n_freqs * 8}};
    const Range outs[] = {rows(dq, n_tok, wq, wq, es), rows(dk, n_tok, wk, wk, es), {dq_weight, (size_t)d * 4},
                          {dk_weight, (size_t)d * 4}, {workspace, need}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    return launched(kda::launch_qk_norm(p, true, (cudaStream_t)stream), "query and key norm backward launch");
}

// ---------------------------------------------------------------- norms

static kda_status check_residual(int64_t n_rows, int32_t d, float eps, int dtype) {
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return api_fail(KDA_ERR_UNSUPPORTED, "dtype must be KDA_F32 or KDA_BF16");
    if (n_rows < 0 || d <= 0) return api_fail(KDA_ERR_INVALID_ARG, "n_rows must be >= 0 and d positive");
    if (n_rows > 0x7fffffffLL) return api_fail(KDA_ERR_UNSUPPORTED, "n_rows above 2^31 - 1");
    if (d > 32768) return api_fail(KDA_ERR_UNSUPPORTED, "d above 32768 is not built");
    if (!(eps > 0.f)) return api_fail(KDA_ERR_INVALID_ARG, "eps must be positive");
    return KDA_OK;
}

kda_status kda_residual_norm_fwd(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                                 const float *scale, const float *weight, void *r, void *y, int64_t n_rows,
                                 int32_t d, float eps, kda_dtype dtype, void *stream) {
    kda_status s = check_residual(n_rows, d, eps, dtype);
    if (s != KDA_OK) return s;
    if (n_rows == 0) return api_ok();
    if (!x || !weight || !y) return api_fail(KDA_ERR_INVALID_ARG, "x, weight and y are required");
    if (x_stride < d || (residual && residual_stride < d))
        return api_fail(KDA_ERR_INVALID_ARG, "a row stride is smaller than d");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    if (misaligned(x, es) || misaligned(residual, es) || misaligned(r, es) || misaligned(y, es) ||
        misaligned(scale, 4) || misaligned(weight, 4))
        return api_fail(KDA_ERR_INVALID_ARG, "every tensor must be aligned to its element size");
    const Range ins[] = {rows(x, n_rows, x_stride, d, es), rows(residual, n_rows, residual_stride, d, es),
                         {scale, (size_t)d * 4}, {weight, (size_t)d * 4}};
    const Range outs[] = {rows(r, n_rows, d, d, es), rows(y, n_rows, d, d, es)};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    kda::ResidualNormArgs p{};
    p.x = x; p.x_stride = x_stride; p.residual = residual; p.residual_stride = residual ? residual_stride : 0;
    p.scale = scale; p.weight = weight; p.r = r; p.y = y;
    p.n_rows = n_rows; p.d = d; p.eps = eps; p.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_residual_norm(p, false, (cudaStream_t)stream), "residual norm launch");
}

size_t kda_residual_norm_bwd_workspace_bytes(int64_t n_rows, int32_t d, int with_scale) {
    if (n_rows < 0 || d <= 0 || d > 32768) return 0;
    return kda::residual_norm_workspace_bytes(n_rows, d, with_scale != 0);
}

kda_status kda_residual_norm_bwd(const void *dy, int64_t dy_stride, const void *dr, int64_t dr_stride,
                                 const void *r, int64_t r_stride, const void *x, int64_t x_stride,
                                 const float *scale, const float *weight, void *dx, void *dresidual,
                                 float *dscale, float *dweight, void *workspace, size_t workspace_bytes,
                                 int64_t n_rows, int32_t d, float eps, kda_dtype dtype, void *stream) {
    kda_status s = check_residual(n_rows, d, eps, dtype);
    if (s != KDA_OK) return s;
    if (!weight || !dweight) return api_fail(KDA_ERR_INVALID_ARG, "weight and dweight are required");
    if (scale ? !dscale : (dscale || dx))
        return api_fail(KDA_ERR_INVALID_ARG, "dscale and dx go with a scale (without one dx is dresidual)");
    if (n_rows > 0 && (!dy || !r || !dresidual || (scale && (!x || !dx))))
        return api_fail(KDA_ERR_INVALID_ARG, "dy, r and dresidual are required, and x and dx with a scale");
    if (dy_stride < d || r_stride < d || (dr && dr_stride < d) || (scale && x_stride < d))
        return api_fail(KDA_ERR_INVALID_ARG, "a row stride is smaller than d");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    const void *elems[] = {dy, dr, r, x, dx, dresidual};
    for (const void *e : elems)
        if (misaligned(e, es)) return api_fail(KDA_ERR_INVALID_ARG, "every tensor must be aligned to its element size");
    if (misaligned(scale, 4) || misaligned(weight, 4) || misaligned(dscale, 4) || misaligned(dweight, 4))
        return api_fail(KDA_ERR_INVALID_ARG, "scale, weight and their gradients must be 4-byte aligned");
    const size_t need = kda::residual_norm_workspace_bytes(n_rows, d, scale != nullptr);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != KDA_OK) return s;
    const Range ins[] = {rows(dy, n_rows, dy_stride, d, es), rows(dr, n_rows, dr_stride, d, es),
                         rows(r, n_rows, r_stride, d, es), rows(scale ? x : nullptr, n_rows, x_stride, d, es),
                         {scale, (size_t)d * 4}, {weight, (size_t)d * 4}};
    const Range outs[] = {rows(dx, n_rows, d, d, es), rows(dresidual, n_rows, d, d, es), {dscale, (size_t)d * 4},
                          {dweight, (size_t)d * 4}, {workspace, need}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    kda::ResidualNormArgs p{};
    p.x = scale ? x : nullptr; p.x_stride = scale ? x_stride : 0;
    p.dy = dy; p.dy_stride = dy_stride; p.dr = dr; p.dr_stride = dr ? dr_stride : 0;
    p.r = const_cast<void *>(r); p.r_stride = r_stride;
    p.scale = scale; p.weight = weight; p.dx = dx; p.dresidual = dresidual; p.dw = dweight; p.dscale = dscale;
    p.partial = static_cast<float *>(workspace);
    p.n_rows = n_rows; p.d = d; p.eps = eps; p.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_residual_norm(p, true, (cudaStream_t)stream), "residual norm backward launch");
}

static kda_status check_gated(int64_t n_tok, int32_t n_heads, int32_t d, float eps, int32_t act, int dtype) {
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return api_fail(KDA_ERR_UNSUPPORTED, "dtype must be KDA_F32 or KDA_BF16");
    if (act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU)
        return api_fail(KDA_ERR_INVALID_ARG, "activation must be KDA_ACT_SIGMOID or KDA_ACT_SILU");
    if (n_tok < 0 || n_heads <= 0 || d <= 0)
        return api_fail(KDA_ERR_INVALID_ARG, "n_tok must be >= 0, n_heads and d positive");
    if (d > 256) return api_fail(KDA_ERR_UNSUPPORTED, "d above 256 is not built");
    if (n_tok > 0x7fffffffLL / n_heads) return api_fail(KDA_ERR_UNSUPPORTED, "n_tok * n_heads above 2^31 - 1");
    if (!(eps > 0.f)) return api_fail(KDA_ERR_INVALID_ARG, "eps must be positive");
    return KDA_OK;
}

kda_status kda_gated_norm_fwd(const void *x, int64_t x_stride, const void *gate, int64_t gate_stride,
                              const float *weight, void *y, int64_t n_tok, int32_t n_heads, int32_t d,
                              float eps, int32_t activation, kda_dtype dtype, void *stream) {
    kda_status s = check_gated(n_tok, n_heads, d, eps, activation, dtype);
    if (s != KDA_OK) return s;
    if (n_tok == 0) return api_ok();
    if (!x || !gate || !weight || !y) return api_fail(KDA_ERR_INVALID_ARG, "x, gate, weight and y are required");
    const int64_t w = (int64_t)n_heads * d;
    if (x_stride < w || gate_stride < w) return api_fail(KDA_ERR_INVALID_ARG, "a token stride is smaller than a token's row");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    if (misaligned(x, es) || misaligned(gate, es) || misaligned(y, es) || misaligned(weight, 4))
        return api_fail(KDA_ERR_INVALID_ARG, "every tensor must be aligned to its element size");
    const Range ins[] = {rows(x, n_tok, x_stride, w, es), rows(gate, n_tok, gate_stride, w, es), {weight, (size_t)d * 4}};
    const Range outs[] = {rows(y, n_tok, w, w, es)};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    kda::GatedNormArgs p{};
    p.x = x; p.x_stride = x_stride; p.gate = gate; p.gate_stride = gate_stride; p.weight = weight; p.y = y;
    p.n_tok = n_tok; p.n_heads = n_heads; p.d = d; p.eps = eps; p.silu = activation == KDA_ACT_SILU;
    p.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_gated_norm(p, false, (cudaStream_t)stream), "gated norm launch");
}

size_t kda_gated_norm_bwd_workspace_bytes(int64_t n_tok, int32_t n_heads, int32_t d) {
    if (n_tok < 0 || n_heads <= 0 || d <= 0 || d > 256) return 0;
    return kda::gated_norm_workspace_bytes(n_tok, n_heads, d);
}

kda_status kda_gated_norm_bwd(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride,
                              const void *gate, int64_t gate_stride, const float *weight, void *dx, void *dgate,
                              float *dweight, void *workspace, size_t workspace_bytes, int64_t n_tok,
                              int32_t n_heads, int32_t d, float eps, int32_t activation, kda_dtype dtype,
                              void *stream) {
    kda_status s = check_gated(n_tok, n_heads, d, eps, activation, dtype);
    if (s != KDA_OK) return s;
    if (!weight || !dweight) return api_fail(KDA_ERR_INVALID_ARG, "weight and dweight are required");
    if (n_tok > 0 && (!dy || !x || !gate || !dx || !dgate))
        return api_fail(KDA_ERR_INVALID_ARG, "dy, x, gate, dx and dgate are required");
    const int64_t w = (int64_t)n_heads * d;
    if (x_stride < w || gate_stride < w || dy_stride < w)
        return api_fail(KDA_ERR_INVALID_ARG, "a token stride is smaller than a token's row");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    const void *elems[] = {dy, x, gate, dx, dgate};
    for (const void *e : elems)
        if (misaligned(e, es)) return api_fail(KDA_ERR_INVALID_ARG, "every tensor must be aligned to its element size");
    if (misaligned(weight, 4) || misaligned(dweight, 4))
        return api_fail(KDA_ERR_INVALID_ARG, "weight and dweight must be 4-byte aligned");
    const size_t need = kda::gated_norm_workspace_bytes(n_tok, n_heads, d);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != KDA_OK) return s;
    const Range ins[] = {rows(dy, n_tok, dy_stride, w, es), rows(x, n_tok, x_stride, w, es),
                         rows(gate, n_tok, gate_stride, w, es), {weight, (size_t)d * 4}};
    const Range outs[] = {rows(dx, n_tok, w, w, es), rows(dgate, n_tok, w, w, es), {dweight, (size_t)d * 4},
                          {workspace, need}};
    if (clash(ins, outs)) return api_fail(KDA_ERR_INVALID_ARG, kOverlap);
    kda::GatedNormArgs p{};
    p.x = x; p.x_stride = x_stride; p.gate = gate; p.gate_stride = gate_stride; p.dy = dy; p.dy_stride = dy_stride;
    p.weight = weight; p.dx = dx; p.dgate = dgate; p.dw = dweight; p.partial = static_cast<float *>(workspace);
    p.n_tok = n_tok; p.n_heads = n_heads; p.d = d; p.eps = eps; p.silu = activation == KDA_ACT_SILU;
    p.bf16 = dtype == KDA_BF16;
    return launched(kda::launch_gated_norm(p, true, (cudaStream_t)stream), "gated norm backward launch");
}

}  // extern "C"
