// C-ABI front end of libgdntree.so: host-side argument validation, kernel
// selection and asynchronous launch on the caller's stream.  The declared
// contract (layouts, ownership, errors) is in include/gdn_tree.h.
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <cmath>

#include "serving.hpp"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool dim_ok(int d) { return d >= 8 && d <= GDN_MAX_DIM && d % 8 == 0; }

gdn_status shape_status(int batch, int n, int H, int dk, int dv) {
    if (batch < 1 || n < 1 || H < 1 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
    if (n > GDN_MAX_NODES || !dim_ok(dk) || !dim_ok(dv)) return GDN_ERR_UNSUPPORTED;
    // element offsets are formed in 64-bit, but grid.x = batch * H must fit
    if ((long long)batch * H > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// log2 of a power of two, -1 for anything else
int log2_exact(int x) { return x >= 1 && (x & (x - 1)) == 0 ? __builtin_ctz((unsigned)x) : -1; }

template <typename... P>
bool all_aligned(const P *...p) {
    return (... && (!p || aligned16(p)));
}

gdn_status rule_status(const gdn::RuleArgs &a) {
    if (!a.S || !a.src || !a.dst) return GDN_ERR_INVALID_ARG;
    if (a.rows > 0 && (!a.q || !a.k || !a.v || !a.alpha || !a.beta || !a.out))
        return GDN_ERR_INVALID_ARG;
    if (a.dtype != GDN_DTYPE_F32 && a.dtype != GDN_DTYPE_BF16) return GDN_ERR_INVALID_ARG;
    if (a.out_dtype != GDN_DTYPE_F32 && a.out_dtype != GDN_DTYPE_BF16) return GDN_ERR_INVALID_ARG;
    if (!all_aligned((const char *)a.q, (const char *)a.k, (const char *)a.v, a.alpha, a.beta,
                     a.cu, a.S, a.src, a.dst, (const char *)a.out, (const char *)a.workspace,
                     a.status))
        return GDN_ERR_INVALID_ARG;
    if (a.batch < 1 || a.rows < 0 || a.slots < 1 || a.H < 1 || a.Hk < 1 || a.dk < 1 || a.dv < 1)
        return GDN_ERR_INVALID_ARG;
    if (a.H % a.Hk != 0 || !dim_ok(a.dk) || !dim_ok(a.dv)) return GDN_ERR_UNSUPPORTED;
    // a chunk's rows are addressed with 32-bit byte offsets
    if (a.H > 16384) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// threads of a launch are counted in 32 bits
bool grid_ok(long long workgroups, long long threads) {
    return workgroups <= 0xffffffffLL / threads;
}

// ---- heads of queries and keys
int64_t element_bytes(gdn_dtype t) { return t == GDN_DTYPE_F32 ? 4 : 2; }

bool dtype_ok(gdn_dtype t) {
    return t == GDN_DTYPE_F32 || t == GDN_DTYPE_BF16 || t == GDN_DTYPE_F16;
}

bool aligned_to(const void *p, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0;
}

template <typename... P>
bool all_aligned4(const P *...p) {
    return (... && (!p || aligned_to(p, 4)));
}

// rows [rows][heads][d] to read: strides not negative, offsets in 63 bits
bool strides_ok(int64_t row, int64_t head) {
    return row >= 0 && head >= 0 && row <= (1LL << 40) && head <= (1LL << 40);
}

// and to write: no two elements in one place
bool apart(int rows, int64_t row, int heads, int64_t head, int d) {
    if (rows <= 1) return heads <= 1 || head >= d;
    if (heads <= 1) return row >= d;
    return (head >= d && row >= d && (row - d) / head >= heads - 1) ||
           (row >= d && head >= d && (head - d) / row >= rows - 1);
}

// What a call does not use may be anything: it goes before the checks, so that no
// kernel sees it.
gdn::HeadsArgs used(gdn::HeadsArgs a) {
    for (gdn::HeadsPart *x : {&a.q, &a.k}) {
        if (x->heads == 0 || a.norm == GDN_NORM_NONE) x->weight = nullptr;
        if (!x->weight) x->weight_head = 0;
    }
    if (a.rot == 0) a.pos = a.base = nullptr, a.inv_freq = nullptr;
    return a;
}

gdn_status part_status(const gdn::HeadsPart &x, const gdn::HeadsArgs &a, bool out_needed) {
    if (x.heads == 0) return GDN_OK;
    if (!x.in || (out_needed && !x.out)) return GDN_ERR_INVALID_ARG;
    const int64_t e = element_bytes(a.dtype);
    if (!aligned_to(x.in, e) || !aligned_to(x.out, e) ||
        !aligned_to(x.weight, a.wide_weight ? 4 : e))
        return GDN_ERR_INVALID_ARG;
    if (!strides_ok(x.in_row, x.in_head)) return GDN_ERR_INVALID_ARG;
    if (x.out && (!strides_ok(x.out_row, x.out_head) ||
                  !apart(a.rows, x.out_row, x.heads, x.out_head, a.d)))
        return GDN_ERR_INVALID_ARG;
    if (x.weight && x.weight_head != 0 && x.weight_head != a.d) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// pointers are of no interest where there are no rows; `weight_dtype` as the caller gave it
gdn_status heads_status(const gdn::HeadsArgs &a, gdn_dtype weight_dtype, bool own_positions,
                        bool k_out_needed) {
    if (!dtype_ok(a.dtype)) return GDN_ERR_INVALID_ARG;
    if (a.norm != GDN_NORM_NONE && a.norm != GDN_NORM_RMS && a.norm != GDN_NORM_L2)
        return GDN_ERR_INVALID_ARG;
    if (a.layout != GDN_ROPE_HALF && a.layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_INVALID_ARG;
    if (a.norm != GDN_NORM_NONE && (a.q.weight || a.k.weight) && weight_dtype != a.dtype &&
        weight_dtype != GDN_DTYPE_F32)
        return GDN_ERR_INVALID_ARG;
    if (a.rows < 0 || a.q.heads < 0 || a.k.heads < 0 || a.q.heads + (int64_t)a.k.heads < 1 ||
        a.d < 1 || a.rot < 0 || a.rot > a.d || a.rot % 2 != 0)
        return GDN_ERR_INVALID_ARG;
    if (a.d > GDN_MAX_HEAD_DIM || a.q.heads > 65535 || a.k.heads > 65535)
        return GDN_ERR_UNSUPPORTED;
    if (a.base && a.base_rows < 1) return GDN_ERR_INVALID_ARG;
    if (a.rows == 0) return GDN_OK;
    if (a.rot > 0 && (!a.inv_freq || (own_positions && !a.pos))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned4(a.pos, a.base, a.inv_freq)) return GDN_ERR_INVALID_ARG;
    gdn_status st = part_status(a.q, a, true);
    if (st == GDN_OK) st = part_status(a.k, a, k_out_needed);
    return st;
}

// pointers are of no interest where there are no requests
gdn_status count_status(const gdn::CountArgs &a) {
    if (a.m < 0 || a.slots < 1 || a.vocab < 1 || a.stride < a.vocab) return GDN_ERR_INVALID_ARG;
    if (a.vocab > GDN_MAX_VOCAB || a.m > GDN_MAX_REQUESTS || a.stride > (1LL << 40))
        return GDN_ERR_UNSUPPORTED;
    if (a.m > 0 && (!a.counts || !a.slot || !aligned_to(a.counts, 2) ||
                    !all_aligned4(a.slot, a.status)))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn_status page_status(const gdn::PageArgs &a, int m, int page) {
    if (!a.table || !a.length || !a.ref) return GDN_ERR_INVALID_ARG;
    if (!all_aligned(a.table, a.length, a.ref, a.status)) return GDN_ERR_INVALID_ARG;
    if (m < 0 || a.seqs < 1 || a.width < 1 || a.pool < 1 || page < 1) return GDN_ERR_INVALID_ARG;
    // tokens and pages are counted in 32 bits, by loops that step past their end
    if (a.page_log < 0 || (long long)a.width * page > GDN_MAX_TOKENS || a.pool > GDN_MAX_PAGES)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status from_hip(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

}  // namespace

namespace gdn {

int device_cu_count() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v <= 0) {
        if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            v <= 0)
            v = 256;
        cache[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

}  // namespace gdn

extern "C" {

gdn_status gdn_tree_verify(const void *q, const void *k, const void *v, gdn_dtype qkv_dtype,
                           const float *alpha, const float *beta, const int32_t *parent,
                           const float *S0, float *out, int batch, int n, int H, int d_k,
                           int d_v, int32_t *status, void *stream) {
    if (!q || !k || !v || !alpha || !beta || !parent || !S0 || !out) return GDN_ERR_INVALID_ARG;
    if (qkv_dtype != GDN_DTYPE_F32 && qkv_dtype != GDN_DTYPE_BF16) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, beta, parent, S0, out, status};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    const gdn_status st = shape_status(batch, n, H, d_k, d_v);
    if (st != GDN_OK) return st;
    gdn::VerifyArgs a{q, k, v, qkv_dtype, alpha, beta, parent, S0, out,
                      batch, n, H, d_k, d_v, status};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (gdn::verify_split_supports(a)) return from_hip(gdn::launch_verify_split(a, s));
    if (gdn::verify_mfma_supports(a)) return from_hip(gdn::launch_verify_mfma(a, s));
    if (gdn::verify_mfma128_supports(a)) return from_hip(gdn::launch_verify_mfma128(a, s));
    if (gdn::verify_f32_supports(a)) return from_hip(gdn::launch_verify_f32(a, s));
    return from_hip(gdn::launch_verify_generic(a, s));
}

gdn_status gdn_branch_verify(const void *q, const void *k, const void *v, gdn_dtype qkv_dtype,
                             const float *alpha, const float *beta, const int32_t *parent,
                             const float *S0, float *out, int batch, int n, int H, int d_k,
                             int d_v, int32_t *status, void *stream) {
    if (!q || !k || !v || !alpha || !beta || !parent || !S0 || !out) return GDN_ERR_INVALID_ARG;
    if (qkv_dtype != GDN_DTYPE_F32 && qkv_dtype != GDN_DTYPE_BF16) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, beta, parent, S0, out, status};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    const gdn_status st = shape_status(batch, n, H, d_k, d_v);
    if (st != GDN_OK) return st;
    gdn::VerifyArgs a{q, k, v, qkv_dtype, alpha, beta, parent, S0, out,
                      batch, n, H, d_k, d_v, status};
    return from_hip(gdn::launch_branch_verify(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_tree_commit(float *S, const int32_t *path, const int32_t *path_len, int max_path,
                           const void *k, const void *v, gdn_dtype qkv_dtype, const float *alpha,
                           const float *beta, const int32_t *parent, int batch, int n, int H,
                           int d_k, int d_v, int32_t *status, void *stream) {
    if (!S || !path || !path_len || !k || !v || !alpha || !beta || !parent)
        return GDN_ERR_INVALID_ARG;
    if (qkv_dtype != GDN_DTYPE_F32 && qkv_dtype != GDN_DTYPE_BF16) return GDN_ERR_INVALID_ARG;
    if (max_path < 1) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {S, path, path_len, k, v, alpha, beta, parent, status};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    const gdn_status st = shape_status(batch, n, H, d_k, d_v);
    if (st != GDN_OK) return st;
    gdn::CommitArgs a{S, path, path_len, max_path, k, v, qkv_dtype, alpha, beta, parent,
                      batch, n, H, d_k, d_v, status};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (gdn::commit_split_supports(a)) return from_hip(gdn::launch_commit_split(a, s));
    if (gdn::commit_mfma_supports(a)) return from_hip(gdn::launch_commit_mfma(a, s));
    if (gdn::commit_f32_supports(a)) return from_hip(gdn::launch_commit_f32(a, s));
    return from_hip(gdn::launch_commit(a, s));
}

gdn_status gdn_tree_commit_verify(float *S, const int32_t *path, const int32_t *path_len,
                                  int max_path, const void *k_prev, const void *v_prev,
                                  const float *alpha_prev, const float *beta_prev,
                                  const int32_t *parent_prev, const void *u_prev, int n_prev,
                                  const void *q, const void *k, const void *v,
                                  gdn_dtype qkv_dtype, const float *alpha, const float *beta,
                                  const int32_t *parent, float *out, void *u_out,
                                  gdn_dtype u_dtype, int batch, int n, int H, int d_k, int d_v,
                                  int32_t *status, void *stream) {
    if (!S || !path || !path_len || !k_prev || !v_prev || !alpha_prev || !beta_prev ||
        !parent_prev || !q || !k || !v || !alpha || !beta || !parent || !out)
        return GDN_ERR_INVALID_ARG;
    if (qkv_dtype != GDN_DTYPE_F32 && qkv_dtype != GDN_DTYPE_BF16) return GDN_ERR_INVALID_ARG;
    if (max_path < 1) return GDN_ERR_INVALID_ARG;
    if ((u_prev || u_out) && u_dtype != GDN_DTYPE_F32 && u_dtype != GDN_DTYPE_F16)
        return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {S,    path, path_len, k_prev, v_prev, alpha_prev, beta_prev, parent_prev,
                          u_prev, q,  k,        v,      alpha,  beta,       parent,    out,
                          u_out, status};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    gdn_status st = shape_status(batch, n_prev, H, d_k, d_v);
    if (st == GDN_OK) st = shape_status(batch, n, H, d_k, d_v);
    if (st != GDN_OK) return st;
    gdn::CommitVerifyArgs a{
        {S, path, path_len, max_path, k_prev, v_prev, qkv_dtype, alpha_prev, beta_prev,
         parent_prev, batch, n_prev, H, d_k, d_v, status},
        {q, k, v, qkv_dtype, alpha, beta, parent, S, out, batch, n, H, d_k, d_v, status, true},
        u_prev,
        u_out,
        u_dtype == GDN_DTYPE_F16};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (gdn::commit_verify_split_supports(a))
        return from_hip(gdn::launch_commit_verify_split(a, s));
    if (gdn::commit_verify_mfma_supports(a)) return from_hip(gdn::launch_commit_verify_mfma(a, s));
    // 65..128 new nodes: one launch, the commit solving for its
    // pseudo-values (u_prev not needed)
    if (gdn::commit_verify_mfma128_supports(a))
        return from_hip(gdn::launch_commit_verify_mfma128(a, s));
    if (u_out) return GDN_ERR_UNSUPPORTED;
    // other shapes: the two halves as separate launches on the same stream
    // (the commit solves for the pseudo-values itself, so u_prev is not
    // needed), the verify ORing its flag into what the commit wrote
    const hipError_t e = gdn::commit_mfma_supports(a.c) ? gdn::launch_commit_mfma(a.c, s)
                         : gdn::commit_f32_supports(a.c) ? gdn::launch_commit_f32(a.c, s)
                                                         : gdn::launch_commit(a.c, s);
    if (e != hipSuccess) return GDN_ERR_HIP;
    if (gdn::verify_mfma128_supports(a.v)) return from_hip(gdn::launch_verify_mfma128(a.v, s));
    if (gdn::verify_f32_supports(a.v)) return from_hip(gdn::launch_verify_f32(a.v, s));
    return from_hip(gdn::launch_verify_generic(a.v, s));
}

gdn_status gdn_tree_path(const int32_t *parent, const int32_t *accepted, int32_t *path,
                         int32_t *path_len, int batch, int n, int max_path, int32_t *status,
                         void *stream) {
    if (!parent || !accepted || !path || !path_len) return GDN_ERR_INVALID_ARG;
    if (batch < 1 || n < 1 || max_path < 1) return GDN_ERR_INVALID_ARG;
    if (n > GDN_MAX_NODES) return GDN_ERR_UNSUPPORTED;
    const void *ptrs[] = {parent, accepted, path, path_len, status};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_path(parent, accepted, path, path_len, batch, n, max_path, status,
                                     static_cast<hipStream_t>(stream)));
}

gdn_status gdn_tree_build(const float *cand_logp, const int32_t *cand_tok, const int32_t *root_tok,
                          int32_t *parent, int32_t *token, float *score, int32_t *n_built,
                          int batch, int n, int K, int width, int max_depth, void *stream) {
    if (!cand_logp || !cand_tok || !parent || !token || !score) return GDN_ERR_INVALID_ARG;
    if (batch < 1 || n < 1 || K < 1 || width < 1 || max_depth < 0) return GDN_ERR_INVALID_ARG;
    if (n > GDN_MAX_NODES || K > GDN_MAX_CANDIDATES) return GDN_ERR_UNSUPPORTED;
    const void *ptrs[] = {cand_logp, cand_tok, root_tok, parent, token, score, n_built};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_tree_build(cand_logp, cand_tok, root_tok, parent, token, score,
                                           n_built, batch, n, K, width, max_depth,
                                           static_cast<hipStream_t>(stream)));
}

gdn_status gdn_tree_accept(const int32_t *parent, const int32_t *draft_tok,
                           const int32_t *verify_tok, int32_t *accepted, int32_t *accept_len,
                           int32_t *bonus_tok, int batch, int n, int32_t *status, void *stream) {
    if (!parent || !draft_tok || !verify_tok || !accepted) return GDN_ERR_INVALID_ARG;
    if (batch < 1 || n < 1) return GDN_ERR_INVALID_ARG;
    if (n > GDN_MAX_NODES) return GDN_ERR_UNSUPPORTED;
    const void *ptrs[] = {parent, draft_tok, verify_tok, accepted, accept_len, bonus_tok, status};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_accept(parent, draft_tok, verify_tok, accepted, accept_len,
                                       bonus_tok, batch, n, status,
                                       static_cast<hipStream_t>(stream)));
}

gdn_status gdn_tree_index(const int32_t *parent, int32_t *depth, uint32_t *anc, int batch, int n,
                          int32_t *status, void *stream) {
    if (!parent || !depth || !anc) return GDN_ERR_INVALID_ARG;
    if (batch < 1 || n < 1) return GDN_ERR_INVALID_ARG;
    if (n > GDN_MAX_NODES) return GDN_ERR_UNSUPPORTED;
    const void *ptrs[] = {parent, depth, anc, status};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_index(parent, depth, anc, batch, n, status,
                                      static_cast<hipStream_t>(stream)));
}

int64_t gdn_prefill_workspace(gdn_dtype qkv_dtype, int batch, int rows, int H, int Hk, int d_k,
                              int d_v) {
    if (batch < 1 || rows < 0 || H < 1 || Hk < 1 || H % Hk != 0 || !dim_ok(d_k) || !dim_ok(d_v))
        return 0;
    gdn::RuleArgs a{};
    a.dtype = qkv_dtype;
    a.batch = batch, a.rows = rows, a.H = H, a.Hk = Hk, a.dk = d_k, a.dv = d_v;
    return gdn::prefill_workspace(a);
}

gdn_status gdn_prefill(const void *q, const void *k, const void *v, gdn_dtype qkv_dtype,
                       const float *alpha, const float *beta, const int32_t *cu, float *S,
                       const int32_t *src, const int32_t *dst, void *out, gdn_dtype out_dtype,
                       int batch, int rows, int slots, int H, int Hk, int d_k, int d_v,
                       void *workspace, int64_t workspace_bytes, int32_t *status, void *stream) {
    gdn::RuleArgs a{q,   k,         v,     qkv_dtype, alpha, beta, cu, S,   src,  dst,
                    out, out_dtype, batch, rows,      slots, H,    Hk, d_k, d_v,  workspace,
                    status};
    if (!cu) return GDN_ERR_INVALID_ARG;
    const gdn_status st = rule_status(a);
    if (st != GDN_OK) return st;
    // chunks of 64 tokens and heads; sequences, heads and 16 columns
    if (!grid_ok(((long long)rows / 64 + batch) * H, 256) ||
        !grid_ok((long long)batch * H * ((d_v + 15) / 16), 512))
        return GDN_ERR_UNSUPPORTED;
    const int64_t need = gdn::prefill_workspace(a);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_prefill(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_step(const void *q, const void *k, const void *v, gdn_dtype qkv_dtype,
                    const float *alpha, const float *beta, float *S, const int32_t *src,
                    const int32_t *dst, void *out, gdn_dtype out_dtype, int batch, int slots,
                    int H, int Hk, int d_k, int d_v, int32_t *status, void *stream) {
    gdn::RuleArgs a{q,   k,         v,     qkv_dtype, alpha, beta, nullptr, S,   src,  dst,
                    out, out_dtype, batch, batch,     slots, H,    Hk,      d_k, d_v,  nullptr,
                    status};
    const gdn_status st = rule_status(a);
    if (st != GDN_OK) return st;
    if (!grid_ok((long long)batch * H * ((d_v + 31) / 32), 256)) return GDN_ERR_UNSUPPORTED;
    return from_hip(gdn::launch_step(a, static_cast<hipStream_t>(stream)));
}

int64_t gdn_tree_attention_workspace(int batch, int n, int Hq, int Hkv, int d, int page,
                                     int max_pages, int groups) {
    if (batch < 1 || n < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d < 1 || max_pages < 1 ||
        log2_exact(page) < 0)
        return 0;
    gdn::AttentionArgs a{};
    a.batch = batch, a.n = n, a.Hq = Hq, a.Hkv = Hkv, a.d = d, a.page_log = log2_exact(page);
    a.max_pages = max_pages, a.groups = groups;
    return gdn::attention_workspace(a);
}

gdn_status gdn_tree_attention(const void *q, const void *k, const void *v, gdn_dtype dtype,
                              const int32_t *parent, const void *k_cache, const void *v_cache,
                              int64_t page_stride, const int32_t *pages, const int32_t *length,
                              const int32_t *group_start, const int32_t *group_shared, int groups,
                              float scale, void *out, int batch, int n, int Hq, int Hkv, int d,
                              int page, int num_pages, int max_pages, void *workspace,
                              int64_t workspace_bytes, int32_t *status, void *stream) {
    if (!q || !k || !v || !parent || !k_cache || !v_cache || !pages || !length || !out)
        return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F16) return GDN_ERR_INVALID_ARG;
    if (groups < 0 || (groups > 0 && (!group_start || !group_shared))) return GDN_ERR_INVALID_ARG;
    if (!all_aligned((const char *)q, (const char *)k, (const char *)v, parent,
                     (const char *)k_cache, (const char *)v_cache, pages, length, group_start,
                     group_shared, (const char *)out, (const char *)workspace, status))
        return GDN_ERR_INVALID_ARG;
    if (batch < 1 || n < 1 || Hq < 1 || Hkv < 1 || d < 1 || page < 1 || num_pages < 1 ||
        max_pages < 1)
        return GDN_ERR_INVALID_ARG;
    const int page_log = log2_exact(page);
    if (n > GDN_MAX_NODES || Hq % Hkv != 0 || d % 8 != 0 || d > GDN_MAX_HEAD_DIM || page_log < 0 ||
        batch > GDN_MAX_SEQUENCES || groups > GDN_MAX_SEQUENCES)
        return GDN_ERR_UNSUPPORTED;
    // tokens, and the query rows of a group, are counted in 32 bits
    if ((long long)max_pages * page > GDN_MAX_TOKENS ||
        (long long)batch * n * Hq > 0x3fffffffLL)
        return GDN_ERR_UNSUPPORTED;
    // the joining kernel: a workgroup of 256 for every 4 rows (d > 128) to 16 (d <= 64)
    if (!grid_ok((long long)batch * (((long long)n * Hq + 3) / 4), 256)) return GDN_ERR_UNSUPPORTED;
    if (page_stride % 8 != 0 || page_stride < (int64_t)Hkv * page * d) return GDN_ERR_INVALID_ARG;
    // rows inside a page, or inside a tree, are addressed with 32-bit byte offsets
    if (page_stride > 0x7fffffffLL || (long long)Hkv * d > 0xffffffLL) return GDN_ERR_UNSUPPORTED;
    gdn::AttentionArgs a{q,      k,      v,           dtype,        parent, k_cache, v_cache,
                         page_stride, pages, length,  group_start,  group_shared, groups,
                         scale,  out,    batch,       n,            Hq,     Hkv,     d,
                         page_log, num_pages, max_pages, workspace, status};
    if (!workspace || workspace_bytes < gdn::attention_workspace(a)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_tree_attention(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_page_fork(int32_t *table, int32_t *length, int32_t *ref, const int32_t *src,
                         const int32_t *dst, int32_t *copies, int m, int seqs, int max_pages,
                         int pool, int page, int32_t *status, void *stream) {
    const gdn::PageArgs a{table, length, ref, seqs, max_pages, pool, log2_exact(page), status};
    const gdn_status st = page_status(a, m, page);
    if (st != GDN_OK) return st;
    if (m == 0) return GDN_OK;
    if (!src || !dst || !copies || !all_aligned(src, dst, copies)) return GDN_ERR_INVALID_ARG;
    if (m > GDN_MAX_REQUESTS) return GDN_ERR_UNSUPPORTED;
    return from_hip(
        gdn::launch_page_fork(a, src, dst, copies, m, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_page_extend(int32_t *table, int32_t *length, int32_t *ref, const int32_t *dst,
                           const int32_t *add, int32_t *begin, int m, int seqs, int max_pages,
                           int pool, int page, int32_t *status, void *stream) {
    const gdn::PageArgs a{table, length, ref, seqs, max_pages, pool, log2_exact(page), status};
    const gdn_status st = page_status(a, m, page);
    if (st != GDN_OK) return st;
    if (m == 0) return GDN_OK;
    if (!dst || !add || !begin || !all_aligned(dst, add, begin)) return GDN_ERR_INVALID_ARG;
    if (m > GDN_MAX_REQUESTS) return GDN_ERR_UNSUPPORTED;
    return from_hip(
        gdn::launch_page_extend(a, dst, add, begin, m, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_page_free(int32_t *table, int32_t *length, int32_t *ref, const int32_t *done, int m,
                         int seqs, int max_pages, int pool, int page, int32_t *status,
                         void *stream) {
    const gdn::PageArgs a{table, length, ref, seqs, max_pages, pool, log2_exact(page), status};
    const gdn_status st = page_status(a, m, page);
    if (st != GDN_OK) return st;
    if (m == 0) return GDN_OK;
    if (!done || !all_aligned(done)) return GDN_ERR_INVALID_ARG;
    if (!grid_ok(m, gdn::kRowThreads)) return GDN_ERR_UNSUPPORTED;
    return from_hip(gdn::launch_page_free(a, done, m, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_page_compact(int32_t *table, const int32_t *length, int32_t *ref, int32_t *copies,
                            int32_t *count, int32_t *workspace, int seqs, int max_pages, int pool,
                            int page, void *stream) {
    const gdn::PageArgs a{table, const_cast<int32_t *>(length), ref,    seqs, max_pages,
                          pool,  log2_exact(page),              nullptr};
    const gdn_status st = page_status(a, 0, page);
    if (st != GDN_OK) return st;
    if ((pool > 1 && !copies) || !count || !workspace) return GDN_ERR_INVALID_ARG;
    if (!all_aligned(copies, count, workspace)) return GDN_ERR_INVALID_ARG;
    if (!grid_ok(seqs, gdn::kRowThreads)) return GDN_ERR_UNSUPPORTED;
    return from_hip(
        gdn::launch_page_compact(a, copies, count, workspace, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_page_copy(void *cache, const int32_t *copies, const int32_t *count, int m,
                         int planes, int pool, int64_t page_bytes, void *stream) {
    if (m < 0 || planes < 1 || pool < 1 || page_bytes < 16) return GDN_ERR_INVALID_ARG;
    if (m == 0) return GDN_OK;
    if (!cache || !copies || !all_aligned((const char *)cache, copies, count) ||
        page_bytes % 16 != 0)
        return GDN_ERR_INVALID_ARG;
    const int64_t parts = gdn::page_copy_parts(page_bytes);
    if (planes > 65535 || parts > 0xffffffffLL || !grid_ok(parts * m, gdn::kCopyThreads))
        return GDN_ERR_UNSUPPORTED;
    return from_hip(gdn::launch_page_copy(cache, copies, count, m, planes, pool, page_bytes,
                                          static_cast<hipStream_t>(stream)));
}

gdn_status gdn_kv_commit(void *k_cache, void *v_cache, int64_t page_stride, const int32_t *table,
                         const int32_t *dst, const int32_t *begin, const void *k, const void *v,
                         const int32_t *path, const int32_t *add, int m, int n, int max_path,
                         int Hkv, int d, int elem_bytes, int seqs, int max_pages, int pool,
                         int page, int32_t *status, void *stream) {
    if (m < 0 || n < 1 || max_path < 1 || Hkv < 1 || d < 1 || seqs < 1 || max_pages < 1 ||
        pool < 1 || page < 1 || (elem_bytes != 2 && elem_bytes != 4))
        return GDN_ERR_INVALID_ARG;
    if (m == 0) return GDN_OK;
    if (!k_cache || !v_cache || !table || !dst || !begin || !k || !v || !path || !add)
        return GDN_ERR_INVALID_ARG;
    if (!all_aligned((const char *)k_cache, (const char *)v_cache, table, dst, begin,
                     (const char *)k, (const char *)v, path, add, status))
        return GDN_ERR_INVALID_ARG;
    const int page_log = log2_exact(page);
    // rows are moved in 16-byte pieces; tokens and a token's pieces are counted
    // in 32 bits
    if (page_log < 0 || d % 8 != 0 || (long long)max_pages * page > GDN_MAX_TOKENS ||
        (long long)Hkv * d > 0xffffffLL)
        return GDN_ERR_UNSUPPORTED;
    if (page_stride % 8 != 0 || page_stride < (int64_t)Hkv * page * d) return GDN_ERR_INVALID_ARG;
    if (!grid_ok(gdn::kv_commit_parts(max_path) * m, gdn::kCommitThreads))
        return GDN_ERR_UNSUPPORTED;
    const gdn::KvCommitArgs a{k_cache, v_cache, page_stride, table, dst,        begin, k,
                              v,       path,    add,         m,     n,          max_path, Hkv,
                              d,       elem_bytes, seqs,     max_pages, pool,   page_log, status};
    return from_hip(gdn::launch_kv_commit(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_rope_frequencies(int rot, double base, gdn_rope_scaling scaling, double factor,
                                double original, double low, double high, float *inv_freq,
                                float *magnitude) {
    if (!inv_freq || !magnitude || !all_aligned4(inv_freq, magnitude)) return GDN_ERR_INVALID_ARG;
    if (rot < 2 || rot % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
        return GDN_ERR_INVALID_ARG;
    if (rot > GDN_MAX_HEAD_DIM) return GDN_ERR_UNSUPPORTED;
    if (scaling < GDN_ROPE_PLAIN || scaling > GDN_ROPE_YARN) return GDN_ERR_INVALID_ARG;
    const bool parts = scaling == GDN_ROPE_PARTS || scaling == GDN_ROPE_YARN;
    if (scaling != GDN_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return GDN_ERR_INVALID_ARG;
    if (scaling == GDN_ROPE_NTK && rot <= 2) return GDN_ERR_INVALID_ARG;
    if (parts && (!(original > 0.0) || !std::isfinite(original) || !(low < high) ||
                  !std::isfinite(high - low)))
        return GDN_ERR_INVALID_ARG;
    if (scaling == GDN_ROPE_NTK) base *= std::pow(factor, rot / (rot - 2.0));
    for (int i = 0; i < rot / 2; ++i) {
        double t = std::pow(base, -2.0 * i / rot);
        if (scaling == GDN_ROPE_LINEAR) t /= factor;
        if (parts) {
            const double turns = original * t / (2 * M_PI);
            const double g = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
            t = g * t + (1 - g) * t / factor;
        }
        inv_freq[i] = static_cast<float>(t);
    }
    *magnitude = scaling == GDN_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1) : 1.f;
    return GDN_OK;
}

gdn_status gdn_qk_norm_rope(const void *q, int64_t q_row, int64_t q_head, const void *k,
                            int64_t k_row, int64_t k_head, gdn_dtype dtype, gdn_norm norm,
                            float eps, float offset, const void *q_weight, int64_t q_weight_head,
                            const void *k_weight, int64_t k_weight_head, gdn_dtype weight_dtype,
                            const int32_t *pos, const int32_t *base, int base_rows,
                            const float *inv_freq, int rot, gdn_rope_layout layout, float scale,
                            void *q_out, int64_t q_out_row, int64_t q_out_head, void *k_out,
                            int64_t k_out_row, int64_t k_out_head, int rows, int Hq, int Hk, int d,
                            void *stream) {
    const gdn::HeadsArgs a = used(
        {{q, q_row, q_head, q_out, q_out_row, q_out_head, q_weight, q_weight_head, Hq},
         {k, k_row, k_head, k_out, k_out_row, k_out_head, k_weight, k_weight_head, Hk},
         dtype, weight_dtype == GDN_DTYPE_F32, norm, eps, offset, pos, base, base_rows, inv_freq,
         rot, layout, scale, rows, d});
    const gdn_status st = heads_status(a, weight_dtype, true, true);
    if (st != GDN_OK || rows == 0) return st;
    // a wave a row, or as many as share its heads
    if (!grid_ok(((long long)rows + 3) * gdn::heads_splits(rows, Hq + Hk), 64))
        return GDN_ERR_UNSUPPORTED;
    return from_hip(gdn::launch_heads(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_rope(const void *q, int64_t q_row, int64_t q_head, const void *k, int64_t k_row,
                    int64_t k_head, gdn_dtype dtype, const int32_t *pos, const int32_t *base,
                    int base_rows, const float *inv_freq, int rot, gdn_rope_layout layout,
                    float scale, void *q_out, int64_t q_out_row, int64_t q_out_head, void *k_out,
                    int64_t k_out_row, int64_t k_out_head, int rows, int Hq, int Hk, int d,
                    void *stream) {
    return gdn_qk_norm_rope(q, q_row, q_head, k, k_row, k_head, dtype, GDN_NORM_NONE, 0.f, 0.f,
                            nullptr, 0, nullptr, 0, GDN_DTYPE_F32, pos, base, base_rows, inv_freq,
                            rot, layout, scale, q_out, q_out_row, q_out_head, k_out, k_out_row,
                            k_out_head, rows, Hq, Hk, d, stream);
}

gdn_status gdn_kv_append(void *k_cache, void *v_cache, int64_t page_stride, const int32_t *table,
                         const int32_t *dst, const int32_t *begin, const int32_t *cu,
                         const void *q, int64_t q_row, int64_t q_head, const void *k, int64_t k_row,
                         int64_t k_head, const void *v, int64_t v_row, int64_t v_head,
                         gdn_dtype dtype, gdn_norm norm, float eps, float offset,
                         const void *q_weight, int64_t q_weight_head, const void *k_weight,
                         int64_t k_weight_head, gdn_dtype weight_dtype, const int32_t *pos,
                         const float *inv_freq, int rot, gdn_rope_layout layout, float scale,
                         void *q_out, int64_t q_out_row, int64_t q_out_head, void *k_out,
                         int64_t k_out_row, int64_t k_out_head, int m, int rows, int Hq, int Hkv,
                         int d, int seqs, int max_pages, int pool, int page, int32_t *status,
                         void *stream) {
    const gdn::AppendArgs a{
        used({{q, q_row, q_head, q_out, q_out_row, q_out_head, q_weight, q_weight_head, Hq},
              {k, k_row, k_head, k_out, k_out_row, k_out_head, k_weight, k_weight_head, Hkv},
              dtype, weight_dtype == GDN_DTYPE_F32, norm, eps, offset, pos, nullptr, 1, inv_freq,
              rot, layout, scale, rows, d}),
        v, v_row, v_head, k_cache, v_cache, page_stride, table, dst, begin, cu, m, seqs, max_pages,
        pool, log2_exact(page), status};
    if (m < 0 || Hkv < 1 || seqs < 1 || max_pages < 1 || pool < 1 || page < 1)
        return GDN_ERR_INVALID_ARG;
    const gdn_status st = heads_status(a.h, weight_dtype, false, false);
    if (st != GDN_OK) return st;
    if (!cu && rows != m) return GDN_ERR_INVALID_ARG;
    if (m == 0) return GDN_OK;
    if (!k_cache || !v_cache || !table || !dst || !begin || (rows > 0 && !v))
        return GDN_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !all_aligned4(table, dst, begin, cu, status) ||
        !aligned_to(v, element_bytes(dtype)) || !strides_ok(v_row, v_head))
        return GDN_ERR_INVALID_ARG;
    // tokens of a row and pages are counted in 32 bits
    if (a.page_log < 0 || d % 8 != 0 || (long long)max_pages * page > GDN_MAX_TOKENS ||
        (long long)Hkv * d > 0xffffffLL || pool > GDN_MAX_PAGES || m > GDN_MAX_REQUESTS)
        return GDN_ERR_UNSUPPORTED;
    if (page_stride % 8 != 0 || page_stride < (int64_t)Hkv * page * d) return GDN_ERR_INVALID_ARG;
    if (!grid_ok(((long long)rows + 3) * gdn::heads_splits(rows, Hq + 2 * Hkv) + m + 3, 64))
        return GDN_ERR_UNSUPPORTED;
    return from_hip(gdn::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_count_prompt(int16_t *counts, int64_t stride, const int32_t *slot,
                            const int32_t *cu, const int32_t *tokens, int m, int rows, int slots,
                            int vocab, int32_t *status, void *stream) {
    const gdn::CountArgs a{counts, stride, slot, m, slots, vocab, status};
    const gdn_status st = count_status(a);
    if (st != GDN_OK) return st;
    if (rows < 0) return GDN_ERR_INVALID_ARG;
    if (m == 0) return GDN_OK;
    if (!cu || (rows > 0 && !tokens) || !all_aligned4(cu, tokens)) return GDN_ERR_INVALID_ARG;
    return from_hip(
        gdn::launch_count_prompt(a, cu, tokens, rows, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_count_commit(int16_t *counts, int64_t stride, const int32_t *slot,
                            const int32_t *tokens, const int32_t *path, const int32_t *add, int m,
                            int n, int max_path, int slots, int vocab, int32_t *status,
                            void *stream) {
    const gdn::CountArgs a{counts, stride, slot, m, slots, vocab, status};
    const gdn_status st = count_status(a);
    if (st != GDN_OK) return st;
    if (n < 1 || max_path < 1) return GDN_ERR_INVALID_ARG;
    if (max_path > GDN_MAX_TOKENS) return GDN_ERR_UNSUPPORTED;
    if (m == 0) return GDN_OK;
    if (!tokens || !path || !add || !all_aligned4(tokens, path, add)) return GDN_ERR_INVALID_ARG;
    return from_hip(gdn::launch_count_commit(a, tokens, path, add, n, max_path,
                                             static_cast<hipStream_t>(stream)));
}

int64_t gdn_adjust_logits_workspace(int batch, int n, int vocab) {
    if (batch < 1 || n < 1 || n > GDN_MAX_NODES || vocab < 1 || vocab > GDN_MAX_VOCAB) return 0;
    gdn::LogitsArgs a{};
    a.batch = batch, a.n = n, a.vocab = vocab;
    return gdn::logits_workspace(a);
}

gdn_status gdn_adjust_logits(const void *logits, gdn_dtype dtype, int64_t stride,
                             const int16_t *counts, int64_t counts_stride, const int32_t *slot,
                             int slots, const int32_t *tokens, const int32_t *parent,
                             const float *repetition, const float *presence, const float *frequency,
                             const int32_t *bias_tok, const float *bias, int bias_len,
                             const int32_t *mask, int mask_rows, void *out, gdn_dtype out_dtype,
                             int64_t out_stride, int32_t *best, int batch, int n, int vocab,
                             void *workspace, int64_t workspace_bytes, int32_t *status,
                             void *stream) {
    if (!logits || (!out && !best) || !dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
    if (out && out_dtype != dtype && out_dtype != GDN_DTYPE_F32) return GDN_ERR_INVALID_ARG;
    if (batch < 1 || n < 1 || vocab < 1 || bias_len < 0 || stride < 0)
        return GDN_ERR_INVALID_ARG;
    if ((tokens != nullptr) != (parent != nullptr) || (bias_len > 0 && (!bias_tok || !bias)))
        return GDN_ERR_INVALID_ARG;
    if (counts && (slots < 1 || counts_stride < vocab)) return GDN_ERR_INVALID_ARG;
    if (mask && mask_rows != 1 && mask_rows != n) return GDN_ERR_INVALID_ARG;
    if (!aligned_to(logits, element_bytes(dtype)) ||
        (out && !aligned_to(out, element_bytes(out_dtype))) || !aligned_to(counts, 2) ||
        !aligned16(workspace) ||
        !all_aligned4(slot, tokens, parent, repetition, presence, frequency, bias_tok, bias, mask,
                      best, status))
        return GDN_ERR_INVALID_ARG;
    if (n > GDN_MAX_NODES || vocab > GDN_MAX_VOCAB || bias_len > GDN_MAX_BIASES ||
        (long long)batch * n > 0x3ffffffLL || stride > (1LL << 40) || out_stride > (1LL << 40) ||
        counts_stride > (1LL << 40))
        return GDN_ERR_UNSUPPORTED;
    if (out && (long long)batch * n > 1 && out_stride < vocab) return GDN_ERR_INVALID_ARG;
    const gdn::LogitsArgs a{logits, dtype,    stride,    counts,     counts_stride, slot,
                            slots,  tokens,   parent,    repetition, presence,      frequency,
                            bias_tok, bias,   bias_len,  mask,       mask_rows,     out,
                            out ? out_dtype : dtype,     out_stride, best,          batch,
                            n,      vocab,    workspace, status};
    const int64_t need = best ? gdn::logits_workspace(a) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
    if (!grid_ok(gdn::logits_threads(a), 1)) return GDN_ERR_UNSUPPORTED;
    return from_hip(gdn::launch_adjust_logits(a, static_cast<hipStream_t>(stream)));
}

const char *gdn_status_string(int status) {
    switch (status) {
        case GDN_OK: return "ok";
        case GDN_ERR_INVALID_ARG: return "invalid argument (null or misaligned pointer, bad size)";
        case GDN_ERR_UNSUPPORTED: return "unsupported shape or dtype";
        case GDN_ERR_HIP: return "HIP runtime error at launch";
        default: return "unknown status";
    }
}

int gdn_tree_abi_version(void) { return GDN_TREE_ABI_VERSION; }

}  // extern "C"
