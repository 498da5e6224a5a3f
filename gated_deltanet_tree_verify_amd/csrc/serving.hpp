// Internal interface of the serving operators (prefill, step, attention over
// a paged cache, page bookkeeping) between api.hip and their launchers.
#pragma once

#include "internal.hpp"

namespace gdn {

// fault flags, mirroring GDN_FAULT_* of the public header
constexpr int kFaultBadSlot = 4;
constexpr int kFaultBadLength = 8;
constexpr int kFaultBadPage = 16;
constexpr int kFaultBadGroup = 32;
constexpr int kFaultNoPage = 64;

// the gated delta rule over ragged sequences; the step has no cu: row b is sequence b's
struct RuleArgs {
    const void *q, *k, *v;
    gdn_dtype dtype;
    const float *alpha, *beta;
    const int32_t *cu;
    float *S;
    const int32_t *src, *dst;
    void *out;
    gdn_dtype out_dtype;
    int batch, rows, slots, H, Hk, dk, dv;
    void *workspace;
    int32_t *status;
};

struct AttentionArgs {
    const void *q, *k, *v;
    gdn_dtype dtype;
    const int32_t *parent;
    const void *kc, *vc;
    int64_t page_stride;
    const int32_t *pages, *length, *gstart, *gshared;
    int groups;
    float scale;
    void *out;
    int batch, n, Hq, Hkv, d, page_log, num_pages, max_pages;
    void *workspace;
    int32_t *status;
};

// the page table calls: rows of `width` page ids, pages of 1 << page_log tokens
struct PageArgs {
    int32_t *table, *length, *ref;
    int seqs, width, pool, page_log;
    int32_t *status;
};

struct KvCommitArgs {
    void *kc, *vc;
    int64_t page_stride;
    const int32_t *table, *dst, *begin;
    const void *k, *v;
    const int32_t *path, *add;
    int m, n, max_path, Hkv, d, elem_bytes, seqs, width, pool, page_log;
    int32_t *status;
};

// workgroups of 256 threads: page_copy moves 16 KiB of a page in each (four
// 16-byte pieces a thread), kv_commit 8 tokens of a request
constexpr int kCopyThreads = 256, kCopyPieces = 4;
constexpr int64_t page_copy_parts(int64_t page_bytes) {
    constexpr int64_t kBytes = 16 * kCopyThreads * kCopyPieces;
    return page_bytes / kBytes + (page_bytes % kBytes != 0);
}
constexpr int kCommitThreads = 256, kCommitTokens = 8;
constexpr int64_t kv_commit_parts(int max_path) {
    return ((int64_t)max_path + kCommitTokens - 1) / kCommitTokens;
}
// page_free and the second kernel of page_compact: a wave a row
constexpr int kRowThreads = 64;

int64_t prefill_workspace(const RuleArgs &a);
hipError_t launch_prefill(const RuleArgs &a, hipStream_t s);
hipError_t launch_step(const RuleArgs &a, hipStream_t s);
int64_t attention_workspace(const AttentionArgs &a);
hipError_t launch_tree_attention(const AttentionArgs &a, hipStream_t s);
hipError_t launch_page_fork(const PageArgs &a, const int32_t *src, const int32_t *dst,
                            int32_t *copies, int m, hipStream_t s);
hipError_t launch_page_extend(const PageArgs &a, const int32_t *dst, const int32_t *add,
                              int32_t *begin, int m, hipStream_t s);
hipError_t launch_page_free(const PageArgs &a, const int32_t *done, int m, hipStream_t s);
hipError_t launch_page_compact(const PageArgs &a, int32_t *copies, int32_t *count,
                               int32_t *workspace, hipStream_t s);
hipError_t launch_page_copy(void *cache, const int32_t *copies, const int32_t *count, int m,
                            int planes, int pool, int64_t page_bytes, hipStream_t s);
hipError_t launch_kv_commit(const KvCommitArgs &a, hipStream_t s);

}  // namespace gdn
