// Pages of a paged key/value cache: forking, extending, freeing and
// compacting rows of a page table with reference counts, moving page bytes,
// and appending an accepted branch's key and value rows.
//
// The table calls are integer work over a few kilobytes whose only order is
// that of the requests, so each is one workgroup: prefix sums over the
// requests (which of them get how many pages), one pass over the reference
// counts that hands out the free pages lowest first, then the rows.  Their
// time is a launch and a few dependent passes through L2; splitting them
// would need a second launch, which costs more than it saves.  page_copy is
// bound by HBM (each byte read and written once) and kv_commit by its launch.
#include "device_common.hpp"
#include "serving.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;

__device__ __forceinline__ int wave_inclusive(int x) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(x, o);
        if (l >= o) x += up;
    }
    return x;
}

// sum over the workgroup's earlier threads; total: over all of them.  Two
// barriers; s_part is free again after the next call's first.
__device__ __forceinline__ int block_exclusive(int x, int *s_part, int &total) {
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int inc = wave_inclusive(x);
    __syncthreads();
    if (l == 63) s_part[w] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const int p = s_part[i];
        before += i < w ? p : 0;
        all += p;
    }
    total = all;
    return before + inc - x;
}

// free pages below the first id at which `most` of them have been seen (all
// of them if there are fewer)
__device__ int count_free(const int32_t *ref, int pool, int most, int *s_part) {
    int seen = 0;
    for (int p0 = 0; p0 < pool && seen < most; p0 += kThreads) {
        const int p = p0 + threadIdx.x;
        int total;
        block_exclusive(p < pool && ref[p] == 0, s_part, total);
        seen += total;
    }
    return min(seen, most);
}

// hand(rank, page) for the `most` lowest free pages, most <= number of free
// pages; a page's ref is read before any hand() of its round
template <typename F>
__device__ void hand_out(const int32_t *ref, int pool, int most, int *s_part, F hand) {
    int seen = 0;
    for (int p0 = 0; p0 < pool && seen < most; p0 += kThreads) {
        const int p = p0 + threadIdx.x;
        const bool is_free = p < pool && ref[p] == 0;
        int total;
        const int rank = seen + block_exclusive(is_free, s_part, total);
        if (is_free && rank < most) hand(rank, p);
        seen += total;
    }
}

// first request whose running total passes rank (upto ascending, rank < upto[m - 1])
__device__ __forceinline__ int owner(const int *upto, int m, int rank) {
    int lo = 0, hi = m - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] > rank) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int page_log) {
    return (int)(((long long)tokens + (1LL << page_log) - 1) >> page_log);
}

// a + b for numbers that are not negative; kMany stands for all that do not
// fit (there are fewer pages than that)
constexpr int kMany = 0x7fffffff;
__device__ __forceinline__ int add_up(int a, int b) {
    return (int)min((unsigned)a + (unsigned)b, (unsigned)kMany);
}

// running totals of need(r) over the requests, in upto[]; returns the last.
// Thousands of requests for whole rows pass 32 bits: the totals stop at kMany.
template <typename F>
__device__ int running_totals(int *upto, int m, int *s_part, F need) {
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
    int sum = 0;
    for (int r0 = 0; r0 < m; r0 += kThreads) {
        const int r = r0 + threadIdx.x;
        int x = r < m ? need(r) : 0;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(x, o);
            if (l >= o) x = add_up(x, up);
        }
        __syncthreads();
        if (l == 63) s_part[w] = x;
        __syncthreads();
        long long before = sum, all = sum;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const int p = s_part[i];
            before += i < w ? p : 0;
            all += p;
        }
        if (r < m) upto[r] = (int)min(before + x, (long long)kMany);
        sum = (int)min(all, (long long)kMany);
    }
    __syncthreads();
    return sum;
}

__device__ __forceinline__ bool row_ok(const PageArgs &a, int row) {
    return row >= 0 && row < a.seqs;
}

struct Requests {
    int part[kWaves];
    int upto[GDN_MAX_REQUESTS];       // running totals of the pages wanted
    int len[GDN_MAX_REQUESTS];        // length of the row that is read, before the call
    int16_t fault[GDN_MAX_REQUESTS];
};
struct Forks : Requests {
    int src[GDN_MAX_REQUESTS], dst[GDN_MAX_REQUESTS];
    int last[GDN_MAX_REQUESTS];       // the page of its own, -1: none
};
// Rows that a wave takes at once: their loads do not wait for each other (64
// forks of 1000 to 2000 tokens, medians of a kernel: 11.5 us, one row at a time
// 14; 4 forks: 7 and 6.4 us, below the host's time for the calls around it; with
// the check of sources 12 to 13.5 and 7.7 us).
constexpr int kRowsAtOnce = 4;

// A row that several requests would write goes to the first of them: each
// puts r - m < 0 into the row's length with an atomic minimum (lengths are
// not negative), and whoever finds its own value there has the row.  The
// holder writes the length again before the kernel ends.
__device__ void claim_rows(const PageArgs &a, const int32_t *dst, int m, Requests &q) {
    __syncthreads();
    for (int r = threadIdx.x; r < m; r += kThreads)
        if (q.fault[r] == 0) atomicMin(&a.length[dst[r]], r - m);
    __syncthreads();
    for (int r = threadIdx.x; r < m; r += kThreads)
        if (q.fault[r] == 0 && __hip_atomic_load(&a.length[dst[r]], __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT) != r - m)
            q.fault[r] = kFaultBadSlot;
    __syncthreads();
}

__global__ __launch_bounds__(kThreads) void page_fork_kernel(PageArgs a, const int32_t *src,
                                                             const int32_t *dst, int2 *copies,
                                                             int m) {
    __shared__ Forks q;
    const int tid = threadIdx.x, l = tid & 63, page = 1 << a.page_log;
    constexpr int kRound = kRowsAtOnce * kWaves;
    const int r_first = tid >> 6;

    // every request by itself: rows, length, the ids it would share
    for (int r = tid; r < m; r += kThreads) {
        int fault = 0, len = 0;
        const int s = src[r], d = dst[r];
        if (!row_ok(a, s) || !row_ok(a, d) || s == d || a.length[d] != 0) fault = kFaultBadSlot;
        else {
            len = a.length[s];
            if (len < 0 || len > (long long)a.width << a.page_log) fault = kFaultBadLength;
        }
        q.fault[r] = (int16_t)fault;
        q.len[r] = len;
        q.src[r] = s;
        q.dst[r] = d;
        q.last[r] = -1;
        copies[r] = make_int2(-1, -1);
    }
    __syncthreads();
    for (int r0 = r_first; r0 < m; r0 += kRound) {
        const int32_t *row[kRowsAtOnce];
        int used[kRowsAtOnce], most = 0;
        bool bad[kRowsAtOnce];
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k) {
            const int r = r0 + k * kWaves;
            const bool live = r < m && q.fault[min(r, m - 1)] == 0;
            row[k] = a.table + (live ? (size_t)q.src[r] * a.width : 0);
            used[k] = live ? pages_of(q.len[r], a.page_log) : 0;
            most = max(most, used[k]);
            bad[k] = false;
        }
        for (int c = l; c < most; c += 64) {
            int p[kRowsAtOnce];
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) p[k] = c < used[k] ? row[k][c] : 0;
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) bad[k] |= p[k] < 0 || p[k] >= a.pool;
        }
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k)
            if (__any(bad[k]) && l == 0) q.fault[r0 + k * kWaves] = kFaultBadPage;
    }
    claim_rows(a, dst, m, q);
    // A source that an earlier request writes: what that row will hold is not
    // known here (it may stay empty for want of a page), so the request fails.
    // A claimed row's length is its request less m.
    constexpr int kLate = -2;
    for (int r = tid; r < m; r += kThreads)
        if (q.fault[r] == 0) {
            const int x = __hip_atomic_load(&a.length[q.src[r]], __ATOMIC_RELAXED,
                                            __HIP_MEMORY_SCOPE_AGENT);
            if (x < 0 && x + m < r) q.last[r] = kLate;
        }
    __syncthreads();
    for (int r = tid; r < m; r += kThreads)
        if (q.last[r] == kLate) {
            q.last[r] = -1;
            q.fault[r] = kFaultBadSlot;
            a.length[q.dst[r]] = 0;
        }

    const int sum = running_totals(q.upto, m, q.part, [&](int r) {
        return q.fault[r] == 0 && (q.len[r] & (page - 1)) != 0 ? 1 : 0;
    });
    const int got = count_free(a.ref, a.pool, sum, q.part);
    hand_out(a.ref, a.pool, got, q.part, [&](int rank, int p) {
        const int r = owner(q.upto, m, rank);
        const int whole = q.len[r] >> a.page_log;
        copies[r] = make_int2(a.table[(size_t)q.src[r] * a.width + whole], p);
        q.last[r] = p;
        a.ref[p] = 1;
    });
    __syncthreads();

    // the rows
    for (int r0 = r_first; r0 < m; r0 += kRound) {
        const int32_t *from[kRowsAtOnce];
        int32_t *to[kRowsAtOnce];
        int whole[kRowsAtOnce], last[kRowsAtOnce];
        bool live[kRowsAtOnce];
#pragma unroll
        for (int k = 0; k < kRowsAtOnce; ++k) {
            const int r = r0 + k * kWaves;
            live[k] = r < m && q.fault[min(r, m - 1)] == 0;
            const int len = live[k] ? q.len[r] : 0;
            const bool ok = live[k] && ((len & (page - 1)) == 0 || q.upto[r] <= got);
            from[k] = a.table + (live[k] ? (size_t)q.src[r] * a.width : 0);
            to[k] = a.table + (live[k] ? (size_t)q.dst[r] * a.width : 0);
            whole[k] = ok ? len >> a.page_log : 0;
            last[k] = ok ? q.last[r] : -1;
            if (l == 0 && r < m) {
                if (live[k]) a.length[q.dst[r]] = ok ? len : 0;
                if (a.status) a.status[r] = live[k] ? (ok ? 0 : kFaultNoPage) : q.fault[r];
            }
        }
        for (int c = l; c < a.width; c += 64) {
            int p[kRowsAtOnce];
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k)
                p[k] = c < whole[k] ? from[k][c] : c == whole[k] ? last[k] : -1;
#pragma unroll
            for (int k = 0; k < kRowsAtOnce; ++k) {
                if (c < whole[k]) atomicAdd(&a.ref[p[k]], 1);
                if (live[k]) to[k][c] = p[k];
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void page_extend_kernel(PageArgs a, const int32_t *dst,
                                                               const int32_t *add, int32_t *begin,
                                                               int m) {
    __shared__ Requests q;
    const int tid = threadIdx.x;
    const long long top = (long long)a.width << a.page_log;

    for (int r = tid; r < m; r += kThreads) {
        int fault = 0, len = 0;
        const int d = dst[r];
        if (!row_ok(a, d)) fault = kFaultBadSlot;
        else {
            len = a.length[d];
            if (len < 0 || add[r] < 0 || (long long)len + add[r] > top) fault = kFaultBadLength;
        }
        q.fault[r] = (int16_t)fault;
        q.len[r] = len;
    }
    claim_rows(a, dst, m, q);
    const int sum = running_totals(q.upto, m, q.part, [&](int r) {
        return q.fault[r] ? 0
                          : pages_of(q.len[r] + add[r], a.page_log) - pages_of(q.len[r], a.page_log);
    });
    const int free_pages = count_free(a.ref, a.pool, sum, q.part);
    // pages go to the requests that are served whole: the totals ascend, so
    // these are the ones up to the last total within the free pages
    int serve = 0;
    for (int r = tid; r < m; r += kThreads)
        if (q.upto[r] <= free_pages) serve = max(serve, q.upto[r]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) serve = max(serve, __shfl_xor(serve, o));
    __syncthreads();
    if ((tid & 63) == 0) q.part[tid >> 6] = serve;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) serve = max(serve, q.part[i]);
    hand_out(a.ref, a.pool, serve, q.part, [&](int rank, int p) {
        const int r = owner(q.upto, m, rank);
        const int have = pages_of(q.len[r], a.page_log);
        const int first = r > 0 ? q.upto[r - 1] : 0;
        a.table[(size_t)dst[r] * a.width + have + (rank - first)] = p;
        a.ref[p] = 1;
    });
    for (int r = tid; r < m; r += kThreads) {
        int fault = q.fault[r], at = -1;
        if (!fault) {
            const bool ok = q.upto[r] <= free_pages;
            if (ok) at = q.len[r];
            else fault = kFaultNoPage;
            a.length[dst[r]] = q.len[r] + (ok ? add[r] : 0);
        }
        begin[r] = at;
        if (a.status) a.status[r] = fault;
    }
}

// One wave per row.  The row's ids are checked before anything is written: each
// has to be in the pool and counted.  Then the exchange of the length claims the
// row, so one that is named twice is given back once.  A wave that finds ids
// that cannot be freed looks at the length again: it is 0 where another wave
// has just freed the row (the claim is visible before that wave's writes), and
// only otherwise the ids are at fault.
__global__ __launch_bounds__(kRowThreads) void page_free_kernel(PageArgs a,
                                                       const int32_t *__restrict__ done) {
    const int r = blockIdx.x, l = threadIdx.x;
    const int row = done[r];
    int fault = 0;
    if (!row_ok(a, row)) fault = kFaultBadSlot;
    else {
        const auto length = [&] {
            return __hip_atomic_load(&a.length[row], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        };
        const int len = __builtin_amdgcn_readfirstlane(length());
        int32_t *t = a.table + (size_t)row * a.width;
        if (len < 0 || len > (long long)a.width << a.page_log) fault = kFaultBadLength;
        else if (len > 0) {
            const int used = pages_of(len, a.page_log);
            bool bad = false;
            for (int c = l; c < used; c += 64) {
                const int p = t[c];
                bad |= p < 0 || p >= a.pool || a.ref[min(max(p, 0), a.pool - 1)] <= 0;
            }
            if (__any(bad)) {
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
                if (__builtin_amdgcn_readfirstlane(length()) != 0) fault = kFaultBadPage;
            } else {
                int mine = 0;
                if (l == 0) mine = atomicExch(&a.length[row], 0) != 0;
                mine = __builtin_amdgcn_readfirstlane(mine);
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
                for (int c = l; mine && c < a.width; c += 64) {
                    if (c < used) atomicSub(&a.ref[t[c]], 1);
                    t[c] = -1;
                }
            }
        }
    }
    if (l == 0 && a.status) a.status[r] = fault;
}

// workspace[p]: where used page p is after the call (p itself if it stays)
__global__ __launch_bounds__(kThreads) void page_compact_kernel(PageArgs a, int2 *copies,
                                                                int32_t *__restrict__ count,
                                                                int32_t *workspace) {
    __shared__ int s_part[kWaves];
    const int tid = threadIdx.x;
    int used = 0;
    for (int p0 = 0; p0 < a.pool; p0 += kThreads) {
        const int p = p0 + tid;
        int total;
        block_exclusive(p < a.pool && a.ref[p] != 0, s_part, total);
        used += total;
    }
    int moves = 0, holes = 0;
    for (int p0 = 0; p0 < a.pool; p0 += kThreads) {
        const int p = p0 + tid;
        const bool in = p < a.pool, busy = in && a.ref[p] != 0;
        const bool move = busy && p >= used, hole = in && !busy && p < used;
        int nm, nh;
        const int im = moves + block_exclusive(move, s_part, nm);
        const int ih = holes + block_exclusive(hole, s_part, nh);
        if (move) copies[im].x = p;
        if (hole) copies[ih].y = p;
        if (in) workspace[p] = p;
        moves += nm;
        holes += nh;
    }
    __syncthreads();
    for (int i = tid; i < moves; i += kThreads) {
        const int2 c = copies[i];
        workspace[c.x] = c.y;
        a.ref[c.y] = a.ref[c.x];
        a.ref[c.x] = 0;
    }
    if (tid == 0) count[0] = moves;
}

__global__ __launch_bounds__(kRowThreads) void page_remap_kernel(PageArgs a,
                                                        const int32_t *__restrict__ to) {
    const int row = blockIdx.x;
    const int len = a.length[row];
    if (len <= 0) return;
    const int used = min(a.width, pages_of(len, a.page_log));
    int32_t *t = a.table + (size_t)row * a.width;
    for (int c = threadIdx.x; c < used; c += 64) {
        const int p = t[c];
        if (p >= 0 && p < a.pool) t[c] = to[p];
    }
}

// a thread's pieces are loaded before any is stored
__global__ __launch_bounds__(kCopyThreads) void page_copy_kernel(
    uint4 *cache, const int2 *__restrict__ copies, const int32_t *__restrict__ count, int pool,
    int64_t pieces, int parts) {
    const int i = blockIdx.x / parts, part = blockIdx.x % parts;
    if (count && i >= *count) return;
    const int2 c = copies[i];
    if (c.x < 0 || c.x >= pool || c.y < 0 || c.y >= pool || c.x == c.y) return;
    const size_t plane = (size_t)blockIdx.y * pool;
    const uint4 *from = cache + (plane + c.x) * pieces;
    uint4 *to = cache + (plane + c.y) * pieces;
    const int64_t p0 = (int64_t)part * (kCopyThreads * kCopyPieces) + threadIdx.x;
    uint4 x[kCopyPieces];
#pragma unroll
    for (int j = 0; j < kCopyPieces; ++j)
        if (p0 + j * kCopyThreads < pieces) x[j] = from[p0 + j * kCopyThreads];
#pragma unroll
    for (int j = 0; j < kCopyPieces; ++j)
        if (p0 + j * kCopyThreads < pieces) to[p0 + j * kCopyThreads] = x[j];
}

// one workgroup per (request, 8 tokens)
__global__ __launch_bounds__(kCommitThreads) void kv_commit_kernel(KvCommitArgs a, int parts) {
    const int r = blockIdx.x / parts, part = blockIdx.x % parts;
    const int row = a.dst[r], at = a.begin[r], add = a.add[r];
    int fault = 0;
    if (row < 0 || row >= a.seqs) fault = kFaultBadSlot;
    else if (add < 0 || add > a.max_path) fault = kFaultBadPath;
    else if (at < -1 || (at >= 0 && (long long)at + add > (long long)a.width << a.page_log))
        fault = kFaultBadLength;
    // the whole request is checked by each of its workgroups: it writes all
    // of its rows or none
    if (!fault && at >= 0) {
        int f = 0;
        for (int j = threadIdx.x; j < add; j += kCommitThreads) {
            const int node = a.path[(size_t)r * a.max_path + j];
            if (node < 0 || node >= a.n) f |= kFaultBadPath;
            const int p = a.table[(size_t)row * a.width + ((at + j) >> a.page_log)];
            if (p < 0 || p >= a.pool) f |= kFaultBadPage;
        }
        if (__syncthreads_or(f & kFaultBadPath)) fault |= kFaultBadPath;
        if (__syncthreads_or(f & kFaultBadPage)) fault |= kFaultBadPage;
    }
    if (a.status && part == 0 && threadIdx.x == 0) a.status[r] = fault;
    if (fault || at < 0) return;

    const int per = a.d * a.elem_bytes / 16;              // pieces of one head's row
    const int rowp = a.Hkv * per;
    const size_t pstride = (size_t)a.page_stride * a.elem_bytes / 16;
    const int n = min(kCommitTokens, add - part * kCommitTokens);
    const uint4 *k = static_cast<const uint4 *>(a.k) + (size_t)r * a.n * rowp;
    const uint4 *v = static_cast<const uint4 *>(a.v) + (size_t)r * a.n * rowp;
    for (int i = threadIdx.x; i < n * rowp; i += kCommitThreads) {
        const int j = part * kCommitTokens + i / rowp, x = i % rowp, h = x / per;
        const int node = a.path[(size_t)r * a.max_path + j], pos = at + j;
        const int p = a.table[(size_t)row * a.width + (pos >> a.page_log)];
        const size_t to = (size_t)p * pstride +
                          (((size_t)h << a.page_log) + (pos & ((1 << a.page_log) - 1))) * per +
                          x % per;
        static_cast<uint4 *>(a.kc)[to] = k[(size_t)node * rowp + x];
        static_cast<uint4 *>(a.vc)[to] = v[(size_t)node * rowp + x];
    }
}

}  // namespace

hipError_t launch_page_fork(const PageArgs &a, const int32_t *src, const int32_t *dst,
                            int32_t *copies, int m, hipStream_t s) {
    hipLaunchKernelGGL(page_fork_kernel, dim3(1), dim3(kThreads), 0, s, a, src, dst,
                       reinterpret_cast<int2 *>(copies), m);
    return hipGetLastError();
}

hipError_t launch_page_extend(const PageArgs &a, const int32_t *dst, const int32_t *add,
                              int32_t *begin, int m, hipStream_t s) {
    hipLaunchKernelGGL(page_extend_kernel, dim3(1), dim3(kThreads), 0, s, a, dst, add, begin, m);
    return hipGetLastError();
}

hipError_t launch_page_free(const PageArgs &a, const int32_t *done, int m, hipStream_t s) {
    hipLaunchKernelGGL(page_free_kernel, dim3((unsigned)m), dim3(kRowThreads), 0, s, a, done);
    return hipGetLastError();
}

hipError_t launch_page_compact(const PageArgs &a, int32_t *copies, int32_t *count,
                               int32_t *workspace, hipStream_t s) {
    hipLaunchKernelGGL(page_compact_kernel, dim3(1), dim3(kThreads), 0, s, a,
                       reinterpret_cast<int2 *>(copies), count, workspace);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(page_remap_kernel, dim3((unsigned)a.seqs), dim3(kRowThreads), 0, s, a,
                       workspace);
    return hipGetLastError();
}

hipError_t launch_page_copy(void *cache, const int32_t *copies, const int32_t *count, int m,
                            int planes, int pool, int64_t page_bytes, hipStream_t s) {
    const int64_t pieces = page_bytes / 16;
    const int64_t parts = page_copy_parts(page_bytes);
    hipLaunchKernelGGL(page_copy_kernel, dim3((unsigned)(parts * m), (unsigned)planes),
                       dim3(kCopyThreads), 0, s, static_cast<uint4 *>(cache),
                       reinterpret_cast<const int2 *>(copies), count, pool, pieces, (int)parts);
    return hipGetLastError();
}

hipError_t launch_kv_commit(const KvCommitArgs &a, hipStream_t s) {
    const int64_t parts = kv_commit_parts(a.max_path);
    hipLaunchKernelGGL(kv_commit_kernel, dim3((unsigned)(parts * a.m)), dim3(kCommitThreads), 0, s,
                       a, (int)parts);
    return hipGetLastError();
}

}  // namespace gdn
