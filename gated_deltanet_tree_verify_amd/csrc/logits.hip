// Logits on their way to acceptance: penalties for repeated tokens, biases and
// grammar masks over a vocabulary, the greedy token of every tree node, and the
// table of counts that the penalties read.
//
// Node i of sequence b, token t, in fp32 with every step rounded:
//   c  = occurrences of t in the output (table) and on the path root .. i
//   z1 = z                           where c = 0 and the prompt has no t
//        z > 0 ? z / rep : z rep     elsewhere
//   d  = bias(t) - (c > 0 ? freq c + pres : 0)
//   z' = z1 + d, or -inf where the mask has no t
//   best = the lowest t with the largest z' (NaN and -inf are never it)
// The order of z' decides integers, so nothing here is contracted or
// reassociated.  A logit is read once; the counts are 2 bytes a token and
// sequence, the mask 1 / 8 byte a token and node.
#include "heads.hpp"

#pragma clang fp contract(off)

namespace gdn {
namespace {

using heads::Bf16;
using heads::F16;
using heads::F32;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kLane = 8;                       // tokens of a lane
constexpr int kSlice = 64 * kLane;             // and of a wave
constexpr int kMarkTokens = 1 << 15;           // of a workgroup of count_prompt
constexpr int kNone = 0x7fffffff;

// ---------------------------------------------------------------------------
// counts
// ---------------------------------------------------------------------------
// request r's slot: outside the table, or named by an earlier request, is a
// fault.  The whole workgroup.
__device__ __forceinline__ int slot_fault(const CountArgs &a, int r) {
    const int slot = a.slot[r];
    bool bad = slot < 0 || slot >= a.slots;
    for (int i = threadIdx.x; i < r; i += blockDim.x) bad |= a.slot[i] == slot;
    return __syncthreads_or(bad) ? kFaultBadSlot : 0;
}

// A workgroup makes one part of one row: a bit for every token of the part,
// set by a pass over the prompt, then the row's values.
__global__ __launch_bounds__(kThreads) void count_prompt_kernel(
    CountArgs a, const int32_t *__restrict__ cu, const int32_t *__restrict__ tokens, int rows) {
    __shared__ uint32_t s_bits[kMarkTokens / 32];
    const int r = blockIdx.x, tid = threadIdx.x;
    const int first = cu[r], end = cu[r + 1];
    int fault = slot_fault(a, r);
    if (first < 0 || end < first || end > rows) fault |= kFaultBadLength;
    if (a.status && blockIdx.y == 0 && tid == 0) a.status[r] = fault;
    if (fault) return;
    const int v0 = (int)blockIdx.y * kMarkTokens, n = min(kMarkTokens, a.vocab - v0);
    for (int i = tid; i < (n + 31) / 32; i += kThreads) s_bits[i] = 0;
    __syncthreads();
    for (int i = first + tid; i < end; i += kThreads) {
        const uint32_t t = (uint32_t)tokens[i] - (uint32_t)v0;
        if (t < (uint32_t)n) atomicOr(&s_bits[t >> 5], 1u << (t & 31));
    }
    __syncthreads();
    int16_t *row = a.counts + a.slot[r] * a.stride + v0;
    for (int i = tid; i < n; i += kThreads)
        row[i] = (s_bits[i >> 5] >> (i & 31) & 1) ? (int16_t)-32768 : (int16_t)0;
}

// A workgroup for every request; its first wave counts 64 tokens of the path
// at a time: the lowest of the lanes that have a token adds them all.
__global__ __launch_bounds__(kThreads) void count_commit_kernel(
    CountArgs a, const int32_t *__restrict__ tokens, const int32_t *__restrict__ path,
    const int32_t *__restrict__ add, int n, int max_path) {
    const int r = blockIdx.x, tid = threadIdx.x;
    const int m = add[r];
    const int32_t *p = path + (size_t)r * max_path;
    int fault = slot_fault(a, r);
    if (m < 0 || m > max_path) fault |= kFaultBadPath;
    else {
        bool bad = false;
        for (int j = tid; j < m; j += kThreads) bad |= p[j] < 0 || p[j] >= n;
        if (__syncthreads_or(bad)) fault |= kFaultBadPath;
    }
    if (a.status && tid == 0) a.status[r] = fault;
    if (fault || tid >= 64) return;
    volatile int16_t *row = a.counts + a.slot[r] * a.stride;
    for (int j0 = 0; j0 < m; j0 += 64) {
        const int t = j0 + tid < m ? tokens[(size_t)r * n + p[j0 + tid]] : -1;
        int same = 0, lowest = 64;
        for (int i = 63; i >= 0; --i)
            if (__shfl(t, i) == t) ++same, lowest = i;
        if (t >= 0 && t < a.vocab && lowest == tid) {
            const int16_t c = row[t];
            row[t] = (int16_t)((c & -32768) | min((c & 32767) + same, 32767));
        }
        __threadfence_block();
    }
}

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------
struct Best {
    float value;
    int token;           // kNone: nothing above -inf
};

__device__ __forceinline__ void better(Best &x, float value, int token) {
    if (value > x.value || (value == x.value && token < x.token)) x.value = value, x.token = token;
}

__device__ __forceinline__ Best wave_best(Best x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const float v = __shfl_xor(x.value, o);
        const int t = __shfl_xor(x.token, o);
        better(x, v, t);
    }
    return x;
}

// the table's row of sequence b, -1: none such
__device__ __forceinline__ int slot_of(const LogitsArgs &a, int b) {
    if (!a.counts) return 0;
    const int slot = a.slot ? a.slot[b] : b;
    return slot < 0 || slot >= a.slots ? -1 : slot;
}

// A wave for every node and 512 tokens, lane l having tokens l, l + 64, ..
template <typename E, typename O>
__global__ __launch_bounds__(kThreads) void logits_kernel(LogitsArgs a, int slices) {
    const int l = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int slice = (int)(unit % slices);
    const int64_t node = unit / slices;
    if (node >= (int64_t)a.batch * a.n) return;
    const int b = (int)(node / a.n), i = (int)(node % a.n);
    const int v0 = slice * kSlice;

    int fault = 0;
    const int32_t *parent = a.parent + (size_t)b * a.n;
    if (a.parent) {
        bool bad = false;
        for (int j = l; j < a.n; j += 64) bad |= !parent_ok(parent[j], j);
        if (__any(bad)) fault |= kFaultBadParent;
    }
    const int slot = slot_of(a, b);
    if (slot < 0) fault |= kFaultBadSlot;
    if (a.status && slice == 0 && i == 0 && l == 0) a.status[b] = fault;

    const typename E::type *z = static_cast<const typename E::type *>(a.logits) + node * a.stride;
    typename O::type *out =
        a.out ? static_cast<typename O::type *>(a.out) + node * a.out_stride : nullptr;
    const float rep = a.repetition ? a.repetition[b] : 1.f;
    const float pres = a.presence ? a.presence[b] : 0.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f;

    int c[kLane] = {}, prompt[kLane] = {};
    float bias[kLane] = {};
    if (!fault) {
        // tokens of the slice are (t - v0) = 64 e + l
        if (a.counts) {
            const int16_t *row = a.counts + slot * a.counts_stride;
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                const int t = v0 + 64 * e + l, x = t < a.vocab ? row[t] : 0;
                c[e] = x & 32767, prompt[e] = x < 0;
            }
        }
        if (a.tokens) {
            const int32_t *tok = a.tokens + (size_t)b * a.n;
            for (int j0 = 0; j0 <= i; j0 += 64) {
                const int t = j0 + l <= i ? tok[j0 + l] : -1;
                uint64_t hits = __ballot((uint32_t)t - (uint32_t)v0 < (uint32_t)kSlice);
                while (hits) {
                    const int j = __builtin_ctzll(hits);
                    hits &= hits - 1;
                    int up = i;
                    while (up > j0 + j) up = parent[up];
                    const int at = __shfl(t, j) - v0;
                    if (up == j0 + j && (at & 63) == l)
#pragma unroll
                        for (int e = 0; e < kLane; ++e) c[e] += at >> 6 == e;
                }
            }
        }
        for (int j0 = 0; j0 < a.bias_len; j0 += 64) {
            const size_t at0 = (size_t)b * a.bias_len + j0 + l;
            const bool in = j0 + l < a.bias_len;
            const int t = in ? a.bias_tok[at0] : -1;
            const float x = in ? a.bias[at0] : 0.f;
            uint64_t hits = __ballot((uint32_t)t - (uint32_t)v0 < (uint32_t)kSlice);
            while (hits) {
                const int j = __builtin_ctzll(hits);
                hits &= hits - 1;
                const int at = __shfl(t, j) - v0;
                const float y = __shfl(x, j);
                if ((at & 63) == l)
#pragma unroll
                    for (int e = 0; e < kLane; ++e)
                        if (at >> 6 == e) bias[e] += y;
            }
        }
    }
    const int words = (a.vocab + 31) / 32;
    const int32_t *mask =
        a.mask ? a.mask + ((size_t)b * a.mask_rows + (a.mask_rows > 1 ? i : 0)) * words : nullptr;
    Best best = {-__builtin_inff(), kNone};
#pragma unroll
    for (int e = 0; e < kLane; ++e) {
        const int t = v0 + 64 * e + l;
        if (t >= a.vocab) continue;
        float y = E::widen(z[t]);
        if (c[e] > 0 || prompt[e]) y = y > 0.f ? y / rep : y * rep;
        float less = 0.f;
        if (c[e] > 0) less = freq * (float)c[e] + pres;
        y = y + (bias[e] - less);
        if (mask && !(mask[t >> 5] >> (t & 31) & 1)) y = -__builtin_inff();
        if (fault) y = __builtin_nanf("");
        if (out) out[t] = O::bits(y);
        if (y > best.value) best.value = y, best.token = t;
    }
    if (!a.best) return;
    best = wave_best(best);
    if (l == 0) static_cast<Best *>(a.workspace)[unit] = best;
}

// a wave for every node: the best of its slices
__global__ __launch_bounds__(64) void logits_join_kernel(LogitsArgs a, int slices) {
    const int l = threadIdx.x;
    const int64_t node = blockIdx.x;
    const Best *part = static_cast<const Best *>(a.workspace) + node * slices;
    Best best = {-__builtin_inff(), kNone};
    for (int i = l; i < slices; i += 64) better(best, part[i].value, part[i].token);
    best = wave_best(best);
    if (l == 0) a.best[node] = best.token == kNone ? -1 : best.token;
}

int logits_slices(const LogitsArgs &a) { return (a.vocab + kSlice - 1) / kSlice; }

template <typename E, typename O>
hipError_t launch(const LogitsArgs &a, hipStream_t s) {
    const int slices = logits_slices(a);
    const int64_t units = (int64_t)a.batch * a.n * slices;
    hipLaunchKernelGGL((logits_kernel<E, O>), dim3((unsigned)((units + kWaves - 1) / kWaves)),
                       dim3(kThreads), 0, s, a, slices);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.best) return e;
    hipLaunchKernelGGL(logits_join_kernel, dim3((unsigned)(a.batch * a.n)), dim3(64), 0, s, a,
                       slices);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_count_prompt(const CountArgs &a, const int32_t *cu, const int32_t *tokens,
                               int rows, hipStream_t s) {
    const int parts = (a.vocab + kMarkTokens - 1) / kMarkTokens;
    hipLaunchKernelGGL(count_prompt_kernel, dim3((unsigned)a.m, (unsigned)parts), dim3(kThreads), 0,
                       s, a, cu, tokens, rows);
    return hipGetLastError();
}

hipError_t launch_count_commit(const CountArgs &a, const int32_t *tokens, const int32_t *path,
                               const int32_t *add, int n, int max_path, hipStream_t s) {
    hipLaunchKernelGGL(count_commit_kernel, dim3((unsigned)a.m), dim3(kThreads), 0, s, a, tokens,
                       path, add, n, max_path);
    return hipGetLastError();
}

int64_t logits_units(const LogitsArgs &a) { return (int64_t)a.batch * a.n * logits_slices(a); }

int64_t logits_workspace(const LogitsArgs &a) { return logits_units(a) * (int64_t)sizeof(Best); }

hipError_t launch_adjust_logits(const LogitsArgs &a, hipStream_t s) {
    const bool same = a.out_dtype == a.dtype;
    if (a.dtype == GDN_DTYPE_BF16) return same ? launch<Bf16, Bf16>(a, s) : launch<Bf16, F32>(a, s);
    if (a.dtype == GDN_DTYPE_F16) return same ? launch<F16, F16>(a, s) : launch<F16, F32>(a, s);
    return launch<F32, F32>(a, s);
}

}  // namespace gdn
