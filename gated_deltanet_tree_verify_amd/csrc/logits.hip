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
//
// Most tokens of a vocabulary have no count, no bias and no place on a path:
// their z' is z, and what bounds a row is its bytes and one comparison for every
// token.  So the loop takes maxima of eight tokens a lane, looks up at the end
// which of the eight it was, and gives the touched ones the long way.
//   16 trees of 32 nodes, 131072 tokens, bf16, masks, counts of 1200 tokens:
//     41 us, 3.6 TB/s (touched tokens in their slices: 48), vector units active 79 % of
//     the time; without counts and masks 30
//   64 rows of 100003 tokens, bf16 read and written, counts of 1500: 13 us and
//     4 us of joining the parts; one row of 32000: 5 and 2 us
//   the trees with a hundredth, a tenth, all of the vocabulary counted: 47, 87,
//     155 us for the whole call; with an output 57, 76, 77
#include "heads.hpp"

#pragma clang fp contract(off)

namespace gdn {
namespace {

using heads::Bf16;
using heads::F16;
using heads::F32;

constexpr int kThreads = 256;
constexpr int kMostThreads = 1024;              // of a workgroup of the logits
constexpr int kLane = 8;                       // tokens of a lane
constexpr int kSlice = 64 * kLane;             // and of a wave
constexpr int kMarkTokens = 1 << 13;           // of a workgroup of count_prompt
constexpr int kNone = 0x7fffffff;
constexpr int kPutOffTokens = 128;             // of a wave
constexpr int kPutOffSlices = 8;               // of a wave that puts tokens off, at least
// lanes with touched tokens in a slice that puts none off: 64 of them cost the wave
// about as much as the one or two of each lane (a tenth of the vocabulary counted:
// 94 us without this, 87 with; all of it 514 and 155; a hundredth 47 both ways)
constexpr int kInPlaceLanes = 24;
constexpr int kAhead = 2;                      // slices on their way, the one in work among them

// 8 adjacent values as they lie in memory, at any address of their type
struct __attribute__((packed, aligned(2))) Half8 {
    uint32_t x[4];
};
struct __attribute__((packed, aligned(4))) Full8 {
    float x[8];
};

typedef uint32_t Half8Vector __attribute__((ext_vector_type(4), aligned(2)));
typedef float Full4Vector __attribute__((ext_vector_type(4), aligned(4)));

template <typename E>
struct Eight {
    Half8 raw;
    __device__ __forceinline__ void load(const uint16_t *p) {
        raw = *reinterpret_cast<const Half8 *>(p);
    }
    __device__ __forceinline__ void load(const uint16_t *p, int n) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            raw.x[i] = (2 * i < n ? p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] : 0u)
                                                        << 16;
    }
    __device__ __forceinline__ float at(int i) const {
        return E::widen((uint16_t)(raw.x[i >> 1] >> (i & 1 ? 16 : 0)));
    }
    __device__ __forceinline__ void set(const float (&y)[kLane]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) raw.x[i] = E::two_bits(y[2 * i], y[2 * i + 1]);
    }
    __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<Half8 *>(p) = raw; }
    // Results pass the lines of the L2 that are still to be read (16 trees of 32
    // nodes, 131072 tokens: 59.5 -> 47.2 us; logits that pass it too: no change)
    __device__ __forceinline__ void store_once(uint16_t *p) const {
        const Half8Vector x = {raw.x[0], raw.x[1], raw.x[2], raw.x[3]};
        __builtin_nontemporal_store(x, reinterpret_cast<Half8Vector *>(p));
    }
    __device__ __forceinline__ void store(uint16_t *p, int n) const {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (i < n) p[i] = (uint16_t)(raw.x[i >> 1] >> (i & 1 ? 16 : 0));
    }
};
template <>
struct Eight<F32> {
    Full8 raw;
    __device__ __forceinline__ void load(const float *p) {
        raw = *reinterpret_cast<const Full8 *>(p);
    }
    __device__ __forceinline__ void load(const float *p, int n) {
#pragma unroll
        for (int i = 0; i < kLane; ++i) raw.x[i] = i < n ? p[i] : 0.f;
    }
    __device__ __forceinline__ float at(int i) const { return raw.x[i]; }
    __device__ __forceinline__ void set(const float (&y)[kLane]) {
#pragma unroll
        for (int i = 0; i < kLane; ++i) raw.x[i] = y[i];
    }
    __device__ __forceinline__ void store_once(float *p) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Full4Vector x = {raw.x[4 * k], raw.x[4 * k + 1], raw.x[4 * k + 2], raw.x[4 * k + 3]};
            __builtin_nontemporal_store(x, reinterpret_cast<Full4Vector *>(p) + k);
        }
    }
    __device__ __forceinline__ void store(float *p, int n) const {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
            if (i < n) p[i] = raw.x[i];
    }
};
struct None {            // no output
    typedef char type;
};

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
// set by a pass over the prompt, then the row's values, 8 tokens a thread.
__global__ __launch_bounds__(kThreads) void count_prompt_kernel(
    CountArgs a, const int32_t *__restrict__ cu, const int32_t *__restrict__ tokens, int rows) {
    __shared__ uint32_t s_bits[kMarkTokens / 32];
    const int r = blockIdx.x, tid = threadIdx.x;
    const int first = cu[r], end = cu[r + 1];
    for (int i = tid; i < kMarkTokens / 32; i += kThreads) s_bits[i] = 0;
    int fault = slot_fault(a, r);                // a barrier: the bits are cleared
    if (first < 0 || end < first || end > rows) fault |= kFaultBadLength;
    if (a.status && blockIdx.y == 0 && tid == 0) a.status[r] = fault;
    if (fault) return;
    const int v0 = (int)blockIdx.y * kMarkTokens, n = min(kMarkTokens, a.vocab - v0);
    for (int64_t i = (int64_t)first + tid; i < end; i += kThreads) {
        const uint32_t t = (uint32_t)tokens[i] - (uint32_t)v0;
        if (t < (uint32_t)n) atomicOr(&s_bits[t >> 5], 1u << (t & 31));
    }
    __syncthreads();
    uint16_t *row = reinterpret_cast<uint16_t *>(a.counts) + a.slot[r] * a.stride + v0;
    for (int t = tid * kLane; t < n; t += kThreads * kLane) {
        const uint32_t bits = s_bits[t >> 5] >> (t & 31);
        Eight<Bf16> x;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x.raw.x[k] = (bits >> 2 * k & 1) << 15 | (bits >> (2 * k + 1) & 1) << 31;
        if (t + kLane <= n) x.store(row + t);
        else x.store(row + t, n - t);
    }
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
        for (int i = min(64, m - j0) - 1; i >= 0; --i)
            if (__builtin_amdgcn_readlane(t, i) == t) ++same, lowest = i;
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

__device__ __forceinline__ void better(Best &x, const Best &y) {
    if (y.value > x.value || (y.value == x.value && y.token < x.token)) x = y;
}

constexpr Best kNothing = {-__builtin_inff(), kNone};

// y of another lane, x where that lane is none
template <int kControl>
__device__ __forceinline__ int other_lane(int x) {
    return __builtin_amdgcn_update_dpp(x, x, kControl, 0xf, 0xf, false);
}

// f over the values of all lanes: neighbours, the other two of four, the other
// four of eight, the other eight of sixteen, then from one sixteen to the next
template <typename F>
__device__ __forceinline__ int wave_over(int x, F f) {
    x = f(x, other_lane<0xb1>(x));
    x = f(x, other_lane<0x4e>(x));
    x = f(x, other_lane<0x141>(x));
    x = f(x, other_lane<0x140>(x));
    x = f(x, other_lane<0x142>(x));
    x = f(x, other_lane<0x143>(x));
    return __builtin_amdgcn_readlane(x, 63);
}

// of values that are no NaN
__device__ __forceinline__ float wave_largest(float x) {
    return __builtin_bit_cast(
        float, wave_over(__builtin_bit_cast(int, x), [](int a, int b) {
            return __builtin_bit_cast(int, fmaxf(__builtin_bit_cast(float, a),
                                                 __builtin_bit_cast(float, b)));
        }));
}

__device__ __forceinline__ int wave_smallest(int x) {
    return wave_over(x, [](int a, int b) { return min(a, b); });
}

// How a launch is cut: `parts` workgroups share a node's row, each wave of them
// takes `per` slices of 512 tokens, one after the other.
struct Cut {
    int slices, per, parts;
    int threads;
    int listed;              // biases of a wave that its list in LDS has room for
};

struct Biased {
    int token;
    float bias;
};

// Biases of a wave's list: the lists of 16 waves and the rest stay below 64 KiB.  With
// more of them the sequence's are gone over in memory for every slice (one wave a node,
// 32000 tokens, 8192 nodes: 432 biases 0.9 ms, 1000 3.6, 4096 154).
constexpr int kListed = 432;

// What a wave knows of its node.
struct Node {
    float rep, inverse;      // the repetition penalty, and its reciprocal
    bool plain;              // far from the ends of fp32: a quotient by fused steps is exact
    float pres, freq;
    int token[2];            // of the nodes l and 64 + l, if they are on the node's path, or -1
    int bias_tok;            // the biases of the wave's slices, in order, up to 64 of them;
    float bias;              // none here where they are more
    uint64_t many;           // then: the slices, counted from the wave's first, modulo 64, that have some,
    const Biased *list;      // and the list of them in LDS,
    int listed;              // so many; -1: more than it has room for, the sequence's are gone over
    int first;
    bool any;                // any of these lies in the wave's slices
    __device__ __forceinline__ bool many_in(int slice) const { return many >> (slice - first & 63) & 1; }
};

// f(token, bias) of 64 biases of the wave at a time, in order (token -1: none)
template <typename F>
__device__ __forceinline__ void each_bias(const LogitsArgs &a, const Node &n, int64_t bias0, F f) {
    const int l = threadIdx.x & 63;
    if (n.listed >= 0)
        for (int j = l; j - l < n.listed; j += 64) {
            const Biased x = j < n.listed ? n.list[j] : Biased{-1, 0.f};
            f(x.token, x.bias);
        }
    else
        for (int j = l; j - l < a.bias_len; j += 64) {
            const bool in = j < a.bias_len;
            f(in ? a.bias_tok[bias0 + j] : -1, in ? a.bias[bias0 + j] : 0.f);
        }
}

// z / rep for z above 0, z rep otherwise, correctly rounded.  With r the
// rounded reciprocal and q = z r, the residue z - q rep is exact in a fused
// step and q + residue r is the rounded quotient (Markstein), as long as
// nothing leaves the range of normal numbers: 3 instructions instead of 12.
__device__ __forceinline__ float repeated(const Node &n, float z) {
    float q = z * n.inverse;
    q = fmaf(fmaf(-q, n.rep, z), n.inverse, q);
    // z in [2^-60, 2^60)
    const bool usual = __float_as_uint(z) - 0x21800000u < 0x5d800000u - 0x21800000u;
    if (z > 0.f && !(usual && n.plain)) q = z / n.rep;
    return z > 0.f ? q : z * n.rep;
}

// z' of a token with z, its entry x of the table, its count on the path, its bias
__device__ __forceinline__ float adjusted(const Node &n, float z, uint32_t x, uint32_t path,
                                          float bias) {
    const int c = (int)((x & 32767u) + path);
    const float less = n.freq * (float)c + n.pres, r = repeated(n, z);
    return (x | path ? r : z) + (c > 0 ? bias - less : bias);
}

// The lane's tokens with a count, a bit each.  Only those that the mask has are
// of interest: the others are -inf, whatever their count.
__device__ __forceinline__ uint32_t counted(const Eight<Bf16> &count) {
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        bits |= __builtin_bit_cast(uint32_t, __builtin_elementwise_min(
                    __builtin_bit_cast(u16x2, count.raw.x[k]), u16x2{1, 1})) << 2 * k;
    }
    return (bits | bits >> 15) & 255u;
}

// y where the lane's mask has token e, -inf elsewhere
__device__ __forceinline__ float allowed(float y, uint32_t mask, int e) {
    const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)mask, e, 1);
    const uint32_t none = __float_as_uint(-__builtin_inff());
    return __uint_as_float((__float_as_uint(y) & keep) | (none & ~keep));
}

struct Running {
    float value;             // the largest of a lane's groups of 8 tokens, the group's
    int slice;               // slice, and what it is the largest of
    float of[kLane];
};

constexpr float kLeast = -__builtin_inff();
constexpr Running kNoneYet = {kLeast, 0, {kLeast, kLeast, kLeast, kLeast, kLeast, kLeast, kLeast,
                                          kLeast}};

// the lane's first token with its largest value
__device__ __forceinline__ Best best_of(const Running &x) {
    int at = 0;
#pragma unroll
    for (int e = kLane - 1; e >= 0; --e) at = x.of[e] == x.value ? e : at;
    if (!(x.value > kLeast)) return kNothing;
    return {x.value, x.slice * kSlice + kLane * (int)(threadIdx.x & 63) + at};
}

// Touched tokens of a wave that are put off until there are 64 of them: a slice
// has few, and each takes its lane as many instructions as 64 take all lanes.
// A wave of few slices, and one that writes its logits, does them in place.
struct Later {
    int *list;               // in LDS, room for kPutOffTokens
    int held;                // the same in all lanes
    Best best;               // of those that the lane has done
};

// token t of each lane, with logit z0 and entry x of the table; of the node's path
// and biases only the lanes in path0, path1 and biased can have it
__device__ __forceinline__ void settle_one(const LogitsArgs &a, const Node &n, int64_t bias0, bool in,
                                           int t, float z0, uint32_t x, uint64_t path0,
                                           uint64_t path1, uint64_t biased, bool many,
                                           Later &later) {
    uint32_t path = 0;
    float bias = 0.f;
    for (; path0; path0 &= path0 - 1)
        path += __builtin_amdgcn_readlane(n.token[0], __builtin_ctzll(path0)) == t ? 1u : 0u;
    for (; path1; path1 &= path1 - 1)
        path += __builtin_amdgcn_readlane(n.token[1], __builtin_ctzll(path1)) == t ? 1u : 0u;
    auto add = [&](uint64_t on, int tok, float y) {
        for (; on; on &= on - 1) {
            const int j = __builtin_ctzll(on);
            const float b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(y), j));
            if (__builtin_amdgcn_readlane(tok, j) == t) bias += b;
        }
    };
    add(biased, n.bias_tok, n.bias);
    if (many)
        each_bias(a, n, bias0, [&](int tok, float y) { add(__ballot(tok >= 0), tok, y); });
    const float y = adjusted(n, z0, x, path, bias);
    // the tokens of a lane do not ascend: the second ones of all follow the first
    if (in && y > kLeast) better(later.best, {y, t});
}

// the first `count` of those put off, one a lane; the others move up
template <typename E>
__device__ __forceinline__ void settle(const LogitsArgs &a, const Node &n, int64_t bias0,
                                       const typename E::type *z, const uint16_t *counts,
                                       uint32_t keep, int count, Later &later) {
    const int l = threadIdx.x & 63;
    heads::exchange();
    const bool in = l < count;
    const int t = in ? later.list[l] : -1;
    const int rest = later.held - count, up = l < rest ? later.list[count + l] : 0;
    heads::exchange();
    if (l < rest) later.list[l] = up;
    later.held = rest;
    const float z0 = in ? __builtin_canonicalizef(E::widen(z[t])) : 0.f;
    const uint32_t x = in ? counts[t] & keep : 0u;
    settle_one(a, n, bias0, in, t, z0, x, n.any ? __ballot(n.token[0] >= 0) : 0,
               n.any ? __ballot(n.token[1] >= 0) : 0, n.any ? __ballot(n.bias_tok >= 0) : 0,
               n.many != 0, later);
}

// all touched tokens of a slice at once, each lane its own one after the other
template <typename E>
__device__ __forceinline__ void settle_slice(const LogitsArgs &a, const Node &n, int64_t bias0,
                                             const Eight<E> &z, const Eight<Bf16> &count,
                                             uint32_t touched, int slice, Later &later) {
    const int v0 = slice * kSlice + kLane * (int)(threadIdx.x & 63);
    auto inside = [&](int t) {
        return n.any ? __ballot((uint32_t)t - (uint32_t)(slice * kSlice) < (uint32_t)kSlice) : 0;
    };
    const uint64_t path0 = inside(n.token[0]), path1 = inside(n.token[1]);
    const uint64_t biased = inside(n.bias_tok);
    while (__any(touched != 0)) {
        const uint32_t one = touched & -touched;
        touched ^= one;
        float z0 = 0.f;
        uint32_t x = 0;
#pragma unroll
        for (int e = 0; e < kLane; ++e) z0 = one == 1u << e ? z.at(e) : z0;
#pragma unroll
        for (int k = 0; k < 4; ++k) x = one >> 2 * k & 3 ? count.raw.x[k] : x;
        x = one & 0xaau ? x >> 16 : x & 65535u;
        settle_one(a, n, bias0, one != 0, v0 + __builtin_ctz(one | 128u), __builtin_canonicalizef(z0),
                   x, path0, path1, biased, n.many_in(slice), later);
    }
}

// The same tokens by their bits: those with a count, on the node's path or biased.
__device__ __forceinline__ uint32_t touched_of(const LogitsArgs &a, const Node &n, int64_t bias0,
                                               const Eight<Bf16> &count, uint32_t mask, int slice) {
    const int l = threadIdx.x & 63, v0 = slice * kSlice + kLane * l;
    uint32_t bits = counted(count);
    auto add = [&](int t) {
        for (uint64_t on = __ballot((uint32_t)t - (uint32_t)(slice * kSlice) < (uint32_t)kSlice); on;
             on &= on - 1) {
            const int at = __builtin_amdgcn_readlane(t, __builtin_ctzll(on)) - v0;
            if ((uint32_t)at < (uint32_t)kLane) bits |= 1u << at;
        }
    };
    if (n.any) {
        add(n.token[0]), add(n.token[1]), add(n.bias_tok);
        if (n.many_in(slice)) each_bias(a, n, bias0, [&](int t, float) { add(t); });
    }
    return bits & mask;
}

// The lane's 8 tokens v0 + 8 l .. of a slice, of which the first `left` are in
// the row; the mask has no others.
template <typename E, typename O>
__device__ __forceinline__ void slice_of(const LogitsArgs &a, const Node &n, int64_t bias0,
                                         const Eight<E> &z, const Eight<Bf16> &count, uint32_t mask,
                                         int slice, int left, void *out, Running &best) {
    const int l = threadIdx.x & 63, v0 = slice * kSlice;
    float y[kLane];
#pragma unroll
    for (int e = 0; e < kLane; ++e) y[e] = __builtin_canonicalizef(z.at(e));   // NaNs are quiet
    auto count_at = [&](int e) { return count.raw.x[e >> 1] >> (e & 1 ? 16 : 0) & 65535u; };
    auto inside = [&](int t) { return __ballot((uint32_t)t - (uint32_t)v0 < (uint32_t)kSlice); };
    uint64_t on_path[2] = {0, 0}, biased = 0;
    if (n.any) {
        on_path[0] = inside(n.token[0]), on_path[1] = inside(n.token[1]);
        biased = inside(n.bias_tok);
    }
    uint32_t touched = counted(count) & mask;
    const bool many = n.many_in(slice);
    if (__any(touched != 0) || (on_path[0] | on_path[1] | biased) || many) {
        uint64_t more = 0;                       // a byte for each of the lane's tokens
        const bool any_path = (on_path[0] | on_path[1]) != 0;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            for (uint64_t hits = on_path[k]; hits; hits &= hits - 1) {
                const int to = __builtin_amdgcn_readlane(n.token[k], __builtin_ctzll(hits)) - v0;
                if (to / kLane == l) more += 1ull << 8 * (to % kLane), touched |= 1u << to % kLane;
            }
        float bias[kLane] = {};
        bool any_bias = false;
        auto add = [&](uint64_t hits, int t, float x) {
            any_bias |= hits != 0;
            for (; hits; hits &= hits - 1) {
                const int j = __builtin_ctzll(hits);
                const int to = __builtin_amdgcn_readlane(t, j) - v0;
                const float b = __builtin_bit_cast(
                    float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), j));
                if (to / kLane == l) {
                    touched |= 1u << to % kLane;
#pragma unroll
                    for (int e = 0; e < kLane; ++e)
                        if (to % kLane == e) bias[e] += b;
                }
            }
        };
        add(biased, n.bias_tok, n.bias);
        if (many) each_bias(a, n, bias0, [&](int t, float x) { add(inside(t), t, x); });
        if (!__any(__popc(touched) > 2)) {
            // Few tokens of a slice are touched, seldom more than one of a lane:
            // the lanes take theirs one after the other.
            while (__any(touched != 0)) {
                const uint32_t one = touched & -touched;
                touched ^= one;
                bool is[kLane];
                float z0 = 0.f, d = 0.f;
                uint32_t x = 0, path = 0;
#pragma unroll
                for (int e = 0; e < kLane; ++e) is[e] = one == 1u << e, z0 = is[e] ? y[e] : z0;
#pragma unroll
                for (int k = 0; k < 4; ++k) x = is[2 * k] || is[2 * k + 1] ? count.raw.x[k] : x;
                x = one & 0xaau ? x >> 16 : x & 65535u;
                if (any_bias)
#pragma unroll
                    for (int e = 0; e < kLane; ++e) d = is[e] ? bias[e] : d;
                if (any_path) path = (uint32_t)(more >> 8 * __builtin_ctz(one | 128u)) & 255u;
                z0 = adjusted(n, z0, x, path, d);
#pragma unroll
                for (int e = 0; e < kLane; ++e) y[e] = is[e] ? z0 : y[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                const float z1 = adjusted(n, y[e], count_at(e), (uint32_t)(more >> 8 * e) & 255u,
                                          bias[e]);
                y[e] = touched >> e & 1 ? z1 : y[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kLane; ++e) y[e] = allowed(y[e], mask, e);
    if constexpr (!__is_same(O, None)) {
        typename O::type *o = static_cast<typename O::type *>(out) + v0 + kLane * l;
        Eight<O> r;
        r.set(y);
        if ((slice + 1) * kSlice > a.vocab) r.store(o, left);
        else r.store_once(o);
    }
    float top = y[0];
#pragma unroll
    for (int e = 1; e < kLane; ++e) top = fmaxf(top, y[e]);
    // slices ascend: an equal one is not better
    const bool up = top > best.value;
    best.value = up ? top : best.value;
    best.slice = up ? slice : best.slice;
#pragma unroll
    for (int e = 0; e < kLane; ++e) best.of[e] = up ? y[e] : best.of[e];
}

// Workgroups go to the eight XCDs in turn; neighbours in a sequence share its
// counts, so each XCD gets a run of them (its L2 then has what they share).
__device__ __forceinline__ int item_of(int block, int blocks) {
    const int xcd = block & 7, each = blocks >> 3, more = blocks & 7;
    return xcd * each + min(xcd, more) + (block >> 3);
}

// Loads run a slice ahead of the work (two ahead: 49 us for the trees instead of
// 47, registers).  Which of a lane's 8 tokens is the largest is looked up once, at
// the end.  Six waves a SIMD where tokens are put off: two workgroups of 12 on a
// compute unit (79 registers).
template <typename E, typename O, bool kPutOff>
__global__ __launch_bounds__(kMostThreads, kPutOff ? 6 : 4) void logits_kernel(LogitsArgs a, Cut cut) {
    typedef typename E::type T;
    __shared__ int s_later[kPutOff ? kMostThreads / 64 : 1][kPutOff ? kPutOffTokens : 1];
    __shared__ Best s_best[kMostThreads / 64];
    extern __shared__ Biased s_biased[];
    const int l = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);      // the same in all lanes
    const int item = item_of((int)blockIdx.x, (int)gridDim.x);
    const int part = item % cut.parts, node = item / cut.parts;
    const int b = node / a.n, i = node % a.n, waves = cut.threads / 64;
    const int first = (part * waves + w) * cut.per, end = min(first + cut.per, cut.slices);
    int slot = 0, fault = 0;
    if (a.counts) {
        slot = a.slot ? a.slot[b] : b;
        if (slot < 0 || slot >= a.slots) fault = kFaultBadSlot, slot = 0;
    }
    const T *z = static_cast<const T *>(a.logits) + node * a.stride;
    // without a table any bytes, none of them kept: loads have no branch
    const uint16_t *counts =
        a.counts ? reinterpret_cast<const uint16_t *>(a.counts) + slot * a.counts_stride
                 : reinterpret_cast<const uint16_t *>(z);
    const uint32_t keep = a.counts ? ~0u : 0u;
    // a lane's 8 tokens are a byte of the mask; without one any byte, all bits set
    const uint8_t *mask = static_cast<const uint8_t *>(a.logits);
    if (a.mask)
        mask = reinterpret_cast<const uint8_t *>(
            a.mask + ((int64_t)b * a.mask_rows + (a.mask_rows > 1 ? i : 0)) * ((a.vocab + 31) / 32));
    const int mask_lane = a.mask ? l : 0, mask_step = a.mask ? kSlice / 8 : 0;
    const uint32_t all = a.mask ? 0u : 255u;
    // tokens of a lane in slice s
    auto left = [&](int s) { return min(max(a.vocab - s * kSlice - kLane * l, 0), kLane); };
    struct Loaded {
        Eight<E> z;
        Eight<Bf16> count;
        uint32_t mask;
    };
    Loaded x[kAhead] = {};
    const int full = a.vocab / kSlice;           // the row may end inside a slice
    auto load = [&](int s, Loaded &x) {          // of the whole ones
        s = min(s, full - 1);
        x.z.load(z + (int64_t)s * kSlice + kLane * l);
        x.count.load(counts + (int64_t)s * kSlice + kLane * l);
        x.mask = mask[s * mask_step + mask_lane];
    };
    auto load_cut = [&](Loaded &x) {             // the one that is not
        const int64_t at = (int64_t)full * kSlice + kLane * l;
        const int n = left(full);
        x.z.load(z + at, n);
        x.count.load(counts + at, n);
        x.mask = n > 0 ? (mask[full * mask_step + mask_lane] | all) & ((1u << n) - 1) : 0u;
    };
    // the largest of a lane's 8 logits that the mask has
    auto largest = [&](const Eight<E> &z, uint32_t mask) {
        float top = -__builtin_inff();
#pragma unroll
        for (int e = 0; e < kLane; ++e)
            top = fmaxf(top, allowed(__builtin_canonicalizef(z.at(e)), mask, e));
        return top;
    };
    if (first < end && full > 0)
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) load(first + k, x[k]);

    // lanes 0, 1 and 2 fetch the penalties; nothing is used before all loads are out
    float penalty = l == 0 ? 1.f : 0.f;
    const float *const from = l == 0 ? a.repetition : l == 1 ? a.presence : a.frequency;
    if (l < 3 && from) penalty = from[b];
    Node n;
    const int64_t bias0 = (int64_t)b * a.bias_len;
    n.bias_tok = -1, n.bias = 0.f, n.many = 0, n.first = first;
    n.list = nullptr, n.listed = 0;
    if (l < a.bias_len && a.bias_len <= 64)
        n.bias_tok = a.bias_tok[bias0 + l], n.bias = a.bias[bias0 + l];
    int parent[2] = {-1, -1}, token[2] = {-1, -1};
    if (a.parent)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (64 * k + l < a.n) {
                parent[k] = a.parent[(int64_t)b * a.n + 64 * k + l];
                token[k] = a.tokens[(int64_t)b * a.n + 64 * k + l];
            }
    auto fetched = [&](int lane) {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, penalty), lane));
    };
    n.rep = fetched(0), n.pres = fetched(1), n.freq = fetched(2);
    n.inverse = 1.f / n.rep;
    n.plain = n.rep >= 0x1p-30f && n.rep <= 0x1p30f;
    n.token[0] = n.token[1] = -1;
    if (a.parent) {
        if (__any(!parent_ok(parent[0], l) || !parent_ok(parent[1], 64 + l)))
            fault |= kFaultBadParent;
        uint64_t path[2] = {0, 0};
        for (int up = fault ? -1 : i; up >= 0;) {
            path[up >> 6] |= 1ull << (up & 63);
            up = up < 64 ? __builtin_amdgcn_readlane(parent[0], up)
                         : __builtin_amdgcn_readlane(parent[1], up - 64);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (path[k] >> l & 1) n.token[k] = token[k];
    }
    auto ours = [&](int t) { return t >= first * kSlice && t < end * kSlice; };
    if (a.bias_len > 64) {
        Biased *list = s_biased + w * cut.listed;
        int held = 0;
        uint64_t in_slices = 0;
#pragma unroll 1
        for (int j = l; j - l < a.bias_len; j += 64) {
            const bool in = j < a.bias_len;
            const Biased x = {in ? a.bias_tok[bias0 + j] : -1, in ? a.bias[bias0 + j] : 0.f};
            const uint64_t hits = __ballot(ours(x.token));
            const int at = held + __builtin_amdgcn_mbcnt_hi(
                                      (uint32_t)(hits >> 32),
                                      __builtin_amdgcn_mbcnt_lo((uint32_t)hits, 0));
            if (ours(x.token)) {
                if (at < cut.listed) list[at] = x;
                in_slices |= 1ull << (x.token / kSlice - first & 63);
            }
            held += __popcll(hits);
        }
        heads::exchange();
        if (held > 64) {
            auto either = [](int x, int y) { return x | y; };
            n.many = (uint64_t)(uint32_t)wave_over((int)(in_slices >> 32), either) << 32 |
                     (uint32_t)wave_over((int)in_slices, either);
            n.list = list, n.listed = held <= cut.listed ? held : -1;
        } else if (l < held) {
            n.bias_tok = list[l].token, n.bias = list[l].bias;
        }
    }
    n.any = n.many != 0 || __any(ours(n.token[0]) || ours(n.token[1]) || ours(n.bias_tok));
    if (a.status && part == 0 && i == 0 && threadIdx.x == 0) a.status[b] = fault;

    typename O::type *out = nullptr;
    if constexpr (!__is_same(O, None))
        out = static_cast<typename O::type *>(a.out) + node * a.out_stride;
    Running best = kNoneYet;
    Later later = {s_later[kPutOff ? w : 0], 0, kNothing};
    auto settle64 = [&] { settle<E>(a, n, bias0, z, counts, keep, 64, later); };
    if (fault) {
        if constexpr (!__is_same(O, None))
            for (int64_t t = (int64_t)first * kSlice + l; t < min((int64_t)end * kSlice, (int64_t)a.vocab);
                 t += 64)
                out[t] = O::bits(__builtin_nanf(""));
    } else {
        for (int s0 = first; s0 < end; s0 += kAhead)
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int s = s0 + k;
                if (s >= end) break;
                if (full > 0) load(s + kAhead - 1, x[(k + kAhead - 1) % kAhead]);
                if (s == full) load_cut(x[k]);
                x[k].mask |= s == full ? 0u : all;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[k].count.raw.x[j] &= keep;
                if constexpr (!kPutOff) {
                    slice_of<E, O>(a, n, bias0, x[k].z, x[k].count, x[k].mask, s, left(s), out, best);
                    continue;
                }
                uint32_t touched = touched_of(a, n, bias0, x[k].count, x[k].mask, s);
                const float top = largest(x[k].z, x[k].mask & ~touched);
                // slices ascend: an equal one is not better
                best.slice = top > best.value ? s : best.slice;
                best.value = top > best.value ? top : best.value;
                if (__popcll(__ballot(touched != 0)) > kInPlaceLanes) {
                    settle_slice<E>(a, n, bias0, x[k].z, x[k].count, touched, s, later);
                    continue;
                }
                while (__any(touched != 0)) {
                    if (later.held > kPutOffTokens - 64) settle64();
                    const uint64_t have = __ballot(touched != 0);
                    const int at = later.held + __builtin_amdgcn_mbcnt_hi(
                                                    (uint32_t)(have >> 32),
                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)have, 0));
                    if (touched) later.list[at] = s * kSlice + kLane * l + __builtin_ctz(touched);
                    later.held += __popcll(have);
                    touched &= touched - 1;
                }
            }
        if constexpr (kPutOff)
            while (later.held > 0)
                settle<E>(a, n, bias0, z, counts, keep, min(later.held, 64), later);
    }
    if (!a.best) return;
    // the lane's first token with its largest value, then the wave's, then the workgroup's
    Best own = kNothing;
    if constexpr (kPutOff) {
        // looked up once, in the lowest eight that have it: the logits are as they were
        own = later.best;
        const float most = wave_largest(fmaxf(own.value, best.value));
        const int eight = wave_smallest(best.value == most && most > -__builtin_inff()
                                            ? best.slice * 64 + l
                                            : kNone);
        if (eight != kNone) {
            const int s = eight >> 6;
            if (s == full) load_cut(x[0]);
            else load(s, x[0]);
            x[0].mask |= s == full ? 0u : all;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[0].count.raw.x[j] &= keep;
            const uint32_t mask = x[0].mask & ~touched_of(a, n, bias0, x[0].count, x[0].mask, s);
            int at = kLane;
#pragma unroll
            for (int e = kLane - 1; e >= 0; --e)
                at = (mask >> e & 1) && x[0].z.at(e) == most ? e : at;
            if (l == (eight & 63)) better(own, {most, s * kSlice + kLane * l + at});
        }
    } else {
        own = best_of(best);
    }
    Best mine;
    mine.value = wave_largest(own.value);
    mine.token = wave_smallest(own.value == mine.value ? own.token : kNone);
    if (l == 0) s_best[w] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < waves; ++k) better(mine, s_best[k]);
        if (cut.parts == 1) a.best[node] = mine.token == kNone ? -1 : mine.token;
        else static_cast<Best *>(a.workspace)[(int64_t)node * cut.parts + part] = mine;
    }
}

// a wave for every node: the best of its parts
__global__ __launch_bounds__(64) void logits_join_kernel(LogitsArgs a, int parts) {
    const int l = threadIdx.x;
    const int64_t node = blockIdx.x;
    const Best *from = static_cast<const Best *>(a.workspace) + node * parts;
    Best best = kNothing;
    for (int i = l; i < parts; i += 64) better(best, from[i]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        better(best, {__shfl_xor(best.value, o), __shfl_xor(best.token, o)});
    if (l == 0) a.best[node] = best.token == kNone ? -1 : best.token;
}

// About 6144 waves, 24 a compute unit: enough loads in flight, and no more of
// what each of them does once.  Up to 16 waves of a node are one workgroup and
// need no joining, as many on each of a compute unit's four SIMDs and so many
// that two workgroups fit (12 without, 8 with an output: registers); more are
// groups of four.
// 512 nodes of 256 slices: 12 waves each 40 us, 8 44, 16 49, 32 (groups) 58;
// the same with an output: 8 waves 48, 12 56, 16 52;
// 64 nodes of 196 slices: 17 groups of three slices a wave 15.4 us, of one
// slice 18.2, of eight 18.9, one workgroup of 16 waves 25.5;
// one node of 63 slices: 16 groups 9.1 us, one workgroup of 16 waves 10.2.
Cut cut_of(const LogitsArgs &a) {
    Cut c;
    const int64_t nodes = (int64_t)a.batch * a.n;
    c.slices = (a.vocab + kSlice - 1) / kSlice;
    int64_t waves = nodes < 6144 ? 6144 / nodes : 1;
    if (waves <= 16)
        waves = waves > 13 ? 16 : waves > 8 ? (a.out ? 8 : 12) : waves > 4 ? 8 : waves;
    if (waves > c.slices) waves = c.slices;
    c.per = (int)((c.slices + waves - 1) / waves);
    waves = (c.slices + c.per - 1) / c.per;
    c.parts = waves <= 16 ? 1 : (int)((waves + 3) / 4);
    c.threads = 64 * (waves > 16 ? 4 : waves > 4 ? ((int)waves + 3) / 4 * 4 : (int)waves);
    c.listed = a.bias_len <= 64 ? 0 : a.bias_len < kListed ? a.bias_len : kListed;
    return c;
}

template <typename E, typename O>
hipError_t launch(const LogitsArgs &a, hipStream_t s) {
    const Cut c = cut_of(a);
    const dim3 grid((unsigned)(a.batch * a.n * c.parts)), block((unsigned)c.threads);
    const unsigned lds = (unsigned)(c.threads / 64 * c.listed * (int)sizeof(Biased));
    if (__is_same(O, None) && c.per >= kPutOffSlices)
        hipLaunchKernelGGL((logits_kernel<E, O, __is_same(O, None)>), grid, block, lds, s, a, c);
    else
        hipLaunchKernelGGL((logits_kernel<E, O, false>), grid, block, lds, s, a, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.best || c.parts == 1) return e;
    hipLaunchKernelGGL(logits_join_kernel, dim3((unsigned)(a.batch * a.n)), dim3(64), 0, s, a,
                       c.parts);
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

int64_t logits_threads(const LogitsArgs &a) {
    const Cut c = cut_of(a);
    return (int64_t)a.batch * a.n * c.parts * c.threads;
}

int64_t logits_workspace(const LogitsArgs &a) {
    const Cut c = cut_of(a);
    return c.parts == 1 ? 0 : (int64_t)a.batch * a.n * c.parts * (int64_t)sizeof(Best);
}

hipError_t launch_adjust_logits(const LogitsArgs &a, hipStream_t s) {
    const bool same = a.out_dtype == a.dtype;
    if (a.dtype == GDN_DTYPE_BF16)
        return !a.out ? launch<Bf16, None>(a, s)
                      : same ? launch<Bf16, Bf16>(a, s) : launch<Bf16, F32>(a, s);
    if (a.dtype == GDN_DTYPE_F16)
        return !a.out ? launch<F16, None>(a, s)
                      : same ? launch<F16, F16>(a, s) : launch<F16, F32>(a, s);
    return !a.out ? launch<F32, None>(a, s) : launch<F32, F32>(a, s);
}

}  // namespace gdn
