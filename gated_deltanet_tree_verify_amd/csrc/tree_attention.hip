// Softmax attention of a draft tree over a paged cache whose prefix may be
// shared by groups of sequences (gfx950).
//
// A row (sequence, node, query head) attends to the tokens of its sequence's
// cache and to its node's ancestors-or-self.  The softmax is split over the
// keys: any part of them gives m (any number near max z), l = sum e^{z - m} and
// o = sum e^{z - m} v, and parts join by
//     m = max m_i,   out = sum e^{m_i - m} o_i / sum e^{m_i - m} l_i,
// so a prefix that several sequences share is one part, computed for all
// their rows together with each key and value read once, and a long context
// is split over workgroups.
//
// Work: a unit is (group, key head, 128 rows) over the shared tokens or
// (sequence, key head, 128 rows) over its own tokens and tree nodes, cut into
// tiles of 64 keys.  All units' tiles form one line, and workgroup i takes
// the places [i c, (i + 1) c) of it, whatever units they belong to: workgroups
// have the same work as long as no unit is cut into more parts than there is
// room for partials (Layout: grid / units + 2 a row).  One context that is much
// longer than the others of a batch with many rows passes that: c grows until
// it fits, and the line ends before the last workgroups (64-node trees, 43000
// tokens in all, medians of whole calls: 16 equal contexts 108 us, one of 32768
// and 15 of 700 505 us; 77000 tokens: 64 equal ones 229 us, one of 32768 and 63
// of 700 1525 us; with one token a sequence 69 and 86 us).  Lengths are
// device data, so every workgroup forms the line's prefix sums by itself (a
// scan over the batch).  Each unit a workgroup meets leaves one partial
// (m, l, o) in the workspace; a second kernel joins a row's partials.
//
// Tile: Z^T = K Q^T puts a query row into a lane's column and its keys into
// the lane's registers, so maxima and sums are in-register plus one exchange
// between the wave's halves, and e^{z - m} is, rounded, the B operand of
// O^T += V^T P^T as it stands (mfma_tile.hpp).  Keys and values go from memory
// to LDS directly (no registers), the next tile while this one is computed;
// the values' transpose is the LDS read's (ds_read_b64_tr_b16).  A unit of more
// than 64 rows gives each of its four waves 32 of them and all keys; up to 64
// rows, two waves and half the keys each; up to 32 rows (decoding), a wave has
// half the keys and half the value columns, and the halves merge through LDS
// at the unit's end.
//
// Times here are of this kernel, the shortest of 20 dispatches unless called
// medians: those are 2 to 7 % above (draft trees 116 to 120, median 121 to 130).
#include <type_traits>

#include "device_common.hpp"
#include "serving.hpp"
#include "mfma_tile.hpp"

namespace gdn {
namespace {

using namespace tile;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kKeys = 64;                 // keys of a tile
constexpr int kRows = 128;                // rows of a unit at most
constexpr float kLog2e = 1.4426950408889634f;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// the two element types: operand vectors, rounding of weights and outputs
struct Bf16 {
    typedef bf16x8 vec;
    static __device__ __forceinline__ f32x16 mma(vec a, vec b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ vec round8(const float *x) {
        vec v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = static_cast<__bf16>(x[i]);
        return v;
    }
    static __device__ __forceinline__ uint16_t bits(float x) { return bf16_bits(x); }
    static __device__ __forceinline__ float widen(uint16_t x) { return to_f32(x); }
    static constexpr uint32_t kExponent = 0x7f80u;     // all ones: infinite or NaN
    // Weights are 2^x relative to a reference that follows the scores: it is
    // set kLift below the largest, and set again once a score passes it by
    // kTop.  bf16 has fp32's range: any reference does.
    static constexpr float kLift = 0.f, kTop = 8.f;
};
struct F16 {
    typedef f16x8 vec;
    static __device__ __forceinline__ f32x16 mma(vec a, vec b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ vec round8(const float *x) {
        vec v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = static_cast<_Float16>(x[i]);
        return v;
    }
    static __device__ __forceinline__ uint16_t bits(float x) { return f16_bits(x); }
    static __device__ __forceinline__ float widen(uint16_t x) {
        return static_cast<float>(__builtin_bit_cast(_Float16, x));
    }
    static constexpr uint32_t kExponent = 0x7c00u;
    // fp16 has five exponent bits: weights of up to 2^15 leave all of them to
    // the small ones.  A weight is a normal number down to 2^-26 of the
    // largest, and never off by more than 2^-37 of it.  (With the largest at 1,
    // everything below 2^-25 of it went missing from the product with V while
    // the sum counted it.)
    static constexpr float kLift = 12.f, kTop = 15.f;
};

// ---------------------------------------------------------------------------
// the line of tiles
// ---------------------------------------------------------------------------
// one entry of the line: a group's shared tokens or a sequence's own
struct Entry {
    int first;       // first sequence of its rows
    int rows;        // query rows per key head
    int pos0;        // cache position of key 0
    int cached;      // keys that are cached tokens
    int keys;        // all keys: cached tokens, then the tree's nodes (own entries)
    int tiles;       // ceil(keys / kKeys)
    int row_tiles;   // ceil(rows / kRows)
    int weight;      // places of the line that a tile takes
};

// what the first kernel leaves for the second
struct Plan {
    long long per_wg;      // places of the line per workgroup
};
struct GroupLine {
    long long pre;         // places before the group's units
    int shared, whole;     // as in Batch
};

struct Slots {
    int own, shared;   // partials kept per row: of its own tokens, of its group's
    long long rows;    // batch * n * Hq
};

struct Layout {
    Slots slots;
    int grid;
    int64_t off_gpre, off_bpre, off_group, off_ml, off_o, bytes;
};

// The lengths and groups, as every workgroup keeps them in LDS: lengths that
// do not fit count as 0, and without sound groups there are none.
struct Batch {
    int length[GDN_MAX_SEQUENCES];
    uint16_t start[GDN_MAX_SEQUENCES + 1];
    uint16_t whole[GDN_MAX_SEQUENCES]; // the group's longest member (the first of them): its
                                       // page row holds every shared token that anyone sees
    int shared[GDN_MAX_SEQUENCES];     // tokens computed once for a group, no more than that
                                       // member has
};

__device__ __forceinline__ int fit_length(const AttentionArgs &a, int len) {
    return len < 0 || len > (a.max_pages << a.page_log) ? 0 : len;
}

// tokens computed once for a group that says it shares `said`: none for a
// group of one sequence (its own part covers them)
__device__ __forceinline__ int fit_shared(const AttentionArgs &a, int members, int said) {
    return members < 2 ? 0 : max(0, min(said, a.max_pages << a.page_log));
}

// group of sequence b, or -1.  start ascends within [0, batch] (checked).
__device__ __forceinline__ int group_of(const uint16_t *start, int groups, int b) {
    if (groups == 0 || b < start[0] || b >= start[groups]) return -1;
    int lo = 0, hi = groups - 1;            // last g with start[g] <= b
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// what follows from an entry's rows and keys
__device__ __forceinline__ void shape(Entry &x) {
    x.tiles = (x.keys + kKeys - 1) / kKeys;
    x.row_tiles = (x.rows + kRows - 1) / kRows;
    // a wave with all of a tile's keys takes about twice as long as one that
    // shares them (3.4 and 1.8 us a tile, two workgroups on a compute unit)
    x.weight = x.rows > 64 ? 2 : 1;
}

__device__ __forceinline__ Entry entry(const AttentionArgs &a, const Batch &y, int groups, int e) {
    Entry x;
    const int heads = a.Hq / a.Hkv;
    if (e < groups) {
        x.first = y.start[e];
        x.rows = (y.start[e + 1] - y.start[e]) * a.n * heads;
        x.pos0 = 0;
        x.cached = y.shared[e];
        x.keys = x.cached;
    } else {
        const int b = e - groups, g = group_of(y.start, groups, b);
        const int len = y.length[b];
        x.first = b;
        x.rows = a.n * heads;
        x.pos0 = g < 0 ? 0 : min(len, y.shared[g]);
        x.cached = len - x.pos0;
        x.keys = x.cached + a.n;
    }
    shape(x);
    return x;
}

// Length of an entry on the line.  A unit begins with the places of kUnit
// tiles, for what it costs apart from its tiles (queries, partial, a masked
// tile).  Without them the workgroups that meet many short units end last
// (16 users' draft trees: 191 us; with 3: 155 us).
constexpr int kUnit = 3;

__device__ __forceinline__ long long unit_length(const Entry &x) {
    return x.tiles > 0 ? (long long)x.weight * (kUnit + x.tiles) : 0;
}
__device__ __forceinline__ long long line_length(const AttentionArgs &a, const Entry &x) {
    return unit_length(x) * x.row_tiles * a.Hkv;
}

// Sums and maxima over a wave by lane moves inside the vector unit: row shifts
// by 1, 2, 4 and 8, then lane 15 of a row of 16 to the next row, lane 31 to the
// upper half.  (Exchanges through LDS cost a round trip each; a single token's
// call spends 1 us less on its line this way.)
template <typename F>
__device__ __forceinline__ int wave_scan(int x, F op) {
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
    return op(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
}
__device__ __forceinline__ int wave_max(int x) {       // of numbers that are not negative
    return __builtin_amdgcn_readlane(wave_scan(x, [](int a, int b) { return max(a, b); }), 63);
}
// 0 <= x < 2^52, in two parts whose sums fit 32 bits
__device__ __forceinline__ long long wave_inclusive64(long long x) {
    auto add = [](int a, int b) { return (int)((uint32_t)a + (uint32_t)b); };
    const uint32_t lo = (uint32_t)wave_scan((int)(x & 0x3ffffff), add);
    const uint32_t hi = (uint32_t)wave_scan((int)(x >> 26), add);
    return ((long long)hi << 26) + lo;
}

template <int D>
struct Tile {
    uint16_t k[kKeys * D];               // rows of keys, 16-byte pieces turned (k_piece)
    uint16_t v[kKeys * D];               // rows of values (v_piece)
};

struct Smem {
    float ml[2][2][32];                  // m and l of the waves that are merged
    uint32_t anc[GDN_MAX_NODES][4];      // ancestor-or-self bits
    int up[GDN_MAX_NODES];
    Batch batch;
    long long part[kWaves];
    long long first_off;
    int first_entry, max_own, max_shared, heavy;
    int flags[kWaves];                   // bad groups, shared tokens
    int lim[kWaves];                     // fewest cached keys seen, over a wave's rows
};

// Place of 16-byte piece c (8 elements) in a row: turned by the key, so that
// 32 keys read at one piece (keys) and 8 keys at four neighbouring pieces
// (values) spread over the 256 bytes that LDS serves at once.
template <int D>
__device__ __forceinline__ int k_piece(int key, int c) {
    return D >= 128 ? c ^ (key & 15) : c ^ ((key >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int v_piece(int key, int c) {
    return D >= 128 ? c ^ (4 * (key & 3)) : c ^ (4 * ((key >> 1) & 1));
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

// four elements of a column: lane i of 16 gives the address of piece i % 4 (4
// elements) of row i / 4 and receives column i of the four rows
__device__ __forceinline__ uint2 lds_transposed(const uint16_t *p) {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4 *)(p)));
}

// 16 bytes from memory to LDS, lane l to base + 16 l; counted by vmcnt
__device__ __forceinline__ void load_to_lds(const void *from, uint16_t *base) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)base, 16, 0, 0);
}

// the larger of lane l's and lane l ^ 32's
__device__ __forceinline__ float max_of_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// x, but not a constant of the loop around: what is computed from it is
// computed again, a few instructions, instead of held in registers throughout
__device__ __forceinline__ int keep_in_loop(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// a value that all lanes share, where the compiler cannot know: into a scalar
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ long long uniform(long long x) {
    const uint32_t lo = uniform((int)(uint32_t)x), hi = uniform((int)(x >> 32));
    return (long long)((uint64_t)hi << 32 | lo);
}

// a tile of the line
template <bool kLooks>
struct Cursor {
    // looks the keys up: x.first is the sequence whose page row names them
    static constexpr bool looks = kLooks;
    int e;               // entry
    int tile, rt, hk;    // tile of the unit, unit of the entry
    Entry x;
};

template <bool kLooks>
__device__ __forceinline__ void seek(const AttentionArgs &a, const Batch &y, int groups,
                                     int entries, Cursor<kLooks> &c, int e) {
    c.tile = c.rt = c.hk = 0;
    for (c.e = e; c.e < entries; ++c.e) {
        const Entry x = entry(a, y, groups, c.e);
        const int first = c.looks && c.e < groups ? y.whole[c.e] : x.first;
        c.x = {uniform(first),   uniform(x.rows),  uniform(x.pos0),     uniform(x.cached),
               uniform(x.keys),  uniform(x.tiles), uniform(x.row_tiles), uniform(x.weight)};
        if (c.x.tiles > 0 && c.x.row_tiles > 0) return;
    }
}

template <bool kLooks>
__device__ __forceinline__ void advance(const AttentionArgs &a, const Batch &y, int groups,
                                        int entries, Cursor<kLooks> &c) {
    if (c.e >= entries || ++c.tile < c.x.tiles) return;
    c.tile = 0;
    if (++c.rt < c.x.row_tiles) return;
    c.rt = 0;
    if (++c.hk < a.Hkv) return;
    seek(a, y, groups, entries, c, c.e + 1);
}

// Where the rows of a tile's keys are, lane l of a wave for key l.  Four tiles
// at once, one by each wave, every fourth tile; their page ids have been
// loaded (to LDS) four tiles before.  The value row is as far from the key row
// as the caches (or the tree's tensors) are from each other.
constexpr int kAhead = 4;                // kWaves
constexpr int kRing = 2 * kAhead;
constexpr unsigned long long kAbsent = 1;    // the key is not there: any row will do (its
                                             // score is masked, its value cleared)
constexpr unsigned long long kTree = 2;      // a row of the tree
struct Rows {
    unsigned long long k[kKeys];         // the key row's address and its flags
};

// Address of the tree's keys, and how far the cache's lie from them: added or
// not, where a choice between two kernel arguments would be compiled into a
// load of the chosen one, waiting for all loads before it.
struct Bases {
    unsigned long long k, to_kc;
};
__device__ __forceinline__ unsigned long long address(const void *p) {
    return reinterpret_cast<unsigned long long>(p);
}

__device__ __forceinline__ void load_pages(const AttentionArgs &a, const Cursor<true> &c, int key,
                                           int *to) {
    const int pos = c.x.pos0 + c.tile * kKeys + key;
    const int32_t *from = a.pages + (size_t)c.x.first * a.max_pages +
                          min(pos >> a.page_log, a.max_pages - 1);
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 4, 0, 0);
}

__device__ __forceinline__ void put_rows(const AttentionArgs &a, const Bases &y, const Cursor<true> &c,
                                         int key, const int *pages, Rows &rows) {
    const int j = c.tile * kKeys + key, pos = c.x.pos0 + j, tj = j - c.x.cached;
    const int page = pages[key];
    const bool there = tj < 0 ? page >= 0 && page < a.num_pages : j < c.x.keys;
    // bytes from the cache's or the tree's first, the parts that all keys
    // share in scalars (a page holds less than 2^31 elements)
    const unsigned long long cached0 = (2ULL * c.hk * a.d) << a.page_log;
    const unsigned long long tree0 = 2ULL * (((unsigned long long)c.x.first * a.n) * a.Hkv + c.hk) *
                                     a.d;
    const uint32_t in_page = 2u * (uint32_t)(pos & ((1 << a.page_log) - 1)) * a.d;
    const uint32_t in_tree = 2u * (uint32_t)tj * (uint32_t)(a.Hkv * a.d);
    const unsigned long long at =
        tj < 0 ? (unsigned long long)(uint32_t)page * (uint32_t)(2 * a.page_stride) + cached0 +
                     in_page
               : tree0 + in_tree;
    const unsigned long long cache = tj < 0 ? ~0ULL : 0ULL;
    rows.k[key] = y.k + (y.to_kc & cache) + (there ? at : kAbsent) + (kTree & ~cache);
}

template <typename E, int D>
__global__ __launch_bounds__(kThreads, D > 128 ? 1 : 2) void attention_kernel(AttentionArgs a,
                                                                             Layout lay) {
    typedef typename E::vec vec;
    constexpr int P = D / 8;                       // 16-byte pieces of a row
    constexpr int kLoads = kKeys * P / kThreads;   // pieces a thread loads of K, and of V
    constexpr int DT = D / 32;                     // 32-column tiles of the values
    // The two tiles are objects of their own, and the code names which one it
    // reads: the compiler then knows that the loads into the other one need
    // no wait.
    __shared__ __attribute__((aligned(16))) Tile<D> tile_0, tile_1;
    __shared__ Rows ring[kRing];         // by tile, modulo kRing
    __shared__ int page_ids[kAhead][kKeys];
    __shared__ Smem sm;

    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    // consecutive workgroups of the line share keys: give each XCD (block
    // index modulo 8) a run of them
    const int grid = gridDim.x;
    const int wg = grid % 8 == 0 ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
    char *ws = static_cast<char *>(a.workspace);

    // ---- lengths and groups; groups ascend within [0, batch], else none
    int groups = a.groups;
    // a group's longest member: its length, then the first that has it (the
    // ring is not in use yet)
    unsigned long long *longest = &ring[0].k[0];
    static_assert(sizeof(ring) >= 8 * GDN_MAX_SEQUENCES, "");
    Batch &bat = sm.batch;
    if (tid == 0) sm.max_own = 0, sm.max_shared = 0, sm.heavy = 1;
    for (int b = tid; b < a.batch; b += kThreads) bat.length[b] = fit_length(a, a.length[b]);
    bool bad = false, any_shared = false;
    for (int g = tid; g < groups; g += kThreads) {
        const int from = a.gstart[g], to = a.gstart[g + 1];
        bat.start[g] = (uint16_t)from;
        if (g == groups - 1) bat.start[groups] = (uint16_t)to;
        bat.shared[g] = fit_shared(a, to - from, a.gshared[g]);
        bat.whole[g] = (uint16_t)from;
        longest[g] = 0;
        any_shared |= bat.shared[g] > 0;
        bad |= from < 0 || to < from || to > a.batch;
    }
    // pieces past the head size are never loaded: zero for good
    if (a.d != D)
        for (int i = tid; i < (int)sizeof(Tile<D>) / 16; i += kThreads) {
            reinterpret_cast<uint4 *>(&tile_0)[i] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4 *>(&tile_1)[i] = make_uint4(0, 0, 0, 0);
        }
    if (const int f = (__any(bad) ? 1 : 0) | (__any(any_shared) ? 2 : 0); l == 0) sm.flags[w] = f;
    __syncthreads();
    const int flags = uniform(sm.flags[0] | sm.flags[1] | sm.flags[2] | sm.flags[3]);
    bad = flags & 1;
    if (bad) groups = 0;
    if (flags == 2) {
        for (int b = tid; b < a.batch; b += kThreads) {
            const int g = group_of(bat.start, groups, b);
            if (g >= 0)
                atomicMax(&longest[g], (unsigned long long)bat.length[b] << 9 |
                                           (unsigned)(GDN_MAX_SEQUENCES - 1 - b));
        }
        __syncthreads();
        for (int g = tid; g < groups; g += kThreads) {
            const unsigned long long x = longest[g];
            bat.whole[g] = (uint16_t)(GDN_MAX_SEQUENCES - 1 - (int)(x & 511));
            bat.shared[g] = min(bat.shared[g], (int)(x >> 9));
        }
        __syncthreads();
    }
    static_assert(GDN_MAX_SEQUENCES == 512, "nine bits of a sequence");
    const int entries = groups + a.batch;

    // ---- length of the line and of its longest units
    long long sum = 0;
    int own = 0, shared = 0, heavy = 1;
    for (int e = tid; e < entries; e += kThreads) {
        const Entry x = entry(a, bat, groups, e);
        sum += line_length(a, x);
        const int span = x.weight * (x.tiles - 1);      // from the first tile to the last
        if (e < groups) shared = max(shared, span);
        else own = max(own, span);
        heavy = max(heavy, x.weight);
    }
    sum = wave_inclusive64(sum);
    own = wave_max(own);
    shared = wave_max(shared);
    heavy = wave_max(heavy);
    if (l == 63) {
        sm.part[w] = sum;
        atomicMax(&sm.max_own, own);
        atomicMax(&sm.max_shared, shared);
        atomicMax(&sm.heavy, heavy);
    }
    __syncthreads();
    const long long total =
        uniform((sm.part[0] + sm.part[1]) + (sm.part[2] + sm.part[3]));
    // a unit whose tiles span s places meets at most (s - 1) / c + 2
    // workgroups: c keeps that within the partials there is room for.  With c
    // no less than a tile's places, none of these workgroups goes without.
    long long c = (total + grid - 1) / grid;
    c = max(c, (long long)(uniform(sm.max_own) + lay.slots.own - 2) / (lay.slots.own - 1));
    c = max(c, (long long)(uniform(sm.max_shared) + lay.slots.shared - 2) / (lay.slots.shared - 1));
    c = max(c, (long long)uniform(sm.heavy));
    const long long t0 = wg * c, t1 = min(total, t0 + c);
    if (t0 >= t1 && wg != 0) return;

    // ---- where this workgroup's tiles begin; workgroup 0 writes the line
    // down for the second kernel
    {
        GroupLine *gpre = reinterpret_cast<GroupLine *>(ws + lay.off_gpre);
        long long *bpre = reinterpret_cast<long long *>(ws + lay.off_bpre);
        int *group = reinterpret_cast<int *>(ws + lay.off_group);
        if (wg == 0 && tid == 0) {
            reinterpret_cast<Plan *>(ws)->per_wg = c;
        }
        long long before = 0;
        for (int e0 = 0; e0 < entries; e0 += kThreads) {
            const int e = e0 + tid;
            const long long x = e < entries ? line_length(a, entry(a, bat, groups, e)) : 0;
            const long long inc = wave_inclusive64(x);
            __syncthreads();
            if (l == 63) sm.part[w] = inc;
            __syncthreads();
            long long pre = before + inc - x;
            for (int i = 0; i < w; ++i) pre += sm.part[i];
            before += (sm.part[0] + sm.part[1]) + (sm.part[2] + sm.part[3]);
            if (e < entries && t0 >= pre && t0 < pre + x) {
                sm.first_entry = e;
                sm.first_off = t0 - pre;
            }
            if (wg == 0 && e < entries) {
                if (e < groups) gpre[e] = {pre, bat.shared[e], bat.whole[e]};
                else {
                    const int b = e - groups;
                    bpre[b] = pre;
                    group[b] = bad ? -2 : group_of(bat.start, groups, b);
                }
            }
        }
        __syncthreads();
    }
    if (t0 >= t1) return;

    const int heads = a.Hq / a.Hkv;
    float sc = a.scale * kLog2e;
    const bool flip = sc < 0.f;        // z = scale q.k: the sign goes into q, exactly
    const uint32_t keep = sc == 0.f ? 0u : ~0u;   // and a scale of zero: masked scores stay -inf
    sc = sc == 0.f ? 1.f : fabsf(sc);

    // the tile that is computed (its place on the line and its unit's, its
    // number in this workgroup), and the one whose rows this wave looks up
    Cursor<false> cur;
    Cursor<true> ahead;
    long long t, v0;
    int ti = 0;
    {
        seek(a, bat, groups, entries, cur, uniform(sm.first_entry));
        const long long off = uniform(sm.first_off), len = unit_length(cur.x);
        const long long unit = off / len;
        const int place = (int)(off - unit * len);
        cur.hk = (int)(unit / cur.x.row_tiles);
        cur.rt = (int)(unit % cur.x.row_tiles);
        v0 = t0 - place;
        cur.tile = max(0, (place + cur.x.weight - 1) / cur.x.weight - kUnit);
        if (cur.tile >= cur.x.tiles) {
            v0 += len;
            cur.tile = cur.x.tiles - 1;
            advance(a, bat, groups, entries, cur);
        }
        ahead = {cur.e, cur.tile, cur.rt, cur.hk, cur.x};
        if (cur.e < groups) ahead.x.first = uniform((int)bat.whole[cur.e]);
        t = cur.e < entries ? v0 + cur.x.weight * (kUnit + cur.tile) : t1;
    }
    if (t >= t1) return;               // places without a tile
    const Bases bases{address(a.k), address(a.kc) - address(a.k)};
    // from a cached key's row to its value's, and how much further in the tree
    const unsigned long long to_v = address(a.vc) - address(a.kc);
    const unsigned long long tree_v = address(a.v) - address(a.k) - to_v;
    auto fetch = [&](Tile<D> &to, const Rows &rows) {
        const unsigned lane = keep_in_loop(l);
        unsigned long long kr[kLoads], vr[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const unsigned key = ((w * kLoads + i) * 64 + lane) / P;
            kr[i] = rows.k[key];
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const unsigned long long tree = kr[i] & kTree ? ~0ULL : 0ULL;
            kr[i] &= ~(kAbsent | kTree);
            vr[i] = kr[i] + to_v + (tree_v & tree);
        }
        auto go = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int s0 = (w * kLoads + i) * 64;          // the wave's first piece
                const unsigned key = (s0 + lane) / P, c1 = lane % P;
                const int ck = k_piece<D>(key, c1), cv = v_piece<D>(key, c1);
                if (whole || 8 * ck < a.d)
                    load_to_lds(reinterpret_cast<const void *>(kr[i] + 16 * ck), &to.k[8 * s0]);
                if (whole || 8 * cv < a.d)
                    load_to_lds(reinterpret_cast<const void *>(vr[i] + 16 * cv), &to.v[8 * s0]);
            }
        };
        if (a.d == D) go(std::true_type{});
        else go(std::false_type{});
    };

    // ---- pipeline: page ids eight tiles ahead, the rows' places four, their
    // bytes one.  `ahead` is the wave's own tile of the four.
    auto skip = [&](int tiles) {
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) advance(a, bat, groups, entries, ahead);
    };
    auto look_ahead = [&](int first) {   // tiles first .. first + 3 from t0 on
        const int lane = keep_in_loop(l);
        if (ahead.e < entries)
            put_rows(a, bases, ahead, lane, page_ids[w], ring[(first + w) & (kRing - 1)]);
        skip(kAhead);
        if (ahead.e < entries) load_pages(a, ahead, lane, page_ids[w]);
    };
    skip(w);
    if (ahead.e < entries) load_pages(a, ahead, l, page_ids[w]);
    __builtin_amdgcn_s_waitcnt(kVmcntZero);
    look_ahead(0);
    lds_barrier();
    fetch(tile_0, ring[0]);

    int anc_of = -1;
    while (t < t1) {
        const Entry x = cur.x;
        const int tile0 = cur.tile, hk = cur.hk, r0 = cur.rt * kRows;
        const int count =
            (int)min((long long)(x.tiles - tile0), (t1 - t + x.weight - 1) / x.weight);
        const int slot = wg - (int)((v0 + x.weight * kUnit) / c);
        const bool is_own = cur.e >= groups;
        const int nrows = min(kRows, x.rows - r0);
        const int row_waves = nrows <= 32 ? 1 : nrows <= 64 ? 2 : 4;
        const int l = keep_in_loop(tid) & 63, m = l & 31, h = l >> 5;
        const int wr = w & (row_waves - 1);
        const int part = row_waves == 1 ? w & 1 : w >> 1;  // its keys (fewer than 4 row waves)
        // one row wave: half of the columns, in the first half of O
        const int col0 = row_waves == 1 ? (w >> 1) * (D / 2) : 0;

        // ---- the tree's ancestor bits, once per sequence: after step i
        // every node knows its 2^i nearest ancestors and jumps that far
        if (is_own && (tile0 + count) * kKeys > x.cached && anc_of != x.first) {
            anc_of = x.first;
            lds_barrier();
            int up = -1;
            if (tid < a.n) {
                up = a.parent[(size_t)x.first * a.n + tid];
                if (!parent_ok(up, tid)) up = -1;
                sm.up[tid] = up;
                for (int i = 0; i < 4; ++i) sm.anc[tid][i] = i == tid >> 5 ? 1u << (tid & 31) : 0u;
            }
            for (int far = 1; far < a.n; far <<= 1) {
                lds_barrier();
                uint32_t more[4] = {};
                int next = -1;
                if (tid < a.n && up >= 0) {
                    for (int i = 0; i < 4; ++i) more[i] = sm.anc[up][i];
                    next = sm.up[up];
                }
                lds_barrier();
                if (tid < a.n && up >= 0) {
                    for (int i = 0; i < 4; ++i) sm.anc[tid][i] |= more[i];
                    sm.up[tid] = up = next;
                }
            }
        }

        // ---- this lane's row: its query as B operands
        const int lr = r0 + 32 * wr + m;                       // row within the entry
        const bool rlive = 32 * wr + m < nrows;
        const int rr = rlive ? lr : r0;
        const size_t qrow =
            ((size_t)x.first * a.n + rr / heads) * a.Hq + (size_t)hk * heads + rr % heads;
        const int node = is_own ? rr / heads : 0;
        const int len_b = bat.length[x.first + rr / heads / a.n];
        const int lim = is_own ? x.cached : min(x.cached, len_b);   // cached keys it sees
        vec qf[D / 16];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint4 q4 = make_uint4(0, 0, 0, 0);
            const int d0 = 16 * kk + 8 * h;
            if (rlive && d0 < a.d)
                q4 = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) +
                                                      qrow * a.d + d0);
            const uint32_t sign = flip ? 0x80008000u : 0u;
            q4.x = (q4.x ^ sign) & keep, q4.y = (q4.y ^ sign) & keep;
            q4.z = (q4.z ^ sign) & keep, q4.w = (q4.w ^ sign) & keep;
            qf[kk] = __builtin_bit_cast(vec, q4);
        }
        int lim_min = lim;                                     // over the wave's rows
        if (!is_own) {
            for (int o = 1; o < 32; o <<= 1) lim_min = min(lim_min, __shfl_xor(lim_min, o));
            if (l == 0) sm.lim[w] = lim_min;
            lds_barrier();
        }
        const int lim_unit =
            uniform(is_own ? lim_min : min(min(sm.lim[0], sm.lim[1]), min(sm.lim[2], sm.lim[3])));

        f32x16 O[DT];
#pragma unroll
        for (int i = 0; i < DT; ++i) O[i] = f32x16{};
        float mx = -__builtin_inff(), ls = 0.f;
        bool odd = false;                  // values were cleared that are not finite

        auto one_tile = [&](Tile<D> &tile, Tile<D> &other, int tl) {
            // this tile has arrived, and everyone is done with the other one
            __builtin_amdgcn_s_waitcnt(kVmcntZero);
            lds_barrier();
            // ---- a tile that not all rows see whole (the last ones): clear
            // the values of keys that are not there, and infinities and NaN,
            // which a weight of zero would not keep out of the product; the
            // second kernel gives them back to the rows that see them
            if (__builtin_expect((tl + 1) * kKeys > lim_unit, 0)) {
                bool found = false;
                for (int i = keep_in_loop(tid); i < kKeys * P; i += kThreads) {
                    uint4 *p = reinterpret_cast<uint4 *>(&tile.v[8 * i]);
                    uint32_t x4[4] = {p->x, p->y, p->z, p->w};
                    const bool there = !(ring[ti & (kRing - 1)].k[i / P] & kAbsent);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t lo = E::kExponent, hi = E::kExponent << 16;
                        const uint32_t keep_lo = (x4[j] & lo) == lo ? 0u : 0xffffu;
                        const uint32_t keep_hi = (x4[j] & hi) == hi ? 0u : 0xffff0000u;
                        found |= there & ((keep_lo == 0) | (keep_hi == 0));
                        x4[j] = there ? x4[j] & (keep_lo | keep_hi) : 0u;
                    }
                    *p = make_uint4(x4[0], x4[1], x4[2], x4[3]);
                }
                if (__syncthreads_or(found)) odd = true;
            }
            if (ti % kAhead == 0) look_ahead(ti + kAhead);
            // the next tile, if there may be one (past the unit its weight is
            // not known here)
            if ((tl + 1 < x.tiles ? t + x.weight : t + x.weight + kUnit) < t1)
                fetch(other, ring[(ti + 1) & (kRing - 1)]);

#pragma unroll 1
            for (int st = 0; st < kKeys / 32; ++st) {
                if ((row_waves < 4 && st != part) || tl * kKeys + 32 * st >= x.keys) continue;
                // All reads of a product are issued before its first step: the
                // keys' before the scores, the values' before the softmax.
                // Key row m, piece 2 kk + h, turned: one exclusive or from kk = 0.
                const int ka = (32 * st + keep_in_loop(m)) * D + 8 * k_piece<D>(m, h);
                vec kf[D / 16];
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    kf[kk] = *reinterpret_cast<const vec *>(&tile.k[ka ^ (16 * kk)]);
                __builtin_amdgcn_sched_barrier(0);
                f32x16 z = {};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) z = E::mma(kf[kk], qf[kk], z);
                // values: columns 32 i + (m & 16) + 4 (l & 3) of key 4 h + (l >> 2) & 3,
                // turned: one exclusive or from i = 0
                const int vkey = 4 * h + ((keep_in_loop(l) >> 2) & 3);
                const int vcol = (m & 16) + 4 * (l & 3);
                const int va = ((32 * st + vkey) * D + 8 * v_piece<D>(vkey, vcol >> 3) +
                                (vcol & 7)) ^ col0;
                // this lane's column of tile i, keys 8 s + 4 h + (0..3)
                uint32_t vv[DT][8];
                auto read_values = [&](int i, uint32_t *y) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint2 x2 = lds_transposed(&tile.v[(va ^ (32 * i)) + 8 * s * D]);
                        y[2 * s] = x2.x, y[2 * s + 1] = x2.y;
                    }
                };
#pragma unroll
                for (int i = 0; i < DT / 2; ++i) read_values(i, vv[i]);
                if (row_waves > 1) {
#pragma unroll
                    for (int i = DT / 2; i < DT; ++i) read_values(i, vv[i]);
                }
                __builtin_amdgcn_sched_barrier(0);
                const int j0 = tl * kKeys + 32 * st;
                if (__builtin_expect(j0 + 32 > lim_unit, 0)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int j = j0 + crow(r, h), tj = j - x.cached;
                        const uint32_t up = sm.anc[node][min(max(tj, 0) >> 5, 3)] >> (tj & 31);
                        const bool see = ((j < lim) & (tj < 0)) |
                                         (is_own & (tj >= 0) & (tj < a.n) & ((up & 1u) != 0));
                        z[r] = see ? z[r] : -__builtin_inff();
                    }
                }
                float top = z[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
                top = max_of_halves(top) * sc;
                // The reference of the weights follows the scores only when
                // one passes it by kTop (in powers of two): weights stay below
                // 2^kTop, sums and partials are right for any reference, and O
                // is seldom multiplied.  A row that has seen no key yet keeps
                // -inf; its weights are zero.
                if (__builtin_expect(__any(top > mx + E::kTop), 0)) {
                    const float mn = fmaxf(mx, top - E::kLift);
                    const float f = __builtin_amdgcn_exp2f(mx - (mn == -__builtin_inff() ? 0.f : mn));
                    ls *= f;
#pragma unroll
                    for (int i = 0; i < DT; ++i) O[i] *= f;
                    mx = mn;
                }
                const float base = mx == -__builtin_inff() ? 0.f : mx;
                float p[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    p[r] = __builtin_amdgcn_exp2f(fmaf(z[r], sc, -base));
                    ls += p[r];
                }
                // weights rounded to the operand type: half a step each
                // (2^-8 or 2^-11 of a weight at most, and for fp16 2^-37 of the
                // largest), independent over the keys.  That is as much as
                // the rounding of the outputs again: 0.0020 to 0.0023 of them
                // in the 2-norm, 0.0017 without.  Two parts a weight would
                // take it away for half as many products again (medians: draft
                // trees 126 -> 152 us, a shared prompt 63 -> 71 us), and where the
                // second part is not positive, inf * weight would be NaN.
                const vec p0 = E::round8(p), p1 = E::round8(p + 8);
                auto times = [&](const uint32_t *y, f32x16 o) {
                    o = E::mma(__builtin_bit_cast(vec, make_uint4(y[0], y[1], y[2], y[3])), p0, o);
                    return E::mma(__builtin_bit_cast(vec, make_uint4(y[4], y[5], y[6], y[7])), p1,
                                  o);
                };
#pragma unroll
                for (int i = 0; i < DT / 2; ++i) O[i] = times(vv[i], O[i]);
                if (row_waves > 1) {
#pragma unroll
                    for (int i = DT / 2; i < DT; ++i) O[i] = times(vv[i], O[i]);
                }
            }
        };
        for (int tl = tile0; tl < tile0 + count; ++tl, t += x.weight, ++ti) {
            if (ti & 1) one_tile(tile_1, tile_0, tl);
            else one_tile(tile_0, tile_1, tl);
        }
        ls += __shfl_xor(ls, 32);

        // ---- join the two halves of the keys through the last tile's LDS
        bool writes = true;
        auto join_keys = [&](Tile<D> &tile) {
            const int l = keep_in_loop(tid) & 63, m = l & 31, h = l >> 5;
            float *buf = reinterpret_cast<float *>(&tile);
            const int which = row_waves == 1 ? w >> 1 : wr;
            static_assert(sizeof(Tile<D>) >= 4u * 2 * 32 * D, "");
            float *o = buf + (size_t)which * (32 * D);
            writes = part == 0;
            lds_barrier();
            if (!writes) {
#pragma unroll
                for (int i = 0; i < DT; ++i) {
                    if (row_waves == 1 && i >= DT / 2) break;
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[(i * 16 + r) * 64 + l] = O[i][r];
                }
                if (h == 0) {
                    sm.ml[which][0][m] = mx;
                    sm.ml[which][1][m] = ls;
                }
            }
            lds_barrier();
            if (writes) {
                const float mo = sm.ml[which][0][m], lo = sm.ml[which][1][m];
                const float mn = fmaxf(mx, mo), base = mn == -__builtin_inff() ? 0.f : mn;
                const float f = __builtin_amdgcn_exp2f(mx - base);
                const float g = __builtin_amdgcn_exp2f(mo - base);
                ls = ls * f + lo * g;
                mx = mn;
#pragma unroll
                for (int i = 0; i < DT; ++i) {
                    if (row_waves == 1 && i >= DT / 2) break;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        O[i][r] = O[i][r] * f + o[(i * 16 + r) * 64 + l] * g;
                }
            }
            if (a.d != D) {
                lds_barrier();
                for (int i = tid; i < (int)sizeof(Tile<D>) / 16; i += kThreads)
                    reinterpret_cast<uint4 *>(buf)[i] = make_uint4(0, 0, 0, 0);
            }
        };
        if (row_waves < 4) {
            if ((ti - 1) & 1) join_keys(tile_1);
            else join_keys(tile_0);
        }
        // ---- the partial: m, l (its sign bit set where values were cleared,
        // also on a sum of zero: all scores -inf) and o of the unit's rows
        if (writes && rlive) {
            const int s = is_own ? slot : lay.slots.own + slot;
            const size_t at = (size_t)s * lay.slots.rows + qrow;
            if (h == 0 && col0 == 0)
                reinterpret_cast<float2 *>(ws + lay.off_ml)[at] = make_float2(mx, odd ? -ls : ls);
            float *o = reinterpret_cast<float *>(ws + lay.off_o) + at * D;
#pragma unroll
            for (int i = 0; i < DT; ++i) {
                if (row_waves == 1 && i >= DT / 2) break;
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4)
                    *reinterpret_cast<float4 *>(&o[col0 + 32 * i + 8 * r4 + 4 * h]) =
                        make_float4(O[i][4 * r4], O[i][4 * r4 + 1], O[i][4 * r4 + 2],
                                    O[i][4 * r4 + 3]);
            }
        }
        // on to the next unit
        v0 += unit_length(x);
        cur.tile = x.tiles - 1;
        advance(a, bat, groups, entries, cur);
        if (t >= t1 || cur.e >= entries) break;
        t = v0 + cur.x.weight * kUnit;
    }
    // nothing may still be on its way into LDS that the next workgroup gets
    __builtin_amdgcn_s_waitcnt(kVmcntZero);
}

// Joins the partials of every row and checks the sequence: one workgroup per
// 1024 / D rows of a sequence, D / 4 lanes a row.
template <typename E, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(AttentionArgs a, Layout lay, int parts) {
    constexpr int kLanes = D / 4, kPer = kThreads / kLanes;
    __shared__ int s_fault;
    const int b = blockIdx.x / parts, part = blockIdx.x % parts, tid = threadIdx.x;
    const char *ws = static_cast<const char *>(a.workspace);
    const int heads = a.Hq / a.Hkv;
    // what does not depend on another load first: each round trip to memory
    // is a tenth of a single token's time
    const int g = reinterpret_cast<const int *>(ws + lay.off_group)[b];
    const long long c = reinterpret_cast<const Plan *>(ws)->per_wg;
    const long long own0 = reinterpret_cast<const long long *>(ws + lay.off_bpre)[b];
    const int raw = a.length[b];
    if (tid == 0) s_fault = g == -2 ? kFaultBadGroup : 0;
    int fault = 0;
    const bool len_ok = raw >= 0 && raw <= a.max_pages << a.page_log;
    if (!len_ok) fault = kFaultBadLength;
    const int len = len_ok ? raw : 0;
    for (int i = tid; i < a.n; i += kThreads)
        if (!parent_ok(a.parent[(size_t)b * a.n + i], i)) fault |= kFaultBadParent;
    const int gs = g >= 0 ? a.gstart[g] : b;
    const int members = g >= 0 ? a.gstart[g + 1] - gs : 1;
    const int said = g >= 0 ? a.gshared[g] : 0;
    const GroupLine line =
        g < 0 ? GroupLine{0, 0, b} : reinterpret_cast<const GroupLine *>(ws + lay.off_gpre)[g];
    const int sh = line.shared;

    // ---- the row's partials.  What the first kernel did with lengths that
    // do not fit is done here: there are as many partials as are counted, and
    // a fault found below only replaces the result.
    const int lr = part * kPer + tid / kLanes, d0 = 4 * (tid % kLanes);
    const bool live = lr < a.n * a.Hq && d0 < a.d;
    const int hq = lr % a.Hq, node = min(lr / a.Hq, a.n - 1), hk = hq / heads;
    const size_t qrow = (size_t)b * a.n * a.Hq + (live ? lr : 0);
    // the unit's first tile on the line and its tiles: its partials are one
    // per workgroup between
    auto partials = [&](long long start, int rows, int keys, int r) {
        Entry x;
        x.rows = rows;
        x.keys = keys;
        shape(x);
        const long long first =
            start + ((long long)hk * x.row_tiles + r / kRows) * unit_length(x) + x.weight * kUnit;
        return (int)((first + x.weight * (x.tiles - 1)) / c - first / c) + 1;
    };
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.f;
    bool odd = false;
    if (live) {
        const int r = node * heads + hq % heads, rows = a.n * heads;
        const int no = partials(own0, rows, len - min(len, sh) + a.n, r);
        const int ns = sh > 0 ? partials(line.pre, members * rows, sh, (b - gs) * rows + r) : 0;
        const float2 *ml = reinterpret_cast<const float2 *>(ws + lay.off_ml) + qrow;
        const float *o = reinterpret_cast<const float *>(ws + lay.off_o) + qrow * D + d0;
        // eight partials at a time: their loads do not wait for each other
        constexpr int kAtOnce = 8;
        float mx = -__builtin_inff();
        const int count = no + ns;
        for (int i0 = 0; i0 < count; i0 += kAtOnce) {
            float2 p[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int x = min(i0 + i, count - 1);
                const size_t s = (size_t)(x < no ? x : lay.slots.own + x - no) * lay.slots.rows;
                p[i] = ml[s];
                v[i] = *reinterpret_cast<const float4 *>(&o[s * D]);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (i0 + i >= count) break;
                const float mn = fmaxf(mx, p[i].x), base = mn == -__builtin_inff() ? 0.f : mn;
                const float f = __builtin_amdgcn_exp2f(mx - base);
                const float e = __builtin_amdgcn_exp2f(p[i].x - base);
                odd |= (int)__float_as_uint(p[i].y) < 0;
                ls = ls * f + fabsf(p[i].y) * e;
                acc.x = acc.x * f + v[i].x * e, acc.y = acc.y * f + v[i].y * e;
                acc.z = acc.z * f + v[i].z * e, acc.w = acc.w * f + v[i].w * e;
                mx = mn;
            }
        }
    }

    // ---- the sequence's pages
    const int32_t *row = a.pages + (size_t)b * a.max_pages;
    const int used = (int)(((long long)len + (1 << a.page_log) - 1) >> a.page_log);
    const int same_tokens = min(len, max(0, said));
    const int same = (int)(((long long)same_tokens + (1 << a.page_log) - 1) >> a.page_log);
    for (int c = tid; c < used; c += kThreads) {
        const int p = row[c];
        if (p < 0 || p >= a.num_pages) fault |= kFaultBadPage;
        if (c < same && p != a.pages[(size_t)line.whole * a.max_pages + c]) fault |= kFaultBadGroup;
    }
    if (said < 0) fault |= kFaultBadGroup;
    __syncthreads();                     // s_fault has its first value
    if (fault) atomicOr(&s_fault, fault);
    __syncthreads();
    fault = s_fault;
    if (a.status && part == 0 && tid == 0) a.status[b] = fault;
    if (!live) return;

    uint16_t *out = static_cast<uint16_t *>(a.out) + qrow * a.d + d0;
    float inv;
    if (fault) {
        inv = __builtin_nanf("");
    } else {
        inv = 1.f / ls;
        if (odd) {
            // The sequence's tiles that not all rows saw whole were computed
            // without infinities and NaN.  What this row sees of them decides
            // its columns: one sign of infinity, or NaN.  Of the shared tokens
            // these are the tiles from the shortest member's end on, the one
            // where the shared part ends inside a tile among them.
            const int pos0 = min(len, sh), from_own = pos0 + (len - pos0) / kKeys * kKeys;
            int shortest = sh;
            for (int i = 0; i < members && sh > 0; ++i)
                shortest = min(shortest, fit_length(a, a.length[gs + i]));
            const int from = sh > 0 ? shortest / kKeys * kKeys : from_own;
            float x[4] = {};
            auto see = [&](const void *base, size_t at) {
                const uint16_t *v = static_cast<const uint16_t *>(base) + at + d0;
                for (int e = 0; e < 4; ++e) {
                    const float y = E::widen(v[e]);
                    if (!(fabsf(y) < __builtin_inff())) x[e] += y;
                }
            };
            for (int pos = from; pos < len; ++pos)
                if (pos < pos0 || pos >= from_own)
                    see(a.vc, (size_t)row[pos >> a.page_log] * a.page_stride +
                                  (((size_t)hk << a.page_log) +
                                   (pos & ((1 << a.page_log) - 1))) * a.d);
            for (int i = node; i >= 0; i = a.parent[(size_t)b * a.n + i])
                see(a.v, (((size_t)b * a.n + i) * a.Hkv + hk) * a.d);
            acc.x += x[0], acc.y += x[1], acc.z += x[2], acc.w += x[3];
        }
    }
    const uint32_t lo = E::bits(acc.x * inv) | (uint32_t)E::bits(acc.y * inv) << 16;
    const uint32_t hi = E::bits(acc.z * inv) | (uint32_t)E::bits(acc.w * inv) << 16;
    *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
}

int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

int64_t up16(int64_t x) { return (x + 15) & ~(int64_t)15; }

Layout layout(const AttentionArgs &a) {
    Layout y;
    const int D = padded_dim(a.d), heads = a.Hq / a.Hkv;
    const int64_t unit_rows = ((int64_t)a.n * heads + kRows - 1) / kRows;
    const int64_t most = ((((int64_t)a.max_pages << a.page_log) + a.n + kKeys - 1) / kKeys) *
                         unit_rows * a.Hkv * a.batch;
    // two workgroups fit a compute unit (one for heads of 256)
    y.grid = device_cu_count() * (D > 128 ? 1 : 2);
    if (2 * most < y.grid) y.grid = (int)(2 * most);
    y.slots.rows = (int64_t)a.batch * a.n * a.Hq;
    // an even load splits a unit over about grid / units workgroups
    const int64_t tiles = (((int64_t)a.max_pages << a.page_log) + a.n + kKeys - 1) / kKeys;
    const int64_t units = (y.slots.rows + kRows - 1) / kRows;
    int64_t slots = y.grid / units + 2;
    if (slots > tiles) slots = tiles;
    if (slots < 2) slots = 2;
    y.slots.own = (int)slots;
    y.slots.shared = (int)slots;
    const int64_t held = y.slots.rows * (a.groups > 0 ? 2 * slots : slots);
    y.off_gpre = up16(sizeof(Plan));
    y.off_bpre = up16(y.off_gpre + (int64_t)sizeof(GroupLine) * a.groups);
    y.off_group = up16(y.off_bpre + 8LL * a.batch);
    y.off_ml = up16(y.off_group + 4LL * a.batch);
    y.off_o = up16(y.off_ml + 8 * held);
    y.bytes = y.off_o + 4 * held * D;
    return y;
}

template <typename E, int D>
hipError_t launch(const AttentionArgs &a, hipStream_t s) {
    const Layout y = layout(a);
    hipLaunchKernelGGL((attention_kernel<E, D>), dim3((unsigned)y.grid), dim3(kThreads), 0, s, a,
                       y);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int kPer = kThreads / (D / 4);
    const int parts = (a.n * a.Hq + kPer - 1) / kPer;
    hipLaunchKernelGGL((join_kernel<E, D>), dim3((unsigned)a.batch * parts), dim3(kThreads), 0, s,
                       a, y, parts);
    return hipGetLastError();
}

}  // namespace

int64_t attention_workspace(const AttentionArgs &a) { return layout(a).bytes; }

hipError_t launch_tree_attention(const AttentionArgs &a, hipStream_t s) {
    const int D = padded_dim(a.d);
    if (a.dtype == GDN_DTYPE_BF16)
        return D == 64 ? launch<Bf16, 64>(a, s) : D == 128 ? launch<Bf16, 128>(a, s)
                                                           : launch<Bf16, 256>(a, s);
    return D == 64 ? launch<F16, 64>(a, s) : D == 128 ? launch<F16, 128>(a, s)
                                                      : launch<F16, 256>(a, s);
}

}  // namespace gdn
