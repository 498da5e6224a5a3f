// Softmax attention of a draft tree over a paged cache whose prefix may be
// shared by groups of sequences (gfx950).
//
// A row (sequence, node, query head) attends to the tokens of its sequence's
// cache and to its node's ancestors-or-self.  The softmax is split over the
// keys: any part of them gives m = max z, l = sum e^{z - m} and
// o = sum e^{z - m} v, and parts join by
//     m = max m_i,   out = sum e^{m_i - m} o_i / sum e^{m_i - m} l_i,
// so a prefix that several sequences share is one part, computed for all
// their rows together with each key and value read once, and a long context
// is split over workgroups.
//
// Work: a unit is (group, key head, 128 rows) over the shared tokens or
// (sequence, key head, 128 rows) over its own tokens and tree nodes, cut into
// tiles of 128 keys.  All units' tiles form one line, and workgroup i takes
// the tiles [i c, (i + 1) c) of it, whatever units they belong to: every
// workgroup has the same number of tiles for any mix of lengths.  Lengths are
// device data, so every workgroup forms the line's prefix sums by itself (a
// scan over the batch).  Each unit a workgroup meets leaves one partial
// (m, l, o) in the workspace; a second kernel joins a row's partials.
//
// Tile: Z^T = K Q^T puts a query row into a lane's column and its keys into
// the lane's registers, so maxima and sums are in-register plus one exchange
// between the wave's halves, and e^{z - m} is, rounded, the B operand of
// O^T += V^T P^T as it stands (mfma_tile.hpp).  A unit of up to 32 rows has
// its four waves take different keys of the tile (merged through LDS at the
// unit's end), one of more rows has them take 32 rows each.
#include "device_common.hpp"
#include "serving.hpp"
#include "mfma_tile.hpp"

namespace gdn {
namespace {

using namespace tile;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kKeys = 128;                // keys of a tile
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
};

// what the first kernel leaves for the second
struct Plan {
    long long tiles_per_wg;
    long long total;
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

__device__ __forceinline__ int clamp_length(const AttentionArgs &a, int b) {
    const int len = a.length[b];
    return len < 0 || len > (a.max_pages << a.page_log) ? 0 : len;
}

// group of sequence b, or -1.  start ascends within [0, batch] (checked).
__device__ __forceinline__ int group_of(const int *start, int groups, int b) {
    if (groups == 0 || b < start[0] || b >= start[groups]) return -1;
    int lo = 0, hi = groups - 1;            // last g with start[g] <= b
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// tokens computed once for the group: none for a group of one sequence (its
// own part covers them)
__device__ __forceinline__ int shared_tokens(const AttentionArgs &a, const int *start, int g) {
    if (start[g + 1] - start[g] < 2) return 0;
    const int sh = a.gshared[g];
    return max(0, min(sh, a.max_pages << a.page_log));
}

__device__ __forceinline__ Entry entry(const AttentionArgs &a, const int *start, int groups,
                                       int e) {
    Entry x;
    const int heads = a.Hq / a.Hkv;
    if (e < groups) {
        x.first = start[e];
        x.rows = (start[e + 1] - start[e]) * a.n * heads;
        x.pos0 = 0;
        x.cached = shared_tokens(a, start, e);
        x.keys = x.cached;
    } else {
        const int b = e - groups, g = group_of(start, groups, b);
        const int len = clamp_length(a, b);
        x.first = b;
        x.rows = a.n * heads;
        x.pos0 = g < 0 ? 0 : min(len, shared_tokens(a, start, g));
        x.cached = len - x.pos0;
        x.keys = x.cached + a.n;
    }
    x.tiles = (x.keys + kKeys - 1) / kKeys;
    x.row_tiles = (x.rows + kRows - 1) / kRows;
    return x;
}

__device__ __forceinline__ long long line_tiles(const AttentionArgs &a, const Entry &x) {
    return (long long)x.tiles * x.row_tiles * a.Hkv;
}

__device__ __forceinline__ long long wave_inclusive64(long long x) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const long long up = __shfl_up(x, o);
        if (l >= o) x += up;
    }
    return x;
}

template <int D>
struct Smem {
    uint16_t k[kKeys * D];               // rows of keys, 16-byte pieces swizzled
    uint16_t vt[D * kKeys];              // values transposed, 8-byte pieces swizzled
    long long off[2][kKeys];             // element offset of a key's row, by tile parity
    uint32_t anc[GDN_MAX_NODES][4];      // ancestor-or-self bits
    int up[GDN_MAX_NODES];
    int start[GDN_MAX_SEQUENCES + 1];
    long long part[kWaves];
    long long total, first_off;
    int first_entry, max_own, max_shared, bad;
    int lim[kWaves];                     // fewest cached keys seen, over a wave's rows
    int odd[2];                          // a masked tile has values that are not finite
};

// Offsets carry their source: cache rows as they are, tree rows with kTree
// set, keys that are not there -1.
constexpr long long kTree = 1LL << 62;

// 16-byte piece c (8 elements) of a key row: rows of D elements, the piece's
// place turned by the key so that 32 keys read at one piece spread over all
// banks
template <int D>
__device__ __forceinline__ int k_at(int key, int c) {
    constexpr int P = D / 8;                       // pieces of a row
    const int turn = D >= 128 ? key & 15 : (key >> 1) & 7;
    return key * D + 8 * ((c & ~15) | ((c ^ turn) & (P < 16 ? P - 1 : 15)));
}

// four keys (8 bytes, quad = place in contraction order) of value column d:
// the place turned by d so that both the transposing stores (lanes 8 columns
// apart) and the reads (lanes one column apart) spread over the banks
__device__ __forceinline__ int v_at(int d, int quad) {
    const int turn = 2 * (((d >> 3) ^ (2 * (d & 7))) & 15);
    return d * kKeys + 4 * (quad ^ turn);
}

template <typename E, int D>
__global__ __launch_bounds__(kThreads, D > 128 ? 1 : 2) void attention_kernel(AttentionArgs a,
                                                                             Layout lay) {
    typedef typename E::vec vec;
    constexpr int P = D / 8;                       // 16-byte pieces of a row
    constexpr int kQuads = kKeys / 4;
    constexpr int kStep = kThreads / P;            // key quads staged at once
    constexpr int kPasses = kQuads / kStep;
    __shared__ Smem<D> sm;

    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const int m = l & 31, h = l >> 5;
    // consecutive workgroups of the line share keys: give each XCD (block
    // index modulo 8) a run of them
    const int grid = gridDim.x;
    const int wg = grid % 8 == 0 ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
    char *ws = static_cast<char *>(a.workspace);

    // ---- groups: ascending within [0, batch], else none
    int groups = a.groups;
    if (tid == 0) sm.bad = 0, sm.max_own = 0, sm.max_shared = 0;
    for (int g = tid; g <= groups && groups > 0; g += kThreads) sm.start[g] = a.gstart[g];
    __syncthreads();
    for (int g = tid; g < groups; g += kThreads)
        if (sm.start[g] < 0 || sm.start[g + 1] < sm.start[g] || sm.start[g + 1] > a.batch)
            sm.bad = 1;
    __syncthreads();
    if (sm.bad) groups = 0;
    const int entries = groups + a.batch;

    // ---- length of the line and of its longest units
    long long sum = 0;
    int own = 0, shared = 0;
    for (int e = tid; e < entries; e += kThreads) {
        const Entry x = entry(a, sm.start, groups, e);
        sum += line_tiles(a, x);
        if (e < groups) shared = max(shared, x.tiles);
        else own = max(own, x.tiles);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        sum += __shfl_xor(sum, o);
        own = max(own, __shfl_xor(own, o));
        shared = max(shared, __shfl_xor(shared, o));
    }
    if (l == 0) {
        sm.part[w] = sum;
        atomicMax(&sm.max_own, own);
        atomicMax(&sm.max_shared, shared);
    }
    __syncthreads();
    const long long total = (sm.part[0] + sm.part[1]) + (sm.part[2] + sm.part[3]);
    // a unit of T tiles meets at most (T - 2) / c + 2 workgroups: c keeps
    // that within the partials there is room for
    long long c = (total + grid - 1) / grid;
    c = max(c, (long long)(sm.max_own + lay.slots.own - 3) / (lay.slots.own - 1));
    c = max(c, (long long)(sm.max_shared + lay.slots.shared - 3) / (lay.slots.shared - 1));
    c = max(c, 1LL);
    const long long t0 = wg * c, t1 = min(total, t0 + c);
    if (t0 >= t1 && wg != 0) return;

    // ---- where this workgroup's tiles begin; workgroup 0 writes the line
    // down for the second kernel
    {
        long long *gpre = reinterpret_cast<long long *>(ws + lay.off_gpre);
        long long *bpre = reinterpret_cast<long long *>(ws + lay.off_bpre);
        int *group = reinterpret_cast<int *>(ws + lay.off_group);
        if (wg == 0 && tid == 0) {
            Plan *p = reinterpret_cast<Plan *>(ws);
            p->tiles_per_wg = c;
            p->total = total;
        }
        long long before = 0;
        for (int e0 = 0; e0 < entries; e0 += kThreads) {
            const int e = e0 + tid;
            const long long x = e < entries ? line_tiles(a, entry(a, sm.start, groups, e)) : 0;
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
                if (e < groups) gpre[e] = pre;
                else {
                    const int b = e - groups;
                    bpre[b] = pre;
                    group[b] = sm.bad ? -2 : group_of(sm.start, groups, b);
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
    const int d8 = tid % P, qd0 = tid / P;        // staging: this thread's piece and first quad
    const bool dlive = 8 * d8 < a.d;
    const uint16_t *kc = static_cast<const uint16_t *>(a.kc);
    const uint16_t *vc = static_cast<const uint16_t *>(a.vc);
    const uint16_t *kt = static_cast<const uint16_t *>(a.k);
    const uint16_t *vtree = static_cast<const uint16_t *>(a.v);

    int e = sm.first_entry;
    long long off = sm.first_off;
    int anc_of = -1;
    long long t = t0;
    while (t < t1) {
        const Entry x = entry(a, sm.start, groups, e);
        const long long in_entry = line_tiles(a, x);
        if (off >= in_entry) {
            ++e;
            off = 0;
            continue;
        }
        const long long unit = off / x.tiles;
        const int tile0 = (int)(off - unit * x.tiles);
        const int count = (int)min((long long)(x.tiles - tile0), t1 - t);
        const int hk = (int)(unit / x.row_tiles), r0 = (int)(unit % x.row_tiles) * kRows;
        const int slot = wg - (int)((t - tile0) / c);
        const bool is_own = e >= groups;
        const int nrows = min(kRows, x.rows - r0);
        const int row_waves = nrows <= 32 ? 1 : nrows <= 64 ? 2 : 4;
        const int key_waves = kWaves / row_waves;
        const int wr = w & (row_waves - 1), wk = w / row_waves;
        const int32_t *prow = a.pages + (size_t)x.first * a.max_pages;
        const bool tree = is_own && (tile0 + count) * kKeys > x.cached;

        // ---- the tree's ancestor bits, once per sequence: after step i
        // every node knows its 2^i nearest ancestors and jumps that far
        if (tree && anc_of != x.first) {
            anc_of = x.first;
            __syncthreads();
            int up = -1;
            uint32_t bits[4] = {};
            if (tid < a.n) {
                up = a.parent[(size_t)x.first * a.n + tid];
                if (!parent_ok(up, tid)) up = -1;
                bits[tid >> 5] = 1u << (tid & 31);
                sm.up[tid] = up;
                for (int i = 0; i < 4; ++i) sm.anc[tid][i] = i == tid >> 5 ? 1u << (tid & 31) : 0u;
            }
            for (int far = 1; far < a.n; far <<= 1) {
                __syncthreads();
                uint32_t more[4] = {};
                int next = -1;
                if (tid < a.n && up >= 0) {
                    for (int i = 0; i < 4; ++i) more[i] = sm.anc[up][i];
                    next = sm.up[up];
                }
                __syncthreads();
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
        const size_t qrow = ((size_t)x.first * a.n + rr / heads) * a.Hq + (size_t)hk * heads + rr % heads;
        const int node = is_own ? rr / heads : 0;
        const int len_b = clamp_length(a, x.first + rr / heads / a.n);
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
        int lim_min = lim;                                     // over the unit's rows
        if (!is_own) {
            for (int o = 1; o < 32; o <<= 1) lim_min = min(lim_min, __shfl_xor(lim_min, o));
        }
        __syncthreads();
        if (l == 0) sm.lim[w] = lim_min;
        if (tid < 2) sm.odd[tid] = 0;

        // element offset of a key's row (thread tid < kKeys: key tid of the tile)
        auto key_offset = [&](int tl) -> long long {
            const int j = tl * kKeys + tid;
            if (tid >= kKeys || j >= x.keys) return -1;
            if (j < x.cached) {
                const int pos = x.pos0 + j;
                const int p = prow[pos >> a.page_log];
                if (p < 0 || p >= a.num_pages) return -1;
                return (long long)p * a.page_stride +
                       (((long long)hk << a.page_log) + (pos & ((1 << a.page_log) - 1))) * a.d;
            }
            return kTree | ((((long long)x.first * a.n + (j - x.cached)) * a.Hkv + hk) * a.d);
        };
        uint4 kx[kPasses][4], vx[kPasses][4];
        auto fetch = [&](int tl) {
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long o = sm.off[tl & 1][4 * (qd0 + p * kStep) + i];
                    const bool ok = o >= 0 && dlive, tr = ok && (o & kTree);
                    const size_t at = ok ? (size_t)(o & ~kTree) + 8 * d8 : 0;
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    const uint4 kv = *reinterpret_cast<const uint4 *>((tr ? kt : kc) + at);
                    const uint4 vv = *reinterpret_cast<const uint4 *>((tr ? vtree : vc) + at);
                    kx[p][i] = ok ? kv : zero;
                    vx[p][i] = ok ? vv : zero;
                }
        };

        f32x16 O[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) O[i] = f32x16{};
        float mx = -__builtin_inff(), ls = 0.f;

        // ---- pipeline: row offsets two tiles ahead, rows one tile ahead
        if (tid < kKeys) sm.off[tile0 & 1][tid] = key_offset(tile0);
        long long next_off = key_offset(tile0 + 1);
        if (tid < kKeys) sm.off[(tile0 + 1) & 1][tid] = next_off;
        __syncthreads();
        fetch(tile0);
        const int lim_unit = min(min(sm.lim[0], sm.lim[1]), min(sm.lim[2], sm.lim[3]));

        for (int tl = tile0; tl < tile0 + count; ++tl) {
            __syncthreads();                      // the last tile's readers are done
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                const int quad = qd0 + p * kStep;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(&sm.k[k_at<D>(4 * quad + i, d8)]) = kx[p][i];
                // place of the quad in contraction order: bits 0, 1 swap
                const int place = (quad & ~3) | ((quad & 1) << 1) | ((quad >> 1) & 1);
                const uint32_t *a0 = reinterpret_cast<const uint32_t *>(&vx[p][0]);
                const uint32_t *a1 = reinterpret_cast<const uint32_t *>(&vx[p][1]);
                const uint32_t *a2 = reinterpret_cast<const uint32_t *>(&vx[p][2]);
                const uint32_t *a3 = reinterpret_cast<const uint32_t *>(&vx[p][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {     // columns 2 i, 2 i + 1 of the piece
                    const uint2 even = make_uint2(__builtin_amdgcn_perm(a1[i], a0[i], 0x05040100u),
                                                  __builtin_amdgcn_perm(a3[i], a2[i], 0x05040100u));
                    const uint2 odd = make_uint2(__builtin_amdgcn_perm(a1[i], a0[i], 0x07060302u),
                                                 __builtin_amdgcn_perm(a3[i], a2[i], 0x07060302u));
                    *reinterpret_cast<uint2 *>(&sm.vt[v_at(8 * d8 + 2 * i, place)]) = even;
                    *reinterpret_cast<uint2 *>(&sm.vt[v_at(8 * d8 + 2 * i + 1, place)]) = odd;
                }
            }
            // a key that only some rows see may hold anything: weights of zero
            // do not keep an infinity or a NaN out of the matrix product
            if ((tl + 1) * kKeys > lim_unit) {
                bool odd = false;
#pragma unroll
                for (int p = 0; p < kPasses; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t *x4 = reinterpret_cast<const uint32_t *>(&vx[p][i]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t lo = E::kExponent, hi = E::kExponent << 16;
                            odd |= (x4[j] & lo) == lo || (x4[j] & hi) == hi;
                        }
                    }
                if (odd) sm.odd[tl & 1] = 1;
            }
            const bool more = tl + 1 < tile0 + count;
            if (more) {
                fetch(tl + 1);
                next_off = key_offset(tl + 2);
            }
            __syncthreads();
            // readers of this parity's offsets fetched before the barrier above
            if (more && tid < kKeys) sm.off[tl & 1][tid] = next_off;
            const bool odd = __builtin_amdgcn_readfirstlane(sm.odd[tl & 1]) != 0;
            if (tid == 0) sm.odd[(tl + 1) & 1] = 0;

            const int keys = min(kKeys, x.keys - tl * kKeys);
            for (int st = wk; 32 * st < keys; st += key_waves) {
                f32x16 z = {};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const vec ka = *reinterpret_cast<const vec *>(
                        &sm.k[k_at<D>(32 * st + m, 2 * kk + h)]);
                    z = E::mma(ka, qf[kk], z);
                }
                const int j0 = tl * kKeys + 32 * st;
                if (j0 + 32 > lim_min) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int j = j0 + crow(r, h), tj = j - x.cached;
                        bool see = j < lim;
                        if (is_own && tj >= 0 && tj < a.n)
                            see = (sm.anc[node][tj >> 5] >> (tj & 31)) & 1u;
                        z[r] = see ? z[r] : -__builtin_inff();
                    }
                }
                float top = z[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, z[r]);
                top = fmaxf(top, __shfl_xor(top, 32)) * sc;
                const float mn = fmaxf(mx, top);
                // a row that has seen no key yet keeps -inf; its weights are zero
                const float base = mn == -__builtin_inff() ? 0.f : mn;
                if (__any(mn > mx)) {
                    const float f = __builtin_amdgcn_exp2f(mx - base);
                    ls *= f;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) O[i] *= f;
                    mx = mn;
                }
                float p[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    p[r] = __builtin_amdgcn_exp2f(fmaf(z[r], sc, -base));
                    ls += p[r];
                }
                if (odd) {
                    // key by key, leaving out what has no weight (rare)
                    for (int key = 0; key < 32; ++key) {
                        float pk = 0.f;
                        // register of the key in either half's lanes
                        const int rk = 4 * (key >> 3) + (key & 3);
#pragma unroll
                        for (int r = 0; r < 16; ++r) pk = r == rk ? p[r] : pk;
                        pk = E::widen(E::bits(__shfl(pk, m + 32 * ((key >> 2) & 1))));
                        const int quad = 8 * st + (key >> 2);
                        const int place =
                            (quad & ~3) | ((quad & 1) << 1) | ((quad >> 1) & 1);
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
#pragma unroll
                            for (int r = 0; r < 16; ++r) {
                                const float x1 = E::widen(
                                    sm.vt[v_at(32 * i + crow(r, h), place) + (key & 3)]);
                                O[i][r] = pk != 0.f ? fmaf(pk, x1, O[i][r]) : O[i][r];
                            }
                    }
                    continue;
                }
                // weights rounded to the operand type: half a step each
                // (2^-9 or 2^-12 of a weight), independent over the keys
                const vec p0 = E::round8(p), p1 = E::round8(p + 8);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int d = 32 * i + m;
                    const vec v0 = *reinterpret_cast<const vec *>(&sm.vt[v_at(d, 8 * st + 2 * h)]);
                    const vec v1 =
                        *reinterpret_cast<const vec *>(&sm.vt[v_at(d, 8 * st + 4 + 2 * h)]);
                    O[i] = E::mma(v0, p0, O[i]);
                    O[i] = E::mma(v1, p1, O[i]);
                }
            }
        }
        ls += __shfl_xor(ls, 32);

        // ---- join the key waves of a row through LDS, in wave order
        if (key_waves > 1) {
            float *buf = reinterpret_cast<float *>(&sm);       // [wave][D/32][16][64], then m, l
            static_assert(sizeof(sm.k) + sizeof(sm.vt) >= 4u * (kWaves - 1) * (32 * D + 64), "");
            __syncthreads();
            if (wk > 0) {
                float *o = buf + (size_t)(w - row_waves) * (32 * D + 64);
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[(i * 16 + r) * 64 + l] = O[i][r];
                if (h == 0) {
                    o[32 * D + m] = mx;
                    o[32 * D + 32 + m] = ls;
                }
            }
            __syncthreads();
            if (wk == 0) {
                for (int k2 = 1; k2 < key_waves; ++k2) {
                    const float *o = buf + (size_t)(k2 * row_waves + wr - row_waves) * (32 * D + 64);
                    const float mo = o[32 * D + m], lo = o[32 * D + 32 + m];
                    const float mn = fmaxf(mx, mo), base = mn == -__builtin_inff() ? 0.f : mn;
                    const float f = __builtin_amdgcn_exp2f(mx - base);
                    const float g = __builtin_amdgcn_exp2f(mo - base);
                    ls = ls * f + lo * g;
                    mx = mn;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            O[i][r] = O[i][r] * f + o[(i * 16 + r) * 64 + l] * g;
                }
            }
        }
        // ---- the partial: m, l and o of the unit's rows
        if (wk == 0 && rlive) {
            const int s = is_own ? slot : lay.slots.own + slot;
            const size_t at = (size_t)s * lay.slots.rows + qrow;
            if (h == 0)
                reinterpret_cast<float2 *>(ws + lay.off_ml)[at] = make_float2(mx, ls);
            float *o = reinterpret_cast<float *>(ws + lay.off_o) + at * D;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4)
                    *reinterpret_cast<float4 *>(&o[32 * i + 8 * r4 + 4 * h]) =
                        make_float4(O[i][4 * r4], O[i][4 * r4 + 1], O[i][4 * r4 + 2],
                                    O[i][4 * r4 + 3]);
        }
        t += count;
        off += count;
    }
}

// Joins the partials of every row and checks the sequence: one workgroup per
// 1024 / D rows of a sequence, D / 4 lanes a row.
template <typename E, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(AttentionArgs a, Layout lay, int parts) {
    constexpr int kLanes = D / 4, kPer = kThreads / kLanes;
    __shared__ int s_fault;
    const int b = blockIdx.x / parts, part = blockIdx.x % parts, tid = threadIdx.x;
    const char *ws = static_cast<const char *>(a.workspace);
    const Plan *plan = reinterpret_cast<const Plan *>(ws);
    const int g = reinterpret_cast<const int *>(ws + lay.off_group)[b];
    const int heads = a.Hq / a.Hkv;

    // ---- the sequence's own faults
    if (tid == 0) s_fault = g == -2 ? kFaultBadGroup : 0;
    __syncthreads();
    const int raw = a.length[b];
    int fault = 0;
    const bool len_ok = raw >= 0 && raw <= a.max_pages << a.page_log;
    if (!len_ok) fault = kFaultBadLength;
    const int len = len_ok ? raw : 0;
    for (int i = tid; i < a.n; i += kThreads)
        if (!parent_ok(a.parent[(size_t)b * a.n + i], i)) fault |= kFaultBadParent;
    const int32_t *row = a.pages + (size_t)b * a.max_pages;
    const int used = (int)(((long long)len + (1 << a.page_log) - 1) >> a.page_log);
    const int gs = g >= 0 ? a.gstart[g] : b;
    const int members = g >= 0 ? a.gstart[g + 1] - gs : 1;
    const int said = g >= 0 ? min(len, max(0, a.gshared[g])) : 0;
    const int same = (int)(((long long)said + (1 << a.page_log) - 1) >> a.page_log);
    for (int c = tid; c < used; c += kThreads) {
        const int p = row[c];
        if (p < 0 || p >= a.num_pages) fault |= kFaultBadPage;
        if (c < same && p != a.pages[(size_t)gs * a.max_pages + c]) fault |= kFaultBadGroup;
    }
    if (g >= 0 && a.gshared[g] < 0) fault |= kFaultBadGroup;
    if (fault) atomicOr(&s_fault, fault);
    __syncthreads();
    fault = s_fault;
    if (a.status && part == 0 && tid == 0) a.status[b] = fault;

    const int lr = part * kPer + tid / kLanes, d0 = 4 * (tid % kLanes);
    if (lr >= a.n * a.Hq || d0 >= a.d) return;
    const size_t qrow = (size_t)b * a.n * a.Hq + lr;
    uint16_t *out = static_cast<uint16_t *>(a.out) + qrow * a.d + d0;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float inv;
    if (fault) {
        inv = __builtin_nanf("");
    } else {
        const int hq = lr % a.Hq, node = lr / a.Hq, hk = hq / heads;
        const long long c = plan->tiles_per_wg;
        const long long *gpre = reinterpret_cast<const long long *>(ws + lay.off_gpre);
        const long long *bpre = reinterpret_cast<const long long *>(ws + lay.off_bpre);
        const int sh = members < 2 ? 0 : min(max(0, a.gshared[g]), a.max_pages << a.page_log);
        // the unit's first tile on the line and its tiles: its partials are
        // one per workgroup between
        const int row_tiles = (a.n * heads + kRows - 1) / kRows;
        const int own_tiles = (len - min(len, sh) + a.n + kKeys - 1) / kKeys;
        const int rt = (node * heads + hq % heads) / kRows;
        const long long o0 = bpre[b] + ((long long)hk * row_tiles + rt) * own_tiles;
        const int no = (int)((o0 + own_tiles - 1) / c - o0 / c) + 1;
        int ns = 0;
        if (sh > 0) {
            const int srow_tiles = (int)(((long long)members * a.n * heads + kRows - 1) / kRows);
            const int stiles = (sh + kKeys - 1) / kKeys;
            const int srt = (((b - gs) * a.n + node) * heads + hq % heads) / kRows;
            const long long s0 = gpre[g] + ((long long)hk * srow_tiles + srt) * stiles;
            ns = (int)((s0 + stiles - 1) / c - s0 / c) + 1;
        }
        const float2 *ml = reinterpret_cast<const float2 *>(ws + lay.off_ml) + qrow;
        const float *o = reinterpret_cast<const float *>(ws + lay.off_o) + qrow * D + d0;
        float mx = -__builtin_inff(), ls = 0.f;
        for (int i = 0; i < no + ns; ++i) {
            const size_t s = (size_t)(i < no ? i : lay.slots.own + i - no) * lay.slots.rows;
            const float2 p = ml[s];
            const float4 v = *reinterpret_cast<const float4 *>(&o[s * D]);
            const float mn = fmaxf(mx, p.x), base = mn == -__builtin_inff() ? 0.f : mn;
            const float f = __builtin_amdgcn_exp2f(mx - base), e = __builtin_amdgcn_exp2f(p.x - base);
            ls = ls * f + p.y * e;
            acc.x = acc.x * f + v.x * e, acc.y = acc.y * f + v.y * e;
            acc.z = acc.z * f + v.z * e, acc.w = acc.w * f + v.w * e;
            mx = mn;
        }
        inv = 1.f / ls;
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
    y.off_bpre = up16(y.off_gpre + 8LL * a.groups);
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
