// Rotary positions, norms of queries and keys, and both on the way into the
// paged cache.
//
// For a row (token) at position p and a head x of d elements:
//   norm     y = x / sqrt(mean x^2 + eps) (offset + w)     RMS, w: weights
//            y = x / sqrt(sum x^2 + eps) (offset + w)      L2 (no w: times 1)
//   rotation pair i of the first rot elements, (y_i, y_{i + rot/2}) or
//            (y_{2i}, y_{2i+1}), by the angle p f_i:
//            (y, y') -> scale (y cos - y' sin, y' cos + y sin)
// Every element is read once and written once (a key that also goes to its
// page: twice); 3 flops a rotated element and 4 a normed one: memory bounds long
// calls, the chain of dependent loads (place, page, angle, head) short ones.
//   8192 rows of 40 heads of 128, bf16: rotation (half of each, 27 us in a loop over
//     one input set) and norm with rotation (29 us): 29 and 32 us among other
//     passes, 5.7 and 5.3 TB/s; a copy of the same bytes 33 us
//   the same into pages of 64, 8 more heads of values, ragged: 53 us, a copy 46
//   one row: 3.4 us, with a norm 4.2, into its page 5.3
#include "heads.hpp"

namespace gdn {
namespace {

using namespace heads;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPairs = GDN_MAX_HEAD_DIM / 2 / 64;   // rotated pairs of a lane
constexpr int kRest = GDN_MAX_HEAD_DIM / 64;        // elements past the rotated ones

// One head in one wave: lane l has the pairs l and l + 64, and the elements
// rot + l, rot + l + 64, ...  Takes any size and alignment.
template <typename E>
struct Head {
    typedef typename E::type T;
    float a[kPairs] = {}, b[kPairs] = {}, r[kRest];

    __device__ __forceinline__ static int first(const HeadsArgs &g, int i) {
        return g.layout == GDN_ROPE_HALF ? i : 2 * i;
    }
    __device__ __forceinline__ static int second(const HeadsArgs &g, int i) {
        return g.layout == GDN_ROPE_HALF ? i + g.rot / 2 : 2 * i + 1;
    }
    template <typename F>
    __device__ __forceinline__ void each(const HeadsArgs &g, F f) {
        const int l = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
            if (l + 64 * j < g.rot / 2) {
                f(a[j], first(g, l + 64 * j));
                f(b[j], second(g, l + 64 * j));
            }
#pragma unroll
        for (int j = 0; j < kRest; ++j)
            if (g.rot + l + 64 * j < g.d) f(r[j], g.rot + l + 64 * j);
    }
    __device__ __forceinline__ void load(const HeadsArgs &g, const T *x) {
        each(g, [&](float &y, int i) { y = E::widen(x[i]); });
    }
    __device__ __forceinline__ void norm(const HeadsArgs &g, const void *w, int64_t at) {
        float s = 0.f;
        each(g, [&](float &y, int) { s = fmaf(y, y, s); });
        const float inv = inverse_norm(g, wave_sum(s));
        each(g, [&](float &y, int i) {
            y *= inv * (w ? g.offset + weight_at<E>(w, g.wide_weight, at + i) : 1.f);
        });
    }
    __device__ __forceinline__ void rotate(const float2 (&cs)[kPairs]) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const float x = a[j], y = b[j];
            a[j] = fmaf(x, cs[j].x, -(y * cs[j].y));
            b[j] = fmaf(y, cs[j].x, x * cs[j].y);
        }
    }
    __device__ __forceinline__ void store(const HeadsArgs &g, T *x) {
        each(g, [&](float &y, int i) { x[i] = E::bits(y); });
    }
};

__device__ __forceinline__ void angles(const HeadsArgs &g, int64_t p, float2 (&cs)[kPairs]) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
        cs[j] = l + 64 * j < g.rot / 2 ? turn(p, g.inv_freq[l + 64 * j], g.scale)
                                       : make_float2(0.f, 0.f);
}

template <typename E>
__device__ __forceinline__ void one_head(const HeadsArgs &g, const HeadsPart &x, int64_t row, int h,
                                         const float2 (&cs)[kPairs], Head<E> &y) {
    typedef typename E::type T;
    y.load(g, static_cast<const T *>(x.in) + row * x.in_row + h * x.in_head);
    if (g.norm != GDN_NORM_NONE) y.norm(g, x.weight, h * x.weight_head);
    y.rotate(cs);
}

// a wave for every row and `splits`-th part of its heads
template <typename E>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsArgs a, int splits) {
    typedef typename E::type T;
    const int64_t unit = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int64_t row = unit / splits;
    if (row >= a.rows) return;
    float2 cs[kPairs] = {};
    if (a.rot > 0)
        angles(a, (int64_t)a.pos[row] + (a.base ? a.base[row / a.base_rows] : 0), cs);
    for (int h = (int)(unit % splits); h < a.q.heads + a.k.heads; h += splits) {
        const bool k = h >= a.q.heads;
        const HeadsPart &x = k ? a.k : a.q;
        const int hx = k ? h - a.q.heads : h;
        Head<E> y;
        one_head<E>(a, x, row, hx, cs, y);
        y.store(a, static_cast<T *>(x.out) + row * x.out_row + hx * x.out_head);
    }
}

// The same with the keys, and the values beside them, written to their pages.
// Workgroups past the rows' report the requests' faults, a wave each.
template <typename E>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, int splits, int row_blocks) {
    typedef typename E::type T;
    const int w = threadIdx.x >> 6;
    const bool bad = a.cu && rows_bad(a);
    if ((int)blockIdx.x >= row_blocks) {
        const int r = ((int)blockIdx.x - row_blocks) * kWaves + w;
        if (r >= a.m) return;
        const int fault = bad ? kFaultBadLength
                              : request(a, r, a.cu ? a.cu[r + 1] - a.cu[r] : 1).fault;
        if ((threadIdx.x & 63) == 0) a.status[r] = fault;
        return;
    }
    const int64_t unit = (int64_t)blockIdx.x * kWaves + w;
    const int row = (int)(unit / splits);
    if (bad || row >= a.h.rows) return;
    int r = row, t = 0, len = 1;
    if (a.cu) {
        if (row < a.cu[0] || row >= a.cu[a.m]) return;
        r = find_request(a, 0, row);
        t = row - a.cu[r], len = a.cu[r + 1] - a.cu[r];
    }
    const Request q = request(a, r, len);
    const bool lost = q.fault || q.at < 0;
    const HeadsArgs &g = a.h;
    const int place = q.at + t;
    float2 cs[kPairs] = {};
    if (g.rot > 0 && !lost) angles(g, g.pos ? g.pos[row] : place, cs);
    size_t cell = 0;
    if (!lost) {
        const int p = a.table[(size_t)q.row * a.width + (place >> a.page_log)];
        cell = (size_t)p * a.page_stride + (size_t)(place & ((1 << a.page_log) - 1)) * g.d;
    }
    const int Hq = g.q.heads, Hk = g.k.heads;
    for (int h = (int)(unit % splits); h < Hq + 2 * Hk; h += splits) {
        Head<E> y;
        if (h >= Hq + Hk) {
            if (lost) continue;
            const int hv = h - Hq - Hk;
            y.load(g, static_cast<const T *>(a.v) + (int64_t)row * a.v_row + hv * a.v_head);
            y.store(g, static_cast<T *>(a.vc) + cell + ((size_t)hv << a.page_log) * g.d);
            continue;
        }
        const bool k = h >= Hq;
        const HeadsPart &x = k ? g.k : g.q;
        const int hx = k ? h - Hq : h;
        T *out = x.out ? static_cast<T *>(x.out) + row * x.out_row + hx * x.out_head : nullptr;
        if (lost) {
            y.each(g, [&](float &z, int) { z = __builtin_nanf(""); });
            if (out) y.store(g, out);
            continue;
        }
        one_head<E>(g, x, row, hx, cs, y);
        if (out) y.store(g, out);
        if (k) y.store(g, static_cast<T *>(a.kc) + cell + ((size_t)hx << a.page_log) * g.d);
    }
}

// ---------------------------------------------------------------------------
// The same in 16-byte pieces: a lane has two pieces of 8 elements of a head, and
// 64 / lanes(d) heads of queries, keys or values lie side by side in a wave, so
// that its loads and stores cover whole lines.  In the half layout the two
// pieces are the two sides of 8 pairs: no lane needs another's elements but for
// the norm's sum.  Angles are a row's, not a head's: each is formed by one lane,
// once, and handed to the lanes that need it through LDS.  The next heads are
// loaded while the present ones are worked on, the first ones before the row's
// place and angles are known.
//
// kSplit: half layout, sides of whole pieces.  kAdjacent: interleaved, whole
// pieces turn.  kMixed: either, where pieces turn in part; a lane has two of them
// as they lie, and the other side of its pairs comes through LDS.
// ---------------------------------------------------------------------------
enum Mode { kSplit, kAdjacent, kMixed };

struct Part {
    const void *in;
    int64_t in_row, in_head;
    void *out;           // null: not written
    int64_t out_row, out_head;
    const void *weight;  // null: ones
    int64_t weight_head;
    void *page;          // the cache that its heads go to, or null
    int heads, before;   // its heads, and the groups of heads before its own
};

struct Pieces {
    Part part[3];        // queries, keys, values (neither normalised nor turned)
    AppendArgs a;
    int log, need;       // lanes of a head: 1 << log, of which the first `need` have a part of it
    int groups, splits;  // groups of heads, and the waves that share a row's
    int rows;            // rows of a wave, kWaves apart
    int tiles;           // workgroups of one split, kWaves * rows rows each
};

typedef float f32x4 __attribute__((ext_vector_type(4)));

// 8 adjacent elements as they lie in memory
template <typename E>
struct Raw {
    uint4 x;
    __device__ __forceinline__ void load(const uint16_t *p) {
        x = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void widen(float (&y)[8]) const {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = E::widen((uint16_t)(w[i] & 0xffffu));
            y[2 * i + 1] = E::widen((uint16_t)(w[i] >> 16));
        }
    }
    __device__ __forceinline__ void narrow(const float (&y)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = E::two_bits(y[2 * i], y[2 * i + 1]);
        x = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Written once, past the lines of the L2 that are still to be read: 8192 rows of
    // 40 heads, rotation 35.9 -> 29.6 us, with a norm 39.9 -> 33.4, ragged into pages
    // 59.2 -> 53.4 (loads that pass it too: 32.2, 35.0, 52.9)
    __device__ __forceinline__ void store(uint16_t *p) const {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        __builtin_nontemporal_store(u32x4{x.x, x.y, x.z, x.w}, reinterpret_cast<u32x4 *>(p));
    }
};
template <>
struct Raw<F32> {
    f32x4 x, z;
    __device__ __forceinline__ void load(const float *p) {
        x = *reinterpret_cast<const f32x4 *>(p);
        z = *reinterpret_cast<const f32x4 *>(p + 4);
    }
    __device__ __forceinline__ void widen(float (&y)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[i], y[4 + i] = z[i];
    }
    __device__ __forceinline__ void narrow(const float (&y)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = y[i], z[i] = y[4 + i];
    }
    __device__ __forceinline__ void store(float *p) const {
        __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(p));
        __builtin_nontemporal_store(z, reinterpret_cast<f32x4 *>(p + 4));
    }
    __device__ __forceinline__ void put(float *p) const {         // to LDS
        *reinterpret_cast<f32x4 *>(p) = x;
        *reinterpret_cast<f32x4 *>(p + 4) = z;
    }
};

template <int kControl>
__device__ __forceinline__ float lane_move(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), kControl,
                                                              0xf, 0xf, true));
}

// the sum over the 1 << log lanes of a head, in each of them
__device__ __forceinline__ float head_sum(float s, int log) {
    if (log > 0) s += lane_move<0xb1>(s);        // neighbour
    if (log > 1) s += lane_move<0x4e>(s);        // the other two of four
    if (log > 2) s += lane_move<0x141>(s);       // eight, mirrored
    if (log > 3) s += lane_move<0x140>(s);       // sixteen, mirrored
    return s;
}

__device__ __forceinline__ void turn8(float (&x)[8], float (&y)[8], const float2 (&cs)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = x[i], b = y[i];
        x[i] = fmaf(a, cs[i].x, -(b * cs[i].y));
        y[i] = fmaf(b, cs[i].x, a * cs[i].y);
    }
}

__device__ __forceinline__ void turn4(float (&x)[8], const float2 *cs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = fmaf(a, cs[i].x, -(b * cs[i].y));
        x[2 * i + 1] = fmaf(b, cs[i].x, a * cs[i].y);
    }
}

// 8 weights, the offset added
template <typename E>
__device__ __forceinline__ void weigh(const HeadsArgs &g, const void *w, int64_t at,
                                      float (&y)[8]) {
    if (g.wide_weight) {
        Raw<F32> r;
        r.load(static_cast<const float *>(w) + at);
        r.widen(y);
    } else {
        Raw<E> r;
        r.load(static_cast<const typename E::type *>(w) + at);
        r.widen(y);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += g.offset;
}

// The lane's two pieces of a head.  Lanes past its end repeat its last piece and
// lanes past the last head that head: they load, compute and store the same
// bytes as another lane of their wave does, so that no access hides behind a
// branch and the loads ahead stay in flight.  `own`: whether a piece counts in
// the head's sum.
struct Place {
    int at[2];
    bool own[2], turns[2];
};

template <Mode kMode>
__device__ __forceinline__ Place place_of(const HeadsArgs &g, int lane, int need) {
    Place p;
    const int c = min(lane, need - 1);
    if (kMode == kSplit) {
        const int rest = c - (g.rot >> 4);
        p.at[0] = rest < 0 ? 8 * c : g.rot + 16 * rest;
        p.at[1] = p.at[0] + (rest < 0 ? g.rot >> 1 : 8);
        p.turns[0] = p.turns[1] = rest < 0;
    } else {
        p.at[0] = 8 * c, p.at[1] = 8 * (c + need);
        p.turns[0] = p.at[0] < g.rot, p.turns[1] = p.at[1] < g.rot;
    }
    p.own[0] = lane < need, p.own[1] = lane < need && p.at[1] < g.d;
    if (p.at[1] >= g.d) p.at[1] = p.at[0], p.turns[1] = p.turns[0];
    return p;
}

// row's place in its request, and the cell of the cache that it goes to
struct Row {
    bool mine, lost;     // a request has it; the request is not served
    int64_t place;
    size_t cell;
};

struct Cursor {
    Request q;
    int r, known;
};

__device__ __forceinline__ Row find_row(const AppendArgs &a, int row, Cursor &c) {
    Row x = {};
    int t = 0, len = 1;
    if (a.cu) {
        if (row < a.cu[0] || row >= a.cu[a.m]) return x;
        c.r = find_request(a, c.r, row);
        t = row - a.cu[c.r], len = a.cu[c.r + 1] - a.cu[c.r];
    } else {
        c.r = row;
    }
    if (c.r != c.known) c.q = request(a, c.r, len), c.known = c.r;
    x.mine = true;
    x.lost = c.q.fault || c.q.at < 0;
    const int place = c.q.at + t;
    if (!x.lost) {
        const int p = a.table[(size_t)c.q.row * a.width + (place >> a.page_log)];
        x.cell = (size_t)p * a.page_stride + (size_t)(place & ((1 << a.page_log) - 1)) * a.h.d;
    }
    x.place = a.h.pos ? a.h.pos[row] : place;
    return x;
}

template <typename E, bool kAppend, Mode kMode, bool kNorm>
__global__ __launch_bounds__(kThreads) void pieces_kernel(Pieces n) {
    typedef typename E::type T;
    __shared__ float2 s_turn[kWaves][GDN_MAX_HEAD_DIM / 2];
    __shared__ float s_weight[kNorm ? 2 : 1][kNorm ? GDN_MAX_HEAD_DIM : 1];
    // a wave's heads: 64 lanes of 16 elements
    __shared__ __attribute__((aligned(16))) float s_head[kWaves][kMode == kMixed ? 64 * 16 : 4];
    const AppendArgs &a = n.a;
    const HeadsArgs &g = a.h;
    const int l = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);      // the same in all lanes
    if (kAppend) {
        const bool bad = a.cu && rows_bad(a);
        const int r = ((int)blockIdx.x - n.tiles * n.splits) * kWaves + w;
        if ((int)blockIdx.x >= n.tiles * n.splits) {
            if (r >= a.m) return;
            const int fault = bad ? kFaultBadLength
                                  : request(a, r, a.cu ? a.cu[r + 1] - a.cu[r] : 1).fault;
            if (l == 0) a.status[r] = fault;
            return;
        }
        if (bad) return;
    }
    const Place pl = place_of<kMode>(g, l & ((1 << n.log) - 1), n.need);
    const int mine = l >> n.log, per = 64 >> n.log;      // the lane's head of a group's
    const int tile = (int)blockIdx.x / n.splits, split = (int)blockIdx.x % n.splits;
    const int keys = n.part[1].before, values = n.part[2].before;

    auto head = [&](const Part &p, int group) {
        return min((group - p.before) * per + mine, p.heads - 1);
    };
    // where there is no such group, 16 bytes of the last one: one line for the wave
    auto load = [&](int row, int group, Raw<E> (&raw)[2]) {
        const bool more = group < n.groups;
        group = min(group, n.groups - 1);
        const Part &p = n.part[group < keys ? 0 : group < values ? 1 : 2];
        const T *x = static_cast<const T *>(p.in) + row * p.in_row;
        const int64_t at = more ? head(p, group) * p.in_head + pl.at[0] : 0;
        raw[0].load(x + at);
        raw[1].load(x + at + (more ? pl.at[1] - pl.at[0] : 0));
    };
    auto store = [&](void *base, int64_t at, const Raw<E> (&raw)[2]) {
        T *x = static_cast<T *>(base) + at;
        raw[0].store(x + pl.at[0]);
        raw[1].store(x + pl.at[1]);
    };
    auto position = [&](int row) {
        if (g.rot == 0) return (int64_t)0;
        return (int64_t)g.pos[row] + (g.base ? g.base[row / g.base_rows] : 0);
    };

    int row = tile * n.rows * kWaves + w;
    Raw<E> next[2];
    Row x = {true, false, 0, 0};
    if (row < g.rows) {
        load(row, split, next);
        if (!kAppend) x.place = position(row);
    }
    if (kNorm) {
        // weights that the heads share, the offset added; ones where there are none
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Part &p = n.part[i];
            for (int j = threadIdx.x; j < g.d; j += kThreads)
                s_weight[i][j] = p.weight ? g.offset + weight_at<E>(p.weight, g.wide_weight, j) : 1.f;
        }
        __syncthreads();
    }
    Cursor c = {{}, 0, -1};
    for (int j = 0; j < n.rows && row < g.rows; ++j, row += kWaves) {
        if (j > 0) load(row, split, next);
        if (kAppend) x = find_row(a, row, c);
        else if (j > 0) x.place = position(row);
        if (!x.mine) continue;
        int group = split;
        if (kAppend && x.lost) {       // the rows of a request that is not served: NaN
            Raw<E> nan[2];
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __builtin_nanf("");
            nan[0].narrow(y), nan[1].narrow(y);
            for (; group < values; group += n.splits) {
                const Part &p = n.part[group < keys ? 0 : 1];
                if (p.out) store(p.out, row * p.out_row + head(p, group) * p.out_head, nan);
            }
            continue;
        }
        float2 cs[kMode == kMixed ? 16 : 8] = {};
        const int half = g.rot >> 1;
        const bool adjacent = g.layout == GDN_ROPE_INTERLEAVED;
        if (g.rot > 0) {
            for (int i = l; i < half; i += 64) s_turn[w][i] = turn(x.place, g.inv_freq[i], g.scale);
            exchange();
            if (kMode == kMixed) {               // (cos, the sine with the other's sign)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = pl.at[e] + i;
                        if (at >= g.rot) continue;
                        const float2 t = s_turn[w][adjacent ? at >> 1 : at < half ? at : at - half];
                        const bool first = adjacent ? at % 2 == 0 : at < half;
                        cs[8 * e + i] = make_float2(t.x, first ? -t.y : t.y);
                    }
            } else if (kMode == kSplit) {
                if (pl.turns[0])
#pragma unroll
                    for (int i = 0; i < 8; ++i) cs[i] = s_turn[w][pl.at[0] + i];
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (pl.turns[e])
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            cs[4 * e + i] = s_turn[w][pl.at[e] / 2 + i];
            }
            __builtin_amdgcn_wave_barrier();
        }
        for (; group < values; group += n.splits) {
            const Part &p = n.part[group < keys ? 0 : 1];
            const int h = head(p, group);
            float by[2][8];
            if (kNorm && p.weight_head != 0) {
                weigh<E>(g, p.weight, h * p.weight_head + pl.at[0], by[0]);
                weigh<E>(g, p.weight, h * p.weight_head + pl.at[1], by[1]);
            }
            const Raw<E> raw[2] = {next[0], next[1]};
            load(row, group + n.splits, next);
            float y[2][8];
            raw[0].widen(y[0]);
            raw[1].widen(y[1]);
            if (kNorm) {
                if (p.weight_head == 0)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            by[e][i] = s_weight[group < keys ? 0 : 1][pl.at[e] + i];
                float s = 0.f, z = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(y[0][i], y[0][i], s);
#pragma unroll
                for (int i = 0; i < 8; ++i) z = fmaf(y[1][i], y[1][i], z);
                s = (pl.own[0] ? s : 0.f) + (pl.own[1] ? z : 0.f);
                const float inv = inverse_norm(g, head_sum(s, n.log));
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[e][i] *= inv * by[e][i];
            }
            if constexpr (kMode == kSplit) {
                if (pl.turns[0]) turn8(y[0], y[1], cs);
            } else if constexpr (kMode == kAdjacent) {
                if (pl.turns[0]) turn4(y[0], &cs[0]);
                if (pl.turns[1]) turn4(y[1], &cs[4]);
            } else {
                float *mate = &s_head[w][mine * g.d];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (pl.turns[e]) {
                        Raw<F32> r;
                        r.narrow(y[e]);
                        r.put(mate + pl.at[e]);
                    }
                exchange();
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = pl.at[e] + i;
                        if (at >= g.rot) continue;
                        const float other =
                            mate[adjacent ? at ^ 1 : at < half ? at + half : at - half];
                        y[e][i] = fmaf(y[e][i], cs[8 * e + i].x, other * cs[8 * e + i].y);
                    }
                exchange();
            }
            Raw<E> done[2];
            done[0].narrow(y[0]);
            done[1].narrow(y[1]);
            if (p.out) store(p.out, row * p.out_row + h * p.out_head, done);
            if (kAppend && group >= keys)
                store(p.page, x.cell + ((size_t)h << a.page_log) * g.d, done);
        }
        if (kAppend)
            for (; group < n.groups; group += n.splits) {
                const Raw<E> raw[2] = {next[0], next[1]};
                load(row, group + n.splits, next);
                const Part &p = n.part[2];
                store(p.page, x.cell + ((size_t)head(p, group) << a.page_log) * g.d, raw);
            }
    }
}

// whether rows, heads and weights are in 16-byte pieces.  8192 rows of 40 heads
// with a norm: 33 us (d 80, rot 20; 96, 24) in pieces, 133 and 156 without.
bool in_pieces(const HeadsArgs &a) {
    const int step = a.dtype == GDN_DTYPE_F32 ? 4 : 8;
    if (a.d % 8 != 0) return false;
    for (const HeadsPart *x : {&a.q, &a.k}) {
        if (x->heads == 0) continue;
        if (((uintptr_t)x->in | (uintptr_t)x->out | (uintptr_t)x->weight) % 16 != 0) return false;
        if ((x->in_row | x->in_head) % step != 0) return false;
        if (x->out && (x->out_row | x->out_head) % step != 0) return false;
    }
    return true;
}

bool in_pieces(const AppendArgs &a) {
    const int step = a.h.dtype == GDN_DTYPE_F32 ? 4 : 8;
    return in_pieces(a.h) && (uintptr_t)a.v % 16 == 0 && (a.v_row | a.v_head) % step == 0;
}

// Rows of a wave of kv_append.  Every wave checks its requests' pages, and its
// workgroup all of cu, before it writes: a row each is best where that is little
// (131072 rows of 48 heads of 128, 64 requests: 596 us, with eight rows 682), and
// eight rows where it is more than a row's own bytes (one request in pages of 16:
// 1235 and 778 us; 4096 requests: 923 and 702 us), as far as the chip stays full.
int append_rows(const AppendArgs &a) {
    const int64_t checks = ((int64_t)a.width + (a.cu ? 2 * a.m : 0)) / 1024;
    const int64_t most = a.h.rows / 4096;
    const int64_t rows = checks < most ? checks : most;
    return rows < 1 ? 1 : rows > 16 ? 16 : (int)rows;
}

template <typename E, bool kAppend>
void launch_pieces(const AppendArgs &a, hipStream_t s) {
    const HeadsArgs &g = a.h;
    Pieces n{};
    const Mode mode = g.layout == GDN_ROPE_HALF ? g.rot % 16 == 0 ? kSplit : kMixed
                      : g.rot % 8 == 0          ? kAdjacent
                                                : kMixed;
    n.need = mode == kSplit ? g.rot / 16 + (g.d - g.rot + 15) / 16 : (g.d + 15) / 16;
    while (1 << n.log < n.need) ++n.log;
    n.a = a;
    const HeadsPart v{a.v, a.v_row, a.v_head, nullptr, 0, 0, nullptr, 0, kAppend ? g.k.heads : 0};
    void *const page[3] = {nullptr, a.kc, a.vc};
    const HeadsPart *const from[3] = {&g.q, &g.k, &v};
    for (int i = 0; i < 3; ++i) {
        const HeadsPart &x = *from[i];
        n.part[i] = {x.in, x.in_row, x.in_head, x.out, x.out_row, x.out_head, x.weight,
                     x.weight_head, page[i], x.heads, n.groups};
        n.groups += (x.heads + (64 >> n.log) - 1) / (64 >> n.log);
    }
    n.splits = heads_splits(g.rows, n.groups);
    n.rows = kAppend ? append_rows(a) : 1;
    n.tiles = (g.rows + kWaves * n.rows - 1) / (kWaves * n.rows);
    const int report = kAppend && a.status ? (a.m + kWaves - 1) / kWaves : 0;
    const int blocks = n.tiles * n.splits + report;
    if (blocks == 0) return;
    const dim3 grid((unsigned)blocks), block(kThreads);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, n); };
    if (g.norm != GDN_NORM_NONE) {
        if (mode == kSplit) go(pieces_kernel<E, kAppend, kSplit, true>);
        else if (mode == kAdjacent) go(pieces_kernel<E, kAppend, kAdjacent, true>);
        else go(pieces_kernel<E, kAppend, kMixed, true>);
    } else {
        if (mode == kSplit) go(pieces_kernel<E, kAppend, kSplit, false>);
        else if (mode == kAdjacent) go(pieces_kernel<E, kAppend, kAdjacent, false>);
        else go(pieces_kernel<E, kAppend, kMixed, false>);
    }
}

template <typename E>
void launch_heads(const HeadsArgs &a, hipStream_t s) {
    if (in_pieces(a)) {
        AppendArgs x{};
        x.h = a;
        return launch_pieces<E, false>(x, s);
    }
    const int splits = heads_splits(a.rows, a.q.heads + a.k.heads);
    const int64_t units = (int64_t)a.rows * splits;
    hipLaunchKernelGGL((heads_kernel<E>), dim3((unsigned)((units + kWaves - 1) / kWaves)),
                       dim3(kThreads), 0, s, a, splits);
}

template <typename E>
void launch_append(const AppendArgs &a, hipStream_t s) {
    if (in_pieces(a)) return launch_pieces<E, true>(a, s);
    const int splits = heads_splits(a.h.rows, a.h.q.heads + 2 * a.h.k.heads);
    const int64_t units = (int64_t)a.h.rows * splits;
    const int blocks = (int)((units + kWaves - 1) / kWaves);
    const int report = a.status ? (a.m + kWaves - 1) / kWaves : 0;
    if (blocks + report > 0)
        hipLaunchKernelGGL((append_kernel<E>), dim3((unsigned)(blocks + report)), dim3(kThreads), 0,
                           s, a, splits, blocks);
}

}  // namespace

hipError_t launch_heads(const HeadsArgs &a, hipStream_t s) {
    if (a.dtype == GDN_DTYPE_BF16) launch_heads<Bf16>(a, s);
    else if (a.dtype == GDN_DTYPE_F16) launch_heads<F16>(a, s);
    else launch_heads<F32>(a, s);
    return hipGetLastError();
}

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t s) {
    if (a.h.dtype == GDN_DTYPE_BF16) launch_append<Bf16>(a, s);
    else if (a.h.dtype == GDN_DTYPE_F16) launch_append<F16>(a, s);
    else launch_append<F32>(a, s);
    return hipGetLastError();
}

}  // namespace gdn
