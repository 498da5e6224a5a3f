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
// page: twice); 3 flops a rotated element and 4 a normed one.
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

template <typename E>
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
        angles<E>(a, (int64_t)a.pos[row] + (a.base ? a.base[row / a.base_rows] : 0), cs);
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
    if (g.rot > 0 && !lost) angles<E>(g, g.pos ? g.pos[row] : place, cs);
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

template <typename E>
void launch_heads(const HeadsArgs &a, hipStream_t s) {
    const int splits = heads_splits(a.rows, a.q.heads + a.k.heads);
    const int64_t units = (int64_t)a.rows * splits;
    hipLaunchKernelGGL((heads_kernel<E>), dim3((unsigned)((units + kWaves - 1) / kWaves)),
                       dim3(kThreads), 0, s, a, splits);
}

template <typename E>
void launch_append(const AppendArgs &a, hipStream_t s) {
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
