// What the kernels over heads of queries and keys share: element types, the
// angle of a position, the request that a row of a ragged batch belongs to.
#pragma once

#include "device_common.hpp"
#include "serving.hpp"

namespace gdn {
namespace heads {

// Element types.  Products, sums and norms are fp32; a result is rounded once,
// to the nearest.
struct Bf16 {
    typedef uint16_t type;
    static __device__ __forceinline__ float widen(uint16_t x) { return to_f32(x); }
    static __device__ __forceinline__ uint16_t bits(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    }
    static __device__ __forceinline__ uint32_t two_bits(float x, float y) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t,
                                  bf16x2{static_cast<__bf16>(x), static_cast<__bf16>(y)});
    }
};
struct F16 {
    typedef uint16_t type;
    static __device__ __forceinline__ float widen(uint16_t x) {
        return static_cast<float>(__builtin_bit_cast(_Float16, x));
    }
    static __device__ __forceinline__ uint16_t bits(float x) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
    }
    static __device__ __forceinline__ uint32_t two_bits(float x, float y) {
        return bits(x) | (uint32_t)bits(y) << 16;
    }
};
struct F32 {
    typedef float type;
    static __device__ __forceinline__ float widen(float x) { return x; }
    static __device__ __forceinline__ float bits(float x) { return x; }
};

// element i of a norm's weights, in the heads' own type or in fp32
template <typename E>
__device__ __forceinline__ float weight_at(const void *w, bool wide, int64_t i) {
    if (wide) return static_cast<const float *>(w)[i];
    return E::widen(static_cast<const typename E::type *>(w)[i]);
}

// cos and sin, times the scale, of position p at frequency f (radians a
// position).  The product p f is held in two parts and so is 1 / (2 pi): the
// turns are exact to 2^-50 after whole ones are taken off, and an angle's error
// is its rounding to fp32 alone, 2^-25 of half a turn at any position (in one
// part each: 2^-24.1 at 2^29, 2^-21.8 at 2^32).
__device__ __forceinline__ float2 turn(int64_t p, float f, float scale) {
    const double high = 0x1.45f306dc9c883p-3, low = -0x1.6b01ec5417056p-57;
    const double x = (double)p, y = (double)f, product = x * y, rest = fma(x, y, -product);
    double t = fma(product, high, -rint(product * high));
    t = fma(rest, high, fma(product, low, t));
    float s, c;
    sincospif((float)(2.0 * t), &s, &c);
    return make_float2(c * scale, s * scale);
}

// what a lane of the wave has written to LDS before is there for the others
__device__ __forceinline__ void exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

// 1 / the norm of a head whose squares sum to s
__device__ __forceinline__ float inverse_norm(const HeadsArgs &a, float s) {
    return rsqrtf((a.norm == GDN_NORM_RMS ? s / (float)a.d : s) + a.eps);
}

// ---- ragged batches of kv_append

struct Request {
    int row, at, len;     // its row of the table, its first token's place, its tokens
    int fault;
};

// request r with its len tokens, checked by a whole wave: slot, length, and
// every page that its tokens go to
__device__ __forceinline__ Request request(const AppendArgs &a, int r, int len) {
    Request q;
    q.row = a.dst[r], q.at = a.begin[r], q.len = len;
    q.fault = 0;
    if (q.row < 0 || q.row >= a.seqs) q.fault = kFaultBadSlot;
    else if (q.at < -1 || (q.at >= 0 && (long long)q.at + len > (long long)a.width << a.page_log))
        q.fault = kFaultBadLength;
    else if (q.at >= 0 && len > 0) {
        const int32_t *row = a.table + (size_t)q.row * a.width;
        const int last = (q.at + len - 1) >> a.page_log;
        bool bad = false;
        for (int c = (q.at >> a.page_log) + (int)(threadIdx.x & 63); c <= last; c += 64) {
            const int p = row[c];
            bad |= p < 0 || p >= a.pool;
        }
        if (__any(bad)) q.fault = kFaultBadPage;
    }
    return q;
}

// whether cu does not ascend within [0, rows]; the whole workgroup
__device__ __forceinline__ bool rows_bad(const AppendArgs &a) {
    bool bad = false;
    for (int i = threadIdx.x; i < a.m; i += blockDim.x)
        bad |= a.cu[i] < 0 || a.cu[i + 1] < a.cu[i] || a.cu[i + 1] > a.h.rows;
    return __syncthreads_or(bad);
}

// the last request whose rows start at `row` or before, from request r on,
// found by a whole wave: 64 starts at a time (cu ascends)
__device__ __forceinline__ int find_request(const AppendArgs &a, int r, int row) {
    while (r + 1 < a.m) {
        const int i = r + 1 + (int)(threadIdx.x & 63);
        const int n = __popcll(__ballot(i < a.m && a.cu[i] <= row));
        r += n;
        if (n < 64) break;
    }
    return r;
}

}  // namespace heads
}  // namespace gdn
