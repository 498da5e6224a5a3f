// One token of the gated delta rule for every sequence: the step of decoding.
//
// For one (sequence, head), with M = alpha S (S of shape d_k x d_v, fp32):
//     u = beta (v - M^T k),   S' = M + k u^T,   o = S'^T q = M^T q + (k . q) u,
// so both products with the old state are formed in one pass over it and the
// new state follows from registers: the state is read and written once.
//
// Bound: HBM.  A (sequence, head) moves 2 x 64 KiB of state against 0.4 MFLOP
// (d_k = d_v = 128).  One workgroup owns a 32-column tile of one state: its
// rows are 128-byte segments (whole cache lines), 16 KiB in flight per
// workgroup, and even one sequence of 32 heads gives 128 workgroups.  Thread
// (rg, cg) holds the kR rows from kR rg of four columns; the 32 row groups are summed by
// three lane exchanges and one pass through LDS.
#include "device_common.hpp"
#include "serving.hpp"
#include "rule_common.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;      // d_v columns of a workgroup
constexpr int kSums = 12;      // M^T k (4), M^T q (4), k . q (1) of a column group, padded

template <typename T, typename OT, int kR>
__global__ __launch_bounds__(kThreads) void rule_recurrent_kernel(RuleArgs a, int tiles) {
    __shared__ float red[kThreads / 64][8][kSums];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
    const int cg = tid & 7, rg = tid >> 3;
    const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int c0 = tile * kTile + 4 * cg, r0 = rg * kR;
    const bool live = c0 < a.dv && r0 < a.dk;

    const int src = a.src[b], dst = a.dst[b];
    const int fault = rule::slots_ok(a, src, dst) ? 0 : kFaultBadSlot;
    if (a.status && h == 0 && tile == 0 && tid == 0) a.status[b] = fault;
    OT *out = static_cast<OT *>(a.out) + ((size_t)b * a.H + h) * a.dv + c0;
    if (fault) {
        if (c0 < a.dv && rg == 0)
            for (int e = 0; e < 4; ++e) rule::put(&out[e], __builtin_nanf(""));
        return;
    }

    const size_t slab = (size_t)a.H * a.dk * a.dv;
    const size_t at = ((size_t)h * a.dk + r0) * a.dv + c0;
    float4 S[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && src >= 0)
            S[i] = *reinterpret_cast<const float4 *>(a.S + src * slab + at + (size_t)i * a.dv);
    }

    const T *q = static_cast<const T *>(a.q) + ((size_t)b * a.Hk + hk) * a.dk + r0;
    const T *k = static_cast<const T *>(a.k) + ((size_t)b * a.Hk + hk) * a.dk + r0;
    const T *v = static_cast<const T *>(a.v) + ((size_t)b * a.H + h) * a.dv + c0;
    float kr[kR], qr[kR], vv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        kr[i] = r0 < a.dk ? to_f32(k[i]) : 0.f;
        qr[i] = r0 < a.dk ? to_f32(q[i]) : 0.f;
    }
    if (c0 < a.dv)
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[e] = to_f32(v[e]);
    const float al = a.alpha[(size_t)b * a.H + h], be = a.beta[(size_t)b * a.H + h];

    float s[9] = {};
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        S[i].x *= al, S[i].y *= al, S[i].z *= al, S[i].w *= al;
        s[0] = fmaf(S[i].x, kr[i], s[0]), s[1] = fmaf(S[i].y, kr[i], s[1]);
        s[2] = fmaf(S[i].z, kr[i], s[2]), s[3] = fmaf(S[i].w, kr[i], s[3]);
        s[4] = fmaf(S[i].x, qr[i], s[4]), s[5] = fmaf(S[i].y, qr[i], s[5]);
        s[6] = fmaf(S[i].z, qr[i], s[6]), s[7] = fmaf(S[i].w, qr[i], s[7]);
        s[8] = fmaf(kr[i], qr[i], s[8]);
    }
#pragma unroll
    for (int x = 8; x < 64; x <<= 1)
#pragma unroll
        for (int j = 0; j < 9; ++j) s[j] += __shfl_xor(s[j], x);
    if (l < 8) {
#pragma unroll
        for (int j = 0; j < 9; ++j) red[w][l][j] = s[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 9; ++j)
        s[j] = (red[0][cg][j] + red[1][cg][j]) + (red[2][cg][j] + red[3][cg][j]);
    float u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = be * (vv[e] - s[e]);
    if (rg == 0 && c0 < a.dv)
#pragma unroll
        for (int e = 0; e < 4; ++e) rule::put(&out[e], fmaf(s[8], u[e], s[4 + e]));
    if (live)
#pragma unroll
        for (int i = 0; i < kR; ++i)
            *reinterpret_cast<float4 *>(a.S + dst * slab + at + (size_t)i * a.dv) =
                make_float4(fmaf(kr[i], u[0], S[i].x), fmaf(kr[i], u[1], S[i].y),
                            fmaf(kr[i], u[2], S[i].z), fmaf(kr[i], u[3], S[i].w));
}

template <typename T, typename OT>
void launch(const RuleArgs &a, hipStream_t s) {
    const int tiles = (a.dv + kTile - 1) / kTile;
    const dim3 grid((unsigned)a.batch * a.H * tiles);
    if (a.dk > 64)
        hipLaunchKernelGGL((rule_recurrent_kernel<T, OT, 4>), grid, dim3(kThreads), 0, s, a, tiles);
    else
        hipLaunchKernelGGL((rule_recurrent_kernel<T, OT, 2>), grid, dim3(kThreads), 0, s, a, tiles);
}

}  // namespace

hipError_t launch_step(const RuleArgs &a, hipStream_t s) {
    const bool half = a.dtype == GDN_DTYPE_BF16, ohalf = a.out_dtype == GDN_DTYPE_BF16;
    if (half && ohalf) launch<uint16_t, uint16_t>(a, s);
    if (half && !ohalf) launch<uint16_t, float>(a, s);
    if (!half && ohalf) launch<float, uint16_t>(a, s);
    if (!half && !ohalf) launch<float, float>(a, s);
    return hipGetLastError();
}

}  // namespace gdn
