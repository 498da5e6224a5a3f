// Prompt prefill of the gated delta rule in chunks of 64 tokens (gfx950).
//
// Inside a chunk, with S the state before it, g_i the running sum of
// log alpha and u_i the pseudo-values of S_i = alpha_i S_{i-1} + k_i u_i^T,
//     X_is = beta_i e^{g_i - g_s} k_i . k_s  (s < i),   T = (I + X)^{-1},
//     R = beta (V - e^g (K S)),     U = T R = R + (T - I) R,
//     O = e^g (Q S) + Y U,          Y_is = e^{g_i - g_s} q_i . k_s  (s <= i),
//     S <- e^{g_l} S + K^T W,       W_i = e^{g_l - g_i} u_i,
// so 64 tokens cost five matrix products instead of 64 passes over the state.
// T and Y depend on the chunk alone: one kernel forms them for all chunks at
// once, another carries the state through a sequence's chunks in order.
//
//   plan:  chunk slots of the sequences (prefix sums), sequences by length
//   chunk: a workgroup per (chunk, head): decays, Gram matrices, T, Y, and
//          the chunk's keys transposed, stored as matrix operands
//   scan:  a workgroup per (sequence, head, 16 columns of d_v): the columns
//          of S are independent, and 32 heads of d_v = 128 give the 256
//          workgroups that fill the chip with a single prompt.  Its four
//          waves split the rows of every product (16 tokens or 32 rows of
//          S each) and exchange S, R and U, W through LDS, three barriers a
//          chunk; the operands that do not depend on S come straight from
//          memory into registers, a chunk ahead.
//
// Operands.  A 16x16 result tile holds row 4 q + r, column m in register r of
// lane (m = l & 15, q = l >> 4); the matrix instruction takes 8 consecutive
// contraction indices from each lane.  Rows of S and tokens are therefore
// numbered so that the registers of the tiles 2 j and 2 j + 1 are the
// indices 32 j + 8 q + (0..7): tile i, row p is index
//     rho(i, p) = 32 (i / 2) + 8 (p / 4) + 4 (i % 2) + p % 4,
// and results feed the next product with no exchange inside the wave.
//
// Precision.  bf16 q, k are exact operands.  fp32 factors (S, R, U, W, T - I, Y)
// enter as three bf16 parts, x = hi + mid + lo exactly, and products of two of
// them keep the six part products down to 2^-16 (those left out are below
// 2^-23): the result is that of fp32 products.  Two parts were off by 2e-6 each (measured: 4.6e-6 in the
// output's 2-norm), more than fp32 sums are.  fp32 q, k take the fp32 matrix
// instruction.  g is summed in 64 bits: decays of late tokens are differences
// of large sums.
#include "mfma_tile.hpp"
#include "rule_common.hpp"

namespace gdn {
namespace {

using tile::bf16x8;
using tile::lds_barrier;

constexpr int kC = 64;             // tokens of a chunk
constexpr int kThreads = 256;
constexpr int kCols = 16;          // d_v columns of a scan workgroup
constexpr int kPlanThreads = 1024;
constexpr int kSortMax = 1024;     // sequences ordered by length up to this many
constexpr int kFrags = 6;          // operand pieces of a lower triangle: tiles 0, 1 need the
                                   // first 32 columns, tiles 2, 3 all 64

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int rho(int i, int p) {
    return 32 * (i >> 1) + 8 * (p >> 2) + 4 * (i & 1) + (p & 3);
}

__device__ __forceinline__ int frag_of(int i, int j) { return i < 2 ? i : 2 * i - 2 + j; }

// a lane's 8 elements of an operand: one bf16 part, three of them, or the
// two halves of 8 fp32 values
struct Raw8 {
    uint4 p[3];
};

// bf16 q, k: exact 8-element operands; fp32 factors in three parts
struct Half {
    static constexpr int kParts = 3;     // 16-byte pieces of an fp32 operand
    typedef uint16_t elem;
    static constexpr int kExact = 1;     // 16-byte pieces of an exact operand
    static __device__ __forceinline__ f32x4 mma(bf16x8 x, bf16x8 y, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
    }
    static __device__ __forceinline__ bf16x8 v(const uint4 &x) {
        return __builtin_bit_cast(bf16x8, x);
    }
    // exact . exact
    static __device__ __forceinline__ f32x4 gram(const Raw8 &x, const Raw8 &y, f32x4 c) {
        return mma(v(x.p[0]), v(y.p[0]), c);
    }
    // exact . fp32, two operands x at once: the instructions of one sum wait
    // for each other, those of the two alternate.  Smallest part first.
    static __device__ __forceinline__ void mul(const Raw8 &x0, const Raw8 &x1, const Raw8 &y,
                                               f32x4 &c0, f32x4 &c1) {
#pragma unroll
        for (int p = 2; p >= 0; --p) {
            c0 = mma(v(x0.p[0]), v(y.p[p]), c0);
            c1 = mma(v(x1.p[0]), v(y.p[p]), c1);
        }
    }
    // fp32 . fp32 into c + d: two sums that alternate
    static __device__ __forceinline__ void mul2(const Raw8 &x, const Raw8 &y, f32x4 &c, f32x4 &d) {
        d = mma(v(x.p[1]), v(y.p[1]), d);
        c = mma(v(x.p[2]), v(y.p[0]), c);
        d = mma(v(x.p[0]), v(y.p[2]), d);
        c = mma(v(x.p[1]), v(y.p[0]), c);
        d = mma(v(x.p[0]), v(y.p[1]), d);
        c = mma(v(x.p[0]), v(y.p[0]), c);
    }
    // by truncation: the upper halves of x, of what is left and of what is
    // left then are 8 bits each, 24 together, so the parts sum to x exactly
    static __device__ __forceinline__ void split(const float *x, uint2 *part) {
        float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(r[i]);
            part[p].x = __builtin_amdgcn_perm(u[1], u[0], 0x07060302u);
            part[p].y = __builtin_amdgcn_perm(u[3], u[2], 0x07060302u);
            if (p < 2)
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] -= __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    // registers of tile 2 j + s as half of pair j's operand
    static __device__ __forceinline__ void put_tile(uint4 (*buf)[kParts][64], int j, int s, int l,
                                                    const f32x4 &x) {
        const float f[4] = {x[0], x[1], x[2], x[3]};
        uint2 part[3];
        split(f, part);
#pragma unroll
        for (int p = 0; p < 3; ++p) reinterpret_cast<uint2 *>(&buf[j][p][l])[s] = part[p];
    }
    static __device__ __forceinline__ Raw8 from_f32(const float *x) {
        uint2 a[3], b[3];
        split(x, a);
        split(x + 4, b);
        Raw8 r;
#pragma unroll
        for (int p = 0; p < 3; ++p) r.p[p] = make_uint4(a[p].x, a[p].y, b[p].x, b[p].y);
        return r;
    }
    static __device__ __forceinline__ Raw8 load8(const elem *p, bool ok) {
        Raw8 x = {};
        if (ok) x.p[0] = *reinterpret_cast<const uint4 *>(p);
        return x;
    }
    static __device__ __forceinline__ Raw8 load8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        Raw8 x;
        x.p[0] = tile::load16<0>(r, off);
        return x;
    }
    static __device__ __forceinline__ uint32_t load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
    }
    static __device__ __forceinline__ float widen(uint32_t x) { return __uint_as_float(x << 16); }
};

// fp32 q, k: the fp32 matrix instruction, eight per 32 indices
struct Full {
    typedef float elem;
    static constexpr int kParts = 2;
    static constexpr int kExact = 2;
    static __device__ __forceinline__ f32x4 gram(const Raw8 &x, const Raw8 &y, f32x4 c) {
        const uint32_t xs[8] = {x.p[0].x, x.p[0].y, x.p[0].z, x.p[0].w,
                                x.p[1].x, x.p[1].y, x.p[1].z, x.p[1].w};
        const uint32_t ys[8] = {y.p[0].x, y.p[0].y, y.p[0].z, y.p[0].w,
                                y.p[1].x, y.p[1].y, y.p[1].z, y.p[1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(xs[e]),
                                                     __uint_as_float(ys[e]), c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ void mul(const Raw8 &x0, const Raw8 &x1, const Raw8 &y,
                                               f32x4 &c0, f32x4 &c1) {
        c0 = gram(x0, y, c0);
        c1 = gram(x1, y, c1);
    }
    static __device__ __forceinline__ void mul2(const Raw8 &x, const Raw8 &y, f32x4 &c, f32x4 &) {
        c = gram(x, y, c);
    }
    static __device__ __forceinline__ void put_tile(uint4 (*buf)[kParts][64], int j, int s, int l,
                                                    const f32x4 &x) {
        buf[j][s][l] = __builtin_bit_cast(uint4, x);
    }
    static __device__ __forceinline__ Raw8 from_f32(const float *x) {
        return {{*reinterpret_cast<const uint4 *>(x), *reinterpret_cast<const uint4 *>(x + 4)}};
    }
    static __device__ __forceinline__ Raw8 load8(const elem *p, bool ok) {
        Raw8 x = {};
        if (ok) {
            x.p[0] = reinterpret_cast<const uint4 *>(p)[0];
            x.p[1] = reinterpret_cast<const uint4 *>(p)[1];
        }
        return x;
    }
    static __device__ __forceinline__ Raw8 load8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        Raw8 x;
        x.p[0] = tile::load16<0>(r, off);
        x.p[1] = tile::load16<0>(r, off + 16);
        return x;
    }
    static __device__ __forceinline__ uint32_t load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
    }
    static __device__ __forceinline__ float widen(uint32_t x) { return __uint_as_float(x); }
};

__device__ __forceinline__ void store1(__amdgpu_buffer_rsrc_t r, uint32_t off, float x, uint16_t) {
    __builtin_amdgcn_raw_buffer_store_b16(tile::bf16_bits(x), r, (int)off, 0, 0);
}
__device__ __forceinline__ void store1(__amdgpu_buffer_rsrc_t r, uint32_t off, float x, float) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, (int)off, 0, 0);
}

// an offset past the end of any buffer: loads give zero, stores do nothing
constexpr uint32_t kNowhere = 0x80000000u;

// one (chunk, head) of the workspace
template <typename M>
struct ChunkData {
    uint4 t[kFrags][M::kParts][64];      // T - I as operands
    uint4 y[kFrags][M::kParts][64];      // Y
    float4 vec[kC];              // beta, beta e^g, e^g, e^{g_l - g} of the tokens
};

struct Layout {
    int slots;                   // chunk slots
    int64_t off_pre, off_order, off_seq, off_kt, off_data, bytes;
};

// ---------------------------------------------------------------------------
// plan: pre[i] = first chunk slot of sequence i (-1: bad rows), seq[slot] its
// sequence (-1: unused slot), order = sequences, most chunks first
// ---------------------------------------------------------------------------
__device__ __forceinline__ int chunks_of(const RuleArgs &a, int i) {
    const rule::Sequence s = rule::sequence(a, i);
    return s.fault & kFaultBadLength ? -1 : (s.len + kC - 1) / kC;
}

__global__ __launch_bounds__(kPlanThreads) void prefill_plan_kernel(RuleArgs a, Layout y) {
    __shared__ int s_part[kPlanThreads / 64];
    __shared__ int s_n[kSortMax];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
    char *ws = static_cast<char *>(a.workspace);
    int *pre = reinterpret_cast<int *>(ws + y.off_pre);
    int *order = reinterpret_cast<int *>(ws + y.off_order);
    int *seq = reinterpret_cast<int *>(ws + y.off_seq);
    for (int s = tid; s < y.slots; s += kPlanThreads) seq[s] = -1;
    const bool sorted = a.batch <= kSortMax;
    long long sum = 0;
    for (int i0 = 0; i0 < a.batch; i0 += kPlanThreads) {
        const int i = i0 + tid;
        const int n = i < a.batch ? chunks_of(a, i) : 0;
        if (sorted && i < a.batch) s_n[i] = n;
        int inc = max(n, 0);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(inc, o);
            if (l >= o) inc += up;
        }
        __syncthreads();
        if (l == 63) s_part[w] = inc;
        __syncthreads();
        long long before = sum;
        for (int x = 0; x < kPlanThreads / 64; ++x) {
            if (x < w) before += s_part[x];
            sum += s_part[x];
        }
        const long long at = before + inc - max(n, 0);
        if (i < a.batch) {
            // ascending offsets need at most the slots there are; offsets
            // that overlap may not
            const bool ok = n >= 0 && at + n <= y.slots;
            pre[i] = ok ? (int)at : -1;
            if (ok)
                for (int c = 0; c < n; ++c) seq[at + c] = i;
            if (!sorted) order[i] = i;
        }
    }
    __syncthreads();
    if (sorted && tid < a.batch) {
        const int n = s_n[tid];
        int rank = 0;
        for (int j = 0; j < a.batch; ++j) rank += s_n[j] > n || (s_n[j] == n && j < tid);
        order[rank] = tid;
    }
}

// ---------------------------------------------------------------------------
// chunk: T, Y, decays, transposed keys
// ---------------------------------------------------------------------------
constexpr int kLd = kC + 4;      // LDS row stride of the 64-wide matrices (floats)

template <typename M, int DK>
__global__ __launch_bounds__(kThreads) void prefill_chunk_kernel(RuleArgs a, Layout y) {
    typedef typename M::elem T;
    constexpr int J = DK / 32;
    __shared__ float s_x[kC][kLd], s_t[kC][kLd], s_y[kC][kLd];
    __shared__ double s_g[kC];
    __shared__ float s_beta[kC];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const int m = l & 15, qd = l >> 4;
    char *ws = static_cast<char *>(a.workspace);
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int i = reinterpret_cast<const int *>(ws + y.off_seq)[slot];
    if (i < 0) return;
    const int rep = a.H / a.Hk, hk = h / rep;
    const int row0 = a.cu[i] + kC * (slot - reinterpret_cast<const int *>(ws + y.off_pre)[i]);
    const int n = min(kC, a.cu[i + 1] - row0);
    ChunkData<M> *out =
        reinterpret_cast<ChunkData<M> *>(ws + y.off_data) + (size_t)slot * a.H + h;

    // ---- decays; a token past the end has alpha 1 and beta 0
    if (w == 0) {
        float lg = 0.f, be = 0.f;
        if (l < n) {
            const size_t at = ((size_t)row0 + l) * a.H + h;
            // alpha = 0: far enough below any exponent to clear the state,
            // small enough to keep the other tokens' logarithms exact
            lg = fmaxf(log2f(a.alpha[at]), -1e4f);
            be = a.beta[at];
        }
        double g = lg;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double up = __shfl_up(g, o);
            if (l >= o) g += up;
        }
        const double last = __shfl(g, 63);
        s_g[l] = g;
        s_beta[l] = be;
        const float eg = exp2f((float)g);
        out->vec[l] = make_float4(be, be * eg, eg, exp2f((float)(last - g)));
    }

    const T *kp = static_cast<const T *>(a.k) + ((size_t)row0 * a.Hk + hk) * a.dk;
    const T *qp = static_cast<const T *>(a.q) + ((size_t)row0 * a.Hk + hk) * a.dk;
    const size_t stride = (size_t)a.Hk * a.dk;
    auto rows8 = [&](const T *p, int t, int j) {
        const int d0 = 32 * j + 8 * qd;
        return M::load8(p + t * stride + d0, t < n && d0 < a.dk);
    };
    Raw8 ka[J], qa[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        ka[j] = rows8(kp, 16 * w + m, j);
        qa[j] = rows8(qp, 16 * w + m, j);
    }
    __syncthreads();

    // ---- tiles (w, jb) of X and Y: rows 16 w + 4 qd + r, column 16 jb + m
    for (int jb = 0; jb <= w; ++jb) {
        f32x4 kk = {}, qk = {};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const Raw8 kb = rows8(kp, 16 * jb + m, j);
            kk = M::gram(ka[j], kb, kk);
            qk = M::gram(qa[j], kb, qk);
        }
        const int s = 16 * jb + m;
        const double gs = s_g[s];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * w + 4 * qd + r;
            const float e = exp2f((float)(s_g[t] - gs));
            s_x[t][s] = s < t ? s_beta[t] * e * kk[r] : 0.f;
            s_y[t][s] = s <= t ? e * qk[r] : 0.f;
        }
    }
    __syncthreads();

    // ---- T by blocks of 16: the diagonal block of wave w by substitution,
    // lane column m of it
    float t[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        float acc = r == m ? 1.f : 0.f;
#pragma unroll
        for (int s = 0; s < r; ++s) acc = fmaf(-s_x[16 * w + r][16 * w + s], t[s], acc);
        t[r] = acc;
    }
    f32x4 tb[4];                       // tiles (k, w) of T, by k - w
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float lo = qd & 1 ? t[4 + r] : t[r], hi = qd & 1 ? t[12 + r] : t[8 + r];
        tb[0][r] = qd & 2 ? hi : lo;
        s_t[16 * w + 4 * qd + r][16 * w + m] = tb[0][r];
    }
    __syncthreads();
    // below it, T_iw = -T_ii sum_k X_ik T_kw: fp32 products (contraction
    // index 4 qd + r of a block at step r)
    auto block = [&](const float(*x)[kLd], int bi, int bk, const f32x4 &b, f32x4 c) {
        const f32x4 av = *reinterpret_cast<const f32x4 *>(&x[16 * bi + m][16 * bk + 4 * qd]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(av[r], b[r], c, 0, 0, 0);
        return c;
    };
#pragma unroll
    for (int di = 1; di < 4; ++di) {
        const int bi = w + di;
        if (bi < 4) {
            f32x4 p = {};
#pragma unroll
            for (int dk = 0; dk < di; ++dk) p = block(s_x, bi, w + dk, tb[dk], p);
            const f32x4 z = block(s_t, bi, bi, p, f32x4{});
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                tb[di][r] = -z[r];
                s_t[16 * bi + 4 * qd + r][16 * w + m] = -z[r];
            }
        }
    }
    __syncthreads();

    // ---- out as operands: tile w's rows
    const int tr = rho(w, m);
    for (int j = 0; j <= w >> 1; ++j) {
        const int k0 = 32 * j + 8 * qd, f = frag_of(w, j);
        float tv[8], yv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            tv[e] = k0 + e < tr ? s_t[tr][k0 + e] : 0.f;
            yv[e] = k0 + e <= tr ? s_y[tr][k0 + e] : 0.f;
        }
        const Raw8 tx = M::from_f32(tv), yx = M::from_f32(yv);
#pragma unroll
        for (int p = 0; p < M::kParts; ++p) {
            out->t[f][p][l] = tx.p[p];
            out->y[f][p][l] = yx.p[p];
        }
    }
    // ---- the keys transposed, once per key head: tile i's rows are rows of
    // S, 8 consecutive tokens a lane
    if (h % rep == 0) {
        uint4 *kt = reinterpret_cast<uint4 *>(ws + y.off_kt) +
                    ((size_t)slot * a.Hk + hk) * (DK / 16) * 2 * M::kExact * 64;
        for (int f = w; f < (DK / 16) * 2; f += 4) {
            const int ti = f >> 1, jt = f & 1, d = rho(ti, m);
            alignas(16) T x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int tok = 32 * jt + 8 * qd + e;
                x[e] = tok < n && d < a.dk ? kp[tok * stride + d] : T(0);
            }
#pragma unroll
            for (int p = 0; p < M::kExact; ++p)
                kt[(f * M::kExact + p) * 64 + l] = reinterpret_cast<const uint4 *>(x)[p];
        }
    }
}

// ---------------------------------------------------------------------------
// scan: the state through a sequence's chunks
// ---------------------------------------------------------------------------
template <typename M, int DK, typename OT, int G>
__global__ __launch_bounds__(kThreads, 2) void prefill_scan_kernel(RuleArgs a, Layout y,
                                                                   int tiles) {
    typedef typename M::elem T;
    constexpr int J = DK / 32;
    constexpr int N = M::kParts;
    __shared__ uint4 s_s[G][J][N][64], s_r[G][2][N][64], s_u[G][2][N][64], s_w[G][2][N][64];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const int m = l & 15, qd = l >> 4;
    char *ws = static_cast<char *>(a.workspace);
    // the column tiles of a (sequence, head) read the same chunk data: they
    // go to one XCD (block index modulo 8)
    const int units = a.batch * a.H;
    const int full = units / 8 * 8 * tiles, x = blockIdx.x;
    int u, ct;
    if (x < full) {
        u = x / (8 * tiles) * 8 + x % 8;
        ct = x / 8 % tiles;
    } else {
        u = units / 8 * 8 + (x - full) / tiles;
        ct = (x - full) % tiles;
    }
    const int i = reinterpret_cast<const int *>(ws + y.off_order)[u / a.H], h = u % a.H;
    const int hk = h / (a.H / a.Hk);
    const int col0 = kCols * G * ct + m;              // and kCols further on for each group
    const int pre = reinterpret_cast<const int *>(ws + y.off_pre)[i];
    rule::Sequence sq = rule::sequence(a, i);
    if (pre < 0) sq.fault = kFaultBadLength;
    if (a.status && h == 0 && ct == 0 && tid == 0) a.status[i] = sq.fault;
    const size_t ostride = (size_t)a.H * a.dv;
    if (sq.fault) {
        OT *out = static_cast<OT *>(a.out) + (size_t)h * a.dv + col0;
        if (!(sq.fault & kFaultBadLength))
            for (int t = tid >> 4; t < sq.len; t += kThreads / 16)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    if (col0 + kCols * g < a.dv)
                        rule::put(&out[((size_t)sq.first + t) * ostride + kCols * g],
                                  __builtin_nanf(""));
        return;
    }

    // ---- rows rho(2 w, .) and rho(2 w + 1, .) of the state's columns
    const size_t slab = (size_t)a.H * a.dk * a.dv;
    const size_t sat = (size_t)h * a.dk * a.dv + col0;
    const int sr = 32 * w + 8 * qd;                 // the lane's eight rows
    const bool slive = w < J && sr < a.dk;
    f32x4 st[G][2] = {};
    if (slive && sq.src >= 0) {
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (col0 + kCols * g < a.dv)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    st[g][e >> 2][e & 3] =
                        a.S[sq.src * slab + sat + (size_t)(sr + e) * a.dv + kCols * g];
    }
    auto put_state = [&]() {
        if (w < J)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                M::put_tile(s_s[g], w, 0, l, st[g][0]);
                M::put_tile(s_s[g], w, 1, l, st[g][1]);
            }
    };
    put_state();

    const T *kp = static_cast<const T *>(a.k) + ((size_t)sq.first * a.Hk + hk) * a.dk;
    const T *qp = static_cast<const T *>(a.q) + ((size_t)sq.first * a.Hk + hk) * a.dk;
    const T *vp = static_cast<const T *>(a.v) + (size_t)sq.first * ostride + (size_t)h * a.dv;
    const OT *op = static_cast<const OT *>(a.out) + (size_t)sq.first * ostride + (size_t)h * a.dv;
    const size_t kstride = (size_t)a.Hk * a.dk;
    const ChunkData<M> *data =
        reinterpret_cast<const ChunkData<M> *>(ws + y.off_data) + (size_t)pre * a.H + h;
    const size_t ktsize = (size_t)(DK / 16) * 2 * M::kExact * 64;
    const uint4 *ktp =
        reinterpret_cast<const uint4 *>(ws + y.off_kt) + ((size_t)pre * a.Hk + hk) * ktsize;

    const int tok = rho(w, m);                      // this lane's row of K, Q
    const int tok4 = 32 * (w >> 1) + 8 * qd + 4 * (w & 1);   // its four tokens of R, U, O
    // rows of a chunk are addressed from its first: 32-bit offsets, and what
    // lies past the chunk's tokens reads as zero with no branch, so that a
    // load is waited for where it is used
    uint32_t koff[J], voff[G];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int d0 = 32 * j + 8 * qd;
        koff[j] = d0 < a.dk ? (uint32_t)((tok * kstride + d0) * sizeof(T)) : kNowhere;
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
        voff[g] = col0 + kCols * g < a.dv ? (uint32_t)(tok4 * ostride + col0 + kCols * g) : kNowhere;
    auto tokens = [&](int c) { return min(kC, sq.len - kC * c); };
    auto rsrc = [&](const void *p, size_t row, size_t width, size_t size, int c) {
        return tile::make_rsrc(static_cast<const char *>(p) + (size_t)kC * c * row * size,
                               (uint32_t)(((tokens(c) - 1) * row + width) * size));
    };
    // an element offset of kNowhere stays past the end in bytes
    auto bytes = [&](uint32_t off, int r, uint32_t size) {
        return off == kNowhere ? kNowhere : (off + (uint32_t)(r * ostride)) * size;
    };
    Raw8 kf[J], qf[J], tf[2], yf[2], kt[2][2];
    float4 vec[4];
    uint32_t vv[G][4];
    float egl = 0.f;
    auto load_kq = [&](int c) {
        const __amdgpu_buffer_rsrc_t rk = rsrc(kp, kstride, a.dk, sizeof(T), c);
        const __amdgpu_buffer_rsrc_t rq = rsrc(qp, kstride, a.dk, sizeof(T), c);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            kf[j] = M::load8(rk, koff[j]);
            qf[j] = M::load8(rq, koff[j]);
        }
    };
    auto load_tv = [&](int c) {
        const ChunkData<M> *p = data + (size_t)c * a.H;
        const __amdgpu_buffer_rsrc_t rv = rsrc(vp, ostride, a.dv, sizeof(T), c);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int g = 0; g < G; ++g) vv[g][r] = M::load1(rv, bytes(voff[g], r, sizeof(T)));
            vec[r] = p->vec[tok4 + r];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (j <= w >> 1) {
                const int f = frag_of(w, j);
#pragma unroll
                for (int n = 0; n < N; ++n) tf[j].p[n] = p->t[f][n][l];
            }
    };
    auto load_yk = [&](int c) {
        const ChunkData<M> *p = data + (size_t)c * a.H;
        egl = p->vec[kC - 1].z;
        if (w < J) {
            const uint4 *q = ktp + (size_t)c * a.Hk * ktsize;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int jt = 0; jt < 2; ++jt) {
                    const int f = ((2 * w + s) * 2 + jt) * M::kExact;
#pragma unroll
                    for (int n = 0; n < M::kExact; ++n) kt[s][jt].p[n] = q[(f + n) * 64 + l];
                }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (j <= w >> 1) {
                const int f = frag_of(w, j);
#pragma unroll
                for (int n = 0; n < N; ++n) yf[j].p[n] = p->y[f][n][l];
            }
    };
    auto read = [&](uint4(*buf)[N][64], int j) {
        Raw8 b;
#pragma unroll
        for (int n = 0; n < N; ++n)
            b.p[n] = buf[j][n][l];
        return b;
    };

    // Each phase first reads the operands that the barrier before it made
    // good, then issues the loads whose registers the last phase set free (a
    // chunk ahead of their use, a third of them in each phase), then
    // multiplies.
    const int chunks = (sq.len + kC - 1) / kC;
    if (chunks > 0) {
        load_kq(0);
        load_tv(0);
    }
    lds_barrier();
    for (int c = 0; c < chunks; ++c) {
        const int next = min(c + 1, chunks - 1);
        // ---- R of 16 tokens (and Q S)
        f32x4 ks[G] = {}, qs[G] = {}, uu[G];
        float wl[4];
        load_yk(c);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const Raw8 b = read(s_s[g], j);
                M::mul(kf[j], qf[j], b, ks[g], qs[g]);
            }
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                uu[g][r] = vec[r].x * M::widen(vv[g][r]) - vec[r].y * ks[g][r];
                qs[g][r] *= vec[r].z;
            }
            M::put_tile(s_r[g], w >> 1, w & 1, l, uu[g]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) wl[r] = vec[r].w;
        lds_barrier();

        // ---- U = R + (T - I) R, W
        load_kq(next);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            f32x4 more = {};
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (j <= w >> 1) M::mul2(tf[j], read(s_r[g], j), uu[g], more);
            uu[g] += more;
            f32x4 wv;
#pragma unroll
            for (int r = 0; r < 4; ++r) wv[r] = wl[r] * uu[g][r];
            M::put_tile(s_w[g], w >> 1, w & 1, l, wv);
            M::put_tile(s_u[g], w >> 1, w & 1, l, uu[g]);
        }
        lds_barrier();

        // ---- S <- e^{g_l} S + K^T W, O = e^g Q S + Y U
        load_tv(next);
        if (w < J) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                st[g][0] *= egl;
                st[g][1] *= egl;
#pragma unroll
                for (int jt = 0; jt < 2; ++jt)
                    M::mul(kt[0][jt], kt[1][jt], read(s_w[g], jt), st[g][0], st[g][1]);
            }
            put_state();
        }
        const __amdgpu_buffer_rsrc_t ro = rsrc(op, ostride, a.dv, sizeof(OT), c);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            f32x4 more = {};
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (j <= w >> 1) M::mul2(yf[j], read(s_u[g], j), qs[g], more);
            qs[g] += more;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                store1(ro, bytes(voff[g], r, sizeof(OT)), qs[g][r], OT{});
        }
        lds_barrier();
    }
    if (slive) {
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (col0 + kCols * g < a.dv)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    a.S[sq.dst * slab + sat + (size_t)(sr + e) * a.dv + kCols * g] =
                        st[g][e >> 2][e & 3];
    }
}

int64_t up256(int64_t x) { return (x + 255) & ~(int64_t)255; }

Layout layout(const RuleArgs &a) {
    Layout y;
    const int DK = a.dk > 64 ? 128 : 64;
    const int64_t kt = (int64_t)(DK / 16) * 2 * 64 * 16 * (a.dtype == GDN_DTYPE_BF16 ? 1 : 2);
    y.slots = a.rows / kC + a.batch;      // every sequence may end in a partial chunk
    y.off_pre = 0;
    y.off_order = up256(4LL * a.batch);
    y.off_seq = y.off_order + up256(4LL * a.batch);
    y.off_kt = y.off_seq + up256(4LL * y.slots);
    y.off_data = y.off_kt + kt * y.slots * a.Hk;
    const int64_t data = a.dtype == GDN_DTYPE_BF16 ? sizeof(ChunkData<Half>)
                                                   : sizeof(ChunkData<Full>);
    y.bytes = y.off_data + data * y.slots * a.H;
    return y;
}

// Two column groups a wave load the chunk's operands once for 32 columns; one
// group gives twice the workgroups.
bool wide_scan(const RuleArgs &a) {
    const long long wide = (long long)a.batch * a.H * ((a.dv + 2 * kCols - 1) / (2 * kCols));
    return wide >= device_cu_count();
}

template <typename M, int DK, typename OT, int G>
hipError_t launch_scan(const RuleArgs &a, const Layout &y, hipStream_t s) {
    const int tiles = (a.dv + kCols * G - 1) / (kCols * G);
    hipLaunchKernelGGL((prefill_scan_kernel<M, DK, OT, G>),
                       dim3((unsigned)a.batch * a.H * tiles), dim3(kThreads), 0, s, a, y, tiles);
    return hipGetLastError();
}

template <typename M, int DK>
hipError_t launch(const RuleArgs &a, hipStream_t s) {
    const Layout y = layout(a);
    hipLaunchKernelGGL(prefill_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, y);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((prefill_chunk_kernel<M, DK>), dim3((unsigned)y.slots * a.H),
                       dim3(kThreads), 0, s, a, y);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool half = a.out_dtype == GDN_DTYPE_BF16;
    if (wide_scan(a)) return half ? launch_scan<M, DK, uint16_t, 2>(a, y, s)
                                  : launch_scan<M, DK, float, 2>(a, y, s);
    return half ? launch_scan<M, DK, uint16_t, 1>(a, y, s) : launch_scan<M, DK, float, 1>(a, y, s);
}

}  // namespace

int64_t prefill_workspace(const RuleArgs &a) { return layout(a).bytes; }

hipError_t launch_prefill(const RuleArgs &a, hipStream_t s) {
    if (a.dtype == GDN_DTYPE_BF16)
        return a.dk > 64 ? launch<Half, 128>(a, s) : launch<Half, 64>(a, s);
    return a.dk > 64 ? launch<Full, 128>(a, s) : launch<Full, 64>(a, s);
}

}  // namespace gdn
