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
//   chunk: a workgroup per (chunk, head): decays, Gram matrices, T and Y, and
//          the chunk's keys (also transposed) and queries, stored as matrix
//          operands
//   scan:  a workgroup per (sequence, head, 16 or 64 columns of d_v): the
//          columns of S are independent, and 32 heads of d_v = 128 give the
//          256 workgroups that fill the chip with a single prompt.  Four waves
//          carry the state: they split the rows of every product (16 tokens
//          or 32 rows of S each) and exchange S, R and W through LDS, three
//          barriers a chunk; four more form the outputs beside them.  The
//          operands that do not depend on S come from memory into registers,
//          a chunk ahead.
//
// Times here are of single kernels and, unless called whole calls, the shortest
// of 20 dispatches: medians are 3 to 10 % above (scan of one prompt 231 to 239,
// median 239 to 250).
//
// Bound.  The chunk kernel writes 25 KiB a (chunk, head) and 48 KiB a (chunk,
// key head) and is held by that traffic (8192 tokens, 32 heads over 16 key
// heads: 63 us for 274 MB with its inputs, 4.3 TB/s).  A scan workgroup reads
// 72 KiB of operands a chunk through its L1 besides V: with every chunk read
// from one place, so from the L2, the scan keeps nine tenths of its time; with
// loads two chunks ahead all of it; and the products (36 of 16 cycles on a
// state wave's SIMD, 24 more for the outputs) are a fifth.  What remains is
// the three exchanges through LDS.  A single prompt's chunks follow each
// other: 128 of them take 128 x 1.9 us.
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
// of large sums.  The logarithms themselves are fp32's: one is off by 2^-23 of
// itself at most, so a decay 2^-x by ln 2 2^-23 x 2^-x <= 2^-24.4, less than a
// rounding of what it multiplies.  (In 64 bits the outputs' error was 1.38e-7
// instead of 1.40e-7, and the chunk kernel 3 us slower.)
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
    // exact . fp32, two products at once: the instructions of one sum wait
    // for each other, those of the two alternate.  Smallest part first.
    static __device__ __forceinline__ void mul(const Raw8 &x0, const Raw8 &x1, const Raw8 &y0,
                                               const Raw8 &y1, f32x4 &c0, f32x4 &c1) {
#pragma unroll
        for (int p = 2; p >= 0; --p) {
            c0 = mma(v(x0.p[0]), v(y0.p[p]), c0);
            c1 = mma(v(x1.p[0]), v(y1.p[p]), c1);
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
    static __device__ __forceinline__ void mul(const Raw8 &x0, const Raw8 &x1, const Raw8 &y0,
                                               const Raw8 &y1, f32x4 &c0, f32x4 &c1) {
        c0 = gram(x0, y0, c0);
        c1 = gram(x1, y1, c1);
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

// one (chunk, head) of the workspace; a head's chunks follow each other
template <typename M>
struct ChunkData {
    // T - I and Y as operands, 8 fp32 values a lane: the scan's output waves
    // have the time to split them, and a third less is moved
    uint4 t[kFrags][2][64], y[kFrags][2][64];
    float4 vec[kC];              // beta, beta e^g, e^g, e^{g_l - g} of the tokens
};

// A chunk's keys and queries as matrix operands, per key head, in runs of
// 1 KiB: the scan's workgroups read them 8 times (d_v = 128), and in place
// each run would be 16 pieces in as many lines.
template <typename M, int DK>
struct KeyData {
    uint4 k[4][DK / 32][M::kExact][64];       // token tile i, contraction over rows of S
    uint4 q[4][DK / 32][M::kExact][64];
    uint4 kt[DK / 16][2][M::kExact][64];      // rows of S, contraction over tokens
};

struct Layout {
    int slots;                   // chunk slots
    int64_t off_pre, off_order, off_slot, off_keys, off_data, bytes;
};

// ---------------------------------------------------------------------------
// plan: pre[i] = first chunk slot of sequence i (-1: bad rows), slot[s] = the
// sequence, first row and tokens of a chunk (sequence -1: unused slot), order
// = sequences, most chunks first
// ---------------------------------------------------------------------------
__device__ __forceinline__ int chunks_of(const RuleArgs &a, int i) {
    const rule::Sequence s = rule::sequence(a, i);
    return s.fault & kFaultBadLength ? -1 : (s.len + kC - 1) / kC;
}

__global__ __launch_bounds__(kPlanThreads) void prefill_plan_kernel(RuleArgs a, Layout y) {
    __shared__ int s_part[kPlanThreads / 64];
    __shared__ int s_n[kSortMax], s_start[kSortMax];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63;
    char *ws = static_cast<char *>(a.workspace);
    int *pre = reinterpret_cast<int *>(ws + y.off_pre);
    int *order = reinterpret_cast<int *>(ws + y.off_order);
    int4 *slot = reinterpret_cast<int4 *>(ws + y.off_slot);
    auto chunk = [&](int i, int c) {
        const int row0 = a.cu[i] + kC * c;
        return make_int4(i, row0, min(kC, a.cu[i + 1] - row0), 0);
    };
    const bool sorted = a.batch <= kSortMax;
    if (!sorted) {
        for (int s = tid; s < y.slots; s += kPlanThreads) slot[s] = make_int4(-1, 0, 0, 0);
        __syncthreads();
    }
    long long sum = 0;
    for (int i0 = 0; i0 < a.batch; i0 += kPlanThreads) {
        const int i = i0 + tid;
        const int n = i < a.batch ? chunks_of(a, i) : 0;
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
            if (sorted) {
                s_n[i] = ok ? n : -1;
                s_start[i] = (int)min(at, (long long)y.slots);
            } else {
                order[i] = i;
                if (ok)
                    for (int c = 0; c < n; ++c) slot[at + c] = chunk(i, c);
            }
        }
    }
    if (!sorted) return;
    __syncthreads();
    if (tid < a.batch) {
        const int n = s_n[tid];
        int rank = 0;
        for (int j = 0; j < a.batch; ++j) rank += s_n[j] > n || (s_n[j] == n && j < tid);
        order[rank] = tid;
    }
    for (int s = tid; s < y.slots; s += kPlanThreads) {
        int lo = 0, hi = a.batch - 1;             // last sequence that starts by slot s
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_start[mid] <= s) lo = mid;
            else hi = mid - 1;
        }
        const int c = s - s_start[lo];
        slot[s] = c < s_n[lo] ? chunk(lo, c) : make_int4(-1, 0, 0, 0);
    }
}

// ---------------------------------------------------------------------------
// chunk: T, Y, decays; keys and queries as operands
//
// K and Q rows go through LDS once (whole lines from memory); X and Y take
// their place after the Gram products.  T^T is kept above the diagonal of the
// array that holds X below it, the diagonal blocks of T^T over those of X, so
// that four workgroups fit a compute unit (d_k = 128, bf16).
// ---------------------------------------------------------------------------
constexpr int kLd = kC + 4;      // LDS row stride of the 64-wide matrices (floats)

template <typename M, int DK>
__global__ __launch_bounds__(kThreads) void prefill_chunk_kernel(RuleArgs a, Layout y) {
    typedef typename M::elem T;
    constexpr int J = DK / 32;
    constexpr int P = DK * sizeof(T) / 16;       // 16-byte pieces of a row
    constexpr int kPer = kC * P / kThreads;      // of K, and of Q, a thread loads
    struct Rows {
        uint4 k[kC][P], q[kC][P];
    };
    struct Square {
        float x[kC][kLd], y[kC][kLd];
    };
    __shared__ union {
        Rows in;
        Square sq;
    } sm;
    __shared__ double s_g[kC];
    __shared__ float s_beta[kC];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const int m = l & 15, qd = l >> 4;
    char *ws = static_cast<char *>(a.workspace);
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int4 at = reinterpret_cast<const int4 *>(ws + y.off_slot)[slot];
    if (at.x < 0) return;
    const int rep = a.H / a.Hk, hk = h / rep;
    const int row0 = at.y, n = at.z;
    ChunkData<M> *out =
        reinterpret_cast<ChunkData<M> *>(ws + y.off_data) + (size_t)h * y.slots + slot;

    const T *kp = static_cast<const T *>(a.k) + ((size_t)row0 * a.Hk + hk) * a.dk;
    const T *qp = static_cast<const T *>(a.q) + ((size_t)row0 * a.Hk + hk) * a.dk;
    const size_t stride = (size_t)a.Hk * a.dk;
    constexpr int E = 16 / sizeof(T);            // elements of a piece
    uint4 kin[kPer], qin[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int t = (tid + kThreads * i) / P, c = (tid + kThreads * i) % P;
        kin[i] = qin[i] = make_uint4(0, 0, 0, 0);
        if (t < n && E * c < a.dk) {
            kin[i] = *reinterpret_cast<const uint4 *>(kp + t * stride + E * c);
            qin[i] = *reinterpret_cast<const uint4 *>(qp + t * stride + E * c);
        }
    }
    // ---- decays; a token past the end has alpha 1 and beta 0
    if (w == 0) {
        float lg = 0.f, be = 0.f;
        if (l < n) {
            const size_t at = ((size_t)row0 + l) * a.H + h;
            // alpha = 0: far enough below any exponent to clear the state,
            // small enough to keep the other tokens' logarithms exact
            const float al = a.alpha[at];
            lg = al == 0.f ? -1e4f : log2f(al);
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
    // pieces are turned by the row: 16 rows read at one piece spread over the banks
    auto piece = [&](int t, int c) { return c ^ (t & (P < 16 ? P - 1 : 15)); };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int t = (tid + kThreads * i) / P, c = (tid + kThreads * i) % P;
        sm.in.k[t][piece(t, c)] = kin[i];
        sm.in.q[t][piece(t, c)] = qin[i];
    }
    __syncthreads();
    auto operand = [&](const uint4(*rows)[P], int t, int j) {
        Raw8 x;
#pragma unroll
        for (int p = 0; p < M::kExact; ++p)
            x.p[p] = rows[t][piece(t, (4 * j + qd) * M::kExact + p)];
        return x;
    };

    // ---- tiles (w, jb) of X and Y: rows 16 w + 4 qd + r, column 16 jb + m
    f32x4 kk[4] = {}, qk[4] = {};
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const Raw8 ka = operand(sm.in.k, 16 * w + m, j), qa = operand(sm.in.q, 16 * w + m, j);
#pragma unroll
        for (int jb = 0; jb < 4; ++jb)
            if (jb <= w) {
                const Raw8 kb = operand(sm.in.k, 16 * jb + m, j);
                kk[jb] = M::gram(ka, kb, kk[jb]);
                qk[jb] = M::gram(qa, kb, qk[jb]);
            }
    }
    // ---- operands of the scan, once per key head
    if (h % rep == 0) {
        KeyData<M, DK> *to = reinterpret_cast<KeyData<M, DK> *>(ws + y.off_keys) +
                             (size_t)hk * y.slots + slot;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const Raw8 kx = operand(sm.in.k, rho(w, m), j), qx = operand(sm.in.q, rho(w, m), j);
#pragma unroll
            for (int p = 0; p < M::kExact; ++p) {
                to->k[w][j][p][l] = kx.p[p];
                to->q[w][j][p][l] = qx.p[p];
            }
        }
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {      // a lane: 8 consecutive tokens of one row of S
            const int f = 4 * i + w, ti = f >> 1, jt = f & 1, d = rho(ti, m);
            alignas(16) T x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int t = 32 * jt + 8 * qd + e;
                x[e] = reinterpret_cast<const T *>(&sm.in.k[t][piece(t, d / E)])[d % E];
            }
#pragma unroll
            for (int p = 0; p < M::kExact; ++p)
                to->kt[ti][jt][p][l] = reinterpret_cast<const uint4 *>(x)[p];
        }
    }
    __syncthreads();                             // X and Y take the rows' place
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)
        if (jb <= w) {
            const int s = 16 * jb + m;
            const double gs = s_g[s];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * w + 4 * qd + r;
                const float e = exp2f((float)(s_g[t] - gs));
                sm.sq.x[t][s] = s < t ? s_beta[t] * e * kk[jb][r] : 0.f;
                sm.sq.y[t][s] = s <= t ? e * qk[jb][r] : 0.f;
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
        for (int s = 0; s < r; ++s) acc = fmaf(-sm.sq.x[16 * w + r][16 * w + s], t[s], acc);
        t[r] = acc;
    }
    f32x4 tb[4];                       // tiles (k, w) of T, by k - w
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        // of values: a choice between elements would keep t in memory
        const float t0 = t[r], t1 = t[4 + r], t2 = t[8 + r], t3 = t[12 + r];
        tb[0][r] = qd & 2 ? (qd & 1 ? t3 : t2) : (qd & 1 ? t1 : t0);
    }
    *reinterpret_cast<f32x4 *>(&sm.sq.x[16 * w + m][16 * w + 4 * qd]) = tb[0];
    __syncthreads();
    // below it, T_iw = -T_ii sum_k X_ik T_kw: fp32 products (contraction
    // index 4 qd + r of a block at step r)
    auto product = [&](const f32x4 &av, const f32x4 &b, f32x4 c) {
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
            for (int dk = 0; dk < di; ++dk)
                p = product(*reinterpret_cast<const f32x4 *>(
                                &sm.sq.x[16 * bi + m][16 * (w + dk) + 4 * qd]),
                            tb[dk], p);
            f32x4 tii;
#pragma unroll
            for (int r = 0; r < 4; ++r) tii[r] = sm.sq.x[16 * bi + 4 * qd + r][16 * bi + m];
            tb[di] = -product(tii, p, f32x4{});
            *reinterpret_cast<f32x4 *>(&sm.sq.x[16 * w + m][16 * bi + 4 * qd]) = tb[di];
        }
    }
    __syncthreads();

    // ---- out as operands, three of the twelve pieces a wave
#pragma unroll
    for (int i = 0; i < 2 * kFrags / 4; ++i) {
        const int job = 4 * i + w, f = job % kFrags;
        const int ti = f < 2 ? f : (f + 2) >> 1, j = f < 2 ? 0 : f & 1;
        const int tr = rho(ti, m), k0 = 32 * j + 8 * qd;
        alignas(16) float v[8];
        if (job < kFrags) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = k0 + e < tr ? sm.sq.x[k0 + e][tr] : 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = k0 + e <= tr ? sm.sq.y[tr][k0 + e] : 0.f;
        }
        uint4(*to)[64] = job < kFrags ? out->t[f] : out->y[f];
#pragma unroll
        for (int p = 0; p < 2; ++p) to[p][l] = reinterpret_cast<const uint4 *>(v)[p];
    }
}

// ---------------------------------------------------------------------------
// scan: the state through a sequence's chunks
// ---------------------------------------------------------------------------
// Eight waves: four carry the state, four form the outputs.  The state waves'
// products wait for each other, and a wave that waits to issue a load issues
// no product: the second wave of a SIMD fills these gaps (8192 tokens, 32
// heads, 16 columns a workgroup, when it was built: 280 us; all in four waves: 328 us).
constexpr int kScanThreads = 512;

template <typename M, int DK, typename OT, int G>
__global__ __launch_bounds__(kScanThreads, 2) void prefill_scan_kernel(
    RuleArgs a, Layout y, int tiles) {
    typedef typename M::elem T;
    constexpr int J = DK / 32;
    constexpr int N = M::kParts;
    __shared__ __attribute__((aligned(16))) float s_vec[8][64];
    __shared__ uint4 s_s[G][J][N][64], s_r[G][2][N][64], s_u[G][2][N][64], s_w[G][2][N][64];
    __shared__ uint4 s_t[kFrags][N][64];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    const int w = wave & 3;                         // of the four of its role
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
            for (int t = tid >> 4; t < sq.len; t += kScanThreads / 16)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    if (col0 + kCols * g < a.dv)
                        rule::put(&out[((size_t)sq.first + t) * ostride + kCols * g],
                                  __builtin_nanf(""));
        return;
    }

    const T *vp = static_cast<const T *>(a.v) + (size_t)sq.first * ostride + (size_t)h * a.dv;
    const OT *op = static_cast<const OT *>(a.out) + (size_t)sq.first * ostride + (size_t)h * a.dv;
    const ChunkData<M> *data =
        reinterpret_cast<const ChunkData<M> *>(ws + y.off_data) + (size_t)h * y.slots + pre;
    const KeyData<M, DK> *keys =
        reinterpret_cast<const KeyData<M, DK> *>(ws + y.off_keys) + (size_t)hk * y.slots + pre;

    const int tok4 = 32 * (w >> 1) + 8 * qd + 4 * (w & 1);   // its four tokens of R, U, O
    // rows of V and O are addressed from a chunk's first: 32-bit offsets, and
    // what lies past its tokens reads as zero with no branch, so that a load
    // is waited for where it is used
    uint32_t voff[G];
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
    // tiles 0 and 1 of a triangle have no second operand: zero, from past the
    // end (behind a branch, the loads would be waited for where it ends)
    auto load_frags = [&](const auto &from, Raw8 *to) {
        constexpr uint32_t kPieces = sizeof(from[0]) / sizeof(from[0][0]);
        const __amdgpu_buffer_rsrc_t r = tile::make_rsrc(from, sizeof(from));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t at = j <= w >> 1 ? 16u * (kPieces * 64 * frag_of(w, j) + l) : kNowhere;
#pragma unroll
            for (uint32_t n = 0; n < kPieces; ++n)
                to[j].p[n] = tile::load16<0>(r, at + 1024 * n);
        }
    };
    auto load_rows = [&](const uint4(*from)[J][M::kExact][64], Raw8 *to) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int n = 0; n < M::kExact; ++n) to[j].p[n] = from[w][j][n][l];
    };
    // the wave's 16 tokens' factors: one number a lane, and through LDS four
    // numbers of four tokens
    auto load_vec = [&](int c) {
        return reinterpret_cast<const float *>(
            &data[c].vec[rho(w, l >> 2)])[l & 3];
    };
    auto read = [&](uint4(*buf)[N][64], int j) {
        Raw8 b;
#pragma unroll
        for (int n = 0; n < N; ++n)
            b.p[n] = buf[j][n][l];
        return b;
    };
    // f(g, operands of group g) for the column groups of buf.  All of a
    // group's reads are issued a group ahead of its products, and in one go:
    // left to the compiler, they are issued a few at a time and waited for
    // each time (8192 tokens: 280 us, so 262 us).
    auto groups = [&](auto &buf, auto f) {
        constexpr int K = sizeof(buf[0]) / sizeof(buf[0][0]);
        Raw8 b[2][K];
#pragma unroll
        for (int j = 0; j < K; ++j) b[0][j] = read(buf[0], j);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (g + 1 < G)
#pragma unroll
                for (int j = 0; j < K; ++j) b[(g + 1) & 1][j] = read(buf[g + 1], j);
            __builtin_amdgcn_sched_barrier(0);
            f(g, b[g & 1]);
        }
    };
    // rows of x times the columns of S, two sums that alternate
    auto times_state = [&](const Raw8 *x, const Raw8 *b) {
        f32x4 even = {}, odd = {};
#pragma unroll
        for (int j = 0; j < J; j += 2) M::mul(x[j], x[j + 1], b[j], b[j + 1], even, odd);
        return even + odd;
    };
    // c + the wave's rows of a lower triangle times b
    auto times_lower = [&](const Raw8 *x, const Raw8 *b, f32x4 c) {
        f32x4 more = {};
        M::mul2(x[0], b[0], c, more);
        if (w >> 1) M::mul2(x[1], b[1], c, more);
        return c + more;
    };

    auto split = [&](const Raw8 &x) {
        alignas(16) float v[8];
        *reinterpret_cast<uint4 *>(v) = x.p[0];
        *reinterpret_cast<uint4 *>(v + 4) = x.p[1];
        return M::from_f32(v);
    };

    // An operand's registers are loaded again, for the next chunk, as soon as
    // they have been used for the last time: a chunk ahead of their next use.
    const int chunks = (sq.len + kC - 1) / kC;
    if (wave >= 4) {
        // ---- outputs: e^g Q S while the state waves form U, Y U while they
        // update S
        Raw8 qf[J], tf[2], yf[2];
        float vec1 = 0.f;
        if (chunks > 0) {
            load_rows(keys->q, qf);
            vec1 = load_vec(0);
            load_frags(data->t, tf);
            load_frags(data->y, yf);
        }
        lds_barrier();
        for (int c = 0; c < chunks; ++c) {
            const int next = min(c + 1, chunks - 1);
            s_vec[wave][l] = vec1;
            vec1 = load_vec(next);
            Raw8 yx[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const Raw8 tx = split(tf[j]);
                if (j <= w >> 1)
#pragma unroll
                    for (int n = 0; n < N; ++n) s_t[frag_of(w, j)][n][l] = tx.p[n];
                yx[j] = split(yf[j]);
            }
            load_frags(data[next].t, tf);
            load_frags(data[next].y, yf);
            lds_barrier();
            f32x4 o[G];
            groups(s_s, [&](int g, const Raw8 *b) { o[g] = times_state(qf, b); });
            load_rows(keys[next].q, qf);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float eg = s_vec[wave][4 * (4 * qd + r) + 2];
#pragma unroll
                for (int g = 0; g < G; ++g) o[g][r] *= eg;
            }
            lds_barrier();
            const __amdgpu_buffer_rsrc_t ro = rsrc(op, ostride, a.dv, sizeof(OT), c);
            groups(s_u, [&](int g, const Raw8 *b) { o[g] = times_lower(yx, b, o[g]); });
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    store1(ro, bytes(voff[g], r, sizeof(OT)), o[g][r], OT{});
            lds_barrier();
        }
        return;
    }

    __builtin_amdgcn_s_setprio(3);          // the outputs are never waited for
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
    if (w < J)
#pragma unroll
        for (int g = 0; g < G; ++g) {
            M::put_tile(s_s[g], w, 0, l, st[g][0]);
            M::put_tile(s_s[g], w, 1, l, st[g][1]);
        }

    Raw8 kf[J], kt[2][2];
    float vec1 = 0.f, egl = 0.f;
    uint32_t vv[G][4];
    auto load_v = [&](int c) {
        const __amdgpu_buffer_rsrc_t rv = rsrc(vp, ostride, a.dv, sizeof(T), c);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int g = 0; g < G; ++g) vv[g][r] = M::load1(rv, bytes(voff[g], r, sizeof(T)));
        vec1 = load_vec(c);
    };
    auto load_kt = [&](int c) {
        egl = data[c].vec[kC - 1].z;
        const KeyData<M, DK> *p = keys + c;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int jt = 0; jt < 2; ++jt)
                // waves past the rows of S: any tile will do
#pragma unroll
                for (int n = 0; n < M::kExact; ++n)
                    kt[s][jt].p[n] = p->kt[(2 * w + s) & (DK / 16 - 1)][jt][n][l];
    };
    if (chunks > 0) {
        load_rows(keys->k, kf);
        load_v(0);
        load_kt(0);
    }
    lds_barrier();
    for (int c = 0; c < chunks; ++c) {
        const int next = min(c + 1, chunks - 1);
        // ---- R of 16 tokens
        f32x4 uu[G];
        s_vec[wave][l] = vec1;
        float4 vec[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            vec[r] = reinterpret_cast<const float4 *>(s_vec[wave])[4 * qd + r];
        groups(s_s, [&](int g, const Raw8 *b) { uu[g] = times_state(kf, b); });
        load_rows(keys[next].k, kf);
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                uu[g][r] = vec[r].x * M::widen(vv[g][r]) - vec[r].y * uu[g][r];
            M::put_tile(s_r[g], w >> 1, w & 1, l, uu[g]);
        }
        load_v(next);
        lds_barrier();

        // ---- U = R + (T - I) R, W
        const Raw8 tf[2] = {read(s_t, frag_of(w, 0)), read(s_t, frag_of(w, w >> 1))};
        groups(s_r, [&](int g, const Raw8 *b) {
            uu[g] = times_lower(tf, b, uu[g]);
            f32x4 wv;
#pragma unroll
            for (int r = 0; r < 4; ++r) wv[r] = vec[r].w * uu[g][r];
            M::put_tile(s_w[g], w >> 1, w & 1, l, wv);
            M::put_tile(s_u[g], w >> 1, w & 1, l, uu[g]);
        });
        lds_barrier();

        // ---- S <- e^{g_l} S + K^T W
        if (w < J) {
            groups(s_w, [&](int g, const Raw8 *b) {
                st[g][0] *= egl;
                st[g][1] *= egl;
#pragma unroll
                for (int jt = 0; jt < 2; ++jt)
                    M::mul(kt[0][jt], kt[1][jt], b[jt], b[jt], st[g][0], st[g][1]);
                M::put_tile(s_s[g], w, 0, l, st[g][0]);
                M::put_tile(s_s[g], w, 1, l, st[g][1]);
            });
        }
        load_kt(next);
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
    const int64_t keys = 3LL * kC * DK * (a.dtype == GDN_DTYPE_BF16 ? 2 : 4);
    y.slots = a.rows / kC + a.batch;      // every sequence may end in a partial chunk
    y.off_pre = 0;
    y.off_order = up256(4LL * a.batch);
    y.off_slot = y.off_order + up256(4LL * a.batch);
    y.off_keys = y.off_slot + up256(16LL * y.slots);
    y.off_data = y.off_keys + keys * y.slots * a.Hk;
    const int64_t data = a.dtype == GDN_DTYPE_BF16 ? sizeof(ChunkData<Half>)
                                                   : sizeof(ChunkData<Full>);
    y.bytes = y.off_data + data * y.slots * a.H;
    return y;
}

// Four column groups a wave load a chunk's operands once for 64 columns; one
// group gives four times the workgroups.  A chunk takes 3.9 us with four, 1.9
// us with one, and a compute unit holds one workgroup of either.  32 heads of
// d_v = 128, whole calls, one group and four: 1 prompt of 2048 tokens 84 and
// 149 us, 2 prompts 162 and 173, 3 prompts 263 and 207, 4 prompts 343 and 237,
// 16 of 512 tokens 366 and 249.  Where one prompt is much longer than the
// others, its own chain counts, and one group is better: 4096, 512, 512: 204
// and 301; 8192 and three of one token: 355 and 587; 4096 and fifteen of 64:
// 228 and 308.  Lengths are device data, so a rule on the batch cannot have all
// of these right.  Four are taken from as many workgroups as there are compute
// units, where equal prompts gain most: of the above, the three equal prompts
// and the long ones beside three or more short ones get the slower form.
bool wide_scan(const RuleArgs &a) {
    const long long wide = (long long)a.batch * a.H * ((a.dv + 4 * kCols - 1) / (4 * kCols));
    return wide >= device_cu_count();
}

template <typename M, int DK, typename OT, int G>
hipError_t launch_scan(const RuleArgs &a, const Layout &y, hipStream_t s) {
    const int tiles = (a.dv + kCols * G - 1) / (kCols * G);
    hipLaunchKernelGGL((prefill_scan_kernel<M, DK, OT, G>),
                       dim3((unsigned)a.batch * a.H * tiles), dim3(kScanThreads), 0, s, a, y, tiles);
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
    if (wide_scan(a)) return half ? launch_scan<M, DK, uint16_t, 4>(a, y, s)
                                  : launch_scan<M, DK, float, 4>(a, y, s);
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
