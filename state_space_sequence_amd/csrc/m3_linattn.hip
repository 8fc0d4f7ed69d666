// Linear attention with a decay for each head: chunked forward, gradients and
// the single-token step (gfx950).
//
// Everything but the step is one kernel. With a = exp(log_decay[h]), a chunk of
// nt tokens and the state S (keys x values) before it,
//   out_i = sum_{j<=i} si a^{i-j} (q_i . k_j) v_j + sr a^{i+1} S^T q_i
//   S    <- a^{nt} S + sum_j su a^{nt-1-j} k_j v_j^T
// is the forward (si = sr = scale, su = 1). Time reversed,
//   out_j = sum_{i>=j} si a^{i-j} (q_j . k_i) v_i + sr a^{nt-1-j} D^T q_j
//   D    <- a^{nt} D + sum_i su a^{i+1} k_i v_i^T
// with D the gradient of the state behind the chunk (si = su = scale, sr = 1). The
// gradients are three such passes over other tensors:
//   dq: forwards,  (q, k, v) = (dy, v, k), the state transposed
//   dk: backwards, (q, k, v) = (v, dy, q), the state transposed
//   dv: backwards, (q, k, v) = (k, q, dy)
// and d log_decay is sum_t scale dy_t . (U_t^T q_t) with U = dS / d log_decay,
// U_t = a (U_{t-1} + S_{t-1}), carried the same way by a forward pass that forms
// out with the weights n a^n in place of a^n and takes its product with dy: every
// weight stays local to its chunk, where sums of t (q.dq - k.dk) over a whole
// sequence would cancel.
//
// A workgroup of 4 waves owns one chain (batch, head), 64 of its values (columns of S) and one
// segment of the tokens. Wave w owns 16 columns: its part of S never leaves its
// registers. The accumulators of the update (keys down the rows) are, two row
// tiles at a time, the operand of the product with q, provided that the key
// index of q is stored in the same order: q and k lie in LDS with their columns
// permuted so (perm below), and k and v a second time transposed, tokens
// consecutive, for the products that contract over tokens.
#include <math.h>

#include "m3_internal.h"
#include "m3_linattn.h"

namespace m3i {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kVT = 64;  // value columns of a workgroup
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxDim = 256;
constexpr int64_t kMaxGrid = 0x7fffffff;

enum Mode { kOut = 0, kState = 1, kDecay = 2 };

// one of a pass's three tensors: [b, L, heads, dim], read at head h / per
struct Tensor {
    const void *p;
    int heads, per;
};

struct Args {
    Tensor q, k, v;
    void *o;       // [b, L, H, vd]: io dtype, or fp32 (o32)
    bool o32, rev;
    const float *log_decay;
    const int *lengths;
    const float *s_in;   // initial states: [chains] or, seg_in, [chains, nseg]; NULL: zero
    const float *u_in;   // likewise, kDecay (zero where there is one segment)
    float *s_out;        // kOut: [chains], the state after the last segment, or NULL. kState: [chains, nseg]
    float *u_out;        // kState: [chains, nseg] or NULL
    bool seg_in;
    const void *dy;         // kDecay: [b, L, H, vd]
    const float *dh_final;  // kDecay: [chains] or NULL
    double *part;           // kDecay: [H, b * nseg * nvt]
    int64_t b, L, nchunks, seg_chunks;
    int H, kd, vd, nseg, nvt;
    int sk, sv;  // strides of a key and a value in a stored state
    float si, sr, su;
};

// 8 contraction slots of one operand row or column: lane l holds row l % 16 and
// slots 8 (l / 16) .. + 7. bf16: one 16x16x32 product; fp32: slot e of every lane
// group is one of eight 16x16x4 products. Both give rows 4 (l / 16) + r, column l % 16.
template <typename E>
struct Ops;

template <>
struct Ops<uint16_t> {
    typedef bf16x8 frag;
    typedef u32x4 pack;  // 8 elements as loaded
    static constexpr int C = 64;   // tokens of a chunk
    static constexpr int NS = 2;   // parts of a state operand
    static constexpr int NA = 2;   // parts of a score
    static constexpr int NW = 3;   // parts of a weighted value, whose sums are stored in fp32
    static constexpr int NU = 3;   // parts of a state operand of d log_decay, an fp32 output
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // x as a sum of NP bf16 parts: each takes 8 of its bits, the remainders are exact
    template <int NP>
    static __device__ __forceinline__ void parts(const float *x, frag *p) {
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[n][e] = (__bf16)r[e];
                if (n + 1 < NP) r[e] -= (float)p[n][e];
            }
    }
    static __device__ __forceinline__ float value(frag f, int e) { return (float)f[e]; }
    // 4 values to 4 consecutive elements, in parts `plane` elements apart
    template <int NP>
    static __device__ __forceinline__ void store4(uint16_t *to, int plane, f32x4 x) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            bf16x4 b;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                b[e] = (__bf16)x[e];
                if (n + 1 < NP) x[e] -= (float)b[e];
            }
            *reinterpret_cast<bf16x4 *>(to + n * plane) = b;
        }
    }
};

template <>
struct Ops<float> {
    typedef f32x8 frag;
    typedef f32x8 pack;
    static constexpr int C = 32, NS = 1, NA = 1, NW = 1, NU = 1;
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    template <int NP>
    static __device__ __forceinline__ void parts(const float *x, frag *p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[0][e] = x[e];
    }
    static __device__ __forceinline__ float value(frag f, int e) { return f[e]; }
    template <int NP>
    static __device__ __forceinline__ void store4(float *to, int, f32x4 x) {
        *reinterpret_cast<f32x4 *>(to) = x;
    }
};

// 8 elements of a row, zero from column dim on, packed; VEC: dim is a multiple of 8 and rows are 16-byte aligned
template <bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t *row, int col, int dim, bool live) {
    u32x4 w = {0, 0, 0, 0};
    if constexpr (VEC) {
        if (live && col < dim) w = *reinterpret_cast<const u32x4 *>(row + col);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            unsigned lo = 0, hi = 0;
            if (live && col + 2 * e < dim) lo = row[col + 2 * e];
            if (live && col + 2 * e + 1 < dim) hi = row[col + 2 * e + 1];
            w[e] = lo | (hi << 16);
        }
    }
    return w;
}

template <bool VEC>
__device__ __forceinline__ f32x8 load8(const float *row, int col, int dim, bool live) {
    f32x8 x = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if constexpr (VEC) {
        if (live && col < dim) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(row + col);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(row + col + 4);
            x = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (live && col + e < dim) x[e] = row[col + e];
    }
    return x;
}

// elements 4 half .. + 3 of a packed row
__device__ __forceinline__ void put4(uint16_t *to, u32x4 w, int half) {
    *reinterpret_cast<u32x2 *>(to) = half ? u32x2{w[2], w[3]} : u32x2{w[0], w[1]};
}
__device__ __forceinline__ void put4(float *to, f32x8 x, int half) {
    *reinterpret_cast<f32x4 *>(to) = half ? f32x4{x[4], x[5], x[6], x[7]} : f32x4{x[0], x[1], x[2], x[3]};
}
// element e of four packed rows
__device__ __forceinline__ void put_column(uint16_t *to, const u32x4 (&w)[4], int e) {
    const unsigned sel = e & 1 ? 0x07060302u : 0x05040100u;
    *reinterpret_cast<u32x2 *>(to) = u32x2{__builtin_amdgcn_perm(w[1][e >> 1], w[0][e >> 1], sel),
                                           __builtin_amdgcn_perm(w[3][e >> 1], w[2][e >> 1], sel)};
}
__device__ __forceinline__ void put_column(float *to, const f32x8 (&x)[4], int e) {
    *reinterpret_cast<f32x4 *>(to) = f32x4{x[0][e], x[1][e], x[2][e], x[3][e]};
}

template <typename E>
__device__ __forceinline__ typename Ops<E>::frag frag_at(const E *p) {
    return *reinterpret_cast<const typename Ops<E>::frag *>(p);
}

// LDS tiles, in blocks of 8 elements (one lane's operand slots).
// Row tile [token][key]: keys permuted so that a block holds what the state's
// accumulators hold of it: block 4s + g of a row is keys 32s + 4g + 0..3 and
// 32s + 16 + 4g + 0..3. Blocks are exchanged by the row's low bits, so that the 16 rows
// which a fragment read touches lie in different banks.
template <int KD>
__device__ __forceinline__ int row_at(int row, int block) {
    return row * KD + ((block ^ (row & 7)) << 3);
}
// Transposed tile [key or value][token]
template <int C>
__device__ __forceinline__ int col_at(int col, int block) {
    return col * C + ((block ^ ((col ^ (col >> 3)) & (C / 8 - 1))) << 3);
}

// 8 consecutive keys from n0 (a multiple of 8) of one token into the row tile
template <int KD, typename E>
__device__ __forceinline__ void put_row(E *tile, int row, int n0, typename Ops<E>::pack x) {
    const int block = 4 * (n0 >> 5) + ((n0 & 15) >> 2), half = (n0 >> 4) & 1;
    put4(tile + row_at<KD>(row, block) + 4 * half, x, 0);
    put4(tile + row_at<KD>(row, block + 1) + 4 * half, x, 1);
}

__device__ __forceinline__ float power(float g2, int n) {
    return n == 0 ? 1.f : __builtin_amdgcn_exp2f(g2 * (float)n);  // a decay of 0 is 2^-inf, and 0 * inf no number
}

// A workgroup's place in the work: consecutive ones (the value tiles of a chain, the
// heads of a group, which read the same tensors) go to one XCD and its L2
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t total) {
    const int64_t q = total / 8, r = total % 8, x = id % 8;
    return x * q + (x < r ? x : r) + id / 8;
}

template <typename E, int KD, int MODE, bool VEC>
__global__ __launch_bounds__(kThreads, KD == 256 || MODE == kDecay ? 1 : 2) void linattn_kernel(const Args a) {
    typedef Ops<E> O;
    typedef typename O::frag frag;
    constexpr int C = O::C, KT = KD / 16, KS = KD / 32, JS = C / 32, IT = C / 16;
    constexpr bool kDec = MODE == kDecay, kSt = MODE == kState;
    constexpr int NA = kDec ? O::NU : O::NA, NS = kDec ? O::NU : O::NS;
    __shared__ __align__(16) E Qs[kSt ? 8 : C * KD];
    __shared__ __align__(16) E Ks[kSt ? 8 : C * KD];
    __shared__ __align__(16) E Kc[KD * C];
    __shared__ __align__(16) E Vc[kVT * C];
    __shared__ __align__(16) E As[kSt ? 8 : NA * C * C];
    __shared__ float wt[C], wu[kDec || kSt ? C : 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, lr = lane & 15, lg = lane >> 4;
    int64_t id = xcd_order(blockIdx.x, gridDim.x);
    const int vt = (int)(id % a.nvt);
    id /= a.nvt;
    const int64_t chains = a.b * a.H, chain = id % chains;
    const int seg = (int)(id / chains);
    const int64_t bi = chain / a.H;
    const int h = (int)(chain % a.H);
    int64_t len = a.L;
    if (a.lengths) {
        const int64_t l = a.lengths[bi];
        len = l < 0 ? 0 : (l < a.L ? l : a.L);
    }
    const float g2 = a.log_decay[h] * kLog2e;
    const int64_t c_lo = seg * a.seg_chunks;
    const int64_t c_hi = c_lo + a.seg_chunks < a.nchunks ? c_lo + a.seg_chunks : a.nchunks;
    const int v0 = vt * kVT, col = v0 + 16 * wave + lr;  // this lane's value column
    const int64_t nstate = (int64_t)a.kd * a.vd;
    const bool with_u = kDec || (kSt && a.u_out != nullptr);

    // the state: rows n = 16 nt + 4 lg + r of column col
    f32x4 S[KT], U[kDec || kSt ? KT : 1];
    const auto load_state = [&](f32x4 *to, const float *from) {
        const float *p = from ? from + (a.seg_in ? chain * a.nseg + seg : chain) * nstate : nullptr;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = 16 * t + 4 * lg + r;
                to[t][r] = p && n < a.kd && col < a.vd ? p[(int64_t)n * a.sk + (int64_t)col * a.sv] : 0.f;
            }
    };
    const auto store_state = [&](const f32x4 *from, float *to, int64_t at) {
        float *p = to + at * nstate;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = 16 * t + 4 * lg + r;
                if (n < a.kd && col < a.vd) p[(int64_t)n * a.sk + (int64_t)col * a.sv] = from[t][r];
            }
    };
    load_state(S, kSt ? nullptr : a.s_in);
    if constexpr (kDec || kSt) load_state(U, kSt ? nullptr : a.u_in);

    // score tile of this wave: output tokens of strip `st`, JW tiles of the others from j0
    constexpr int JW = IT * IT / 4;
    const int st = wave % IT, j0 = (wave / IT) * JW;
    float mask[kSt ? 1 : JW][4];
    if constexpr (!kSt) {
#pragma unroll
        for (int t = 0; t < JW; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * st + lr, j = 16 * (j0 + t) + 4 * lg + r, n = a.rev ? j - i : i - j;
                mask[t][r] = n < 0 ? 0.f : a.si * power(g2, n) * (kDec ? (float)n : 1.f);
                if (kDec && n == 0) mask[t][r] = 0.f;
            }
    }
    const int kh = h / a.k.per, vh = h / a.v.per, qh = kSt ? 0 : h / a.q.per;
    const E *kb = static_cast<const E *>(a.k.p) + ((int64_t)bi * a.L * a.k.heads + kh) * a.kd;
    const E *vb = static_cast<const E *>(a.v.p) + ((int64_t)bi * a.L * a.v.heads + vh) * a.vd;
    const E *qb = kSt ? nullptr : static_cast<const E *>(a.q.p) + ((int64_t)bi * a.L * a.q.heads + qh) * a.kd;
    const int64_t kst = (int64_t)a.k.heads * a.kd, vst = (int64_t)a.v.heads * a.vd,
                  qst = kSt ? 0 : (int64_t)a.q.heads * a.kd;
    double dsum = 0.0;

    // staging units: k and v 4 tokens x 8 columns, q 1 token x 8 columns
    constexpr int KU = (C / 4) * (KD / 8), KN = (KU + kThreads - 1) / kThreads;
    constexpr int VU = (C / 4) * (kVT / 8);
    constexpr int QN = kSt ? 0 : C * (KD / 8) / kThreads;
    static_assert(VU <= kThreads && (kSt || C * (KD / 8) % kThreads == 0), "staging");
    typename O::pack kx[KN][4], vx[4], qx[QN ? QN : 1];

    const auto fetch_k = [&](int64_t t0, int u) {
        const int unit = tid + u * kThreads, n0 = 8 * (unit % (KD / 8)), j = 4 * (unit / (KD / 8));
#pragma unroll
        for (int r = 0; r < 4; ++r)
            kx[u][r] = load8<VEC>(kb + (t0 + j + r) * kst, n0, a.kd, j < C && t0 + j + r < len);
    };
    const auto fetch_v = [&](int64_t t0) {
        const int p0 = 8 * (tid % (kVT / 8)), j = 4 * (tid / (kVT / 8));
#pragma unroll
        for (int r = 0; r < 4; ++r)
            vx[r] = load8<VEC>(vb + (t0 + j + r) * vst, v0 + p0, a.vd, j < C && t0 + j + r < len);
    };
    const auto fetch_q = [&](int64_t t0, int u) {
        const int unit = tid + u * kThreads, n0 = 8 * (unit % (KD / 8)), i = unit / (KD / 8);
        qx[u] = load8<VEC>(qb + (t0 + i) * qst, n0, a.kd, t0 + i < len);
    };
    const auto stage_k = [&](int u) {
        const int unit = tid + u * kThreads, n0 = 8 * (unit % (KD / 8)), j = 4 * (unit / (KD / 8));
        if (KU % kThreads == 0 || unit < KU) {
            if constexpr (!kSt) {
#pragma unroll
                for (int r = 0; r < 4; ++r) put_row<KD>(Ks, j + r, n0, kx[u][r]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) put_column(Kc + col_at<C>(n0 + e, j >> 3) + (j & 4), kx[u], e);
        }
    };
    const auto stage_v = [&]() {
        if (tid < VU) {
            const int p0 = 8 * (tid % (kVT / 8)), j = 4 * (tid / (kVT / 8));
#pragma unroll
            for (int e = 0; e < 8; ++e) put_column(Vc + col_at<C>(p0 + e, j >> 3) + (j & 4), vx, e);
        }
    };
    const auto stage_q = [&](int u) {
        const int unit = tid + u * kThreads;
        put_row<KD>(Qs, unit / (KD / 8), 8 * (unit % (KD / 8)), qx[u]);
    };
    // The next chunk's tensors are loaded while this one is computed. Two states of 256 keys
    // leave no registers for that: there each piece is loaded and staged by itself.
    constexpr bool kAhead = !(kDec && KD == 256);
    const auto fetch = [&](int64_t c) {
#pragma unroll
        for (int u = 0; u < KN; ++u) fetch_k(c * C, u);
        fetch_v(c * C);
#pragma unroll
        for (int u = 0; u < QN; ++u) fetch_q(c * C, u);
    };
    const auto stage = [&](int64_t c, int nt) {
#pragma unroll
        for (int u = 0; u < KN; ++u) {
            if (!kAhead) {
                fetch_k(c * C, u);
                __builtin_amdgcn_sched_barrier(0);
            }
            stage_k(u);
        }
        if (!kAhead) {
            fetch_v(c * C);
            __builtin_amdgcn_sched_barrier(0);
        }
        stage_v();
#pragma unroll
        for (int u = 0; u < QN; ++u) {
            if (!kAhead) {
                fetch_q(c * C, u);
                __builtin_amdgcn_sched_barrier(0);
            }
            stage_q(u);
        }
        if (tid < C) {
            const int n = a.rev ? tid + 1 : nt - 1 - tid;  // steps from this token to the state behind it
            const float p = tid < nt ? a.su * power(g2, n) : 0.f;
            wt[tid] = p;
            if constexpr (kDec || kSt) wu[tid] = n == 0 || p == 0.f ? 0.f : p * (float)n;
        }
    };

    const int64_t nc = c_hi > c_lo ? c_hi - c_lo : 0;
    if (kAhead && nc > 0) fetch(a.rev ? c_hi - 1 : c_lo);
    for (int64_t s = 0; s < nc; ++s) {
        const int64_t c = a.rev ? c_hi - 1 - s : c_lo + s, t0 = c * C;
        const int nt = len - t0 >= C ? C : (len > t0 ? (int)(len - t0) : 0);
        stage(c, nt);
        __syncthreads();
        if (kAhead && s + 1 < nc) fetch(a.rev ? c - 1 : c + 1);
        frag vf[JS];
#pragma unroll
        for (int ks = 0; ks < JS; ++ks) vf[ks] = frag_at(Vc + col_at<C>(16 * wave + lr, 4 * ks + lg));

        if constexpr (!kSt) {
            // scores, transposed: rows j, column i = this lane's token of the strip
            f32x4 sc[JW];
#pragma unroll
            for (int t = 0; t < JW; ++t) sc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const frag qf = frag_at(Qs + row_at<KD>(16 * st + lr, 4 * ks + lg));
#pragma unroll
                for (int t = 0; t < JW; ++t)
                    sc[t] = O::mfma(frag_at(Ks + row_at<KD>(16 * (j0 + t) + lr, 4 * ks + lg)), qf, sc[t]);
            }
#pragma unroll
            for (int t = 0; t < JW; ++t) {
                const int i = 16 * st + lr, jb = 2 * (j0 + t) + (lg >> 1);
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = mask[t][r] == 0.f ? 0.f : sc[t][r] * mask[t][r];
                O::template store4<NA>(As + i * C + ((jb ^ (i & (C / 8 - 1))) << 3) + 4 * (lg & 1), C * C, x);
            }
            // the carried state's part: rows are values, column i
            f32x4 acc[IT], ac2[kDec ? IT : 1];
#pragma unroll
            for (int it = 0; it < IT; ++it) acc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (kDec) {
#pragma unroll
                for (int it = 0; it < IT; ++it) ac2[it] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float x[8];
                frag sp[NS], up[kDec ? NS : 1];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = S[2 * ks + (e >> 2)][e & 3];
                O::template parts<NS>(x, sp);
                if constexpr (kDec) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = U[2 * ks + (e >> 2)][e & 3];
                    O::template parts<NS>(x, up);
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const frag qf = frag_at(Qs + row_at<KD>(16 * it + lr, 4 * ks + lg));
#pragma unroll
                    for (int n = NS - 1; n >= 0; --n) {
                        acc[it] = O::mfma(sp[n], qf, acc[it]);
                        if constexpr (kDec) ac2[it] = O::mfma(up[n], qf, ac2[it]);
                    }
                }
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int i = 16 * it + lr, n = a.rev ? nt - 1 - i : i + 1;
                const float p = i < nt ? a.sr * power(g2, n) : 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (kDec) acc[it][r] = p * (acc[it][r] * (float)n + ac2[it][r]);
                    else acc[it][r] *= p;
                }
            }
            __syncthreads();
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int ks = 0; ks < JS; ++ks)
#pragma unroll
                    for (int n = NA - 1; n >= 0; --n)
                        acc[it] = O::mfma(
                            vf[ks], frag_at(As + n * C * C + (16 * it + lr) * C + (((4 * ks + lg) ^ (lr & (C / 8 - 1))) << 3)),
                            acc[it]);
            const int p0 = v0 + 16 * wave + 4 * lg;
            float csum = 0.f;
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int i = 16 * it + lr;
                const int64_t tok = t0 + i;
                if (tok >= a.L) continue;
                const int64_t at = ((bi * a.L + tok) * a.H + h) * a.vd + p0;
                if constexpr (kDec) {
                    if (i < nt) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (p0 + r < a.vd) csum += acc[it][r] * ld_io<sizeof(E) == 2>(a.dy, at + r);
                    }
                } else {
                    f32x4 x = acc[it];
                    if (i >= nt) x = f32x4{0.f, 0.f, 0.f, 0.f};
                    if (VEC) {
                        if (p0 < a.vd) {
                            if (sizeof(E) == 4 || a.o32)
                                *reinterpret_cast<f32x4 *>(static_cast<float *>(a.o) + at) = x;
                            else
                                Ops<uint16_t>::store4<1>(static_cast<uint16_t *>(a.o) + at, 0, x);
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (p0 + r < a.vd) {
                                if (sizeof(E) == 4 || a.o32) static_cast<float *>(a.o)[at + r] = x[r];
                                else static_cast<__bf16 *>(a.o)[at + r] = (__bf16)x[r];
                            }
                    }
                }
            }
            if constexpr (kDec) dsum += (double)csum;
        }

        // the state behind the chunk
        {
            const float at = power(g2, nt), atn = nt ? at * (float)nt : 0.f;
            frag wv[JS][O::NW], wv2[kDec || kSt ? JS : 1][O::NW];
#pragma unroll
            for (int ks = 0; ks < JS; ++ks) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = wt[32 * ks + 8 * lg + e] * O::value(vf[ks], e);
                O::template parts<O::NW>(x, wv[ks]);
                if constexpr (kDec || kSt) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = wu[32 * ks + 8 * lg + e] * O::value(vf[ks], e);
                    O::template parts<O::NW>(x, wv2[ks]);
                }
            }
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                if constexpr (kDec || kSt) {
                    if (with_u) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) U[t][r] = at * U[t][r] + (atn == 0.f ? 0.f : atn * S[t][r]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) S[t][r] *= at;
#pragma unroll
                for (int ks = 0; ks < JS; ++ks) {
                    const frag kf = frag_at(Kc + col_at<C>(16 * t + lr, 4 * ks + lg));
#pragma unroll
                    for (int n = O::NW - 1; n >= 0; --n) {
                        S[t] = O::mfma(kf, wv[ks][n], S[t]);
                        if constexpr (kDec || kSt) {
                            if (with_u) U[t] = O::mfma(kf, wv2[ks][n], U[t]);
                        }
                    }
                }
            }
        }
        __syncthreads();
    }

    if constexpr (kSt) {
        store_state(S, a.s_out, chain * a.nseg + seg);
        if (with_u) store_state(U, a.u_out, chain * a.nseg + seg);
    }
    const bool last = a.rev ? seg == 0 : seg == a.nseg - 1;
    if constexpr (MODE == kOut) {
        if (last && a.s_out) store_state(S, a.s_out, chain);
    }
    if constexpr (kDec) {
        if (last && a.dh_final) {
            const float *p = a.dh_final + chain * nstate;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = 16 * t + 4 * lg + r;
                    if (n < a.kd && col < a.vd) dsum += (double)U[t][r] * p[(int64_t)n * a.sk + (int64_t)col * a.sv];
                }
        }
        // sum over the workgroup, in a fixed order
        __shared__ double sums[kThreads];
        sums[tid] = dsum;
        __syncthreads();
        for (int n = kThreads / 2; n > 0; n >>= 1) {
            if (tid < n) sums[tid] += sums[tid + n];
            __syncthreads();
        }
        if (tid == 0) a.part[((int64_t)h * a.b + bi) * a.nseg * a.nvt + seg * a.nvt + vt] = sums[0];
    }
}

// Segment states into incoming states, in place: st[c][seg] <- the state before the
// segment (in the order of the sweep), from init [c] or zero. One thread a state element.
struct ChainArgs {
    float *st, *ut;
    const float *init, *log_decay;
    const int *lengths;
    int64_t chains, nstate, L, seg_tokens;
    int H, nseg;
    bool rev;
};

__global__ __launch_bounds__(kThreads) void linattn_chain_kernel(const ChainArgs a) {
    const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= a.chains * a.nstate) return;
    const int64_t chain = e / a.nstate, i = e % a.nstate, bi = chain / a.H;
    int64_t len = a.L;
    if (a.lengths) {
        const int64_t l = a.lengths[bi];
        len = l < 0 ? 0 : (l < a.L ? l : a.L);
    }
    const float g2 = a.log_decay[chain % a.H] * kLog2e;
    float s = a.init ? a.init[e] : 0.f, u = 0.f;
    for (int k = 0; k < a.nseg; ++k) {
        const int seg = a.rev ? a.nseg - 1 - k : k;
        int64_t n = len - seg * a.seg_tokens;
        n = n < 0 ? 0 : (n < a.seg_tokens ? n : a.seg_tokens);
        const float p = n == 0 ? 1.f : __builtin_amdgcn_exp2f(g2 * (float)n);
        const int64_t at = (chain * a.nseg + seg) * a.nstate + i;
        const float own = a.st[at];
        a.st[at] = s;
        if (a.ut) {
            const float ou = a.ut[at];
            a.ut[at] = u;
            u = p * u + (p == 0.f ? 0.f : p * (float)n * s) + ou;
        }
        s = p * s + own;
    }
}

// out[row][g][d] = sum over the heads of group g of part[row][h][d]
template <bool BF16>
__global__ __launch_bounds__(kThreads) void linattn_heads_kernel(const float *part, void *out, int64_t rows, int G,
                                                                 int per, int d) {
    const int64_t n = rows * G * d;
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < n; e += (int64_t)gridDim.x * kThreads) {
        const int64_t rg = e / d;
        const float *p = part + rg * per * d + e % d;
        float s = 0.f;
        for (int k = 0; k < per; ++k) s += p[(int64_t)k * d];
        if constexpr (BF16) static_cast<__bf16 *>(out)[e] = (__bf16)s;
        else static_cast<float *>(out)[e] = s;
    }
}

__global__ __launch_bounds__(kThreads) void linattn_decay_kernel(const double *part, float *out, int64_t n) {
    __shared__ double sums[kThreads];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += part[blockIdx.x * n + i];
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int k = kThreads / 2; k > 0; k >>= 1) {
        if ((int)threadIdx.x < k) sums[threadIdx.x] += sums[threadIdx.x + k];
        __syncthreads();
    }
    if (threadIdx.x == 0) out[blockIdx.x] = (float)sums[0];
}

// ------------------------------------------------------------------ launch ---
template <typename E, int MODE, bool VEC>
hipError_t launch_dims(const Args &a, int64_t grid, hipStream_t s) {
    const dim3 g((unsigned)grid), t(kThreads);
    if (a.kd <= 64) hipLaunchKernelGGL((linattn_kernel<E, 64, MODE, VEC>), g, t, 0, s, a);
    else if (a.kd <= 128) hipLaunchKernelGGL((linattn_kernel<E, 128, MODE, VEC>), g, t, 0, s, a);
    else hipLaunchKernelGGL((linattn_kernel<E, 256, MODE, VEC>), g, t, 0, s, a);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_pass(const Args &a, bool bf16, hipStream_t s) {
    const int64_t grid = a.b * a.H * a.nseg * a.nvt;
    if (grid == 0) return hipSuccess;
    const bool vec = a.kd % 8 == 0 && a.vd % 8 == 0;
    if (bf16)
        return vec ? launch_dims<uint16_t, MODE, true>(a, grid, s) : launch_dims<uint16_t, MODE, false>(a, grid, s);
    return vec ? launch_dims<float, MODE, true>(a, grid, s) : launch_dims<float, MODE, false>(a, grid, s);
}

struct LinPlan {
    int64_t nchunks, seg_chunks, chains;
    int nseg, C;
};

int tiles(int64_t d) { return (int)((d + kVT - 1) / kVT); }

// Segments: enough workgroups for two on each of the 256 CUs, of four chunks at least
LinPlan make_lin_plan(const m3_shape &s) {
    LinPlan p{};
    p.C = s.io_dtype == M3_BF16 ? Ops<uint16_t>::C : Ops<float>::C;
    p.chains = s.batch * s.nheads;
    p.nchunks = (s.seqlen + p.C - 1) / p.C;
    int64_t n = s.nsegments;
    if (n == 0) {
        const int64_t have = p.chains * tiles(s.headdim);
        n = have >= 384 || have == 0 ? 1 : (512 + have - 1) / have;
        if (n > p.nchunks / 4) n = p.nchunks / 4;
    }
    if (n > p.nchunks) n = p.nchunks;
    if (n < 1) n = 1;
    p.seg_chunks = p.nchunks ? (p.nchunks + n - 1) / n : 1;
    p.nseg = p.nchunks ? (int)((p.nchunks + p.seg_chunks - 1) / p.seg_chunks) : 1;
    return p;
}

bool al16(const void *p) { return (((uintptr_t)p) & 15u) == 0; }

m3_status lin_check(const m3_shape *s, uint32_t flags) {
    if (!s) return M3_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->nheads < 1 || s->ngroups < 1 || s->headdim < 1 || s->dstate < 1 ||
        s->rank < 1 || s->nsegments < 0)
        return M3_ERR_INVALID_ARG;
    if (s->nheads % s->ngroups != 0) return M3_ERR_INVALID_ARG;
    if (s->io_dtype != M3_F32 && s->io_dtype != M3_BF16) return M3_ERR_INVALID_ARG;
    if (s->flags & ~flags) return M3_ERR_INVALID_ARG;
    if (s->rank != 1 || s->dstate > kMaxDim || s->headdim > kMaxDim || s->nheads > 65536) return M3_ERR_UNSUPPORTED;
    if (s->batch > (1LL << 31) || s->seqlen > (1LL << 31) || s->batch * s->nheads > kMaxGrid / 4 ||
        (s->seqlen > 0 && s->batch > (1LL << 40) / s->seqlen))
        return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

m3_status lin_plan(const m3_shape *s, LinPlan *p) {
    const m3_status st = lin_check(s, 0);
    if (st != M3_OK) return st;
    *p = make_lin_plan(*s);
    if (p->chains * p->nseg > kMaxGrid / 4) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

size_t up(size_t n) { return (n + 255) & ~size_t(255); }

// workspace of the backward, in this order
struct BwdWs {
    size_t seg;          // one set of segment states
    size_t dk, dv;       // per-head partials where heads share keys and values
    size_t part;         // d log_decay partials
    size_t total;
};

BwdWs bwd_ws(const m3_shape &s, const LinPlan &p) {
    BwdWs w{};
    const size_t rows = (size_t)(s.batch * s.seqlen * s.nheads);
    if (p.nseg > 1) w.seg = up((size_t)p.chains * p.nseg * s.headdim * s.dstate * 4);
    if (s.nheads != s.ngroups) {
        w.dk = up(rows * s.dstate * 4);
        w.dv = up(rows * s.headdim * 4);
    }
    w.part = up((size_t)p.chains * p.nseg * tiles(s.headdim) * 8);
    w.total = 3 * w.seg + w.dk + w.dv + w.part;
    return w;
}

Args base_args(const m3_shape &s, const LinPlan &p, const float *log_decay, const int32_t *lengths) {
    Args a{};
    a.log_decay = log_decay;
    a.lengths = lengths;
    a.b = s.batch; a.L = s.seqlen; a.H = (int)s.nheads;
    a.nchunks = p.nchunks; a.seg_chunks = p.seg_chunks; a.nseg = p.nseg;
    return a;
}

// kd keys, vd values; a stored state is [P][N], so the keys are its fast axis unless `swapped`
void set_dims(Args &a, int64_t kd, int64_t vd, bool swapped) {
    a.kd = (int)kd; a.vd = (int)vd;
    a.nvt = tiles(vd);
    a.sk = swapped ? (int)vd : 1;
    a.sv = swapped ? 1 : (int)kd;
}

hipError_t chain_states(const Args &a, const LinPlan &p, float *st, float *ut, const float *init, bool rev,
                        hipStream_t s) {
    ChainArgs c{};
    c.st = st; c.ut = ut; c.init = init; c.log_decay = a.log_decay; c.lengths = a.lengths;
    c.chains = p.chains; c.nstate = (int64_t)a.kd * a.vd; c.L = a.L; c.seg_tokens = p.seg_chunks * p.C;
    c.H = a.H; c.nseg = p.nseg; c.rev = rev;
    const int64_t n = c.chains * c.nstate, grid = (n + kThreads - 1) / kThreads;
    if (grid > kMaxGrid) return hipErrorInvalidValue;
    hipLaunchKernelGGL(linattn_chain_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, c);
    return hipGetLastError();
}

hipError_t sum_heads(const float *part, void *out, bool bf16, int64_t rows, int64_t G, int64_t per, int64_t d,
                     hipStream_t s) {
    int64_t grid = (rows * G * d + kThreads - 1) / kThreads;
    if (grid == 0) return hipSuccess;
    if (grid > 65536) grid = 65536;
    if (bf16)
        hipLaunchKernelGGL((linattn_heads_kernel<true>), dim3((unsigned)grid), dim3(kThreads), 0, s, part, out, rows,
                           (int)G, (int)per, (int)d);
    else
        hipLaunchKernelGGL((linattn_heads_kernel<false>), dim3((unsigned)grid), dim3(kThreads), 0, s, part, out, rows,
                           (int)G, (int)per, (int)d);
    return hipGetLastError();
}

// -------------------------------------------------------------------- step ---
// One token. The state is read and written once and bounds the call (HBM): a row of N keys lies
// across LPR lanes, V elements (16 bytes) each; a thread keeps its keys and queries in
// registers for RPT rows, whose loads are all issued before the first is used.
template <typename E, typename T, int LPR, int RPT, bool VEC>
__global__ __launch_bounds__(kThreads) void linattn_step_kernel(const void *q, const void *k, const void *v,
                                                                const float *log_decay, void *state, void *y, int H,
                                                                int per, int P, int N, float scale) {
    constexpr int V = sizeof(T) == 4 ? 4 : 8, RW = kThreads / LPR;  // rows of a workgroup's pass
    constexpr bool BF = sizeof(E) == 2;
    const int h = blockIdx.x % H, c = threadIdx.x % LPR, n0 = c * V;
    const int64_t bh = blockIdx.x, bg = (bh / H) * (H / per) + h / per;
    const int p0 = blockIdx.y * RW * RPT + threadIdx.x / LPR;
    T *st = static_cast<T *>(state) + bh * P * N;
    float x[RPT][V];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int p = p0 + i * RW;
        const T *row = st + (int64_t)p * N + n0;
        if constexpr (VEC) {
            u32x4 w = {0, 0, 0, 0};
            if (p < P && n0 < N) w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(row));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (V == 4) x[i][e] = __uint_as_float(w[e]);
                else {
                    x[i][2 * e] = __uint_as_float(w[e] << 16);
                    x[i][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) x[i][e] = p < P && n0 + e < N ? ld_io<V == 8>(row, e) : 0.f;
        }
    }
    const float a = expf(log_decay[h]);
    float kk[V], qq[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const bool live = n0 + e < N;
        kk[e] = live ? ld_io<BF>(k, bg * N + n0 + e) : 0.f;
        qq[e] = live ? scale * ld_io<BF>(q, bh * N + n0 + e) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int p = p0 + i * RW;
        const float vv = p < P ? ld_io<BF>(v, bg * P + p) : 0.f;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            x[i][e] = __builtin_fmaf(a, x[i][e], vv * kk[e]);
            s = __builtin_fmaf(x[i][e], qq[e], s);
        }
        s = group_sum<LPR>(s);
        if (p < P) {
            T *row = st + (int64_t)p * N + n0;
            if constexpr (VEC) {
                if (n0 < N) {
                    u32x4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (V == 4) w[e] = __float_as_uint(x[i][e]);
                        else {
                            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                            const bf16x2 b = {(__bf16)x[i][2 * e], (__bf16)x[i][2 * e + 1]};
                            w[e] = __builtin_bit_cast(unsigned, b);
                        }
                    }
                    __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(row));
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (n0 + e < N) {
                        if constexpr (V == 4) row[e] = x[i][e];
                        else reinterpret_cast<__bf16 *>(row)[e] = (__bf16)x[i][e];
                    }
            }
            if (c == 0) {
                if constexpr (BF) static_cast<__bf16 *>(y)[bh * P + p] = (__bf16)s;
                else static_cast<float *>(y)[bh * P + p] = s;
            }
        }
    }
}

struct StepArgs {
    const m3_linattn_step_io *io;
    int64_t b;
    int H, per, P, N;
};

template <typename E, typename T, int LPR, bool VEC>
hipError_t launch_step_rows(const StepArgs &a, hipStream_t s) {
    constexpr int RW = kThreads / LPR;
    const m3_linattn_step_io &io = *a.io;
    // few heads: one row a thread, so that more of the card takes part
    const bool wide = a.b * a.H >= 1024;
    const int rows = RW * (wide ? 8 : 1);
    const dim3 grid((unsigned)(a.b * a.H), (unsigned)((a.P + rows - 1) / rows)), t(kThreads);
    if (wide)
        hipLaunchKernelGGL((linattn_step_kernel<E, T, LPR, 8, VEC>), grid, t, 0, s, io.q, io.k, io.v, io.log_decay, io.h,
                           io.y, a.H, a.per, a.P, a.N, io.scale);
    else
        hipLaunchKernelGGL((linattn_step_kernel<E, T, LPR, 1, VEC>), grid, t, 0, s, io.q, io.k, io.v, io.log_decay, io.h,
                           io.y, a.H, a.per, a.P, a.N, io.scale);
    return hipGetLastError();
}

template <typename E, typename T>
hipError_t launch_step(const StepArgs &a, hipStream_t s) {
    constexpr int V = sizeof(T) == 4 ? 4 : 8;
    const int lanes = (a.N + V - 1) / V;
    const bool vec = a.N % V == 0;
    if (lanes <= 8)
        return vec ? launch_step_rows<E, T, 8, true>(a, s) : launch_step_rows<E, T, 8, false>(a, s);
    if (lanes <= 16)
        return vec ? launch_step_rows<E, T, 16, true>(a, s) : launch_step_rows<E, T, 16, false>(a, s);
    if (lanes <= 32)
        return vec ? launch_step_rows<E, T, 32, true>(a, s) : launch_step_rows<E, T, 32, false>(a, s);
    return vec ? launch_step_rows<E, T, 64, true>(a, s) : launch_step_rows<E, T, 64, false>(a, s);
}

m3_status status(hipError_t e) { return e == hipSuccess ? M3_OK : M3_ERR_HIP; }

// Segment states of one direction: each segment's own, then chained from init
hipError_t segment_states(Args a, const LinPlan &p, bool bf16, float *st, float *ut, const float *init, hipStream_t s) {
    a.s_in = nullptr; a.s_out = st; a.u_out = ut;
    const hipError_t e = launch_pass<kState>(a, bf16, s);
    return e == hipSuccess ? chain_states(a, p, st, ut, init, a.rev, s) : e;
}

}  // namespace
}  // namespace m3i

using namespace m3i;

extern "C" {

size_t m3_linattn_workspace_bytes(const m3_shape *shape) {
    LinPlan p;
    if (lin_plan(shape, &p) != M3_OK || p.nseg == 1) return 0;
    return up((size_t)p.chains * p.nseg * shape->headdim * shape->dstate * 4);
}

m3_status m3_linattn_fwd(const m3_shape *shape, const m3_linattn_io *io, void *workspace, size_t ws_bytes,
                         void *stream) {
    LinPlan p;
    const m3_status st = lin_plan(shape, &p);
    if (st != M3_OK) return st;
    if (!io || !isfinite(io->scale)) return M3_ERR_INVALID_ARG;
    const m3_shape &s = *shape;
    if (s.batch == 0) return M3_OK;
    if (!io->log_decay || (s.seqlen > 0 && (!io->q || !io->k || !io->v || !io->y))) return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->q, io->k, io->v, io->log_decay, io->h0, io->lengths, io->y, io->h_final, workspace};
    for (const void *x : ptrs)
        if (!al16(x)) return M3_ERR_MISALIGNED;
    const size_t need = m3_linattn_workspace_bytes(shape);
    if (need && (!workspace || ws_bytes < need)) return M3_ERR_WORKSPACE_TOO_SMALL;
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const bool bf16 = s.io_dtype == M3_BF16;
    const int H = (int)s.nheads, G = (int)s.ngroups;
    Args a = base_args(s, p, io->log_decay, io->lengths);
    set_dims(a, s.dstate, s.headdim, false);
    a.q = {io->q, H, 1}; a.k = {io->k, G, H / G}; a.v = {io->v, G, H / G};
    a.si = a.sr = io->scale; a.su = 1.f;
    a.s_in = io->h0;
    if (p.nseg > 1) {
        float *seg = static_cast<float *>(workspace);
        const hipError_t e = segment_states(a, p, bf16, seg, nullptr, io->h0, hs);
        if (e != hipSuccess) return M3_ERR_HIP;
        a.s_in = seg;
        a.seg_in = true;
    }
    a.o = io->y;
    a.s_out = io->h_final;
    return status(launch_pass<kOut>(a, bf16, hs));
}

size_t m3_linattn_bwd_workspace_bytes(const m3_shape *shape) {
    LinPlan p;
    return lin_plan(shape, &p) == M3_OK ? bwd_ws(*shape, p).total : 0;
}

m3_status m3_linattn_bwd(const m3_shape *shape, const m3_linattn_io *io, const m3_linattn_grads *gr, void *workspace,
                         size_t ws_bytes, void *stream) {
    LinPlan p;
    const m3_status st = lin_plan(shape, &p);
    if (st != M3_OK) return st;
    if (!io || !gr || !isfinite(io->scale)) return M3_ERR_INVALID_ARG;
    const m3_shape &s = *shape;
    const bool work = s.batch * s.seqlen > 0;
    if ((s.batch > 0 && !io->log_decay) ||
        (work && (!io->q || !io->k || !io->v || !gr->dy || !gr->dq || !gr->dk || !gr->dv)))
        return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->q, io->k, io->v, io->log_decay, io->h0, io->lengths, gr->dy, gr->dh_final,
                          gr->dq, gr->dk, gr->dv, gr->dlog_decay, gr->dh0, workspace};
    for (const void *x : ptrs)
        if (!al16(x)) return M3_ERR_MISALIGNED;
    const BwdWs w = bwd_ws(s, p);
    if (w.total && (!workspace || ws_bytes < w.total)) return M3_ERR_WORKSPACE_TOO_SMALL;
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const bool bf16 = s.io_dtype == M3_BF16;
    const int H = (int)s.nheads, G = (int)s.ngroups, per = H / G;
    char *at = static_cast<char *>(workspace);
    float *seg_s = reinterpret_cast<float *>(at), *seg_u = reinterpret_cast<float *>(at + w.seg),
          *seg_d = reinterpret_cast<float *>(at + 2 * w.seg), *pk = reinterpret_cast<float *>(at + 3 * w.seg),
          *pv = reinterpret_cast<float *>(at + 3 * w.seg + w.dk);
    double *part = reinterpret_cast<double *>(at + 3 * w.seg + w.dk + w.dv);
    const Tensor q = {io->q, H, 1}, k = {io->k, G, per}, v = {io->v, G, per}, dy = {gr->dy, H, 1};
    const float sc = io->scale;
    const Args base = base_args(s, p, io->log_decay, io->lengths);
    const bool split = p.nseg > 1;
    hipError_t e = hipSuccess;
    if (s.batch > 0) {
        // the states of both directions, key-major as the forward and dv use them
        Args f = base, r = base;
        set_dims(f, s.dstate, s.headdim, false);
        f.q = q; f.k = k; f.v = v; f.si = f.sr = sc; f.su = 1.f;
        set_dims(r, s.dstate, s.headdim, false);
        r.rev = true;
        r.q = k; r.k = q; r.v = dy; r.si = r.su = sc; r.sr = 1.f;
        if (split) {
            e = segment_states(f, p, bf16, seg_s, gr->dlog_decay ? seg_u : nullptr, io->h0, hs);
            if (e == hipSuccess) e = segment_states(r, p, bf16, seg_d, nullptr, gr->dh_final, hs);
            if (e != hipSuccess) return M3_ERR_HIP;
        }
        const float *s_in = split ? seg_s : io->h0, *d_in = split ? seg_d : gr->dh_final;
        f.seg_in = r.seg_in = split;
        Args dq = f;  // (dy, v, k), the state transposed
        set_dims(dq, s.headdim, s.dstate, true);
        dq.q = dy; dq.k = v; dq.v = k; dq.s_in = s_in; dq.o = gr->dq;
        if ((e = launch_pass<kOut>(dq, bf16, hs)) != hipSuccess) return M3_ERR_HIP;
        Args dk = r;  // (v, dy, q), the state transposed
        set_dims(dk, s.headdim, s.dstate, true);
        dk.q = v; dk.k = dy; dk.v = q; dk.s_in = d_in;
        dk.o32 = per > 1; dk.o = per > 1 ? pk : gr->dk;
        if ((e = launch_pass<kOut>(dk, bf16, hs)) != hipSuccess) return M3_ERR_HIP;
        Args dv = r;  // (k, q, dy)
        dv.s_in = d_in; dv.s_out = gr->dh0;
        dv.o32 = per > 1; dv.o = per > 1 ? pv : gr->dv;
        if ((e = launch_pass<kOut>(dv, bf16, hs)) != hipSuccess) return M3_ERR_HIP;
        if (per > 1) {
            const int64_t rows = s.batch * s.seqlen;
            if ((e = sum_heads(pk, gr->dk, bf16, rows, G, per, s.dstate, hs)) != hipSuccess ||
                (e = sum_heads(pv, gr->dv, bf16, rows, G, per, s.headdim, hs)) != hipSuccess)
                return M3_ERR_HIP;
        }
        if (gr->dlog_decay) {
            f.s_in = s_in; f.u_in = split ? seg_u : nullptr;
            f.dy = gr->dy; f.dh_final = gr->dh_final; f.part = part;
            if ((e = launch_pass<kDecay>(f, bf16, hs)) != hipSuccess) return M3_ERR_HIP;
        }
    }
    if (gr->dlog_decay) {
        hipLaunchKernelGGL(linattn_decay_kernel, dim3((unsigned)H), dim3(kThreads), 0, hs, part, gr->dlog_decay,
                           s.batch * p.nseg * tiles(s.headdim));
        e = hipGetLastError();
    }
    return status(e);
}

m3_status m3_linattn_step(const m3_shape *shape, const m3_linattn_step_io *io, void *stream) {
    const m3_status st = lin_check(shape, M3_FLAG_BF16_STATE);
    if (st != M3_OK) return st;
    if (!io || !isfinite(io->scale)) return M3_ERR_INVALID_ARG;
    const m3_shape &s = *shape;
    if (s.batch == 0) return M3_OK;
    if (!io->q || !io->k || !io->v || !io->log_decay || !io->h || !io->y) return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->q, io->k, io->v, io->log_decay, io->h, io->y};
    for (const void *x : ptrs)
        if (!al16(x)) return M3_ERR_MISALIGNED;
    const StepArgs a = {io, s.batch, (int)s.nheads, (int)(s.nheads / s.ngroups), (int)s.headdim, (int)s.dstate};
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const bool bs = (s.flags & M3_FLAG_BF16_STATE) != 0;
    if (s.io_dtype == M3_BF16)
        return status(bs ? launch_step<uint16_t, uint16_t>(a, hs) : launch_step<uint16_t, float>(a, hs));
    return status(bs ? launch_step<float, uint16_t>(a, hs) : launch_step<float, float>(a, hs));
}

}  // extern "C"
