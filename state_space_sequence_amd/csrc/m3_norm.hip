// Group norm with an activation, channels last: forward and gradients (gfx950).
//
//   u = (x - mean) r w + b,  r = 1/sqrt(var + eps);  y = act(u), or u act(z) with a gate
//   du = dy act'(u) | dy act(z);  dz = dy u act'(z);  d = du w
//   dx = r (d - mean(d) - xh mean(d xh)),  xh = (x - mean) r;  dw = sum du xh;  db = sum du
// Bound by HBM: x (z, dy) read and y (dx, dz) written once. Tokens, bf16 b8 L4096 of 4096 channels with a gate: 154 us, 5.2 TB/s;
// gradients of b4: 136 us, 4.9 TB/s. Sequences read x twice, with gradients three times: bf16 b2 L4000 of 2048
// channels 61 us, six launches, of tensors that the last cache holds.
//
// Tokens by themselves (one position a row): the lanes of a group (L of them, each with 16 bytes of
// its channels) hold it in registers, so one pass is enough: the variance is taken of
// the differences to the mean, and the sums go across lanes by DPP moves. A lane keeps
// its channels from row to row: weights, and the sums for dw and db, stay in registers, and a workgroup's are joined in LDS.
//
// Sequences: partial sums of a slice of the positions (a thread keeps its channels; the sums for dw and db from one
// short slice to the next), joined in a fixed order by one workgroup a group, then one elementwise pass. Slices' means and
// squared differences are joined, not raw squares, which would lose the variance of
// values far from 0. The backward needs the sums of du and du xh of every channel
// only: the group's means of d and d xh are their products with w.
#include <math.h>

#include "m3_internal.h"
#include "m3_norm.h"

namespace m3i {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int64_t kMaxGrid = 0xffffff;  // workgroups along x: 2^32 threads
constexpr int64_t kLastCache = 256 << 20;
// Terms that a thread adds up in fp32, one after another: their error is below 2^-16 of the sum of their sizes
// (2^-17 where they are equal). What is beyond is added in fp64
constexpr int64_t kChain = 256;

struct NormArgs {
    const void *x, *z;
    const float *w, *b;
    const int *lengths;
    void *y;
    const void *dy;  // backward
    void *dx, *dz;
    float *dw, *db;
    int64_t n, S;  // rows, positions
    int C, G, D;
    float eps;
    bool silu;
    bool past;  // stores past the caches
    // tokens: rows of a workgroup. sequences: positions of a slice, slices; vectors of a workgroup,
    // positions it takes at a time, workgroups that share a group
    int64_t rows_wg, slice;
    int nslice, vb, pg, pieces, sweep;  // (sweep: slices of a workgroup that sums gradients)
    float *part, *chan;  // partial sums: of groups, of channels (tokens and sequences)
    float *stats;        // [n, G, 4]: mean, 1/std, mean of d, mean of d xh
};

template <bool BF16>
__device__ __forceinline__ float sigmoid(float x) {
    // (bf16 outputs: the hardware exponential's error, |x| 2^-24, is far below their rounding)
    const float e = BF16 ? __builtin_amdgcn_exp2f(-1.4426950408889634f * x) : expf(-x);
    return __builtin_amdgcn_rcpf(1.f + e);
}
template <bool BF16>
__device__ __forceinline__ float act(float x, bool silu) {
    return silu ? x * sigmoid<BF16>(x) : x;
}
// value and slope
template <bool BF16>
__device__ __forceinline__ void act2(float x, bool silu, float &v, float &s) {
    v = x;
    s = 1.f;
    if (silu) {
        const float g = sigmoid<BF16>(x);
        v = x * g;
        s = g * (1.f + x * (1.f - g));
    }
}

// 16 bytes. Tokens are read once, and past the caches; sequences are read again by the next pass. Where the tensors of a call
// are larger than the last cache the stores go past it too (b8 L4096 of 4096 channels with a gate, one call after
// another: 155 us, loads alone 162, neither 163; gradients of b4 147, 155, 154).
template <bool ONCE>
__device__ __forceinline__ u32x4 load16(const void *p) {
    const u32x4 *q = static_cast<const u32x4 *>(p);
    if constexpr (ONCE) return __builtin_nontemporal_load(q);
    else return *q;
}

// V consecutive elements from p + i: one 16-byte access, or (V == 1, or !VEC) single ones, `live` of them
template <bool BF16, int V, bool VEC, bool ONCE = false>
__device__ __forceinline__ void load(const void *p, int64_t i, int live, float (&x)[V]) {
    if constexpr (VEC && V > 1) {
        u32x4 w = {0, 0, 0, 0};
        if constexpr (BF16) {
            if (live > 0) w = load16<ONCE>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(w[e] << 16);
                x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
        } else {
            if (live > 0) w = load16<ONCE>(static_cast<const float *>(p) + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = e < live ? ld_io<BF16>(p, i + e) : 0.f;
    }
}

// (past: by the caches, where the tensors of the call do not fit them)
template <bool BF16, int V, bool VEC>
__device__ __forceinline__ void store(void *p, int64_t i, int live, const float (&x)[V], bool past) {
    if constexpr (VEC && V > 1) {
        if (live > 0) {
            u32x4 w;
            if constexpr (BF16) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 v = {x[2 * e], x[2 * e + 1]};
                    w[e] = __builtin_bit_cast(unsigned, __builtin_convertvector(v, bf16x2));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(x[e]);
            }
            u32x4 *to = static_cast<u32x4 *>(BF16 ? static_cast<void *>(static_cast<uint16_t *>(p) + i)
                                                  : static_cast<void *>(static_cast<float *>(p) + i));
            if (past) {
                asm volatile("");  // (two equal stores but for their hint would become one)
                __builtin_nontemporal_store(w, to);
                asm volatile("");
            } else {
                *to = w;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < live) {
                if constexpr (BF16) static_cast<__bf16 *>(p)[i + e] = (__bf16)x[e];
                else static_cast<float *>(p)[i + e] = x[e];
            }
    }
}

template <int V, bool VEC>
__device__ __forceinline__ void load_w(const float *p, int64_t i, int live, float none, float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = p && (VEC ? live > 0 : e < live) ? p[i + e] : none;
}

// u and v summed over the `rows` threads of a workgroup that hold the same channels, `stride` threads apart (this
// one is number `row`; `rows` or more: none of them), in LDS and in a fixed order. The first of them gets the
// sums; every thread of the workgroup takes part
template <int N>
__device__ __forceinline__ void join_rows(float (&u)[N], float (&v)[N], int row, int rows, int stride,
                                          float (*lds)[kThreads]) {
    if (rows == 1) return;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < N; ++e) {
        lds[e][threadIdx.x] = u[e];
        lds[N + e][threadIdx.x] = v[e];
    }
    for (int k = kThreads / 2; k > 0; k >>= 1) {
        if (k >= rows) continue;
        __syncthreads();
        if (row < k && row + k < rows) {
#pragma unroll
            for (int e = 0; e < 2 * N; ++e) lds[e][threadIdx.x] += lds[e][threadIdx.x + k * stride];
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        u[e] = lds[e][threadIdx.x];
        v[e] = lds[N + e][threadIdx.x];
    }
}

// ------------------------------------------------------------------ tokens ---
// Slots of L lanes, one group each: slots of a pass cover groups blockIdx.y * slots .. or, with
// fewer groups than slots, several rows. CH pieces of L * V channels a group.
template <bool BF16, int L, int CH, bool VEC>
struct Slot {
    static constexpr int V = BF16 ? 8 : 4, N = kThreads / L;
    int g, row0, rows;  // group, first row's offset, rows of a pass (0: an idle slot)
    int live[CH];       // channels of this lane's pieces
    int c[CH];          // their first channel
    __device__ __forceinline__ Slot(const NormArgs &a) {
        const int s = threadIdx.x / L, l = threadIdx.x % L;
        const int per = a.G < N ? N / a.G : 1;
        g = a.G < N ? s % a.G : (int)blockIdx.y * N + s;
        row0 = a.G < N ? s / a.G : 0;
        rows = per;
        const bool idle = a.G < N ? row0 >= per : g >= a.G;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int at = (k * L + l) * V, left = a.D - at;
            live[k] = idle || left <= 0 ? 0 : (left < V ? left : V);
            c[k] = g * a.D + at;
        }
        if (idle) rows = 0;
    }
};

template <bool BF16, int L, int CH, bool VEC>
__device__ __forceinline__ void token_stats(const NormArgs &a, const Slot<BF16, L, CH, VEC> &s,
                                            const float (&x)[CH][BF16 ? 8 : 4], float &mean, float &r) {
    constexpr int V = BF16 ? 8 : 4;
    const float inv = 1.f / (float)a.D;
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) t += x[k][e];
    mean = group_sum<L>(t) * inv;
    t = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = (VEC ? s.live[k] > 0 : e < s.live[k]) ? x[k][e] - mean : 0.f;
            t = __builtin_fmaf(d, d, t);
        }
    r = 1.f / sqrtf(group_sum<L>(t) * inv + a.eps);
}

template <bool BF16, int L, int CH, bool VEC, bool GATE>
__global__ __launch_bounds__(kThreads) void token_fwd_kernel(const NormArgs a) {
    constexpr int V = BF16 ? 8 : 4;
    const Slot<BF16, L, CH, VEC> s(a);
    float w[CH][V], b[CH][V];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        load_w<V, VEC>(a.w, s.c[k], s.live[k], 1.f, w[k]);
        load_w<V, VEC>(a.b, s.c[k], s.live[k], 0.f, b[k]);
    }
    const int64_t first = (int64_t)blockIdx.x * a.rows_wg, end = first + a.rows_wg < a.n ? first + a.rows_wg : a.n;
    const int step = a.G < s.N ? s.N / a.G : 1;
    for (int64_t row = first + s.row0; row - s.row0 < end; row += step) {
        const bool here = s.rows && row < end;
        float x[CH][V], z[GATE ? CH : 1][V];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int live = here ? s.live[k] : 0;
            load<BF16, V, VEC, true>(a.x, row * a.C + s.c[k], live, x[k]);
            if constexpr (GATE) load<BF16, V, VEC, true>(a.z, row * a.C + s.c[k], live, z[k]);
        }
        float mean, r;
        token_stats<BF16, L, CH, VEC>(a, s, x, mean, r);
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float u = __builtin_fmaf((x[k][e] - mean) * r, w[k][e], b[k][e]);
                if constexpr (GATE) y[e] = u * act<BF16>(z[k][e], a.silu);
                else y[e] = act<BF16>(u, a.silu);
            }
            store<BF16, V, VEC>(a.y, row * a.C + s.c[k], here ? s.live[k] : 0, y, a.past);
        }
    }
}

// chan: [gridDim.x][2][C]
template <bool BF16, int L, int CH, bool VEC, bool GATE>
__global__ __launch_bounds__(kThreads) void token_bwd_kernel(const NormArgs a) {
    constexpr int V = BF16 ? 8 : 4;
    const Slot<BF16, L, CH, VEC> s(a);
    float w[CH][V], b[CH][V], dw[CH][V], db[CH][V];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        load_w<V, VEC>(a.w, s.c[k], s.live[k], 1.f, w[k]);
        load_w<V, VEC>(a.b, s.c[k], s.live[k], 0.f, b[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) dw[k][e] = db[k][e] = 0.f;
    }
    const float inv = 1.f / (float)a.D;
    const int64_t first = (int64_t)blockIdx.x * a.rows_wg, end = first + a.rows_wg < a.n ? first + a.rows_wg : a.n;
    const int step = a.G < s.N ? s.N / a.G : 1;
    for (int64_t row = first + s.row0; row - s.row0 < end; row += step) {
        const bool here = s.rows && row < end;
        float x[CH][V], z[GATE ? CH : 1][V], d[CH][V];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int live = here ? s.live[k] : 0;
            load<BF16, V, VEC, true>(a.x, row * a.C + s.c[k], live, x[k]);
            load<BF16, V, VEC, true>(a.dy, row * a.C + s.c[k], live, d[k]);
            if constexpr (GATE) load<BF16, V, VEC, true>(a.z, row * a.C + s.c[k], live, z[k]);
        }
        float mean, r;
        token_stats<BF16, L, CH, VEC>(a, s, x, mean, r);
        float sa = 0.f, sb = 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const bool in = here && (VEC ? s.live[k] > 0 : e < s.live[k]);
                const float xh = (x[k][e] - mean) * r, u = __builtin_fmaf(xh, w[k][e], b[k][e]);
                float du, v, sl;
                if constexpr (GATE) {
                    act2<BF16>(z[k][e], a.silu, v, sl);
                    z[k][e] = d[k][e] * u * sl;  // dz
                    du = d[k][e] * v;
                } else {
                    act2<BF16>(u, a.silu, v, sl);
                    du = d[k][e] * sl;
                }
                du = in ? du : 0.f;
                x[k][e] = in ? xh : 0.f;
                dw[k][e] = __builtin_fmaf(du, x[k][e], dw[k][e]);
                db[k][e] += du;
                d[k][e] = du * w[k][e];
                sa += d[k][e];
                sb = __builtin_fmaf(d[k][e], x[k][e], sb);
            }
        }
        sa = group_sum<L>(sa) * inv;
        sb = group_sum<L>(sb) * inv;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int live = here ? s.live[k] : 0;
#pragma unroll
            for (int e = 0; e < V; ++e) d[k][e] = r * (d[k][e] - sa - x[k][e] * sb);
            store<BF16, V, VEC>(a.dx, row * a.C + s.c[k], live, d[k], a.past);
            if constexpr (GATE) store<BF16, V, VEC>(a.dz, row * a.C + s.c[k], live, z[k], a.past);
        }
    }
    if (a.chan) {
        __shared__ float lds[2 * V][kThreads];
        float *p = a.chan + (int64_t)blockIdx.x * 2 * a.C;
        const int rows = end - first < step ? (int)(end - first) : step;  // (the others have no sums)
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            join_rows<V>(dw[k], db[k], s.rows ? s.row0 : rows, rows, a.G * L, lds);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (s.row0 == 0 && (VEC ? s.live[k] > 0 : e < s.live[k])) {
                    p[s.c[k] + e] = dw[k][e];
                    p[a.C + s.c[k] + e] = db[k][e];
                }
        }
    }
}

// --------------------------------------------------------------- sequences ---
// A workgroup has one slice of a row's positions and vb vectors of V channels: whole groups (dv vectors
// each), or a piece of up to 256 vectors of one group. With fewer vectors than threads, pg positions at a time.
template <int V>
struct Lane {
    int64_t row, p0, p1;  // row, positions of the slice (those of the length)
    int64_t len;
    int c, po, step;
    int lv, run;   // this thread's vector in its group's part here, and the vectors of that part
    int g, piece;
    int64_t entry; // where the part's partial sums go
    bool idle;
    __device__ __forceinline__ Lane(const NormArgs &a, bool whole) : Lane(a) { take(a, blockIdx.x, whole); }
    // (without a slice yet)
    __device__ __forceinline__ explicit Lane(const NormArgs &a) {
        const int dv = a.D / V, cv = a.C / V;
        const int lane = (int)threadIdx.x % a.vb;
        po = (int)threadIdx.x / a.vb;
        step = a.pg;
        int v;
        piece = 0;
        if (a.pieces == 1) {
            v = (int)blockIdx.y * a.vb + lane;
            g = v / dv;
            lv = lane % dv;
            run = dv;
        } else {
            g = (int)blockIdx.y / a.pieces;
            piece = (int)blockIdx.y % a.pieces;
            lv = lane;
            v = g * dv + piece * a.vb + lane;
            run = dv - piece * a.vb < a.vb ? dv - piece * a.vb : a.vb;
        }
        idle = v >= cv || po >= a.pg || lv >= run;
        c = v * V;
    }
    // slice `id` of all rows' slices
    __device__ __forceinline__ void take(const NormArgs &a, unsigned id, bool whole) {
        const int slice = (int)(id % (unsigned)a.nslice);
        row = id / (unsigned)a.nslice;
        entry = ((row * a.G + g) * a.nslice + slice) * a.pieces + piece;
        len = a.S;
        if (a.lengths) {
            const int64_t l = a.lengths[row];
            len = l < 0 ? 0 : (l < a.S ? l : a.S);
        }
        p0 = slice * a.slice;
        const int64_t most = whole ? a.S : len;
        p1 = p0 + a.slice < most ? p0 + a.slice : most;
    }
    // v summed over the threads of this one's group, in a fixed order; every thread of the workgroup takes part
    template <typename T>
    __device__ __forceinline__ T sum(const NormArgs &a, T v, T *lds) const {
        __syncthreads();
        lds[threadIdx.x] = idle ? T{} : v;
        __syncthreads();
        if (po == 0)
            for (int k = 1; k < a.pg; ++k) lds[threadIdx.x] += lds[threadIdx.x + k * a.vb];
        for (int k = kThreads / 2; k > 0; k >>= 1) {
            if (k >= a.vb) continue;  // (no two vectors are that far apart)
            __syncthreads();
            if (po == 0 && !idle && lv < k && lv + k < run) lds[threadIdx.x] += lds[threadIdx.x + k];
        }
        __syncthreads();
        return lds[threadIdx.x % a.vb - (idle ? 0 : lv)];
    }
};

constexpr int kAhead = 4;  // positions of a thread whose loads are in flight together

// values, mean and squared differences of a group's part of a slice: part [n, G, nslice, pieces, 4]
template <bool BF16, int V>
__global__ __launch_bounds__(kThreads) void seq_stats_kernel(const NormArgs a) {
    __shared__ float lds[kThreads];
    const Lane<V> t(a, false);
    constexpr int B = 8;  // positions taken together
    float mean = 0.f, m2 = 0.f, n = 0.f;
    if (!t.idle)
        for (int64_t p = t.p0 + t.po; p < t.p1; p += B * t.step) {
            float x[B][V], s = 0.f, cnt = 0.f;
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const int64_t at = p + k * t.step;
                load<BF16, V, true>(a.x, (t.row * a.S + at) * a.C + t.c, at < t.p1 ? V : 0, x[k]);
            }
#pragma unroll
            for (int k = 0; k < B; ++k) {
                if (p + k * t.step < t.p1) cnt += V;
#pragma unroll
                for (int e = 0; e < V; ++e) s += x[k][e];
            }
            const float m = s / cnt;
            float q = 0.f;
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const bool in = p + k * t.step < t.p1;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = in ? x[k][e] - m : 0.f;
                    q = __builtin_fmaf(d, d, q);
                }
            }
            const float all = n + cnt, d = m - mean, f = cnt / all;
            m2 += q + d * d * n * f;
            mean += d * f;
            n = all;
        }
    // the group's part: its mean as a difference to one thread's, so that nothing is lost far from 0
    const float all = t.p1 > t.p0 ? (float)((t.p1 - t.p0) * t.run * V) : 0.f;
    __syncthreads();
    lds[threadIdx.x] = mean;
    __syncthreads();
    const float ref = lds[(int)threadIdx.x % a.vb - (t.idle ? 0 : t.lv)];
    const float d = n > 0.f ? mean - ref : 0.f;
    const float sum_d = t.sum(a, n * d, lds), off = all > 0.f ? sum_d / all : 0.f;
    const float sq = t.sum(a, n > 0.f ? m2 + n * (d - off) * (d - off) : 0.f, lds);
    if (!t.idle && t.po == 0 && t.lv == 0)
        *reinterpret_cast<f32x4 *>(a.part + 4 * t.entry) = f32x4{all, ref + off, sq, 0.f};
}

__device__ __forceinline__ int64_t length_of(const NormArgs &a, int64_t row) {
    if (!a.lengths) return a.S;
    const int64_t l = a.lengths[row];
    return l < 0 ? 0 : (l < a.S ? l : a.S);
}

// v summed over the N threads (a wave, or the workgroup) of one (row, group), in a fixed order
template <int N>
__device__ __forceinline__ double join_sum(double v) {
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (N > 64) {
        __shared__ double sums[N / 64];
        __syncthreads();
        if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = v;
        __syncthreads();
        v = 0.0;
#pragma unroll
        for (int k = 0; k < N / 64; ++k) v += sums[k];
    }
    return v;
}

// N threads a (row, group): stats <- mean, 1/std.
template <int N>
__global__ __launch_bounds__(kThreads) void seq_join_kernel(const NormArgs a) {
    const int64_t rg = (int64_t)blockIdx.x * (kThreads / N) + threadIdx.x / N;
    if (rg >= a.n * a.G) return;
    const int lane = threadIdx.x % N, total = a.nslice * a.pieces;
    const float *part = a.part + 4 * rg * total;
    double n = 0.0, s = 0.0, q = 0.0;
    for (int i = lane; i < total; i += N) {
        const f32x4 p = *reinterpret_cast<const f32x4 *>(part + 4 * i);
        n += (double)p[0];
        s += (double)p[0] * (double)p[1];
    }
    n = join_sum<N>(n);
    s = join_sum<N>(s);
    const double mean = n > 0.0 ? s / n : 0.0;
    for (int i = lane; i < total; i += N) {
        const f32x4 p = *reinterpret_cast<const f32x4 *>(part + 4 * i);
        const double d = (double)p[1] - mean;
        q += (double)p[2] + (double)p[0] * d * d;
    }
    q = join_sum<N>(q);
    const double var = n > 0.0 ? q / n : 0.0;
    if (lane == 0) {
        a.stats[4 * rg] = (float)mean;
        a.stats[4 * rg + 1] = (float)(1.0 / sqrt(var + (double)a.eps));
    }
}

template <bool BF16, int V, bool GATE>
__global__ __launch_bounds__(kThreads) void seq_fwd_kernel(const NormArgs a) {
    const Lane<V> t(a, true);
    if (t.idle) return;
    const float *st = a.stats + 4 * (t.row * a.G + t.c / a.D);
    const float mean = st[0], r = st[1];
    float w[V], b[V];
    load_w<V, true>(a.w, t.c, V, 1.f, w);
    load_w<V, true>(a.b, t.c, V, 0.f, b);
    for (int64_t p = t.p0 + t.po; p < t.p1; p += kAhead * t.step) {
        float x[kAhead][V], z[GATE ? kAhead : 1][V];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t q = p + k * t.step, at = (t.row * a.S + q) * a.C + t.c;
            const int live = q < t.p1 && q < t.len ? V : 0;
            load<BF16, V, true>(a.x, at, live, x[k]);
            if constexpr (GATE) load<BF16, V, true>(a.z, at, live, z[k]);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t q = p + k * t.step, at = (t.row * a.S + q) * a.C + t.c;
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float u = __builtin_fmaf((x[k][e] - mean) * r, w[e], b[e]);
                if constexpr (GATE) y[e] = u * act<BF16>(z[k][e], a.silu);
                else y[e] = act<BF16>(u, a.silu);
                if (q >= t.len) y[e] = 0.f;
            }
            store<BF16, V, true>(a.y, at, q < t.p1 ? V : 0, y, a.past);
        }
    }
}

// du of V values; with a gate z becomes dz, x becomes xh
template <bool BF16, int V, bool GATE>
__device__ __forceinline__ void seq_du(const NormArgs &a, float mean, float r, const float (&w)[V], const float (&b)[V],
                                       float (&x)[V], float (&z)[V], float (&d)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float xh = (x[e] - mean) * r, u = __builtin_fmaf(xh, w[e], b[e]);
        float v, sl;
        act2<BF16>(GATE ? z[e] : u, a.silu, v, sl);
        if constexpr (GATE) z[e] = d[e] * u * sl;
        d[e] = GATE ? d[e] * v : d[e] * sl;
        x[e] = xh;
    }
}

// Sums of du xh and du of every channel, chan [gridDim.x][2][C], and of d and d xh of a group's part of a slice,
// part [n, G, nslice, pieces, 4]. A workgroup takes `sweep` slices, one after another
template <bool BF16, int V, bool GATE>
__global__ __launch_bounds__(kThreads) void seq_sums_kernel(const NormArgs a) {
    __shared__ f32x2 lds[kThreads];
    __shared__ float rows[2 * V][kThreads];
    Lane<V> t(a);
    float w[V], b[V], dw[V], db[V];
    load_w<V, true>(a.w, t.c, t.idle ? 0 : V, 1.f, w);
    load_w<V, true>(a.b, t.c, t.idle ? 0 : V, 0.f, b);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[e] = db[e] = 0.f;
    const unsigned total = (unsigned)(a.n * a.nslice), first = blockIdx.x * (unsigned)a.sweep;
    for (unsigned id = first; id < total && id < first + (unsigned)a.sweep; ++id) {
        t.take(a, id, false);
        float sw[V], sb[V];  // of this slice
#pragma unroll
        for (int e = 0; e < V; ++e) sw[e] = sb[e] = 0.f;
        if (!t.idle) {
            const float *st = a.stats + 4 * (t.row * a.G + t.c / a.D);
            const float mean = st[0], r = st[1];
            for (int64_t p = t.p0 + t.po; p < t.p1; p += kAhead * t.step) {
                float x[kAhead][V], z[kAhead][V], d[kAhead][V];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int64_t q = p + k * t.step, at = (t.row * a.S + q) * a.C + t.c;
                    const int live = q < t.p1 ? V : 0;
                    load<BF16, V, true>(a.x, at, live, x[k]);
                    load<BF16, V, true>(a.dy, at, live, d[k]);
                    if constexpr (GATE) load<BF16, V, true>(a.z, at, live, z[k]);
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    seq_du<BF16, V, GATE>(a, mean, r, w, b, x[k], z[k], d[k]);
                    if (p + k * t.step < t.p1) {
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            sw[e] = __builtin_fmaf(d[k][e], x[k][e], sw[e]);
                            sb[e] += d[k][e];
                        }
                    }
                }
            }
        }
        f32x2 s = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s[0] = __builtin_fmaf(w[e], sb[e], s[0]);
            s[1] = __builtin_fmaf(w[e], sw[e], s[1]);
            dw[e] += sw[e];
            db[e] += sb[e];
        }
        s = t.sum(a, s, lds);
        if (!t.idle && t.po == 0 && t.lv == 0) *reinterpret_cast<f32x2 *>(a.part + 4 * t.entry) = s;
    }
    if (a.chan) {
        join_rows<V>(dw, db, t.po, a.pg, a.vb, rows);
        if (!t.idle && t.po == 0) {
            float *o = a.chan + (int64_t)blockIdx.x * 2 * a.C + t.c;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                o[e] = dw[e];
                o[a.C + e] = db[e];
            }
        }
    }
}

// likewise: stats <- means of d and d xh
template <int N>
__global__ __launch_bounds__(kThreads) void seq_join_sums_kernel(const NormArgs a) {
    const int64_t rg = (int64_t)blockIdx.x * (kThreads / N) + threadIdx.x / N;
    if (rg >= a.n * a.G) return;
    const int lane = threadIdx.x % N, total = a.nslice * a.pieces;
    const float *part = a.part + 4 * rg * total;
    double sa = 0.0, sb = 0.0;
    for (int i = lane; i < total; i += N) {
        sa += (double)part[4 * i];
        sb += (double)part[4 * i + 1];
    }
    sa = join_sum<N>(sa);
    sb = join_sum<N>(sb);
    const double n = (double)length_of(a, rg / a.G) * a.D;
    if (lane == 0) {
        a.stats[4 * rg + 2] = n > 0.0 ? (float)(sa / n) : 0.f;
        a.stats[4 * rg + 3] = n > 0.0 ? (float)(sb / n) : 0.f;
    }
}

template <bool BF16, int V, bool GATE>
__global__ __launch_bounds__(kThreads) void seq_bwd_kernel(const NormArgs a) {
    const Lane<V> t(a, true);
    if (t.idle) return;
    const float *st = a.stats + 4 * (t.row * a.G + t.c / a.D);
    const float mean = st[0], r = st[1], ma = st[2], mb = st[3];
    float w[V], b[V];
    load_w<V, true>(a.w, t.c, V, 1.f, w);
    load_w<V, true>(a.b, t.c, V, 0.f, b);
    for (int64_t p = t.p0 + t.po; p < t.p1; p += kAhead * t.step) {
        float x[kAhead][V], z[kAhead][V], d[kAhead][V];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t q = p + k * t.step, at = (t.row * a.S + q) * a.C + t.c;
            const int live = q < t.p1 && q < t.len ? V : 0;
            load<BF16, V, true>(a.x, at, live, x[k]);
            load<BF16, V, true>(a.dy, at, live, d[k]);
            if constexpr (GATE) load<BF16, V, true>(a.z, at, live, z[k]);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t q = p + k * t.step, at = (t.row * a.S + q) * a.C + t.c;
            seq_du<BF16, V, GATE>(a, mean, r, w, b, x[k], z[k], d[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                d[k][e] = q < t.len ? r * (d[k][e] * w[e] - ma - x[k][e] * mb) : 0.f;
                if constexpr (GATE) z[k][e] = q < t.len ? z[k][e] : 0.f;
            }
            store<BF16, V, true>(a.dx, at, q < t.p1 ? V : 0, d[k], a.past);
            if constexpr (GATE) store<BF16, V, true>(a.dz, at, q < t.p1 ? V : 0, z[k], a.past);
        }
    }
}

// dw, db <- sums over the partials [rows][2][C]: 32 of the 2 C columns a workgroup, 32 runs of
// rows, eight loads of each in flight (with 4 runs and one load this took longer than the
// gradients themselves: 300 us for 2048 rows of 2 x 2048)
constexpr int kSumCols = 32, kSumRuns = 32;

__global__ __launch_bounds__(kSumCols * kSumRuns) void channel_sums_kernel(const float *part, int64_t rows, int C,
                                                                            float *dw, float *db) {
    __shared__ double sums[kSumRuns][kSumCols];
    const int col = threadIdx.x % kSumCols, run = threadIdx.x / kSumCols;
    const int64_t i = (int64_t)blockIdx.x * kSumCols + col, width = 2 * (int64_t)C;
    double s = 0.0;
    if (i < width)
        for (int64_t r = run; r < rows; r += 8 * kSumRuns) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = r + k * kSumRuns < rows ? part[(r + k * kSumRuns) * width + i] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += (double)v[k];
        }
    sums[run][col] = s;
    __syncthreads();
    for (int n = kSumRuns / 2; n > 0; n >>= 1) {
        if (run < n) sums[run][col] += sums[run + n][col];
        __syncthreads();
    }
    if (run == 0 && i < width) {
        if (i < C) {
            if (dw) dw[i] = (float)sums[0][col];
        } else if (db) {
            db[i - C] = (float)sums[0][col];
        }
    }
}

// ------------------------------------------------------------------ launch ---
struct NormPlan {
    bool token;
    int L, CH;            // tokens
    int64_t rows_wg, gx;  // tokens: rows of a workgroup, workgroups along the rows
    int gy, pass;         // tokens: workgroups along the groups, rows of a pass
    int64_t slice;        // sequences
    int64_t nslice;
    int vb, pg, pieces, vblocks, V;
    int64_t sweep, sweeps;  // slices of a workgroup of the gradients' sums, and how many such workgroups (times vblocks)
    size_t part_bytes, chan_bytes, stats_bytes, total;
};

size_t up(size_t n) { return (n + 255) & ~size_t(255); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

NormPlan make_plan(const m3_norm_shape &s, bool lengths, bool bwd) {
    NormPlan p{};
    const int V = s.io_dtype == M3_BF16 ? 8 : 4;
    const int64_t C = s.channels, G = s.groups, D = C / G;
    p.token = s.positions == 1 && !lengths && D <= 4 * 64 * V;
    if (p.token) {
        const int64_t vecs = ceil_div(D, V);
        p.L = 1;
        while (p.L < vecs && p.L < 64) p.L *= 2;
        p.CH = vecs <= 64 ? 1 : (vecs <= 128 ? 2 : 4);
        const int slots = kThreads / p.L;
        p.pass = G < slots ? (int)(slots / G) : 1;
        p.gy = G < slots ? 1 : (int)ceil_div(G, slots);
        // Rows of a workgroup: enough passes to pay for the weights (and the partial sums), few
        // enough that the workgroups fill the 256 CUs several times over
        int64_t passes = ceil_div(s.rows, (int64_t)p.pass * 4096) * p.gy;
        const int64_t most = bwd ? 64 : 16;
        passes = passes < 1 ? 1 : (passes > most ? most : passes);
        // A workgroup's partial sums are 8 bytes a channel: two workgroups a CU (b4 L4096 in 64 groups of 64: 137 us, with four
        // 146, with one 205)
        const int64_t wgs = p.gy < 512 ? 512 / p.gy : 1;
        if (bwd && ceil_div(s.rows, p.pass * passes) > wgs) passes = ceil_div(s.rows, p.pass * wgs);
        if (bwd && passes > kChain) passes = kChain;
        if (!bwd && ceil_div(s.rows, p.pass * passes) > (1 << 20)) passes = ceil_div(s.rows, (int64_t)p.pass << 20);
        p.rows_wg = p.pass * passes;
        p.gx = ceil_div(s.rows, p.rows_wg);
        if (bwd) p.total = p.chan_bytes = up((size_t)p.gx * 2 * C * 4);
        return p;
    }
    p.V = D % V == 0 ? V : 1;
    const int64_t cv = C / p.V, dv = D / p.V;
    if (dv <= kThreads) {
        const int64_t whole = kThreads / dv * dv;
        p.vb = (int)(cv < whole ? cv : whole);
        p.pieces = 1;
        p.vblocks = (int)ceil_div(cv, p.vb);
    } else {
        p.vb = kThreads;
        p.pieces = (int)ceil_div(dv, kThreads);
        p.vblocks = (int)(G * p.pieces);
    }
    p.pg = kThreads / p.vb;
    // Slices: two workgroups a CU, of eight positions a thread at least. More slices are more partial sums (gradients of
    // b8 L4096 of 4096 channels with a gate: 455 us, with eight a CU 560, with one 503; b1 of 320 channels 40, 37, 50)
    int64_t n = ceil_div(512, (s.rows > 0 ? s.rows : 1) * p.vblocks);
    const int64_t most = ceil_div(s.positions, 8 * p.pg);
    n = n > most ? most : n;
    n = n < 1 ? 1 : n;
    p.slice = ceil_div(ceil_div(s.positions, n), p.pg) * p.pg;
    if (p.slice > kChain * p.pg) p.slice = kChain * p.pg;
    if (p.slice < 1) p.slice = 1;
    p.nslice = s.positions > 0 ? ceil_div(s.positions, p.slice) : 1;
    // A workgroup that sums gradients takes several short slices, so that about a thousand workgroups (what the CUs have at
    // once) hold all, as long as a thread's additions stay a chain: the partial sums are at most 32 MB, or a sixteenth of x
    // (a workgroup a slice and a partial sum a thread: 100000 rows of 4 positions of 64 channels 44 ms and 1.6 GB, now 1.2 ms
    // and 4 MB; one group of 4096 channels for each of 32768 tokens 1657 us and 1.1 GB, now 765 and 18 MB)
    const int64_t slices = s.rows * p.nslice, chain = ceil_div(p.slice, p.pg);
    p.sweep = slices * p.vblocks / 1024;
    if (p.sweep > kChain / chain) p.sweep = kChain / chain;
    if (p.sweep < 1) p.sweep = 1;
    p.sweeps = ceil_div(slices, p.sweep);
    p.part_bytes = up((size_t)slices * G * p.pieces * 16);
    if (bwd) p.chan_bytes = up((size_t)p.sweeps * 8 * C);
    p.stats_bytes = up((size_t)s.rows * G * 16);
    p.total = p.part_bytes + p.chan_bytes + p.stats_bytes;
    return p;
}

bool al16(const void *p) { return (((uintptr_t)p) & 15u) == 0; }

m3_status norm_check(const m3_norm_shape *s) {
    if (!s) return M3_ERR_INVALID_ARG;
    if (s->rows < 0 || s->positions < 0 || s->channels < 1 || s->groups < 1 || s->channels % s->groups != 0)
        return M3_ERR_INVALID_ARG;
    if (s->io_dtype != M3_F32 && s->io_dtype != M3_BF16) return M3_ERR_INVALID_ARG;
    if (s->activation != M3_ACT_NONE && s->activation != M3_ACT_SILU) return M3_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f) || !isfinite(s->eps) || s->flags) return M3_ERR_INVALID_ARG;
    if (s->channels > (1 << 20) || s->rows > (1LL << 31) || s->positions > (1LL << 40) ||
        (s->positions > 0 && s->rows > (1LL << 40) / s->positions))
        return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

// the launches of one plan stay within a grid
m3_status norm_plan(const m3_norm_shape *s, bool lengths, bool bwd, NormPlan *p) {
    const m3_status st = norm_check(s);
    if (st != M3_OK) return st;
    *p = make_plan(*s, lengths, bwd);
    const int64_t x = p->token ? p->gx : s->rows * p->nslice;
    const int64_t y = p->token ? p->gy : p->vblocks;
    if (x > kMaxGrid || y > 65535 || (!p->token && s->rows * s->groups > 4 * kMaxGrid))
        return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

template <bool BF16, int L, int CH, bool VEC>
void launch_token(const NormArgs &a, const NormPlan &p, bool bwd, hipStream_t s) {
    const dim3 g((unsigned)p.gx, (unsigned)p.gy), t(kThreads);
    if (bwd) {
        if (a.z) hipLaunchKernelGGL((token_bwd_kernel<BF16, L, CH, VEC, true>), g, t, 0, s, a);
        else hipLaunchKernelGGL((token_bwd_kernel<BF16, L, CH, VEC, false>), g, t, 0, s, a);
    } else {
        if (a.z) hipLaunchKernelGGL((token_fwd_kernel<BF16, L, CH, VEC, true>), g, t, 0, s, a);
        else hipLaunchKernelGGL((token_fwd_kernel<BF16, L, CH, VEC, false>), g, t, 0, s, a);
    }
}

template <bool BF16, bool VEC>
hipError_t launch_token_dims(const NormArgs &a, const NormPlan &p, bool bwd, hipStream_t s) {
    switch (p.L * p.CH) {
        case 1: launch_token<BF16, 1, 1, VEC>(a, p, bwd, s); break;
        case 2: launch_token<BF16, 2, 1, VEC>(a, p, bwd, s); break;
        case 4: launch_token<BF16, 4, 1, VEC>(a, p, bwd, s); break;
        case 8: launch_token<BF16, 8, 1, VEC>(a, p, bwd, s); break;
        case 16: launch_token<BF16, 16, 1, VEC>(a, p, bwd, s); break;
        case 32: launch_token<BF16, 32, 1, VEC>(a, p, bwd, s); break;
        case 64: launch_token<BF16, 64, 1, VEC>(a, p, bwd, s); break;
        case 128: launch_token<BF16, 64, 2, VEC>(a, p, bwd, s); break;
        case 256: launch_token<BF16, 64, 4, VEC>(a, p, bwd, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch_tokens(const NormArgs &a, const NormPlan &p, bool bwd, hipStream_t s) {
    return a.D % (BF16 ? 8 : 4) == 0 ? launch_token_dims<BF16, true>(a, p, bwd, s)
                                     : launch_token_dims<BF16, false>(a, p, bwd, s);
}

hipError_t launch_channel_sums(const NormArgs &a, int64_t rows, hipStream_t s) {
    if (!a.dw && !a.db) return hipSuccess;
    hipLaunchKernelGGL(channel_sums_kernel, dim3((unsigned)ceil_div(2 * (int64_t)a.C, kSumCols)),
                       dim3(kSumCols * kSumRuns), 0, s, a.chan,
                       rows, a.C, a.dw, a.db);
    return hipGetLastError();
}

template <bool BF16, int V>
hipError_t launch_seq(const NormArgs &a, const NormPlan &p, bool bwd, hipStream_t s) {
    const dim3 g((unsigned)(a.n * a.nslice), (unsigned)p.vblocks), gs((unsigned)p.sweeps, (unsigned)p.vblocks), t(kThreads);
    // (a workgroup a (row, group) where the partial sums are more than a wave takes at once)
    const bool many = a.nslice * a.pieces > 64 && a.n * a.G <= kMaxGrid;
    const dim3 j((unsigned)(many ? a.n * a.G : ceil_div(a.n * a.G, kThreads / 64)));
    hipError_t e;
    hipLaunchKernelGGL((seq_stats_kernel<BF16, V>), g, t, 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (many) hipLaunchKernelGGL(seq_join_kernel<kThreads>, j, t, 0, s, a);
    else hipLaunchKernelGGL(seq_join_kernel<64>, j, t, 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (!bwd) {
        if (a.z) hipLaunchKernelGGL((seq_fwd_kernel<BF16, V, true>), g, t, 0, s, a);
        else hipLaunchKernelGGL((seq_fwd_kernel<BF16, V, false>), g, t, 0, s, a);
        return hipGetLastError();
    }
    if (a.z) hipLaunchKernelGGL((seq_sums_kernel<BF16, V, true>), gs, t, 0, s, a);
    else hipLaunchKernelGGL((seq_sums_kernel<BF16, V, false>), gs, t, 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (many) hipLaunchKernelGGL(seq_join_sums_kernel<kThreads>, j, t, 0, s, a);
    else hipLaunchKernelGGL(seq_join_sums_kernel<64>, j, t, 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.z) hipLaunchKernelGGL((seq_bwd_kernel<BF16, V, true>), g, t, 0, s, a);
    else hipLaunchKernelGGL((seq_bwd_kernel<BF16, V, false>), g, t, 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    return launch_channel_sums(a, p.sweeps, s);
}

m3_status run(const m3_norm_shape &s, const NormPlan &p, NormArgs &a, bool bwd, void *workspace, hipStream_t hs) {
    a.n = s.rows; a.S = s.positions; a.C = (int)s.channels; a.G = (int)s.groups; a.D = a.C / a.G;
    a.eps = s.eps; a.silu = s.activation == M3_ACT_SILU;
    // x, y and the gate, dy, dx and the gate's
    const int64_t bytes = a.n * a.S * a.C * (s.io_dtype == M3_BF16 ? 2 : 4) * ((bwd ? 3 : 2) + (a.z ? (bwd ? 2 : 1) : 0));
    a.past = bytes > kLastCache;
    a.rows_wg = p.rows_wg; a.slice = p.slice; a.nslice = (int)p.nslice; a.vb = p.vb; a.pg = p.pg; a.pieces = p.pieces;
    a.sweep = (int)p.sweep;
    char *ws = static_cast<char *>(workspace);
    a.part = reinterpret_cast<float *>(ws);
    a.stats = reinterpret_cast<float *>(ws + p.part_bytes);
    a.chan = bwd && (a.dw || a.db) ? reinterpret_cast<float *>(ws + p.part_bytes + p.stats_bytes) : nullptr;
    const bool bf16 = s.io_dtype == M3_BF16;
    hipError_t e = hipSuccess;
    if (a.n * a.S == 0) {
        if (bwd) e = launch_channel_sums(a, 0, hs);  // zeros
    } else if (p.token) {
        e = bf16 ? launch_tokens<true>(a, p, bwd, hs) : launch_tokens<false>(a, p, bwd, hs);
        if (bwd && e == hipSuccess) e = launch_channel_sums(a, p.gx, hs);
    } else if (bf16) {
        e = p.V > 1 ? launch_seq<true, 8>(a, p, bwd, hs) : launch_seq<true, 1>(a, p, bwd, hs);
    } else {
        e = p.V > 1 ? launch_seq<false, 4>(a, p, bwd, hs) : launch_seq<false, 1>(a, p, bwd, hs);
    }
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

}  // namespace
}  // namespace m3i

using namespace m3i;

extern "C" {

size_t m3_group_norm_workspace_bytes(const m3_norm_shape *shape, int lengths) {
    NormPlan p;
    return norm_plan(shape, lengths != 0, false, &p) == M3_OK ? p.total : 0;
}

size_t m3_group_norm_bwd_workspace_bytes(const m3_norm_shape *shape, int lengths) {
    NormPlan p;
    return norm_plan(shape, lengths != 0, true, &p) == M3_OK ? p.total : 0;
}

m3_status m3_group_norm_fwd(const m3_norm_shape *shape, const m3_norm_io *io, void *workspace, size_t ws_bytes,
                            void *stream) {
    m3_status st = norm_check(shape);
    if (st != M3_OK) return st;
    if (!io) return M3_ERR_INVALID_ARG;
    NormPlan p;
    if ((st = norm_plan(shape, io->lengths != nullptr, false, &p)) != M3_OK) return st;
    if (shape->rows * shape->positions > 0 && (!io->x || !io->y)) return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->x, io->z, io->weight, io->bias, io->lengths, io->y, workspace};
    for (const void *q : ptrs)
        if (!al16(q)) return M3_ERR_MISALIGNED;
    const size_t need = p.total;
    if (need && (!workspace || ws_bytes < need)) return M3_ERR_WORKSPACE_TOO_SMALL;
    // (y may be x or z: an element is read before it is written, by the same thread)
    if (clash({io->y}, {io->weight, io->bias, io->lengths, workspace}) ||
        (need && clash({workspace}, {io->x, io->z, io->weight, io->bias, io->lengths})))
        return M3_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = io->x; a.z = io->z; a.w = io->weight; a.b = io->bias; a.lengths = io->lengths; a.y = io->y;
    return run(*shape, p, a, false, workspace, reinterpret_cast<hipStream_t>(stream));
}

m3_status m3_group_norm_bwd(const m3_norm_shape *shape, const m3_norm_io *io, const m3_norm_grads *gr, void *workspace,
                            size_t ws_bytes, void *stream) {
    m3_status st = norm_check(shape);
    if (st != M3_OK) return st;
    if (!io || !gr) return M3_ERR_INVALID_ARG;
    NormPlan p;
    if ((st = norm_plan(shape, io->lengths != nullptr, true, &p)) != M3_OK) return st;
    if (shape->rows * shape->positions > 0 &&
        (!io->x || !gr->dy || !gr->dx || (io->z == nullptr) != (gr->dz == nullptr)))
        return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->x, io->z, io->weight, io->bias, io->lengths, gr->dy, gr->dx, gr->dz,
                          gr->dweight, gr->dbias, workspace};
    for (const void *q : ptrs)
        if (!al16(q)) return M3_ERR_MISALIGNED;
    const size_t need = p.total;
    if (need && (!workspace || ws_bytes < need)) return M3_ERR_WORKSPACE_TOO_SMALL;
    // (likewise dx may be x or dy, and dz may be z)
    if (clash({gr->dx, gr->dz, gr->dweight, gr->dbias}, {io->weight, io->bias, io->lengths, workspace}) ||
        clash({gr->dweight, gr->dbias}, {io->x, io->z, gr->dy}) ||
        (gr->dx != io->x && gr->dx != gr->dy && clash({gr->dx}, {io->z})) ||
        (gr->dz != io->z && clash({gr->dz}, {io->x, gr->dy})) ||
        (need && clash({workspace}, {io->x, io->z, io->weight, io->bias, io->lengths, gr->dy})))
        return M3_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = io->x; a.z = io->z; a.w = io->weight; a.b = io->bias; a.lengths = io->lengths;
    a.dy = gr->dy; a.dx = gr->dx; a.dz = gr->dz; a.dw = gr->dweight; a.db = gr->dbias;
    return run(*shape, p, a, true, workspace, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
