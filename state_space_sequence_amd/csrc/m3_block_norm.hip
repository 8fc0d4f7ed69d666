// The norms around a block with its gate, scale and residual: forward and gradients (gfx950).
//
//   v = x rx w,  rx = 1/sqrt(mean x^2 + eps) (or v = x);  R = alpha r + sc act(z) v;  y = R rR wp
//   dR' = dR + rR (q - R rR mean(q R rR)),  q = dy wp;  dr = alpha dR';  dz = dR' sc v act'(z)
//   g = dR' sc act(z) w;  dx = rx (g - x rx mean(g x rx));  dwp = sum dy R rR;  dsc = sum dR' act(z) v;  dw = sum dR' sc act(z) x rx
//
// Bound by HBM: every tensor is read or written once. The lanes of a row (16 to 1024 of them) hold it in registers, 4 to
// 16 values each; its sums go across a wave by DPP and row swaps, across waves by LDS. A lane keeps its channels from row
// to row, so weights and their gradients stay in registers too, and the next row is loaded while this one is summed. bf16, all parts:
// b8 L4096 of 2048 channels with an fp32 stream 161 us (5.8 TB/s), gradients of b4 L4096 of 4096 191 us (5.6 TB/s).
#include <math.h>

#include "m3_block_norm.h"
#include "m3_internal.h"

namespace m3i {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kChainRows = 256;  // rows whose weight gradients a thread adds up in fp32
constexpr int64_t kMaxThreads = 0xffffffff;  // of a launch
constexpr int64_t kLastCache = 256 << 20;

struct BlockArgs {
    const void *x, *z, *r;
    const float *w, *wp, *sc;
    void *R, *y;
    const void *dy, *dR;
    void *dx, *dz, *dr;
    float *part;   // [workgroups][3][C]: sums of dw, dwp, dsc
    float *stats;  // (wide rows) [n][kStats]
    int64_t n;
    int C;
    float eps, alpha;
    int act;
    bool post, pre, sums;
    bool past;  // stores past the caches
    int rows;   // (wide rows) rows of a workgroup that sums columns
};

// V consecutive values of one dtype as they lie in memory
template <bool BF16, int V>
struct Packed {
    static constexpr int W = BF16 ? V / 2 : V;
    unsigned w[W];
};

// N words at an address that is aligned to the values alone (rows of odd widths): one access all the same
template <bool BF16, int N, bool WHOLE>
struct Words {
    typedef unsigned any __attribute__((ext_vector_type(N), aligned(WHOLE ? 4 * N : BF16 ? 2 : 4)));
};

// `live` of V values: all of them in one access of 8 or 16 bytes, fewer one by one. WHOLE: rows of a whole number of aligned
// accesses, live is 0 or V (the question costs the gradients of b4 L4096 of 4096 channels 196 -> 247 us)
template <bool BF16, int V, bool WHOLE>
__device__ __forceinline__ void load(const void *p, int64_t i, int live, Packed<BF16, V> &o) {
    constexpr int W = Packed<BF16, V>::W;
#pragma unroll
    for (int e = 0; e < W; ++e) o.w[e] = 0;
    const char *at = static_cast<const char *>(p) + i * (BF16 ? 2 : 4);
    if (WHOLE ? live > 0 : live == V) {
        const auto v = __builtin_nontemporal_load(reinterpret_cast<const typename Words<BF16, W, WHOLE>::any *>(at));
#pragma unroll
        for (int e = 0; e < W; ++e) o.w[e] = v[e];
    } else if (!WHOLE && live > 0) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < live) {
                if constexpr (BF16) o.w[e / 2] |= (unsigned)reinterpret_cast<const uint16_t *>(at)[e] << (e % 2 * 16);
                else o.w[e] = reinterpret_cast<const unsigned *>(at)[e];
            }
    }
}
template <bool BF16, int V>
__device__ __forceinline__ void unpack(const Packed<BF16, V> &o, float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if constexpr (!BF16) x[e] = __uint_as_float(o.w[e]);
        else x[e] = __uint_as_float(e % 2 ? o.w[e / 2] & 0xffff0000u : o.w[e / 2] << 16);
    }
}
// Past the caches: forwards where the tensors of the call do not fit them (ASK, past), with gradients always (the question
// changes nothing for b4 L4096 of 4096 channels, 190 us and 189, in fp32 of half the tokens 187 and 188)
template <bool BF16, int V, bool WHOLE, bool ASK>
__device__ __forceinline__ void store(void *p, int64_t i, int live, const float (&x)[V], bool past) {
    constexpr int W = Packed<BF16, V>::W;
    char *at = static_cast<char *>(p) + i * (BF16 ? 2 : 4);
    if (WHOLE ? live > 0 : live == V) {
        typedef typename Words<BF16, W, WHOLE>::any vec;
        vec v;
#pragma unroll
        for (int e = 0; e < W; ++e) {
            if constexpr (BF16) v[e] = __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x[2 * e], x[2 * e + 1]}), bf16x2));
            else v[e] = __float_as_uint(x[e]);
        }
        vec *to = reinterpret_cast<vec *>(at);
        if constexpr (!ASK) {
            __builtin_nontemporal_store(v, to);
        } else if (past) {
            asm volatile("");  // (two equal stores but for their hint would become one)
            __builtin_nontemporal_store(v, to);
            asm volatile("");
        } else {
            *to = v;
        }
    } else if (!WHOLE && live > 0) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < live) {
                if constexpr (BF16) reinterpret_cast<__bf16 *>(at)[e] = (__bf16)x[e];
                else reinterpret_cast<float *>(at)[e] = x[e];
            }
    }
}

// e^-z. ROUGH, for outputs in bf16: the hardware exponential of a rounded argument, off by |z| 2^-23, far below their rounding (with
// gradients the terms of the weights' fp32 sums are off by as much). Forwards beside an fp32 stream, which takes the gate as it is, a z of
// bf16's 8 bits times the upper 16 of log2(e) is an exact argument, and the lower bits are a factor: the gate is off by 3.5 * 2^-24 at
// most, in place of 57, in the same time (b8 L4096 of 2048 channels 160 us; expf as for fp32 blocks 4% more)
template <bool BF, bool ROUGH>
__device__ __forceinline__ float neg_exp(float z) {
    if constexpr (ROUGH) return __builtin_amdgcn_exp2f(-1.4426950408889634f * z);
    else if constexpr (BF) return __builtin_amdgcn_exp2f(-0x1.715400p+0f * z) * __builtin_amdgcn_exp2f(-0x1.d94ae0p-18f * z);
    else return expf(-z);
}

// the gate's value, and its slope
template <bool BF, bool ROUGH>
__device__ __forceinline__ void gate(float z, int act, float &v, float &slope) {
    v = z;
    slope = 1.f;
    if (act != M3_ACT_NONE) {
        const float e = neg_exp<BF, ROUGH>(z);
        const float s = __builtin_amdgcn_rcpf(1.f + e), rest = (e > 0x1p126f ? 0x1p126f : e) * s;  // 1 - s
        if (act == M3_ACT_SILU) {
            v = z * s;
            slope = s * __builtin_fmaf(z, rest, 1.f);
        } else {
            v = s;
            slope = s * rest;
        }
    }
}

// `live` of V channels of a weight from c on, a multiple of V (none given: 1)
template <int V>
__device__ __forceinline__ void read_weight(const float *p, int c, int live, float (&w)[V]) {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = 1.f;
    if (!p) return;
    if (live == V) {
#pragma unroll
        for (int f = 0; f < V; f += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(p + c + f);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[f + e] = v[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < live) w[e] = p[c + e];
    }
}

// Where a thread is: LANES lanes a row, CH pieces of LANES * V channels
template <int LANES, int CH, int V>
struct Lanes {
    static constexpr int kThreads = LANES < 256 ? 256 : LANES, kRows = kThreads / LANES;
    int r;              // its row among those of a pass
    int c[CH], live[CH];  // first channel and channels of a piece
    __device__ __forceinline__ explicit Lanes(int C) {
        r = threadIdx.x / LANES;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            c[k] = (k * LANES + (int)threadIdx.x % LANES) * V;
            const int left = C - c[k];
            live[k] = left <= 0 ? 0 : (left < V ? left : V);
        }
    }
    __device__ __forceinline__ void weights(const float *p, int k, float (&w)[V]) const { read_weight<V>(p, c[k], live[k], w); }
    // N sums over the lanes of a row. `slot` alternates: a slow wave still reads the last one's
    template <int N>
    static __device__ __forceinline__ void sum(float (&s)[N], float (*lds)[kThreads / 64][4], int &slot) {
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] = group_sum<(LANES < 64 ? LANES : 64)>(s[j]);
        if constexpr (LANES > 64) {
            constexpr int W = LANES / 64;
            const int wave = threadIdx.x >> 6, first = wave / W * W;
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int j = 0; j < N; ++j) lds[slot][wave][j] = s[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < N; ++j) {
                s[j] = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) s[j] += lds[slot][first + w][j];
            }
            slot ^= 1;
        }
    }
};

// One of the three weights: in registers for all rows, or (rows of 1024 lanes with gradients) read for each row again, from
// the caches
template <int LANES, int CH, int V, bool KEEP>
struct Weight {
    const float *p;
    float w[KEEP ? CH : 1][V];
    __device__ __forceinline__ Weight(const Lanes<LANES, CH, V> &at, const float *from) : p(from) {
        if constexpr (KEEP)
#pragma unroll
            for (int k = 0; k < CH; ++k) at.weights(p, k, w[k]);
    }
    __device__ __forceinline__ void get(const Lanes<LANES, CH, V> &at, int k, float (&o)[V]) const {
        if constexpr (KEEP) {
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = w[k][e];
        } else {
            at.weights(p, k, o);
        }
    }
};

// BF: x, z, y in bf16; RF: the residual stream in bf16
template <bool BF, bool RF, int V, int LANES, int CH, bool WHOLE>
__global__ __launch_bounds__((Lanes<LANES, CH, V>::kThreads)) void fwd_kernel(const BlockArgs a) {
    using At = Lanes<LANES, CH, V>;
    __shared__ float lds[2][At::kThreads / 64][4];
    const At p(a.C);
    const Weight<LANES, CH, V, true> Kw(p, a.w), Kp(p, a.wp), Ks(p, a.sc);
    const float inv = 1.f / (float)a.C;
    Packed<BF, V> x[CH], z[CH];
    Packed<RF, V> r[CH];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int live = row < a.n ? p.live[k] : 0;
            load<BF, V, WHOLE>(a.x, row * a.C + p.c[k], live, x[k]);
            if (a.z) load<BF, V, WHOLE>(a.z, row * a.C + p.c[k], live, z[k]);
            if (a.r) load<RF, V, WHOLE>(a.r, row * a.C + p.c[k], live, r[k]);
        }
    };
    const int64_t step = (int64_t)gridDim.x * At::kRows;
    int slot = 0;
    fetch((int64_t)blockIdx.x * At::kRows + p.r);
    // (all rows of a workgroup's pass go round together: the barriers are theirs)
    for (int64_t pass = (int64_t)blockIdx.x * At::kRows; pass < a.n; pass += step) {
        const int64_t row = pass + p.r;
        float v[CH][V], R[CH][V];
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            unpack<BF, V>(x[k], v[k]);
            float zs[V], rs[V], w[V], sc[V];
            Kw.get(p, k, w);
            Ks.get(p, k, sc);
            unpack<BF, V>(z[k], zs);
            unpack<RF, V>(r[k], rs);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                R[k][e] = a.r ? a.alpha * rs[e] : 0.f;
                s[0] = __builtin_fmaf(v[k][e], v[k][e], s[0]);
                float on = sc[e] * w[e], slope;
                if (a.z) {
                    float act;
                    gate<BF, BF && RF>(zs[e], a.act, act, slope);
                    on *= act;
                }
                v[k][e] *= on;
            }
        }
        fetch(row + step);
        float rx = 1.f;
        if (a.post) {
            At::sum(s, lds, slot);
            rx = 1.f / sqrtf(s[0] * inv + a.eps);
        }
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                R[k][e] = __builtin_fmaf(v[k][e], rx, R[k][e]);
                s[0] = __builtin_fmaf(R[k][e], R[k][e], s[0]);
            }
        const bool here = row < a.n;
#pragma unroll
        for (int k = 0; k < CH; ++k)
            if (a.R) store<RF, V, WHOLE, true>(a.R, row * a.C + p.c[k], here ? p.live[k] : 0, R[k], a.past);
        if (a.pre) {
            At::sum(s, lds, slot);
            const float rR = 1.f / sqrtf(s[0] * inv + a.eps);
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                float wp[V];
                Kp.get(p, k, wp);
#pragma unroll
                for (int e = 0; e < V; ++e) R[k][e] *= rR * wp[e];
                store<BF, V, WHOLE, true>(a.y, row * a.C + p.c[k], here ? p.live[k] : 0, R[k], a.past);
            }
        }
    }
}

template <bool BF, bool RF, int V, int LANES, int CH, bool WHOLE>
__global__ __launch_bounds__((Lanes<LANES, CH, V>::kThreads)) void bwd_kernel(const BlockArgs a) {
    using At = Lanes<LANES, CH, V>;
    __shared__ float lds[2][At::kThreads / 64][4];
    const At p(a.C);
    float dw[CH][V], dwp[CH][V], dsc[CH][V];
    // (weights in registers and loads ahead where those allow it)
    constexpr bool AHEAD = LANES <= 512;
    const Weight<LANES, CH, V, AHEAD> Kw(p, a.w), Kp(p, a.wp), Ks(p, a.sc);
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[k][e] = dwp[k][e] = dsc[k][e] = 0.f;
    const float inv = 1.f / (float)a.C;
    Packed<BF, V> x[CH], z[CH], y[CH];  // y: dy
    Packed<RF, V> R[CH], D[CH];         // D: the gradient of R
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int live = row < a.n ? p.live[k] : 0;
            const int64_t at = row * a.C + p.c[k];
            load<BF, V, WHOLE>(a.x, at, live, x[k]);
            if (a.z) load<BF, V, WHOLE>(a.z, at, live, z[k]);
            if (a.pre) {
                load<RF, V, WHOLE>(a.R, at, live, R[k]);
                load<BF, V, WHOLE>(a.dy, at, live, y[k]);
            }
            if (a.dR) load<RF, V, WHOLE>(a.dR, at, live, D[k]);
        }
    };
    const int64_t step = (int64_t)gridDim.x * At::kRows;
    int slot = 0;
    if constexpr (AHEAD) fetch((int64_t)blockIdx.x * At::kRows + p.r);
    for (int64_t pass = (int64_t)blockIdx.x * At::kRows; pass < a.n; pass += step) {
        const int64_t row = pass + p.r;
        const bool here = row < a.n;
        if constexpr (!AHEAD) fetch(row);
        float xs[CH][V], zs[CH][V], d[CH][V], Rs[CH][V], q[CH][V];
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            unpack<BF, V>(x[k], xs[k]);
            unpack<BF, V>(z[k], zs[k]);
            unpack<BF, V>(y[k], q[k]);
            unpack<RF, V>(R[k], Rs[k]);
            unpack<RF, V>(D[k], d[k]);
            float wp[V];
            Kp.get(p, k, wp);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[0] = __builtin_fmaf(xs[k][e], xs[k][e], s[0]);
                if (!a.dR) d[k][e] = 0.f;
                if (a.pre) {
                    s[1] = __builtin_fmaf(Rs[k][e], Rs[k][e], s[1]);
                    s[2] = __builtin_fmaf(q[k][e] * wp[e], Rs[k][e], s[2]);
                }
            }
        }
        if constexpr (AHEAD) fetch(row + step);
        float rx = 1.f;
        if (a.post || a.pre) {
            At::sum(s, lds, slot);
            if (a.post) rx = 1.f / sqrtf(s[0] * inv + a.eps);
        }
        if (a.pre) {
            const float rR = 1.f / sqrtf(s[1] * inv + a.eps), mean = s[2] * inv * rR * rR;
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                float wp[V];
                Kp.get(p, k, wp);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float n = here ? Rs[k][e] * rR : 0.f;  // (rows behind the last: 1/sqrt(eps) may be infinite)
                    dwp[k][e] = __builtin_fmaf(q[k][e], n, dwp[k][e]);
                    d[k][e] += rR * (q[k][e] * wp[e] - Rs[k][e] * mean);
                }
            }
        }
        float t[1] = {0.f};
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int64_t at = row * a.C + p.c[k];
            const int live = here ? p.live[k] : 0;
            if (a.dr) {
                float o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] = a.alpha * d[k][e];
                store<RF, V, WHOLE, false>(a.dr, at, live, o, a.past);
            }
            float o[V], w[V], sc[V];
            Kw.get(p, k, w);
            Ks.get(p, k, sc);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!here) d[k][e] = 0.f;
                const float n = here ? xs[k][e] * rx : 0.f, v = n * w[e];
                xs[k][e] = n;
                float act = 1.f, slope = 0.f;
                if (a.z) {
                    gate<BF, BF>(zs[k][e], a.act, act, slope);
                    o[e] = d[k][e] * sc[e] * v * slope;
                }
                const float da = d[k][e] * act;
                dsc[k][e] = __builtin_fmaf(da, v, dsc[k][e]);
                d[k][e] = da * sc[e];
                dw[k][e] = __builtin_fmaf(d[k][e], n, dw[k][e]);
                d[k][e] *= w[e];
                t[0] = __builtin_fmaf(d[k][e], n, t[0]);
            }
            if (a.z) store<BF, V, WHOLE, false>(a.dz, at, live, o, a.past);
        }
        if (a.post) {
            At::sum(t, lds, slot);
            t[0] *= inv;
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            if (a.post)
#pragma unroll
                for (int e = 0; e < V; ++e) d[k][e] = rx * (d[k][e] - xs[k][e] * t[0]);
            store<BF, V, WHOLE, false>(a.dx, row * a.C + p.c[k], here ? p.live[k] : 0, d[k], a.past);
        }
    }
    if (!a.sums) return;
    // the sums of a workgroup's lanes of rows, in a fixed order, and in fp64: they are of up to kRows * kChainRows rows
    float *part = a.part + (int64_t)blockIdx.x * 3 * a.C;
    if constexpr (At::kRows > 1) {
        __shared__ float join[3][At::kThreads];
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                __syncthreads();
                join[0][threadIdx.x] = dw[k][e];
                join[1][threadIdx.x] = dwp[k][e];
                join[2][threadIdx.x] = dsc[k][e];
                __syncthreads();
                for (int i = threadIdx.x; i < 3 * LANES; i += At::kThreads) {
                    const int j = i / LANES, l = i % LANES, c = (k * LANES + l) * V + e;
                    double t = 0.;
                    for (int r = 0; r < At::kRows; ++r) t += join[j][r * LANES + l];
                    if (c < a.C) part[(int64_t)j * a.C + c] = (float)t;
                }
            }
    } else {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < p.live[k]) {
                    part[p.c[k] + e] = dw[k][e];
                    part[a.C + p.c[k] + e] = dwp[k][e];
                    part[2 * a.C + p.c[k] + e] = dsc[k][e];
                }
    }
}

// --------------------------------------------------------------- wide rows ---
// Rows that the registers do not hold: a workgroup goes over its row two or three times, V channels a thread, from the
// caches after the first; gradients of weights by columns, from the rows' factors and means, in a launch of their own. Gradients of
// 4096 bf16 rows of 16384 channels 530 us, bound by its passes (element by element 2140).
constexpr int kWide = 1024;
constexpr int kStats = 4;  // a row's rx, rR, mean(q R rR) rR, mean(g x rx)

// N sums over a workgroup, the same in all threads
template <int N>
__device__ __forceinline__ void wide_sum(float (&s)[N], float (*lds)[N]) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        s[j] = wave_sum(s[j]);
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6][j] = s[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        s[j] = 0.f;
        for (int w = 0; w < kWide / 64; ++w) s[j] += lds[w][j];
    }
}

template <bool BF, int V>
__device__ __forceinline__ void wide_read(const void *p, int64_t i, int live, float (&x)[V]) {
    Packed<BF, V> o;
    load<BF, V, false>(p, i, live, o);
    unpack<BF, V>(o, x);
}

// the stream behind the block, of V channels, before it is rounded
template <bool BF, bool RF, int V>
__device__ __forceinline__ void wide_stream(const BlockArgs &a, int64_t i, int c, int live, float rx, float (&R)[V]) {
    float x[V], z[V], r[V], w[V], sc[V];
    wide_read<BF, V>(a.x, i, live, x);
    if (a.z) wide_read<BF, V>(a.z, i, live, z);
    if (a.r) wide_read<RF, V>(a.r, i, live, r);
    read_weight<V>(a.w, c, live, w);
    read_weight<V>(a.sc, c, live, sc);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float act = 1.f, slope;
        if (a.z) gate<BF, BF && RF>(z[e], a.act, act, slope);
        R[e] = __builtin_fmaf(x[e] * (sc[e] * w[e] * act), rx, a.r ? a.alpha * r[e] : 0.f);
    }
}

template <bool BF, bool RF, int V>
__global__ __launch_bounds__(kWide) void wide_fwd_kernel(const BlockArgs a) {
    __shared__ float lds[kWide / 64][1];
    const float inv = 1.f / (float)a.C;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const int64_t base = row * a.C;
        float rx = 1.f, s[1] = {0.f};
        if (a.post) {
            for (int c = threadIdx.x * V; c < a.C; c += kWide * V) {
                float x[V];
                wide_read<BF, V>(a.x, base + c, a.C - c < V ? a.C - c : V, x);
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] = __builtin_fmaf(x[e], x[e], s[0]);
            }
            wide_sum(s, lds);
            rx = 1.f / sqrtf(s[0] * inv + a.eps);
        }
        if (a.pre) {
            s[0] = 0.f;
            for (int c = threadIdx.x * V; c < a.C; c += kWide * V) {
                float R[V];
                const int live = a.C - c < V ? a.C - c : V;
                wide_stream<BF, RF, V>(a, base + c, c, live, rx, R);
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] = e < live ? __builtin_fmaf(R[e], R[e], s[0]) : s[0];
            }
            wide_sum(s, lds);
        }
        const float rR = a.pre ? 1.f / sqrtf(s[0] * inv + a.eps) : 0.f;
        // (what is overwritten in place is read by the thread itself just before)
        for (int c = threadIdx.x * V; c < a.C; c += kWide * V) {
            float R[V], wp[V];
            const int live = a.C - c < V ? a.C - c : V;
            wide_stream<BF, RF, V>(a, base + c, c, live, rx, R);
            if (a.R) store<RF, V, false, true>(a.R, base + c, live, R, a.past);
            if (a.pre) {
                read_weight<V>(a.wp, c, live, wp);
#pragma unroll
                for (int e = 0; e < V; ++e) R[e] *= rR * wp[e];
                store<BF, V, false, true>(a.y, base + c, live, R, a.past);
            }
        }
    }
}

// V channels of a row: the gradient of R, and x's part
template <bool BF, bool RF, int V>
struct WideStep {
    float D[V], n[V], w[V], sc[V], act[V], slope[V], q[V], N[V];
    __device__ __forceinline__ WideStep(const BlockArgs &a, int64_t i, int c, int live, float rx, float rR, float mean) {
        float R[V], z[V], wp[V];
        wide_read<BF, V>(a.x, i, live, n);
        if (a.dR) wide_read<RF, V>(a.dR, i, live, D);
        if (a.z) wide_read<BF, V>(a.z, i, live, z);
        if (a.pre) {
            wide_read<RF, V>(a.R, i, live, R);
            wide_read<BF, V>(a.dy, i, live, q);
            read_weight<V>(a.wp, c, live, wp);
        }
        read_weight<V>(a.w, c, live, w);
        read_weight<V>(a.sc, c, live, sc);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (!a.dR) D[e] = 0.f;
            if (a.pre) {
                N[e] = R[e] * rR;
                D[e] += rR * (q[e] * wp[e] - R[e] * mean);
            } else {
                q[e] = N[e] = 0.f;
            }
            n[e] *= rx;
            act[e] = 1.f;
            slope[e] = 0.f;
            if (a.z) gate<BF, BF>(z[e], a.act, act[e], slope[e]);
        }
    }
};

template <bool BF, bool RF, int V>
__global__ __launch_bounds__(kWide) void wide_stats_kernel(const BlockArgs a) {
    __shared__ float lds[kWide / 64][3], one[kWide / 64][1];
    const float inv = 1.f / (float)a.C;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const int64_t base = row * a.C;
        float s[3] = {0.f, 0.f, 0.f};
        for (int c = threadIdx.x * V; c < a.C; c += kWide * V) {
            const int live = a.C - c < V ? a.C - c : V;
            float x[V], R[V], q[V], wp[V];
            wide_read<BF, V>(a.x, base + c, live, x);
            if (a.pre) {
                wide_read<RF, V>(a.R, base + c, live, R);
                wide_read<BF, V>(a.dy, base + c, live, q);
                read_weight<V>(a.wp, c, live, wp);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[0] = __builtin_fmaf(x[e], x[e], s[0]);
                if (a.pre) {
                    s[1] = __builtin_fmaf(R[e], R[e], s[1]);
                    s[2] = __builtin_fmaf(q[e] * wp[e], R[e], s[2]);
                }
            }
        }
        wide_sum(s, lds);
        const float rx = a.post ? 1.f / sqrtf(s[0] * inv + a.eps) : 1.f;
        const float rR = a.pre ? 1.f / sqrtf(s[1] * inv + a.eps) : 0.f, mean = s[2] * inv * rR * rR;
        float t[1] = {0.f};
        if (a.post) {
            for (int c = threadIdx.x * V; c < a.C; c += kWide * V) {
                const int live = a.C - c < V ? a.C - c : V;
                const WideStep<BF, RF, V> k(a, base + c, c, live, rx, rR, mean);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e < live) t[0] = __builtin_fmaf(k.D[e] * k.act[e] * k.sc[e] * k.w[e], k.n[e], t[0]);
            }
            wide_sum(t, one);
        }
        if (threadIdx.x == 0) {
            float *to = a.stats + row * kStats;
            to[0] = rx;
            to[1] = rR;
            to[2] = mean;
            to[3] = t[0] * inv;
        }
    }
}

// (behind the sums below: what dx, dz and dr may overwrite is read by the thread itself just before)
template <bool BF, bool RF, int V>
__global__ __launch_bounds__(kWide) void wide_bwd_kernel(const BlockArgs a) {
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const int64_t base = row * a.C;
        const float *s = a.stats + row * kStats;
        const float rx = s[0], rR = s[1], mean = s[2], t = s[3];
        for (int c = threadIdx.x * V; c < a.C; c += kWide * V) {
            const int live = a.C - c < V ? a.C - c : V;
            const WideStep<BF, RF, V> k(a, base + c, c, live, rx, rR, mean);
            float dx[V], dz[V], dr[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float g = k.D[e] * k.act[e] * k.sc[e] * k.w[e];
                dr[e] = a.alpha * k.D[e];
                dz[e] = k.D[e] * k.sc[e] * (k.n[e] * k.w[e]) * k.slope[e];
                dx[e] = a.post ? rx * (g - k.n[e] * t) : g;
            }
            if (a.dr) store<RF, V, false, false>(a.dr, base + c, live, dr, true);
            if (a.z) store<BF, V, false, false>(a.dz, base + c, live, dz, true);
            store<BF, V, false, false>(a.dx, base + c, live, dx, true);
        }
    }
}

// partial sums of the weights' gradients: a thread V columns, up to kChainRows rows
template <bool BF, bool RF, int V>
__global__ __launch_bounds__(64) void wide_sums_kernel(const BlockArgs a) {
    const int c = (blockIdx.x * 64 + threadIdx.x) * V, live = a.C - c < V ? a.C - c : V;
    if (c >= a.C) return;
    const int64_t first = (int64_t)blockIdx.y * a.rows, end = first + a.rows < a.n ? first + a.rows : a.n;
    float dw[V] = {}, dwp[V] = {}, dsc[V] = {};
    for (int64_t row = first; row < end; ++row) {
        const float *s = a.stats + row * kStats;
        const WideStep<BF, RF, V> k(a, row * a.C + c, c, live, s[0], s[1], s[2]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float da = k.D[e] * k.act[e];
            dwp[e] = __builtin_fmaf(k.q[e], k.N[e], dwp[e]);
            dsc[e] = __builtin_fmaf(da, k.n[e] * k.w[e], dsc[e]);
            dw[e] = __builtin_fmaf(da * k.sc[e], k.n[e], dw[e]);
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * 3 * a.C + c;
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (e < live) {
            part[e] = dw[e];
            part[a.C + e] = dwp[e];
            part[2 * (int64_t)a.C + e] = dsc[e];
        }
}

// the weights' gradients: partial sums of all workgroups in a fixed order, 64 columns and kRuns runs a workgroup
constexpr int kRuns = 16;
__global__ __launch_bounds__(64 * kRuns) void weight_sums_kernel(const float *part, int64_t n, int C, float *dw, float *dwp,
                                                                 float *dsc) {
    __shared__ double lds[kRuns][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, at = blockIdx.x * 64 + lane;
    double d = 0.;
    if (at < 3 * C) {
#pragma unroll 4
        for (int64_t r = run; r < n; r += kRuns) d += part[r * 3 * C + at];
    }
    lds[run][lane] = d;
    __syncthreads();
    if (run || at >= 3 * C) return;
    for (int k = 1; k < kRuns; ++k) d += lds[k][lane];
    float *to = at < C ? dw : (at < 2 * C ? dwp : dsc);
    if (to) to[at % C] = (float)d;
}

// --------------------------------------------------------------------- host ---
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct BlockPlan {
    bool whole, wide[2];         // rows of whole aligned accesses; (forward, backward) rows that the registers do not hold
    int V, lanes[2], pieces[2];
    int64_t groups[2], parts;    // workgroups; partial sums of the weights' gradients
    int64_t rows;                // (wide) rows of such a sum
    size_t stats, total;         // bytes of workspace
};

m3_status block_plan(const m3_block_norm_shape *s, BlockPlan *p) {
    if (!s) return M3_ERR_INVALID_ARG;
    if (s->rows < 0 || s->channels < 1 || !(s->eps >= 0.f) || !isfinite(s->eps) || !isfinite(s->residual_scale))
        return M3_ERR_INVALID_ARG;
    if (s->io_dtype != M3_F32 && s->io_dtype != M3_BF16) return M3_ERR_INVALID_ARG;
    if (s->residual_dtype != M3_F32 && s->residual_dtype != s->io_dtype) return M3_ERR_INVALID_ARG;
    if (s->activation < M3_ACT_NONE || s->activation > M3_ACT_SIGMOID) return M3_ERR_INVALID_ARG;
    if (s->flags & ~(uint32_t)(M3_BLOCK_POST_NORM | M3_BLOCK_PRE_NORM)) return M3_ERR_INVALID_ARG;
    if (s->rows > (1LL << 40) || s->channels > (1 << 20) || s->rows > (1LL << 44) / s->channels) return M3_ERR_UNSUPPORTED;
    p->V = s->io_dtype == M3_BF16 && s->residual_dtype == M3_BF16 ? 8 : 4;
    const int64_t need = ceil_div(s->channels, p->V);
    p->whole = s->channels % p->V == 0;
    p->parts = 0;
    int threads[2];
    for (int b = 0; b < 2; ++b) {
        p->wide[b] = s->channels > (b ? 8192 : 16384);
        // Lanes of a row: one access each, of 4 channels two each from 512 lanes on with gradients, whose registers hold three sums a channel
        // too. 1024 lanes leave those no room for weights and loads ahead (16384 rows of 4096 channels, bf16 with an fp32 stream: 273 us
        // with 512 lanes, 574 with 1024 and their weights in registers that spill). A whole number of waves from 256 on
        const int64_t lanes = b && p->V == 4 && need > 512 ? ceil_div(need, 2) : need;
        p->lanes[b] = 16;
        while (p->lanes[b] < lanes && p->lanes[b] < 256) p->lanes[b] *= 2;
        for (int more : {320, 384, 512, 1024})
            if (p->lanes[b] < lanes) p->lanes[b] = more;
        p->pieces[b] = need <= p->lanes[b] ? 1 : (need <= 2 * p->lanes[b] ? 2 : 4);
        threads[b] = p->wide[b] ? kWide : (p->lanes[b] < 256 ? 256 : p->lanes[b]);
        const int64_t passes = p->wide[b] ? s->rows : ceil_div(s->rows, threads[b] / p->lanes[b]);
        // About 1024 threads of them a CU forwards (b8 L4096 of 2048 channels with an fp32 stream 163 us; 2048 175, 4096 171), 640 with
        // gradients, each with its own sums of the weights (b4 L4096 of 4096, 512 lanes a row: one a CU 190 us, two 201)
        const int each = ((b ? 640 : 1024) + threads[b] / 2) / threads[b];
        const int64_t best = p->wide[b] ? 512 : 256 * (each < 1 ? 1 : each);
        p->groups[b] = passes < best ? passes : best;
        if (b && !p->wide[b] && p->groups[b] * kChainRows < passes) p->groups[b] = ceil_div(passes, kChainRows);
    }
    // (wide rows: a wave has 64 V columns of up to kChainRows rows, of fewer where that fills the card)
    const int64_t across = ceil_div(need, 64), want = ceil_div(4096, across), least = ceil_div(s->rows, kChainRows);
    p->rows = s->rows ? ceil_div(s->rows, want > least ? (want < s->rows ? want : s->rows) : least) : 1;
    p->parts = p->wide[1] ? ceil_div(s->rows, p->rows) : p->groups[1];
    if (p->groups[1] > kMaxThreads / threads[1] || (p->wide[1] && p->parts > 65535)) return M3_ERR_UNSUPPORTED;
    p->stats = p->wide[1] ? ((size_t)s->rows * kStats * sizeof(float) + 255) & ~(size_t)255 : 0;
    p->total = p->stats + (size_t)p->parts * 3 * (size_t)s->channels * sizeof(float);
    return M3_OK;
}

template <bool BF, bool RF, int V, int LANES, int CH, bool WHOLE>
hipError_t launch(const BlockArgs &a, const BlockPlan &p, bool bwd, hipStream_t s) {
    const dim3 t((Lanes<LANES, CH, V>::kThreads)), g((unsigned)p.groups[bwd]);
    // (what the plan does not ask for: forwards two pieces of fewer than 1024 lanes, or over 16 channels a lane; with gradients over 8
    // channels a lane, or 1024 lanes of 4)
    constexpr bool forward = CH == 1 || (LANES == 1024 && CH * V <= 16), backward = CH * V <= 8 && !(LANES == 1024 && CH * V == 4);
    if constexpr (backward)
        if (bwd) hipLaunchKernelGGL((bwd_kernel<BF, RF, V, LANES, CH, WHOLE>), g, t, 0, s, a);
    if constexpr (forward)
        if (!bwd) hipLaunchKernelGGL((fwd_kernel<BF, RF, V, LANES, CH, WHOLE>), g, t, 0, s, a);
    return (bwd ? backward : forward) ? hipGetLastError() : hipErrorInvalidValue;
}

template <bool BF, bool RF, int V, bool WHOLE>
hipError_t launch_lanes(const BlockArgs &a, const BlockPlan &p, bool bwd, hipStream_t s) {
    switch (p.lanes[bwd] * 8 + p.pieces[bwd]) {
        case 16 * 8 + 1: return launch<BF, RF, V, 16, 1, WHOLE>(a, p, bwd, s);
        case 32 * 8 + 1: return launch<BF, RF, V, 32, 1, WHOLE>(a, p, bwd, s);
        case 64 * 8 + 1: return launch<BF, RF, V, 64, 1, WHOLE>(a, p, bwd, s);
        case 128 * 8 + 1: return launch<BF, RF, V, 128, 1, WHOLE>(a, p, bwd, s);
        case 256 * 8 + 1: return launch<BF, RF, V, 256, 1, WHOLE>(a, p, bwd, s);
        case 320 * 8 + 1: return launch<BF, RF, V, 320, 1, WHOLE>(a, p, bwd, s);
        case 384 * 8 + 1: return launch<BF, RF, V, 384, 1, WHOLE>(a, p, bwd, s);
        case 512 * 8 + 1: return launch<BF, RF, V, 512, 1, WHOLE>(a, p, bwd, s);
        case 1024 * 8 + 1: return launch<BF, RF, V, 1024, 1, WHOLE>(a, p, bwd, s);
        case 320 * 8 + 2: return launch<BF, RF, V, 320, 2, WHOLE>(a, p, bwd, s);
        case 384 * 8 + 2: return launch<BF, RF, V, 384, 2, WHOLE>(a, p, bwd, s);
        case 512 * 8 + 2: return launch<BF, RF, V, 512, 2, WHOLE>(a, p, bwd, s);
        case 1024 * 8 + 2: return launch<BF, RF, V, 1024, 2, WHOLE>(a, p, bwd, s);
        case 1024 * 8 + 4: return launch<BF, RF, V, 1024, 4, WHOLE>(a, p, bwd, s);
    }
    return hipErrorInvalidValue;
}

template <bool BF, bool RF, int V>
hipError_t launch_rows(const BlockArgs &a, const BlockPlan &p, bool bwd, hipStream_t s) {
    return p.whole ? launch_lanes<BF, RF, V, true>(a, p, bwd, s) : launch_lanes<BF, RF, V, false>(a, p, bwd, s);
}

template <bool BF, bool RF, int V>
hipError_t launch_wide(const BlockArgs &a, const BlockPlan &p, bool bwd, hipStream_t s) {
    const dim3 g((unsigned)p.groups[bwd]);
    if (!bwd) {
        hipLaunchKernelGGL((wide_fwd_kernel<BF, RF, V>), g, dim3(kWide), 0, s, a);
        return hipGetLastError();
    }
    hipError_t e;
    hipLaunchKernelGGL((wide_stats_kernel<BF, RF, V>), g, dim3(kWide), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.sums) {
        hipLaunchKernelGGL((wide_sums_kernel<BF, RF, V>), dim3((unsigned)ceil_div(a.C, 64 * V), (unsigned)p.parts), dim3(64), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL((wide_bwd_kernel<BF, RF, V>), g, dim3(kWide), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_any(const m3_block_norm_shape &s, BlockArgs &a, const BlockPlan &p, bool bwd, hipStream_t hs) {
    const bool bf = s.io_dtype == M3_BF16, rf = s.residual_dtype == M3_BF16;
    // x, y and the gate, with gradients theirs; the stream before and behind, and its gradients
    const int64_t each = (bf ? 2 : 4) * ((bwd ? 3 : 2) + (a.z ? (bwd ? 2 : 1) : 0)) + (rf ? 2 : 4) * (bwd ? 3 : 2);
    a.past = a.n * a.C > kLastCache / each;
    a.rows = (int)p.rows;
    if (p.wide[bwd])
        return bf && rf ? launch_wide<true, true, 8>(a, p, bwd, hs)
                        : (bf ? launch_wide<true, false, 4>(a, p, bwd, hs) : launch_wide<false, false, 4>(a, p, bwd, hs));
    if (bf && rf) return launch_rows<true, true, 8>(a, p, bwd, hs);
    return bf ? launch_rows<true, false, 4>(a, p, bwd, hs) : launch_rows<false, false, 4>(a, p, bwd, hs);
}

BlockArgs block_args(const m3_block_norm_shape &s, const m3_block_norm_io &io) {
    BlockArgs a{};
    a.x = io.x; a.z = io.z; a.r = io.residual; a.w = io.post_weight; a.wp = io.pre_weight; a.sc = io.scale;
    a.R = io.residual_out; a.y = io.y; a.n = s.rows; a.C = (int)s.channels; a.eps = s.eps; a.alpha = s.residual_scale;
    a.act = s.activation; a.post = s.flags & M3_BLOCK_POST_NORM; a.pre = s.flags & M3_BLOCK_PRE_NORM;
    return a;
}

// a weight of a norm that the call does not have
bool stray(const m3_block_norm_shape &s, const void *post, const void *pre) {
    return (post && !(s.flags & M3_BLOCK_POST_NORM)) || (pre && !(s.flags & M3_BLOCK_PRE_NORM));
}

}  // namespace
}  // namespace m3i

using namespace m3i;

extern "C" {

size_t m3_block_norm_bwd_workspace_bytes(const m3_block_norm_shape *shape) {
    BlockPlan p;
    return block_plan(shape, &p) == M3_OK ? p.total : 0;
}

m3_status m3_block_norm_fwd(const m3_block_norm_shape *shape, const m3_block_norm_io *io, void *stream) {
    BlockPlan p;
    const m3_status st = block_plan(shape, &p);
    if (st != M3_OK) return st;
    if (!io) return M3_ERR_INVALID_ARG;
    const bool pre = shape->flags & M3_BLOCK_PRE_NORM;
    if (stray(*shape, io->post_weight, io->pre_weight) || (!pre && io->y)) return M3_ERR_INVALID_ARG;
    if (shape->rows > 0 && (!io->x || (pre ? !io->y : !io->residual_out))) return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->x, io->z, io->residual, io->post_weight, io->pre_weight, io->scale, io->residual_out, io->y};
    for (const void *q : ptrs)
        if (!al16(q)) return M3_ERR_MISALIGNED;
    // (y may be x or z, residual_out may be residual: a lane's part of a row is read before it is written, by itself)
    if (clash({io->residual_out, io->y}, {io->post_weight, io->pre_weight, io->scale}) ||
        clash({io->residual_out}, {io->x, io->z}) || clash({io->y}, {io->residual}))
        return M3_ERR_INVALID_ARG;
    if (shape->rows == 0) return M3_OK;
    BlockArgs a = block_args(*shape, *io);
    const hipError_t e = launch_any(*shape, a, p, false, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

m3_status m3_block_norm_bwd(const m3_block_norm_shape *shape, const m3_block_norm_io *io, const m3_block_norm_grads *gr,
                            void *workspace, size_t ws_bytes, void *stream) {
    BlockPlan p;
    const m3_status st = block_plan(shape, &p);
    if (st != M3_OK) return st;
    if (!io || !gr) return M3_ERR_INVALID_ARG;
    const bool pre = shape->flags & M3_BLOCK_PRE_NORM, sums = gr->dpost_weight || gr->dpre_weight || gr->dscale;
    if (stray(*shape, io->post_weight, io->pre_weight) || stray(*shape, gr->dpost_weight, gr->dpre_weight) || (!pre && gr->dy))
        return M3_ERR_INVALID_ARG;
    if (shape->rows > 0 && (!io->x || !gr->dx || (io->z == nullptr) != (gr->dz == nullptr) ||
                            (pre ? !io->residual_out || !gr->dy : !gr->dresidual_out)))
        return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->x, io->z, io->post_weight, io->pre_weight, io->scale, io->residual_out, gr->dy, gr->dresidual_out,
                          gr->dx, gr->dz, gr->dresidual, gr->dpost_weight, gr->dpre_weight, gr->dscale, workspace};
    for (const void *q : ptrs)
        if (!al16(q)) return M3_ERR_MISALIGNED;
    const size_t need = sums ? p.total : p.stats;
    if (need && (!workspace || ws_bytes < need)) return M3_ERR_WORKSPACE_TOO_SMALL;
    void *ws = need ? workspace : nullptr;
    // (dx may be x or dy, dz may be z, dresidual may be dresidual_out)
    const void *x = io->x, *z = io->z, *R = io->residual_out, *dy = gr->dy, *dR = gr->dresidual_out;
    if (clash({gr->dx, gr->dz, gr->dresidual, gr->dpost_weight, gr->dpre_weight, gr->dscale, ws},
              {io->post_weight, io->pre_weight, io->scale, R}) ||
        clash({gr->dpost_weight, gr->dpre_weight, gr->dscale, ws}, {x, z, dy, dR}) || clash({gr->dx}, {z, dR}) ||
        clash({gr->dz}, {x, dy, dR}) || clash({gr->dresidual}, {x, z, dy}))
        return M3_ERR_INVALID_ARG;
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    BlockArgs a = block_args(*shape, *io);
    a.dy = dy; a.dR = dR; a.dx = gr->dx; a.dz = gr->dz; a.dr = gr->dresidual;
    a.sums = sums;
    a.stats = static_cast<float *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.stats);
    hipError_t e = shape->rows > 0 ? launch_any(*shape, a, p, true, hs) : hipSuccess;
    if (e == hipSuccess && sums) {
        hipLaunchKernelGGL(weight_sums_kernel, dim3((unsigned)ceil_div(3 * shape->channels, 64)), dim3(64 * kRuns), 0, hs, a.part,
                           p.parts, (int)shape->channels, gr->dpost_weight, gr->dpre_weight, gr->dscale);
        e = hipGetLastError();
    }
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

}  // extern "C"
