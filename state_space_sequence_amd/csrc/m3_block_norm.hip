// The norms around a block with its gate, scale and residual: forward and gradients (gfx950).
//
//   v = x rx w,  rx = 1/sqrt(mean x^2 + eps) (or v = x);  R = alpha r + sc act(z) v;  y = R rR wp
//   dR' = dR + rR (q - R rR mean(q R rR)),  q = dy wp;  dr = alpha dR';  dz = dR' sc v act'(z)
//   g = dR' sc act(z) w;  dx = rx (g - x rx mean(g x rx));  dwp = sum dy R rR;  dsc = sum dR' act(z) v;  dw = sum dR' sc act(z) x rx
//
// Bound by HBM: every tensor is read or written once. The lanes of a row (16 to 1024 of them) hold it in registers, up to
// 32 values each; its sums go across a wave by DPP and row swaps, across waves by LDS. A lane keeps its channels from row
// to row, so weights and their gradients stay in registers too, and the next row is loaded while this one is summed.
#include <math.h>

#include "m3_block_norm.h"
#include "m3_internal.h"

namespace m3i {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kChainRows = 256;  // rows whose weight gradients a thread adds up in fp32
constexpr int64_t kMaxGrid = 0x3fffff;  // workgroups of 1024 threads: 2^32 threads
constexpr int64_t kLastCache = 256 << 20;

struct BlockArgs {
    const void *x, *z, *r;
    const float *w, *wp, *sc;
    void *R, *y;
    const void *dy, *dR;
    void *dx, *dz, *dr;
    float *part;  // [workgroups][3][C]: sums of dw, dwp, dsc
    int64_t n;
    int C;
    float eps, alpha;
    int act;
    bool post, pre, sums;
    bool past;  // stores past the caches
};

// V consecutive values of one dtype as they lie in memory
template <bool BF16, int V>
struct Packed {
    static constexpr int W = BF16 ? V / 2 : V;
    unsigned w[W];
};

// VEC: live is 0 or V, one access of 8 or 16 bytes (two of an fp32 V of 8 do not occur)
template <bool BF16, int V, bool VEC>
__device__ __forceinline__ void load(const void *p, int64_t i, int live, Packed<BF16, V> &o) {
    constexpr int W = Packed<BF16, V>::W;
    if constexpr (VEC) {
#pragma unroll
        for (int e = 0; e < W; ++e) o.w[e] = 0;
        if (live > 0) {
            const char *at = static_cast<const char *>(p) + i * (BF16 ? 2 : 4);
            if constexpr (W == 4) {
                const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(at));
#pragma unroll
                for (int e = 0; e < 4; ++e) o.w[e] = v[e];
            } else {
                static_assert(W == 2, "8 or 16 bytes");
                const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(at));
                o.w[0] = v[0];
                o.w[1] = v[1];
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            if constexpr (BF16) {
                const uint16_t *q = static_cast<const uint16_t *>(p) + i;
                const unsigned lo = 2 * e < live ? q[2 * e] : 0, hi = 2 * e + 1 < live ? q[2 * e + 1] : 0;
                o.w[e] = lo | hi << 16;
            } else {
                o.w[e] = e < live ? static_cast<const unsigned *>(p)[i + e] : 0;
            }
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
// Past the caches: forwards where the tensors of the call do not fit them (ASK, past), with gradients always (b4 L4096 of 4096
// channels 222 us by kernel trace, with the question 227)
template <bool BF16, int V, bool VEC, bool ASK>
__device__ __forceinline__ void store(void *p, int64_t i, int live, const float (&x)[V], bool past) {
    constexpr int W = Packed<BF16, V>::W;
    if constexpr (VEC) {
        unsigned w[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
            if constexpr (BF16) w[e] = __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x[2 * e], x[2 * e + 1]}), bf16x2));
            else w[e] = __float_as_uint(x[e]);
        }
        if (live > 0) {
            typedef unsigned vec __attribute__((ext_vector_type(W)));
            vec v;
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = w[e];
            vec *to = reinterpret_cast<vec *>(static_cast<char *>(p) + i * (BF16 ? 2 : 4));
            if constexpr (!ASK) {
                __builtin_nontemporal_store(v, to);
            } else if (past) {
                asm volatile("");  // (two equal stores but for their hint would become one)
                __builtin_nontemporal_store(v, to);
                asm volatile("");
            } else {
                *to = v;
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

// the gate's value, and its slope. (bf16: the hardware exponential's error, |z| 2^-23, is far below the outputs' rounding)
template <bool BF16>
__device__ __forceinline__ void gate(float z, int act, float &v, float &slope) {
    v = z;
    slope = 1.f;
    if (act != M3_ACT_NONE) {
        const float e = BF16 ? __builtin_amdgcn_exp2f(-1.4426950408889634f * z) : expf(-z);
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

// Where a thread is: LANES lanes a row, CH pieces of LANES * V channels
template <int LANES, int CH, int V, bool VEC>
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
    __device__ __forceinline__ void weights(const float *p, float (&w)[CH][V]) const {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) w[k][e] = p && e < live[k] ? p[c[k] + e] : 1.f;
    }
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

// BF: x, z, y in bf16; RF: the residual stream in bf16
template <bool BF, bool RF, int V, int LANES, int CH, bool VEC>
__global__ __launch_bounds__((Lanes<LANES, CH, V, VEC>::kThreads)) void fwd_kernel(const BlockArgs a) {
    using At = Lanes<LANES, CH, V, VEC>;
    __shared__ float lds[2][At::kThreads / 64][4];
    const At p(a.C);
    float w[CH][V], wp[CH][V], sc[CH][V];
    p.weights(a.w, w);
    p.weights(a.wp, wp);
    p.weights(a.sc, sc);
    const float inv = 1.f / (float)a.C;
    Packed<BF, V> x[CH], z[CH];
    Packed<RF, V> r[CH];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int live = row < a.n ? p.live[k] : 0;
            load<BF, V, VEC>(a.x, row * a.C + p.c[k], live, x[k]);
            if (a.z) load<BF, V, VEC>(a.z, row * a.C + p.c[k], live, z[k]);
            if (a.r) load<RF, V, VEC>(a.r, row * a.C + p.c[k], live, r[k]);
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
            float zs[V], rs[V];
            unpack<BF, V>(z[k], zs);
            unpack<RF, V>(r[k], rs);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                R[k][e] = a.r ? a.alpha * rs[e] : 0.f;
                s[0] = __builtin_fmaf(v[k][e], v[k][e], s[0]);
                float on = sc[k][e] * w[k][e], slope;
                if (a.z) {
                    float act;
                    gate<BF>(zs[e], a.act, act, slope);
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
        for (int k = 0; k < CH; ++k) store<RF, V, VEC, true>(a.R, row * a.C + p.c[k], here ? p.live[k] : 0, R[k], a.past);
        if (a.pre) {
            At::sum(s, lds, slot);
            const float rR = 1.f / sqrtf(s[0] * inv + a.eps);
#pragma unroll
            for (int k = 0; k < CH; ++k) {
#pragma unroll
                for (int e = 0; e < V; ++e) R[k][e] *= rR * wp[k][e];
                store<BF, V, VEC, true>(a.y, row * a.C + p.c[k], here ? p.live[k] : 0, R[k], a.past);
            }
        }
    }
}

template <bool BF, bool RF, int V, int LANES, int CH, bool VEC>
__global__ __launch_bounds__((Lanes<LANES, CH, V, VEC>::kThreads)) void bwd_kernel(const BlockArgs a) {
    using At = Lanes<LANES, CH, V, VEC>;
    __shared__ float lds[2][At::kThreads / 64][4];
    const At p(a.C);
    float w[CH][V], wp[CH][V], sc[CH][V], dw[CH][V], dwp[CH][V], dsc[CH][V];
    p.weights(a.w, w);
    p.weights(a.wp, wp);
    p.weights(a.sc, sc);
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
            load<BF, V, VEC>(a.x, at, live, x[k]);
            if (a.z) load<BF, V, VEC>(a.z, at, live, z[k]);
            if (a.pre) {
                load<RF, V, VEC>(a.R, at, live, R[k]);
                load<BF, V, VEC>(a.dy, at, live, y[k]);
            }
            if (a.dR) load<RF, V, VEC>(a.dR, at, live, D[k]);
        }
    };
    const int64_t step = (int64_t)gridDim.x * At::kRows;
    int slot = 0;
    fetch((int64_t)blockIdx.x * At::kRows + p.r);
    for (int64_t pass = (int64_t)blockIdx.x * At::kRows; pass < a.n; pass += step) {
        const int64_t row = pass + p.r;
        const bool here = row < a.n;
        float xs[CH][V], zs[CH][V], d[CH][V], Rs[CH][V], q[CH][V];
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            unpack<BF, V>(x[k], xs[k]);
            unpack<BF, V>(z[k], zs[k]);
            unpack<BF, V>(y[k], q[k]);
            unpack<RF, V>(R[k], Rs[k]);
            unpack<RF, V>(D[k], d[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[0] = __builtin_fmaf(xs[k][e], xs[k][e], s[0]);
                if (!a.dR) d[k][e] = 0.f;
                if (a.pre) {
                    s[1] = __builtin_fmaf(Rs[k][e], Rs[k][e], s[1]);
                    s[2] = __builtin_fmaf(q[k][e] * wp[k][e], Rs[k][e], s[2]);
                }
            }
        }
        fetch(row + step);
        float rx = 1.f;
        if (a.post || a.pre) {
            At::sum(s, lds, slot);
            if (a.post) rx = 1.f / sqrtf(s[0] * inv + a.eps);
        }
        if (a.pre) {
            const float rR = 1.f / sqrtf(s[1] * inv + a.eps), mean = s[2] * inv * rR * rR;
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float n = here ? Rs[k][e] * rR : 0.f;  // (rows behind the last: 1/sqrt(eps) may be infinite)
                    dwp[k][e] = __builtin_fmaf(q[k][e], n, dwp[k][e]);
                    d[k][e] += rR * (q[k][e] * wp[k][e] - Rs[k][e] * mean);
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
                store<RF, V, VEC, false>(a.dr, at, live, o, a.past);
            }
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!here) d[k][e] = 0.f;
                const float n = here ? xs[k][e] * rx : 0.f, v = n * w[k][e];
                xs[k][e] = n;
                float act = 1.f, slope = 0.f;
                if (a.z) {
                    gate<BF>(zs[k][e], a.act, act, slope);
                    o[e] = d[k][e] * sc[k][e] * v * slope;
                }
                const float da = d[k][e] * act;
                dsc[k][e] = __builtin_fmaf(da, v, dsc[k][e]);
                d[k][e] = da * sc[k][e];
                dw[k][e] = __builtin_fmaf(d[k][e], n, dw[k][e]);
                d[k][e] *= w[k][e];
                t[0] = __builtin_fmaf(d[k][e], n, t[0]);
            }
            if (a.z) store<BF, V, VEC, false>(a.dz, at, live, o, a.past);
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
            store<BF, V, VEC, false>(a.dx, row * a.C + p.c[k], here ? p.live[k] : 0, d[k], a.past);
        }
    }
    if (!a.sums) return;
    // the sums of a workgroup's lanes of rows, in a fixed order
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
                    float t = 0.f;
                    for (int r = 0; r < At::kRows; ++r) t += join[j][r * LANES + l];
                    if (c < a.C) part[(int64_t)j * a.C + c] = t;
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
    int V, lanes, pieces;
    bool vec;
    int64_t fwd, bwd;  // workgroups
};

// lanes of a row: one access each where 1024 are enough
m3_status block_plan(const m3_block_norm_shape *s, BlockPlan *p) {
    if (!s) return M3_ERR_INVALID_ARG;
    if (s->rows < 0 || s->channels < 1 || !(s->eps >= 0.f) || !isfinite(s->eps) || !isfinite(s->residual_scale))
        return M3_ERR_INVALID_ARG;
    if (s->io_dtype != M3_F32 && s->io_dtype != M3_BF16) return M3_ERR_INVALID_ARG;
    if (s->residual_dtype != M3_F32 && s->residual_dtype != s->io_dtype) return M3_ERR_INVALID_ARG;
    if (s->activation < M3_ACT_NONE || s->activation > M3_ACT_SIGMOID) return M3_ERR_INVALID_ARG;
    if (s->flags & ~(uint32_t)(M3_BLOCK_POST_NORM | M3_BLOCK_PRE_NORM)) return M3_ERR_INVALID_ARG;
    p->V = s->io_dtype == M3_BF16 && s->residual_dtype == M3_BF16 ? 8 : 4;
    if (s->rows > (1LL << 40) || s->channels > 4096 * p->V) return M3_ERR_UNSUPPORTED;
    p->vec = s->channels % p->V == 0;
    const int64_t need = ceil_div(s->channels, p->V);
    p->lanes = 16;
    while (p->lanes < need && p->lanes < 1024) p->lanes *= 2;
    p->pieces = need <= p->lanes ? 1 : (need <= 2 * p->lanes ? 2 : 4);
    const int threads = p->lanes < 256 ? 256 : p->lanes, rows = threads / p->lanes;
    const int64_t passes = ceil_div(s->rows, rows);
    // A CU with 1024 threads of them forwards (b8 L4096 of 2048 channels with an fp32 stream 165 us; 2048 172, 4096 168), 512 with
    // gradients, each with its own sums of the weights (b4 L4096 of 4096 219 us by kernel trace; 1024 238, 2048 254)
    const int64_t fwd = 256 * 1024 / threads, bwd = 256 * 512 / threads;
    p->fwd = passes < fwd ? passes : fwd;
    p->bwd = passes < bwd ? passes : bwd;
    if (p->bwd * kChainRows < passes) p->bwd = ceil_div(passes, kChainRows);
    if (p->bwd > kMaxGrid) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

template <bool BF, bool RF, int V, int LANES, int CH, bool VEC>
hipError_t launch(const BlockArgs &a, const BlockPlan &p, bool bwd, hipStream_t s) {
    const dim3 t((Lanes<LANES, CH, V, VEC>::kThreads));
    if (bwd) hipLaunchKernelGGL((bwd_kernel<BF, RF, V, LANES, CH, VEC>), dim3((unsigned)p.bwd), t, 0, s, a);
    else hipLaunchKernelGGL((fwd_kernel<BF, RF, V, LANES, CH, VEC>), dim3((unsigned)p.fwd), t, 0, s, a);
    return hipGetLastError();
}

template <bool BF, bool RF, int V, bool VEC>
hipError_t launch_lanes(const BlockArgs &a, const BlockPlan &p, bool bwd, hipStream_t s) {
    switch (p.lanes * p.pieces) {
        case 16: return launch<BF, RF, V, 16, 1, VEC>(a, p, bwd, s);
        case 32: return launch<BF, RF, V, 32, 1, VEC>(a, p, bwd, s);
        case 64: return launch<BF, RF, V, 64, 1, VEC>(a, p, bwd, s);
        case 128: return launch<BF, RF, V, 128, 1, VEC>(a, p, bwd, s);
        case 256: return launch<BF, RF, V, 256, 1, VEC>(a, p, bwd, s);
        case 512: return launch<BF, RF, V, 512, 1, VEC>(a, p, bwd, s);
        case 1024: return launch<BF, RF, V, 1024, 1, VEC>(a, p, bwd, s);
        case 2048: return launch<BF, RF, V, 1024, 2, VEC>(a, p, bwd, s);
        case 4096: return launch<BF, RF, V, 1024, 4, VEC>(a, p, bwd, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_any(const m3_block_norm_shape &s, BlockArgs &a, const BlockPlan &p, bool bwd, hipStream_t hs) {
    const bool bf = s.io_dtype == M3_BF16, rf = s.residual_dtype == M3_BF16;
    // x, y and the gate, with gradients theirs; the stream before and behind, and its gradients
    const int64_t each = (bf ? 2 : 4) * ((bwd ? 3 : 2) + (a.z ? (bwd ? 2 : 1) : 0)) + (rf ? 2 : 4) * (bwd ? 3 : 2);
    a.past = a.n * a.C > kLastCache / each;
    if (bf && rf)
        return p.vec ? launch_lanes<true, true, 8, true>(a, p, bwd, hs) : launch_lanes<true, true, 8, false>(a, p, bwd, hs);
    if (bf)
        return p.vec ? launch_lanes<true, false, 4, true>(a, p, bwd, hs) : launch_lanes<true, false, 4, false>(a, p, bwd, hs);
    return p.vec ? launch_lanes<false, false, 4, true>(a, p, bwd, hs) : launch_lanes<false, false, 4, false>(a, p, bwd, hs);
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
    return block_plan(shape, &p) == M3_OK ? (size_t)p.bwd * 3 * (size_t)shape->channels * sizeof(float) : 0;
}

m3_status m3_block_norm_fwd(const m3_block_norm_shape *shape, const m3_block_norm_io *io, void *stream) {
    BlockPlan p;
    const m3_status st = block_plan(shape, &p);
    if (st != M3_OK) return st;
    if (!io) return M3_ERR_INVALID_ARG;
    const bool pre = shape->flags & M3_BLOCK_PRE_NORM;
    if (stray(*shape, io->post_weight, io->pre_weight) || (!pre && io->y)) return M3_ERR_INVALID_ARG;
    if (shape->rows > 0 && (!io->x || !io->residual_out || (pre && !io->y))) return M3_ERR_INVALID_ARG;
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
    const size_t need = sums ? (size_t)p.bwd * 3 * (size_t)shape->channels * sizeof(float) : 0;
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
    a.part = static_cast<float *>(workspace);
    hipError_t e = shape->rows > 0 ? launch_any(*shape, a, p, true, hs) : hipSuccess;
    if (e == hipSuccess && sums) {
        hipLaunchKernelGGL(weight_sums_kernel, dim3((unsigned)ceil_div(3 * shape->channels, 64)), dim3(64 * kRuns), 0, hs, a.part,
                           p.bwd, (int)shape->channels, gr->dpost_weight, gr->dpre_weight, gr->dscale);
        e = hipGetLastError();
    }
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

}  // extern "C"
