// Gated linear recurrence, one state a channel: prompt, gradients, single token (gfx950).
//
//   s = sigmoid(r), g = sigmoid(i) or 1, a = exp(ld s), m = sqrt(1 - a^2) or 1
//   h_t = a_t h_{t-1} + m_t g_t x_t
//   G_t = a_t (dy_t + G_{t+1}) is the gradient of h_{t-1}; with E_t = dy_t + G_{t+1}, that of h_t:
//   dx = E m g, di = E m x g (1-g), d(ld s) = E (a h_{t-1} - g x a^2 / m), dr = d(ld s) ld s (1-s), dld = sum d(ld s) s
//
// A step is the map h -> A h + B, and maps in a row are one map again: (A2 A1, A2 B1 + B2). A workgroup of kW
// waves owns 64 lanes of channels (one of fp32, two of bf16: 4 bytes each) of a row and walks a segment of its tokens in chunks of
// kW x kT: a wave forms the gates of its kT tokens and their joint map, the maps meet in LDS, and each wave runs its tokens
// from the state that the maps before it give. The next chunk is loaded meanwhile. Backwards the same
// in both directions at once: states forwards from the kept one, G backwards from the chunk behind.
// With few channels the sequence is split: the map of each segment first, then all segments, from the maps before them.
#include <math.h>

#include "m3_internal.h"
#include "m3_recurrence.h"

namespace m3i {
namespace {

constexpr int kT = 8, kW = 8, kChunk = kT * kW, kThreads = 64 * kW;
static_assert(kChunk == M3_REC_KEEP, "a chunk starts at a kept state");
constexpr int64_t kMaxGrid = 0x7fffff;  // workgroups of one launch: 2^32 threads
constexpr unsigned kOutside = 0x80000000u;  // a byte offset behind every buffer (chunks are at most 2^28 bytes)

struct RecArgs {
    const void *x, *r, *i;
    const float *ld, *h0;
    const int *lengths;
    void *y;
    float *hf, *states;
    float *part;  // [b][nseg][2][C]: maps of the segments
    float *start; // [b][C]: with segments, a copy of the state (the gradient) that they start from: the last one's end may
                  // be written over it while the others still begin
    const void *dy;
    const float *dhf;
    void *dx, *dr, *di;
    float *dld, *dh0;
    double *dpart;  // [b][nseg][C]: sums of dld
    int64_t L;
    int C, cols, nseg, nkeep;  // workgroups across the channels, segments, kept states of a row
    int64_t seg;               // tokens of a segment, whole chunks
};

// what a workgroup works on
struct Place {
    int lane, wave, seg, c;
    int64_t row, s0, s1, len;  // tokens of the segment; valid tokens of the row
    bool in;                   // this lane has channels
    template <int V>
    static __device__ __forceinline__ Place make(const RecArgs &a) {
        Place p;
        p.lane = threadIdx.x & 63;
        p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int col = blockIdx.x % a.cols, rest = blockIdx.x / a.cols;
        p.seg = rest % a.nseg;
        p.row = rest / a.nseg;
        p.c = (col * 64 + p.lane) * V;
        p.in = p.c < a.C;
        p.len = a.L;
        if (a.lengths) {
            const int64_t n = a.lengths[p.row];
            p.len = n < 0 ? 0 : (n < a.L ? n : a.L);
        }
        p.s0 = p.seg * a.seg;
        p.s1 = p.s0 + a.seg < a.L ? p.s0 + a.seg : a.L;
        return p;
    }
};

// V channels of one token of a lane, as they lie in memory, by buffer accesses: what lies
// behind the buffer reads as 0 and is not written
template <bool BF16, int V>
struct Io {
    static constexpr int B = BF16 ? 2 * V : 4;  // bytes of a lane and token
    static_assert(BF16 ? V <= 2 : V == 1, "four bytes at most");
    using rsrc_t = decltype(__builtin_amdgcn_make_buffer_rsrc(static_cast<void *>(nullptr), 0, 0, 0));
    // tokens t0 .. t0 + rows - 1 of a row
    static __device__ __forceinline__ rsrc_t rows(const RecArgs &a, const void *p, int64_t row, int64_t t0, int64_t n) {
        constexpr int E = BF16 ? 2 : 4;
        const char *at = static_cast<const char *>(p) + (row * a.L + t0) * a.C * E;
        n = n < 0 ? 0 : (n < kChunk ? n : kChunk);
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(at), 0, (int)n * a.C * E, 0x00020000);
    }
    static __device__ __forceinline__ unsigned load(rsrc_t r, unsigned at) {
        if constexpr (B == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
        else return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
    }
    static __device__ __forceinline__ void unpack(unsigned w, float (&v)[V]) {
        if constexpr (!BF16) {
            v[0] = __uint_as_float(w);
        } else {
            v[0] = __uint_as_float(w << 16);
            if constexpr (V > 1) v[V - 1] = __uint_as_float(w & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(rsrc_t r, unsigned at, const float (&v)[V]) {
        if constexpr (!BF16) {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r, at, 0, 0);
        } else if constexpr (V == 1) {
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[0]), r, at, 0, 0);
        } else {
            const unsigned lo = __builtin_bit_cast(uint16_t, (__bf16)v[0]), hi = __builtin_bit_cast(uint16_t, (__bf16)v[V - 1]);
            __builtin_amdgcn_raw_buffer_store_b32(lo | hi << 16, r, at, 0, 0);
        }
    }
};

// The sigmoid, and 1 - sigmoid without cancellation (where e^-x overflows: any finite factor of 0). bf16: the
// hardware exponential of a rounded argument is off by |x| 2^-23, far below the outputs' rounding
template <bool BF16>
__device__ __forceinline__ float neg_exp(float x) {
    return BF16 ? __builtin_amdgcn_exp2f(-1.4426950408889634f * x) : expf(-x);
}
template <bool BF16>
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + neg_exp<BF16>(x)); }
template <bool BF16>
__device__ __forceinline__ float sigmoid(float x, float &rest) {
    const float e = neg_exp<BF16>(x), s = __builtin_amdgcn_rcpf(1.f + e);
    rest = (e > 0x1p126f ? 0x1p126f : e) * s;
    return s;
}

// a = 2^l and p = 1 - a for l <= 0, both to half a step: 2^f - 1 = f P(f) for the rest f of l from its nearest whole
// number n, P the polynomial of degree 5 that is closest over |f| <= 1/2 (1.1e-8 relative; fitted here). p has no
// cancellation: for n = 0 it is -f P(f), else at least 0.29. A state of slow decay keeps what hundreds of steps
// bring, so a and m must not be off in one direction.
__device__ __forceinline__ void decay(float l, float &a, float &p) {
    const float n = __builtin_rintf(l), f = l - n;
    const float z = __builtin_amdgcn_ldexpf(1.f, (int)n);
    float e = __builtin_fmaf(f, 0x1.4308f8p-13f, 0x1.5f07b4p-10f);
    e = __builtin_fmaf(e, f, 0x1.3b2ba0p-7f);
    e = __builtin_fmaf(e, f, 0x1.c6af6ep-5f);
    e = __builtin_fmaf(e, f, 0x1.ebfbdep-3f);
    e = __builtin_fmaf(e, f, 0x1.62e430p-1f);
    e *= f;
    a = __builtin_fmaf(z, e, z);
    p = __builtin_fmaf(-z, e, 1.f - z);
}

// log_decay in powers of 2 (of the lanes without channels: 0, a state that stays)
template <int V>
__device__ __forceinline__ void load_decay(const RecArgs &a, const Place &p, float (&ld2)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) ld2[v] = p.in ? a.ld[p.c + v] * 1.4426950408889634f : 0.f;
}

// the step's map h -> a h + b of one channel
template <bool BF16, bool GATE, bool UNIT>
__device__ __forceinline__ void step_map(float x, float r, float i, float ld2, float &a, float &b) {
    float p;
    decay(ld2 * sigmoid<BF16>(r), a, p);
    b = GATE ? x * sigmoid<BF16>(i) : x;
    if constexpr (!UNIT) b *= __builtin_amdgcn_sqrtf(p * (2.f - p));  // 1 - a^2 = p (2 - p)
}

// ------------------------------------------------------------------ forward ---
// y, kept states and the final state of a segment, from the state that the maps before it give
template <bool BF16, int V, bool GATE, bool UNIT>
__global__ __launch_bounds__(kThreads) void fwd_kernel(const RecArgs a) {
    using IO = Io<BF16, V>;
    __shared__ float lds[2][kW][2 * V][64];
    const Place p = Place::make<V>(a);
    const unsigned bytes = (unsigned)a.C * (BF16 ? 2 : 4), own = (p.in ? p.c * (BF16 ? 2 : 4) : kOutside) + p.wave * kT * bytes;
    float ld2[V], h[V];
    load_decay<V>(a, p, ld2);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    const float *h0 = a.nseg > 1 && a.h0 ? a.start : a.h0;
    if (p.in && h0)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = h0[p.row * a.C + p.c + v];
    if (p.in) {
        const float *m = a.part + p.row * a.nseg * 2 * a.C + p.c;
        for (int k = 0; k < p.seg; ++k, m += 2 * (int64_t)a.C)
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(m[v], h[v], m[a.C + v]);
    }
    const int64_t end = p.s1 < p.len ? p.s1 : p.len;
    unsigned rx[kT], rr[kT], ri[GATE ? kT : 1];
    auto fetch = [&](int64_t t0) {
        const auto bx = IO::rows(a, a.x, p.row, t0, end - t0), br = IO::rows(a, a.r, p.row, t0, end - t0);
        const auto bi = IO::rows(a, GATE ? a.i : a.r, p.row, t0, end - t0);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            rx[t] = IO::load(bx, own + t * bytes);
            rr[t] = IO::load(br, own + t * bytes);
            if constexpr (GATE) ri[t] = IO::load(bi, own + t * bytes);
        }
    };
    if (p.s0 < end) fetch(p.s0);
    int side = 0;
    for (int64_t t0 = p.s0; t0 < p.s1; t0 += kChunk, side ^= 1) {
        const int n = end - t0 < kChunk ? (int)(end - t0) : kChunk;  // valid tokens (none or fewer behind the length)
        const auto by = IO::rows(a, a.y, p.row, t0, a.y ? p.s1 - t0 : 0);
        if (n <= 0) {
            const float zero[V] = {};
#pragma unroll
            for (int t = 0; t < kT; ++t) IO::store(by, own + t * bytes, zero);
            if (a.states && p.in && p.wave == 0)
#pragma unroll
                for (int v = 0; v < V; ++v) a.states[(p.row * a.nkeep + t0 / kChunk) * a.C + p.c + v] = h[v];
            continue;
        }
        float sa[kT][V], sb[kT][V], A[V], B[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            B[v] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            float x[V], r[V], i[V] = {};
            IO::unpack(rx[t], x);
            IO::unpack(rr[t], r);
            if constexpr (GATE) IO::unpack(ri[t], i);
            const bool valid = p.wave * kT + t < n;  // (what is not: x is 0, and with a decay of 1 the state stays)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                step_map<BF16, GATE, UNIT>(x[v], r[v], i[v], valid ? ld2[v] : 0.f, sa[t][v], sb[t][v]);
                B[v] = __builtin_fmaf(sa[t][v], B[v], sb[t][v]);
                A[v] *= sa[t][v];
            }
        }
        if (t0 + kChunk < end) fetch(t0 + kChunk);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            lds[side][p.wave][v][p.lane] = A[v];
            lds[side][p.wave][V + v][p.lane] = B[v];
        }
        __syncthreads();  // (two sides: the next chunk's maps are written while these are read)
        if (a.states && p.in && p.wave == 0)
#pragma unroll
            for (int v = 0; v < V; ++v) a.states[(p.row * a.nkeep + t0 / kChunk) * a.C + p.c + v] = h[v];
        float hw[V];
#pragma unroll
        for (int k = 0; k < kW; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (k == p.wave) hw[v] = h[v];
                h[v] = __builtin_fmaf(lds[side][k][v][p.lane], h[v], lds[side][k][V + v][p.lane]);
            }
        if (a.y) {
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                float y[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    hw[v] = __builtin_fmaf(sa[t][v], hw[v], sb[t][v]);
                    y[v] = p.wave * kT + t < n ? hw[v] : 0.f;
                }
                IO::store(by, own + t * bytes, y);
            }
        }
    }
    if (a.hf && p.in && p.wave == 0 && p.seg == a.nseg - 1)
#pragma unroll
        for (int v = 0; v < V; ++v) a.hf[p.row * a.C + p.c + v] = h[v];
}

// The map of every segment: of the states (BACK: of their gradients, the last token first). A wave takes a run
// of the segment's tokens by itself; the runs are joined at the end.
template <bool BF16, int V, bool GATE, bool UNIT, bool BACK>
__global__ __launch_bounds__(kThreads) void map_kernel(const RecArgs a) {
    using IO = Io<BF16, V>;
    __shared__ float lds[kW][2 * V][64];
    const Place p = Place::make<V>(a);
    const unsigned bytes = (unsigned)a.C * (BF16 ? 2 : 4), own = p.in ? p.c * (BF16 ? 2 : 4) : kOutside;
    float ld2[V], A[V], B[V];
    load_decay<V>(a, p, ld2);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = 1.f;
        B[v] = 0.f;
    }
    const int64_t end = p.s1 < p.len ? p.s1 : p.len, run = a.seg / kW;  // (a multiple of kT)
    const int64_t r0 = p.s0 + p.wave * run, r1 = r0 + run < end ? r0 + run : end;
    unsigned rx[kT], rr[kT], ri[GATE ? kT : 1];  // (BACK: rx is dy)
    auto fetch = [&](int64_t t0) {
        const auto bx = IO::rows(a, BACK ? a.dy : a.x, p.row, t0, r1 - t0), br = IO::rows(a, a.r, p.row, t0, r1 - t0);
        const auto bi = IO::rows(a, GATE ? a.i : a.r, p.row, t0, r1 - t0);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            rx[t] = IO::load(bx, own + t * bytes);
            rr[t] = IO::load(br, own + t * bytes);
            if constexpr (GATE && !BACK) ri[t] = IO::load(bi, own + t * bytes);
        }
    };
    const int64_t steps = r0 < r1 ? (r1 - r0 + kT - 1) / kT : 0;
    auto start = [&](int64_t k) { return r0 + (BACK ? steps - 1 - k : k) * kT; };
    if (steps) fetch(start(0));
    for (int64_t k = 0; k < steps; ++k) {
        const int64_t t0 = start(k);
        const int n = r1 - t0 < kT ? (int)(r1 - t0) : kT;
        float sa[kT][V], sb[kT][V];
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            float x[V], r[V], i[V] = {};
            IO::unpack(rx[t], x);
            IO::unpack(rr[t], r);
            if constexpr (GATE && !BACK) IO::unpack(ri[t], i);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                step_map<BF16, GATE && !BACK, UNIT || BACK>(x[v], r[v], i[v], t < n ? ld2[v] : 0.f, sa[t][v], sb[t][v]);
                A[v] *= sa[t][v];
            }
        }
        if (k + 1 < steps) fetch(start(k + 1));
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (BACK) B[v] = sa[kT - 1 - t][v] * (B[v] + sb[kT - 1 - t][v]);
                else B[v] = __builtin_fmaf(sa[t][v], B[v], sb[t][v]);
            }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        lds[p.wave][v][p.lane] = A[v];
        lds[p.wave][V + v][p.lane] = B[v];
    }
    __syncthreads();
    const float *from = BACK ? a.dhf : a.h0;
    if (p.seg == 0 && p.wave == 1 && p.in && from)
#pragma unroll
        for (int v = 0; v < V; ++v) a.start[p.row * a.C + p.c + v] = from[p.row * a.C + p.c + v];
    if (p.wave == 0 && p.in) {
        float *to = a.part + (p.row * a.nseg + p.seg) * 2 * a.C + p.c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float m = 1.f, b = 0.f;
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                const int w = BACK ? kW - 1 - k : k;
                b = __builtin_fmaf(lds[w][v][p.lane], b, lds[w][V + v][p.lane]);
                m *= lds[w][v][p.lane];
            }
            to[v] = m;
            to[a.C + v] = b;
        }
    }
}

// ---------------------------------------------------------------- gradients ---
// Chunks of a segment, the last first; the states come from the kept ones
template <bool BF16, int V, bool GATE, bool UNIT>
__global__ __launch_bounds__(kThreads) void bwd_kernel(const RecArgs a) {
    using IO = Io<BF16, V>;
    __shared__ float lds[2][kW][3 * V][64];
    const Place p = Place::make<V>(a);
    const unsigned bytes = (unsigned)a.C * (BF16 ? 2 : 4), own = (p.in ? p.c * (BF16 ? 2 : 4) : kOutside) + p.wave * kT * bytes;
    float ld2[V], ld[V], G[V];
    double sum[V];
    load_decay<V>(a, p, ld2);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ld[v] = p.in ? a.ld[p.c + v] : 0.f;
        G[v] = 0.f;
        sum[v] = 0.;
    }
    const float *last = a.nseg > 1 && a.dhf ? a.start : a.dhf;
    if (p.in && last)
#pragma unroll
        for (int v = 0; v < V; ++v) G[v] = last[p.row * a.C + p.c + v];
    if (p.in) {
        for (int k = a.nseg - 1; k > p.seg; --k) {
            const float *m = a.part + (p.row * a.nseg + k) * 2 * a.C + p.c;
#pragma unroll
            for (int v = 0; v < V; ++v) G[v] = __builtin_fmaf(m[v], G[v], m[a.C + v]);
        }
    }
    const int64_t end = p.s1 < p.len ? p.s1 : p.len;
    unsigned rx[kT], rr[kT], ri[GATE ? kT : 1], rd[kT];
    float hs[V] = {};
    auto fetch = [&](int64_t t0) {
        const auto bx = IO::rows(a, a.x, p.row, t0, end - t0), br = IO::rows(a, a.r, p.row, t0, end - t0);
        const auto bi = IO::rows(a, GATE ? a.i : a.r, p.row, t0, end - t0), bd = IO::rows(a, a.dy, p.row, t0, end - t0);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            rx[t] = IO::load(bx, own + t * bytes);
            rr[t] = IO::load(br, own + t * bytes);
            if constexpr (GATE) ri[t] = IO::load(bi, own + t * bytes);
            rd[t] = IO::load(bd, own + t * bytes);
        }
        if (p.in)
#pragma unroll
            for (int v = 0; v < V; ++v) hs[v] = a.states[(p.row * a.nkeep + t0 / kChunk) * a.C + p.c + v];
    };
    const int64_t nchunk = (p.s1 - p.s0 + kChunk - 1) / kChunk, live = end > p.s0 ? (end - p.s0 + kChunk - 1) / kChunk : 0;
    for (int64_t k = nchunk - 1; k >= live; --k) {
        const int64_t t0 = p.s0 + k * kChunk;
        const float zero[V] = {};
        const auto b1 = IO::rows(a, a.dx, p.row, t0, p.s1 - t0), b2 = IO::rows(a, a.dr, p.row, t0, p.s1 - t0);
        const auto b3 = IO::rows(a, GATE ? a.di : a.dr, p.row, t0, p.s1 - t0);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            IO::store(b1, own + t * bytes, zero);
            IO::store(b2, own + t * bytes, zero);
            if constexpr (GATE) IO::store(b3, own + t * bytes, zero);
        }
    }
    if (live > 0) fetch(p.s0 + (live - 1) * kChunk);
    int side = 0;
    for (int64_t k = live - 1; k >= 0; --k, side ^= 1) {
        const int64_t t0 = p.s0 + k * kChunk;
        const int n = end - t0 < kChunk ? (int)(end - t0) : kChunk;
        // of a step: a, b; E's factors in dx, in di, in d(ld s) and from there in dr; s
        float sa[kT][V], sb[kT][V], fx[kT][V], fi[GATE ? kT : 1][V], fl[kT][V], fr[kT][V], ss[kT][V], dy[kT][V];
        float A[V], B[V], D[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            B[v] = D[v] = 0.f;
            h[v] = hs[v];
        }
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            float x[V], r[V], i[V] = {};
            IO::unpack(rx[t], x);
            IO::unpack(rr[t], r);
            if constexpr (GATE) IO::unpack(ri[t], i);
            IO::unpack(rd[t], dy[t]);
            const bool valid = p.wave * kT + t < n;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float q, s1, g = 1.f, g1 = 0.f;
                const float s = sigmoid<BF16>(r[v], s1);
                decay(valid ? ld2[v] * s : 0.f, sa[t][v], q);
                q *= 2.f - q;
                if constexpr (GATE) g = sigmoid<BF16>(i[v], g1);
                float m = 1.f, inv = 0.f;
                if constexpr (!UNIT) {
                    // (below the smallest normal number the root counts as 0, and its slope too)
                    inv = q < 0x1p-126f ? 0.f : __builtin_amdgcn_rsqf(q);
                    m = q * inv;
                }
                const float u = g * x[v];
                sb[t][v] = m * u;
                fx[t][v] = m * g;
                if constexpr (GATE) fi[t][v] = m * u * g1;
                fl[t][v] = u * sa[t][v] * sa[t][v] * inv;
                fr[t][v] = ld[v] * (s * s1);
                ss[t][v] = valid ? s : 0.f;
                B[v] = __builtin_fmaf(sa[t][v], B[v], sb[t][v]);
                A[v] *= sa[t][v];
            }
        }
        if (k > 0) fetch(t0 - kChunk);
#pragma unroll
        for (int t = kT - 1; t >= 0; --t)
#pragma unroll
            for (int v = 0; v < V; ++v) D[v] = sa[t][v] * (dy[t][v] + D[v]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            lds[side][p.wave][v][p.lane] = A[v];
            lds[side][p.wave][V + v][p.lane] = B[v];
            lds[side][p.wave][2 * V + v][p.lane] = D[v];
        }
        __syncthreads();
        float hw[V], Gw[V];
#pragma unroll
        for (int w = 0; w < kW; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (w == p.wave) hw[v] = h[v];
                h[v] = __builtin_fmaf(lds[side][w][v][p.lane], h[v], lds[side][w][V + v][p.lane]);
            }
#pragma unroll
        for (int w = kW - 1; w >= 0; --w)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (w == p.wave) Gw[v] = G[v];
                G[v] = __builtin_fmaf(lds[side][w][v][p.lane], G[v], lds[side][w][2 * V + v][p.lane]);
            }
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float kept = sa[t][v] * hw[v];
                fl[t][v] = kept - fl[t][v];
                hw[v] = kept + sb[t][v];
            }
        const auto b1 = IO::rows(a, a.dx, p.row, t0, p.s1 - t0), b2 = IO::rows(a, a.dr, p.row, t0, p.s1 - t0);
        const auto b3 = IO::rows(a, GATE ? a.di : a.dr, p.row, t0, p.s1 - t0);
        float dl[V] = {};
#pragma unroll
        for (int t = kT - 1; t >= 0; --t) {
            float ox[V], orr[V], oi[V];
            const bool valid = p.wave * kT + t < n;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float E = valid ? dy[t][v] + Gw[v] : 0.f, d = E * fl[t][v];
                ox[v] = E * fx[t][v];
                orr[v] = d * fr[t][v];
                if constexpr (GATE) oi[v] = E * fi[t][v];
                dl[v] = __builtin_fmaf(d, ss[t][v], dl[v]);
                Gw[v] = valid ? sa[t][v] * E : Gw[v];
            }
            IO::store(b1, own + t * bytes, ox);
            IO::store(b2, own + t * bytes, orr);
            if constexpr (GATE) IO::store(b3, own + t * bytes, oi);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] += dl[v];
    }
    if (a.dh0 && p.in && p.wave == 0 && p.seg == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) a.dh0[p.row * a.C + p.c + v] = G[v];
    if (a.dpart) {
        double(*join)[V][64] = reinterpret_cast<double(*)[V][64]>(&lds[0][0][0][0]);
        static_assert(sizeof(double) * kW * V * 64 <= sizeof(lds), "the sums fit");
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) join[p.wave][v][p.lane] = sum[v];
        __syncthreads();
        if (p.wave == 0 && p.in)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                double d = 0.;
#pragma unroll
                for (int w = 0; w < kW; ++w) d += join[w][v][p.lane];
                a.dpart[(p.row * a.nseg + p.seg) * a.C + p.c + v] = d;
            }
    }
}

// dld[c]: the sums of all rows and segments, in a fixed order
constexpr int kRuns = 4;
__global__ __launch_bounds__(64 * kRuns) void decay_sums_kernel(const double *part, int64_t rows, int C, float *dld) {
    __shared__ double lds[kRuns][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    double d = 0.;
    if (c < C)
        for (int64_t r = run; r < rows; r += kRuns) d += part[r * C + c];
    lds[run][lane] = d;
    __syncthreads();
    if (run == 0 && c < C) dld[c] = (float)(lds[0][lane] + lds[1][lane] + lds[2][lane] + lds[3][lane]);
}

// ------------------------------------------------------------- single token ---
template <bool BF16, int V, bool GATE, bool UNIT>
__global__ __launch_bounds__(256) void step_kernel(const void *x, const void *r, const void *i, const float *ld, float *h,
                                                   void *y, int64_t n, int C) {
    for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; at < n; at += (int64_t)gridDim.x * 256 * V) {
        const int c = (int)(at % C);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a, b;
            step_map<BF16, GATE, UNIT>(ld_io<BF16>(x, at + v), ld_io<BF16>(r, at + v), GATE ? ld_io<BF16>(i, at + v) : 0.f,
                                       ld[c + v] * 1.4426950408889634f, a, b);
            const float s = __builtin_fmaf(a, h[at + v], b);
            h[at + v] = s;
            if constexpr (BF16) static_cast<__bf16 *>(y)[at + v] = (__bf16)s;
            else static_cast<float *>(y)[at + v] = s;
        }
    }
}

// --------------------------------------------------------------------- host ---
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct RecPlan {
    int V;
    int64_t cols, nseg, seg, nkeep, groups;  // groups: workgroups of a launch
    size_t states, part, dpart;              // bytes
};

m3_status rec_check(const m3_rec_shape *s) {
    if (!s) return M3_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1 || s->nsegments < 0 || s->reserved) return M3_ERR_INVALID_ARG;
    if (s->io_dtype != M3_F32 && s->io_dtype != M3_BF16) return M3_ERR_INVALID_ARG;
    if (s->flags & ~(uint32_t)M3_REC_UNSCALED) return M3_ERR_INVALID_ARG;
    if (s->channels > (1 << 20) || s->batch > (1LL << 31) || s->seqlen > (1LL << 40) ||
        (s->seqlen > 0 && s->batch > (1LL << 40) / s->seqlen))
        return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

m3_status rec_plan(const m3_rec_shape *s, RecPlan *p) {
    const m3_status st = rec_check(s);
    if (st != M3_OK) return st;
    p->V = s->io_dtype == M3_BF16 && s->channels % 2 == 0 ? 2 : 1;
    p->cols = ceil_div(s->channels, 64 * p->V);
    p->nkeep = ceil_div(s->seqlen, kChunk);
    const int64_t wide = s->batch * p->cols;
    int64_t k = s->nsegments;
    if (k == 0) k = wide >= 192 || wide == 0 ? 1 : ceil_div(512, wide) < 64 ? ceil_div(512, wide) : 64;
    // whole chunks, four at least where the split is picked here
    int64_t chunks = ceil_div(p->nkeep, k);
    if (s->nsegments == 0 && chunks < 4) chunks = 4;
    if (chunks < 1) chunks = 1;
    p->seg = chunks * kChunk;
    p->nseg = p->nkeep ? ceil_div(p->nkeep, chunks) : 1;
    if (wide > kMaxGrid || wide * p->nseg > kMaxGrid) return M3_ERR_UNSUPPORTED;
    p->groups = wide * p->nseg;
    p->states = up((size_t)(s->batch * p->nkeep * s->channels) * sizeof(float));
    p->part = p->nseg > 1 ? up((size_t)(s->batch * (2 * p->nseg + 1) * s->channels) * sizeof(float)) : 0;
    p->dpart = up((size_t)(s->batch * p->nseg * s->channels) * sizeof(double));
    return M3_OK;
}

RecArgs rec_args(const m3_rec_shape &s, const m3_rec_io &io, const RecPlan &p) {
    RecArgs a{};
    a.x = io.x; a.r = io.decay_gate; a.i = io.input_gate; a.ld = io.log_decay; a.h0 = io.h0; a.lengths = io.lengths;
    a.L = s.seqlen; a.C = (int)s.channels; a.cols = (int)p.cols; a.nseg = (int)p.nseg; a.nkeep = (int)p.nkeep;
    a.seg = p.seg;
    return a;
}

void set_part(RecArgs &a, void *at, int64_t batch) {
    a.part = static_cast<float *>(at);
    a.start = a.part + batch * a.nseg * 2 * a.C;
}

template <bool BF16, int V, bool GATE, bool UNIT>
hipError_t launch_fwd(const RecArgs &a, const RecPlan &p, hipStream_t s) {
    const dim3 g((unsigned)p.groups), t(kThreads);
    if (p.nseg > 1) {
        hipLaunchKernelGGL((map_kernel<BF16, V, GATE, UNIT, false>), g, t, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((fwd_kernel<BF16, V, GATE, UNIT>), g, t, 0, s, a);
    return hipGetLastError();
}

template <bool BF16, int V, bool GATE, bool UNIT>
hipError_t launch_bwd(const RecArgs &a, const RecPlan &p, hipStream_t s) {
    const dim3 g((unsigned)p.groups), t(kThreads);
    if (p.nseg > 1) {
        hipLaunchKernelGGL((map_kernel<BF16, V, GATE, UNIT, true>), g, t, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((bwd_kernel<BF16, V, GATE, UNIT>), g, t, 0, s, a);
    return hipGetLastError();
}

template <bool BF16, int V, bool GATE, bool UNIT>
hipError_t launch_step(const m3_rec_shape &s, const m3_rec_step_io &io, hipStream_t hs) {
    const int64_t n = s.batch * s.channels, g = ceil_div(n, 256 * V);
    hipLaunchKernelGGL((step_kernel<BF16, V, GATE, UNIT>), dim3((unsigned)(g < kMaxGrid ? g : kMaxGrid)), dim3(256), 0, hs, io.x,
                       io.decay_gate, io.input_gate, io.log_decay, io.h, io.y, n, (int)s.channels);
    return hipGetLastError();
}

// f<BF16, V, GATE, UNIT>(...) of the shape at hand
#define M3_REC_PICK(f, shape, V, gate, ...)                                                        \
    [&]() -> hipError_t {                                                                          \
        const bool unit = ((shape).flags & M3_REC_UNSCALED) != 0;                                  \
        if ((shape).io_dtype != M3_BF16)                                                           \
            return gate ? (unit ? f<false, 1, true, true>(__VA_ARGS__) : f<false, 1, true, false>(__VA_ARGS__))    \
                        : (unit ? f<false, 1, false, true>(__VA_ARGS__) : f<false, 1, false, false>(__VA_ARGS__)); \
        if (V == 1)                                                                                \
            return gate ? (unit ? f<true, 1, true, true>(__VA_ARGS__) : f<true, 1, true, false>(__VA_ARGS__))      \
                        : (unit ? f<true, 1, false, true>(__VA_ARGS__) : f<true, 1, false, false>(__VA_ARGS__));   \
        return gate ? (unit ? f<true, 2, true, true>(__VA_ARGS__) : f<true, 2, true, false>(__VA_ARGS__))          \
                    : (unit ? f<true, 2, false, true>(__VA_ARGS__) : f<true, 2, false, false>(__VA_ARGS__));       \
    }()

}  // namespace
}  // namespace m3i

using namespace m3i;

extern "C" {

size_t m3_recurrence_workspace_bytes(const m3_rec_shape *shape) {
    RecPlan p;
    return rec_plan(shape, &p) == M3_OK ? p.part : 0;
}

size_t m3_recurrence_bwd_workspace_bytes(const m3_rec_shape *shape, int states) {
    RecPlan p;
    return rec_plan(shape, &p) == M3_OK ? (states ? 0 : p.states) + p.part + p.dpart : 0;
}

m3_status m3_recurrence_fwd(const m3_rec_shape *shape, const m3_rec_io *io, void *workspace, size_t ws_bytes, void *stream) {
    RecPlan p;
    const m3_status st = rec_plan(shape, &p);
    if (st != M3_OK) return st;
    if (!io) return M3_ERR_INVALID_ARG;
    if (shape->batch > 0 && (!io->log_decay || (shape->seqlen > 0 && (!io->x || !io->decay_gate || !io->y))))
        return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->x, io->decay_gate, io->input_gate, io->log_decay, io->h0, io->lengths, io->y, io->h_final,
                          io->states, workspace};
    for (const void *q : ptrs)
        if (!al16(q)) return M3_ERR_MISALIGNED;
    if (p.part && (!workspace || ws_bytes < p.part)) return M3_ERR_WORKSPACE_TOO_SMALL;
    void *ws = p.part ? workspace : nullptr;
    if (clash({io->y, io->states, ws}, {io->x, io->decay_gate, io->input_gate, io->log_decay, io->h0, io->lengths, io->h_final}) ||
        clash({io->h_final}, {io->x, io->decay_gate, io->input_gate, io->log_decay, io->lengths}))
        return M3_ERR_INVALID_ARG;
    if (p.groups == 0) return M3_OK;
    RecArgs a = rec_args(*shape, *io, p);
    a.y = io->y; a.hf = io->h_final; a.states = io->states;
    set_part(a, workspace, shape->batch);
    const hipError_t e = M3_REC_PICK(launch_fwd, *shape, p.V, a.i != nullptr, a, p, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

m3_status m3_recurrence_bwd(const m3_rec_shape *shape, const m3_rec_io *io, const m3_rec_grads *gr, void *workspace,
                            size_t ws_bytes, void *stream) {
    RecPlan p;
    const m3_status st = rec_plan(shape, &p);
    if (st != M3_OK) return st;
    if (!io || !gr) return M3_ERR_INVALID_ARG;
    if (shape->batch > 0 &&
        (!io->log_decay || (shape->seqlen > 0 && (!io->x || !io->decay_gate || !gr->dy || !gr->dx || !gr->ddecay_gate ||
                                                  (io->input_gate == nullptr) != (gr->dinput_gate == nullptr)))))
        return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->x, io->decay_gate, io->input_gate, io->log_decay, io->h0, io->lengths, io->states, gr->dy,
                          gr->dh_final, gr->dx, gr->ddecay_gate, gr->dinput_gate, gr->dlog_decay, gr->dh0, workspace};
    for (const void *q : ptrs)
        if (!al16(q)) return M3_ERR_MISALIGNED;
    const size_t own_states = io->states ? 0 : p.states, need = own_states + p.part + p.dpart;
    if (need && (!workspace || ws_bytes < need)) return M3_ERR_WORKSPACE_TOO_SMALL;
    void *ws = need ? workspace : nullptr;
    if (clash({gr->dx, gr->ddecay_gate, gr->dinput_gate, gr->dlog_decay, ws},
              {io->x, io->decay_gate, io->input_gate, io->log_decay, io->h0, io->lengths, io->states, gr->dy, gr->dh_final,
               gr->dh0}) ||
        clash({gr->dh0}, {io->x, io->decay_gate, io->input_gate, io->log_decay, io->h0, io->lengths, io->states, gr->dy}))
        return M3_ERR_INVALID_ARG;
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    char *at = static_cast<char *>(workspace);
    RecArgs a = rec_args(*shape, *io, p);
    hipError_t e = hipSuccess;
    a.states = io->states ? io->states : reinterpret_cast<float *>(at);
    set_part(a, at + own_states, shape->batch);
    if (p.groups > 0) {
        if (!io->states && shape->seqlen > 0)
            e = M3_REC_PICK(launch_fwd, *shape, p.V, a.i != nullptr, a, p, hs);
        a.dy = gr->dy; a.dhf = gr->dh_final; a.dx = gr->dx; a.dr = gr->ddecay_gate; a.di = gr->dinput_gate;
        a.dld = gr->dlog_decay; a.dh0 = gr->dh0;
        a.dpart = gr->dlog_decay ? reinterpret_cast<double *>(at + own_states + p.part) : nullptr;
        if (e == hipSuccess) e = M3_REC_PICK(launch_bwd, *shape, p.V, a.i != nullptr, a, p, hs);
    }
    if (e == hipSuccess && gr->dlog_decay) {
        hipLaunchKernelGGL(decay_sums_kernel, dim3((unsigned)ceil_div(shape->channels, 64)), dim3(64 * kRuns), 0, hs, a.dpart,
                           shape->batch * p.nseg, (int)shape->channels, gr->dlog_decay);
        e = hipGetLastError();
    }
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

m3_status m3_recurrence_step(const m3_rec_shape *shape, const m3_rec_step_io *io, void *stream) {
    const m3_status st = rec_check(shape);
    if (st != M3_OK) return st;
    if (!io) return M3_ERR_INVALID_ARG;
    if (shape->batch > 0 && (!io->x || !io->decay_gate || !io->log_decay || !io->h || !io->y)) return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->x, io->decay_gate, io->input_gate, io->log_decay, io->h, io->y};
    for (const void *q : ptrs)
        if (!al16(q)) return M3_ERR_MISALIGNED;
    if (clash({io->h, io->y}, {io->x, io->decay_gate, io->input_gate, io->log_decay})) return M3_ERR_INVALID_ARG;
    if (shape->batch == 0) return M3_OK;
    const int V = shape->io_dtype == M3_BF16 && shape->channels % 2 == 0 ? 2 : 1;
    const hipError_t e =
        M3_REC_PICK(launch_step, *shape, V, io->input_gate != nullptr, *shape, *io, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

}  // extern "C"
