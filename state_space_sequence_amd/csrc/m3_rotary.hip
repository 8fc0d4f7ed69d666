// Rotary positions: queries and keys turned by their positions (gfx950).
//
//   (u', w') = scale (u cos t - w sin t, u sin t + w cos t),  t = pos freqs[i];  backwards with -t
//
// Bound by HBM: q and k read and written once. A lane has an item of a head, 16 bytes of it (two pieces of 16 bytes, their
// distance half of the turned channels, in the layout of halves): it forms the item's cosines and sines once and takes
// head after head of its token with them, q's and then k's. A wave has one token, or several where their heads do not fill it; with few
// tokens their heads go to several waves. The angle is formed in turns, whose whole ones are dropped before it
// is rounded to fp32: b8 L4096, 64 + 8 heads of 128, bf16 215 us (5.6 TB/s); two or four heads ahead, and
// more waves for few tokens, change nothing.
#include <math.h>

#include "m3_internal.h"
#include "m3_rotary.h"

namespace m3i {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256, kAhead = 3;  // heads whose loads are in flight
constexpr int64_t kMaxGrid = 0xffffff, kLastCache = 256 << 20;

struct RotArgs {
    const void *q, *k;
    void *qo, *ko;
    const float *freqs;
    const int *positions, *offsets;
    int64_t L, tokens, units;  // units: waves' pieces of work
    int H, G, D, half;         // half: pairs of a head
    int items, lanes, chunks;  // items of a head; those of a wave at a time, and times it takes
    int heads, toks, split;    // heads and tokens of a wave at a time; waves that share a token's heads
    float scale;
    bool back, past;
};

// V values of one dtype
template <bool BF16, int V>
struct Vec {
    static constexpr int W = V == 1 ? 1 : (BF16 ? V / 2 : V);
    typedef unsigned words __attribute__((ext_vector_type(W)));  // (aligned to its size)
    unsigned w[W];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        if constexpr (V == 1) {
            if constexpr (BF16) w[0] = static_cast<const uint16_t *>(p)[i];
            else w[0] = static_cast<const unsigned *>(p)[i];
        } else {
            const words v = __builtin_nontemporal_load(
                reinterpret_cast<const words *>(static_cast<const char *>(p) + i * (BF16 ? 2 : 4)));
#pragma unroll
            for (int e = 0; e < W; ++e) w[e] = v[e];
        }
    }
    __device__ __forceinline__ void store(void *p, int64_t i, bool past) const {
        if constexpr (V == 1) {
            if constexpr (BF16) static_cast<uint16_t *>(p)[i] = (uint16_t)w[0];
            else static_cast<unsigned *>(p)[i] = w[0];
        } else {
            words v;
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = w[e];
            words *to = reinterpret_cast<words *>(static_cast<char *>(p) + i * (BF16 ? 2 : 4));
            if (past) {
                asm volatile("");  // (two equal stores but for their hint would become one)
                __builtin_nontemporal_store(v, to);
                asm volatile("");
            } else {
                *to = v;
            }
        }
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (!BF16) return __uint_as_float(w[e]);
        else return __uint_as_float(V > 1 && e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
    // x[e] in the place of all values
    __device__ __forceinline__ void set(const float (&x)[V]) {
        if constexpr (!BF16) {
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] = __float_as_uint(x[e]);
        } else if constexpr (V == 1) {
            w[0] = __builtin_bit_cast(uint16_t, (__bf16)x[0]);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e)
                w[e] = __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x[2 * e], x[2 * e + 1]}), bf16x2));
        }
    }
};

// Cosine and sine of pos * freq, times scale. The product and its turns are kept to twice the bits of fp64 until whole turns
// are dropped (1/(2 pi) in two parts, what each product leaves behind by an FMA): of 2^31 positions at a frequency of 1 a
// product of fp64 alone is off by 2^-21 rad. What the fraction loses as an fp32 number goes in behind.
__device__ __forceinline__ void turn(const RotArgs &a, double pos, float freq, float &c, float &s) {
#pragma clang fp contract(off)  // (t - rint(t) of the rounded t)
    constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
    const double p = pos * (double)freq, left = __builtin_fma(pos, (double)freq, -p), t = p * kHigh;
    double f = __builtin_fma(p, kHigh, -t) + __builtin_fma(p, kLow, left * kHigh);
    f += t - __builtin_rint(t);
    f -= __builtin_rint(f);
    const float near = (float)f, d = (float)((f - (double)near) * 6.283185307179586);
    float c0, s0;
    sincospif(2.f * near, &s0, &c0);
    c = __builtin_fmaf(-s0, d, c0) * a.scale;
    s = __builtin_fmaf(c0, d, s0) * (a.back ? -a.scale : a.scale);
}

// PAIRED: pairs are neighbours, an item is V channels (V = 1: two); else an item is V channels and those `half` further.
// Items behind the pairs are copies of V channels (V = 1: one).
template <bool BF16, int V, bool PAIRED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const RotArgs a) {
    constexpr int P = V == 1 ? 1 : (PAIRED ? V / 2 : V);  // pairs of an item
    using X = Vec<BF16, V>;
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * (kThreads / 64);
    const int turned = (a.half + P - 1) / P;  // items with pairs (the last one may have fewer, and copies)
    for (int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < a.units;
         unit += waves) {
        const int chunk = (int)(unit % a.chunks);
        const int part = (int)(unit / a.chunks % a.split);
        const int64_t token = unit / a.chunks / a.split * a.toks + lane / (a.lanes * a.heads);
        const int item = chunk * a.lanes + lane % a.lanes, first = lane / a.lanes % a.heads + part * a.heads;
        if (lane >= a.lanes * a.heads * a.toks || item >= a.items || token >= a.tokens) continue;
        const bool pairs = item < turned;
        float c[P], s[P];
        // first channel of the item, and of its second piece (V = 1, or not PAIRED)
        int at, other;
        if (pairs) {
            double pos;
            if (a.positions) pos = a.positions[token];
            else {
                const int64_t row = token / a.L;
                pos = (double)(token - row * a.L + (a.offsets ? (int64_t)a.offsets[row] : 0));
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const int i = item * P + e;
                turn(a, pos, i < a.half ? a.freqs[i] : 0.f, c[e], s[e]);
            }
            at = V == 1 && PAIRED ? 2 * item : item * V;
            other = PAIRED ? at + 1 : at + a.half;
        } else {
            at = other = PAIRED && V > 1 ? item * V : 2 * a.half + (item - turned) * V;
        }
        const bool two = pairs && (!PAIRED || V == 1);
        const int step = a.heads * a.split, all = a.H + a.G;
        auto place = [&](int h, const void *q, const void *k, const void *&p, int64_t &i) {
            const bool of_q = h < a.H;
            p = of_q ? q : k;
            i = (token * (of_q ? a.H : a.G) + (of_q ? h : h - a.H)) * a.D;
        };
        for (int h0 = first; h0 < all; h0 += kAhead * step) {
            X u[kAhead], w[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
                const int h = h0 + n * step;
                if (h < all) {
                    const void *p;
                    int64_t i;
                    place(h, a.q, a.k, p, i);
                    u[n].load(p, i + at);
                    if (two) w[n].load(p, i + other);
                }
            }
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
                const int h = h0 + n * step;
                if (h >= all) continue;
                const void *p;
                int64_t i;
                place(h, a.qo, a.ko, p, i);
                if (pairs) {
                    float x[V], y[V];
                    if constexpr (PAIRED && V > 1) {
#pragma unroll
                        for (int e = 0; e < P; ++e) {
                            const float g = u[n].get(2 * e), b = u[n].get(2 * e + 1);
                            const bool on = item * P + e < a.half;  // (copies as they are, whatever they hold)
                            x[2 * e] = on ? __builtin_fmaf(g, c[e], -(b * s[e])) : g;
                            x[2 * e + 1] = on ? __builtin_fmaf(g, s[e], b * c[e]) : b;
                        }
                        u[n].set(x);
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float g = u[n].get(e), b = w[n].get(e);
                            x[e] = __builtin_fmaf(g, c[e], -(b * s[e]));
                            y[e] = __builtin_fmaf(g, s[e], b * c[e]);
                        }
                        u[n].set(x);
                        w[n].set(y);
                    }
                }
                u[n].store(const_cast<void *>(p), i + at, a.past);
                if (two) w[n].store(const_cast<void *>(p), i + other, a.past);
            }
        }
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

m3_status rotary_check(const m3_rotary_shape *s, bool k) {
    if (!s) return M3_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->nheads < 1 || (k && s->ngroups < 1) || s->headdim < 1 || s->rotary < 0 ||
        s->rotary > s->headdim || s->rotary % 2 != 0 || s->reserved || !isfinite(s->scale))
        return M3_ERR_INVALID_ARG;
    if (s->io_dtype != M3_F32 && s->io_dtype != M3_BF16) return M3_ERR_INVALID_ARG;
    if (s->flags & ~(uint32_t)(M3_ROTARY_INTERLEAVED | M3_ROTARY_BACKWARD)) return M3_ERR_INVALID_ARG;
    if (s->headdim > 1024 || s->nheads > 4096 || (k && s->ngroups > 4096)) return M3_ERR_UNSUPPORTED;
    const int64_t each = (s->nheads + (k ? s->ngroups : 0)) * s->headdim, most = (1LL << 40) / each;
    if (s->batch > most || s->seqlen > most || (s->seqlen > 0 && s->batch > most / s->seqlen)) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

template <bool BF16, int V>
hipError_t launch(const RotArgs &a, bool paired, hipStream_t s) {
    const int64_t g = ceil_div(a.units, kThreads / 64);
    const dim3 grid((unsigned)(g < kMaxGrid ? g : kMaxGrid)), t(kThreads);
    if (paired) hipLaunchKernelGGL((rotary_kernel<BF16, V, true>), grid, t, 0, s, a);
    else hipLaunchKernelGGL((rotary_kernel<BF16, V, false>), grid, t, 0, s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace m3i

using namespace m3i;

extern "C" m3_status m3_rotary(const m3_rotary_shape *shape, const m3_rotary_io *io, void *stream) {
    const m3_status st = rotary_check(shape, io && io->k);
    if (st != M3_OK) return st;
    if (!io) return M3_ERR_INVALID_ARG;
    const m3_rotary_shape &s = *shape;
    if ((io->k == nullptr) != (io->k_out == nullptr) || (io->positions && io->offsets)) return M3_ERR_INVALID_ARG;
    if (s.batch * s.seqlen > 0 && (!io->q || !io->q_out || (s.rotary > 0 && !io->freqs))) return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->q, io->k, io->freqs, io->positions, io->offsets, io->q_out, io->k_out};
    for (const void *p : ptrs)
        if (!al16(p)) return M3_ERR_MISALIGNED;
    if (clash({io->q_out, io->k_out}, {io->freqs, io->positions, io->offsets}) || clash({io->q_out}, {io->k}) ||
        clash({io->k_out}, {io->q}))
        return M3_ERR_INVALID_ARG;
    RotArgs a{};
    a.tokens = s.batch * s.seqlen;
    if (a.tokens == 0) return M3_OK;
    const bool bf16 = s.io_dtype == M3_BF16, paired = s.flags & M3_ROTARY_INTERLEAVED, in_place = io->q == io->q_out &&
                                                                                              (!io->k || io->k == io->k_out);
    a.q = io->q; a.k = io->k; a.qo = io->q_out; a.ko = io->k_out; a.freqs = io->freqs; a.positions = io->positions;
    a.offsets = io->offsets; a.L = s.seqlen; a.H = (int)s.nheads; a.G = io->k ? (int)s.ngroups : 0; a.D = (int)s.headdim;
    a.half = (int)(s.rotary / 2); a.scale = s.scale; a.back = s.flags & M3_ROTARY_BACKWARD;
    // 16 bytes at a time, in bf16 8 (halves, D 96 with 40 turned, b4 L4096, 16 + 4 heads: 42 us, one value at a time
    // 67; D 72: 26 and 38), where every piece is aligned to them; pieces of two values are slower than single ones
    // (D 100, halves: bf16 56 us and 41, fp32 57 and 50)
    int V = bf16 ? 8 : 4;
    while (V > 1 && (s.headdim % V || (!paired && a.half % V))) V = V > 4 ? 4 : 1;
    const int rest = a.D - 2 * a.half;
    if (paired && V > 1) a.items = in_place ? (int)ceil_div(2 * a.half, V) : a.D / V;
    else a.items = a.half / V + (in_place ? 0 : rest / V);
    if (a.items == 0) return M3_OK;
    const int all = a.H + a.G;
    a.lanes = a.items < 64 ? a.items : 64;
    a.chunks = (int)ceil_div(a.items, a.lanes);
    a.heads = 64 / a.lanes < all ? 64 / a.lanes : all;
    a.toks = 64 / (a.lanes * a.heads);
    const int64_t groups = ceil_div(a.tokens, a.toks) * a.chunks, rounds = ceil_div(all, a.heads);
    // (waves enough for the card's 1024 SIMDs)
    a.split = groups >= 2048 ? 1 : (int)(ceil_div(2048, groups) < rounds ? ceil_div(2048, groups) : rounds);
    a.units = groups * a.split;
    a.past = a.tokens * all * a.D > kLastCache / (bf16 ? 4 : 8);
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = bf16 ? (V == 8   ? launch<true, 8>(a, paired, hs)
                                 : V == 4 ? launch<true, 4>(a, paired, hs)
                                          : launch<true, 1>(a, paired, hs))
                              : (V == 4 ? launch<false, 4>(a, paired, hs) : launch<false, 1>(a, paired, hs));
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}
