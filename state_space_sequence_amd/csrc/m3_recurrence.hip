// Gated linear recurrence, one state a channel: prompt, gradients, single token (gfx950).
//
//   s = sigmoid(r), g = sigmoid(i) or 1, a = exp(ld s), m = sqrt(1 - a^2) or 1
//   h_t = a_t h_{t-1} + m_t g_t x_t
//   G_t = a_t (dy_t + G_{t+1}) is the gradient of h_{t-1}; with E_t = dy_t + G_{t+1}, that of h_t:
//   dx = E m g, di = E m x g (1-g), d(ld s) = E (a h_{t-1} - g x a^2 / m), dr = d(ld s) ld s (1-s), dld = sum d(ld s) s
//
// A step is the map h -> A h + B, and maps in a row are one map again: (A2 A1, A2 B1 + B2). A workgroup of eight waves has a
// column of 64 lanes of channels (4 bytes each) of a row and takes its tokens tile by tile: a wave forms the gates of its
// run of 16 tokens (8 with gradients), all in registers, and their joint map; the maps of the runs meet in LDS, and each wave runs
// its tokens from the state that the maps before it give. One pass over the data. Backwards the same in both
// directions at once: states forwards from the kept one at the tile's start, G backwards.
//
// With few columns several workgroups share one, and the state that a tile starts from comes through memory (CHAIN). A
// tile publishes its map as soon as it has it, and the state behind it later; one that needs its start looks at the
// kWindow tiles before it for the nearest known state and the maps from there (the published scan in a single pass with decoupled
// look-back, of Merrill and Garland, 2016, for these maps). The state behind a tile is
// A h + B of its joint map wherever it is formed, so the bits do not depend on who was first. A word is written and read
// by one atomic access and is there whole or not at all, without fences or flags. A wait ends: the tiles of a column are
// taken in order from a counter, a workgroup does what it took in that order, and a tile needs nothing from later ones.
//
// Bound by HBM and, nearly as much, by vector issue: 34 instructions an element, 5 of them exponentials, reciprocals and roots, 53 ns
// an element of a wave on a SIMD, so 110 us of the prompt's 211. bf16, with an input gate, times of a call: prompt b8 L4096 of
// 4096 channels 211 us (5.1 TB/s), long b2 L32768 of 2560 in a chain 288 (4.7 TB/s), gradients b8 L2048 of 4096 201 (4.7 TB/s).
#include <math.h>

#include <type_traits>

#include "m3_internal.h"
#include "m3_recurrence.h"

namespace m3i {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kW = 8, kThreads = 64 * kW;        // runs of a tile, one a wave
constexpr int kFwd = 16, kBwd = 8;               // tokens of a run
// Tiles before it that a tile looks at: gradients b2 L32768 of 2560 channels 591 us, with eight 621 (more registers), a
// single column of 16384 tokens 37 us, with eight 28
constexpr int kWindow = 4;
constexpr int kSlots = 256;                      // workgroups that run at a time: one a CU
constexpr int64_t kMaxGrid = 0x7fffff;           // workgroups of one launch: 2^32 threads
constexpr unsigned kOutside = 0x80000000u;       // a byte offset behind every buffer (tiles are at most 2^29 bytes)
constexpr uint64_t kEmpty = ~0ull;               // (a word of 64 bits; of 32: its half)
constexpr int kPast = 2;                         // buffer accesses past the caches
static_assert(kW * kBwd == M3_REC_KEEP && M3_REC_KEEP % kFwd == 0, "kept states are at the start of runs and of tiles");

struct RecArgs {
    const void *x, *r, *i;
    const float *ld, *h0;
    const int *lengths;
    void *y;
    float *hf, *states;
    const void *dy;
    const float *dhf;
    void *dx, *dr, *di;
    float *dh0;
    float *dpart;     // [b][ntile][C]: sums of dld
    uint64_t *maps;   // [b][ntile][C]: maps of the tiles, in the order of the chain
    unsigned *ends;   // [b][ntile][C]: the states behind them
    unsigned *begins; // [b][C]: what the chain starts from
    unsigned *taken;  // [b][cols]: tiles taken so far
    int64_t L;
    int C, cols, ntile, nkeep;  // tiles across the channels and along the tokens, kept states of a row
    unsigned columns;           // batch * cols
    int turns;                  // tiles that a workgroup takes at most, one after another
};

// V channels of one token of a lane, as they lie in memory, by buffer accesses: what lies
// behind the buffer reads as 0 and is not written
template <bool BF16, int V>
struct Io {
    static constexpr int B = (BF16 ? 2 : 4) * V, W = (B + 3) / 4;  // bytes and words of a lane and token
    static_assert(B == 2 || B == 4, "an access of two or four bytes");
    struct raw { unsigned w[W]; };
    using rsrc_t = decltype(__builtin_amdgcn_make_buffer_rsrc(static_cast<void *>(nullptr), 0, 0, 0));
    // tokens t0 .. t0 + n - 1 of a row
    static __device__ __forceinline__ rsrc_t rows(const RecArgs &a, const void *p, int64_t row, int64_t t0, int n) {
        constexpr int E = BF16 ? 2 : 4;
        const char *at = static_cast<const char *>(p) + (row * a.L + t0) * a.C * E;
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(at), 0, n * a.C * E, 0x00020000);
    }
    static __device__ __forceinline__ raw load(rsrc_t r, unsigned at) {
        raw o;
        if constexpr (B == 4) o.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, kPast);
        else o.w[0] = __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, kPast);
        return o;
    }
    // (the words stay packed until here: unpacked ahead, as the compiler would, two paths' values spill)
    static __device__ __forceinline__ void unpack(raw o, float (&v)[V]) {
#pragma unroll
        for (int e = 0; e < W; ++e) asm volatile("" : "+v"(o.w[e]));
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if constexpr (!BF16) v[e] = __uint_as_float(o.w[e]);
            else v[e] = __uint_as_float(e % 2 ? o.w[e / 2] & 0xffff0000u : o.w[e / 2] << 16);
        }
    }
    static __device__ __forceinline__ void store(rsrc_t r, unsigned at, const float (&v)[V]) {
        unsigned w[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
            if constexpr (!BF16) w[e] = __float_as_uint(v[e]);
            else if constexpr (V == 1) w[e] = __builtin_bit_cast(uint16_t, (__bf16)v[0]);
            else w[e] = __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{v[2 * e], v[2 * e + 1]}), bf16x2));
        }
        if constexpr (B == 4) __builtin_amdgcn_raw_buffer_store_b32(w[0], r, at, 0, kPast);
        else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)w[0], r, at, 0, 0);
    }
};

// The sigmoid, and 1 - sigmoid without cancellation (where e^-x overflows: any finite factor of 0). bf16: the
// hardware exponential of a rounded argument is off by |x| 2^-23, far below the rounding of outputs in bf16. The fp32 states take it
// as it is, each term off by that much of itself; an exact argument would cost an exponential more a gate, and issue is a bound here
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

// a = 2^l and p = 1 - a for l <= 0: 2^f - 1 = f P(f) for the rest f of l from its nearest whole
// number n, P the polynomial of degree 5 that is closest over |f| <= 1/2 (fitted here; 2.1e-8 relative with fp32 coefficients). p has no
// cancellation: for n = 0 it is -f P(f), else at least 0.29. With all roundings a is off by at most 1.6 * 2^-24 of itself and p by 2.1.
// A state of slow decay keeps what hundreds of steps bring, so a and m must not be off in one direction: on average both
// are by less than 0.12 * 2^-24.
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

// The same for kMild <= l <= 0, where one polynomial of degree 6 gives p (fitted here; 9.8e-9 relative) without a division
// of the range: 8 operations in place of 13. p is off by at most 2.1 * 2^-24, a = 1 - p by 1.5 where l > -1/2, else by 3.8. A channel's l is
// between 0 and its log_decay in powers of 2
constexpr float kMild = -1.5f;
__device__ __forceinline__ void mild_decay(float l, float &a, float &p) {
    float q = __builtin_fmaf(l, -0x1.458340p-17f, -0x1.2c9900p-13f);
    q = __builtin_fmaf(q, l, -0x1.5ab9a6p-10f);
    q = __builtin_fmaf(q, l, -0x1.3afb90p-7f);
    q = __builtin_fmaf(q, l, -0x1.c6ad90p-5f);
    q = __builtin_fmaf(q, l, -0x1.ebfbcep-3f);
    q = __builtin_fmaf(q, l, -0x1.62e430p-1f);
    p = l * q;
    a = 1.f - p;
}

// the step's map h -> a h + b of one channel
template <bool BF16, bool GATE, bool UNIT, bool MILD>
__device__ __forceinline__ void step_map(float x, float r, float i, float ld2, float &a, float &b) {
    float p;
    const float l = ld2 * sigmoid<BF16>(r);
    if constexpr (MILD) mild_decay(l, a, p);
    else decay(l, a, p);
    b = GATE ? x * sigmoid<BF16>(i) : x;
    if constexpr (!UNIT) b *= __builtin_amdgcn_sqrtf(p * (2.f - p));  // 1 - a^2 = p (2 - p)
}

// -------------------------------------------------------------------- tiles ---
// The column of a workgroup, 64 lanes of V channels of a row, and the tiles of it that it takes
template <bool BF16, int V, int T, bool CHAIN>
struct Column {
    static constexpr int kTile = kW * T;
    int row, lane, wave;
    int c;       // this lane's first channel
    bool in;     // (it has channels)
    unsigned at, bytes, own;  // the column's number; bytes of a token; this lane's first offset in a tile
    int64_t len;
    __device__ __forceinline__ explicit Column(const RecArgs &a) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        at = blockIdx.x % a.columns;
        row = at / a.cols;
        c = ((int)(at % a.cols) * 64 + lane) * V;
        in = c < a.C;
        bytes = (unsigned)a.C * (BF16 ? 2 : 4);
        own = (in ? c * (BF16 ? 2 : 4) : kOutside) + wave * T * bytes;
        len = a.L;
        if (a.lengths) {
            const int64_t n = a.lengths[row];
            len = n < 0 ? 0 : (n < a.L ? n : a.L);
        }
    }
    // `own`, which the compiler takes for a new value each time: it would keep the offsets of all tokens in registers
    __device__ __forceinline__ unsigned start() const {
        unsigned o = own;
        asm volatile("" : "+v"(o));
        return o;
    }
    // the column's next tile, for the workgroup's turn-th (one thread)
    __device__ __forceinline__ int take(const RecArgs &a, int turn) const {
        if constexpr (!CHAIN) return turn;
        if (turn >= a.turns) return a.ntile;
        return (int)__hip_atomic_fetch_add(a.taken + at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    // tokens of the tile that starts at t0, of the first n of the row
    static __device__ __forceinline__ int count(int64_t t0, int64_t n) {
        n -= t0;
        return n < 0 ? 0 : (n < kTile ? (int)n : kTile);
    }
};

// Words that other workgroups wait for. (A NaN of all ones would look like an empty one)
__device__ __forceinline__ unsigned word(float x) {
    const unsigned u = __float_as_uint(x);
    return u == (unsigned)kEmpty ? 0x7fc00000u : u;
}
template <class T>
__device__ __forceinline__ void put(T *p, T w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T get(const T *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void give_map(const RecArgs &a, int row, int k, int c, float A, float B) {
    put(a.maps + ((int64_t)row * a.ntile + k) * a.C + c, (uint64_t)__float_as_uint(B) << 32 | word(A));
}
__device__ __forceinline__ void give_end(const RecArgs &a, int row, int k, int c, float h) {
    put(a.ends + ((int64_t)row * a.ntile + k) * a.C + c, word(h));
}

// What tile k starts from, for one channel a lane: the nearest state before it that is known, and the maps from there.
// `meanwhile` runs while the words first come
template <class F>
__device__ __forceinline__ float chain(const RecArgs &a, int row, int k, int c, bool in, F meanwhile) {
    const uint64_t *map = a.maps + ((int64_t)row * a.ntile + k - 1) * a.C + c;
    const unsigned *end = a.ends + ((int64_t)row * a.ntile + k - 1) * a.C + c, *begin = a.begins + (int64_t)row * a.C + c;
    for (bool again = false;; again = true) {
        uint64_t m[kWindow - 1];
        unsigned e[kWindow];
#pragma unroll
        for (int j = 0; j < kWindow; ++j) {
            e[j] = (unsigned)kEmpty;
            if (in && j <= k) e[j] = get(j < k ? end - (int64_t)j * a.C : begin);
        }
#pragma unroll
        for (int j = 0; j < kWindow - 1; ++j) {
            m[j] = kEmpty;
            if (in && j < k) m[j] = get(map - (int64_t)j * a.C);
        }
        if (!again) meanwhile();
        bool known = false;
        float h = 0.f;
#pragma unroll
        for (int j = kWindow - 1; j >= 0; --j) {
            if (j < kWindow - 1) {
                known = known && m[j] != kEmpty;
                h = __builtin_fmaf(__uint_as_float((unsigned)m[j]), h, __uint_as_float((unsigned)(m[j] >> 32)));
            }
            const bool here = e[j] != (unsigned)kEmpty;
            known = known || here;
            h = here ? __uint_as_float(e[j]) : h;
        }
        if (__all(known || !in)) return h;
        __builtin_amdgcn_s_sleep(1);
    }
}

// Two chains before they start: all words empty, no tile taken, what they start from
struct ChainStart {
    u32x4 *words;         // maps and ends, to a whole number of 16 bytes
    int64_t nwords;
    unsigned *begins, *taken;
    const float *from;
    int64_t nbegins, ntaken;
};
__global__ __launch_bounds__(256) void chain_start_kernel(const ChainStart one, const ChainStart two) {
    const int64_t step = (int64_t)gridDim.x * 256, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    constexpr unsigned none = (unsigned)kEmpty;
    for (const ChainStart &s : {one, two}) {
        for (int64_t i = at; i < s.nwords; i += step) s.words[i] = u32x4{none, none, none, none};
        for (int64_t i = at; i < s.nbegins; i += step) s.begins[i] = s.from ? word(s.from[i]) : 0u;
        for (int64_t i = at; i < s.ntaken; i += step) s.taken[i] = 0;
    }
}

// ------------------------------------------------------------------ forward ---
template <bool BF16, int V, bool GATE, bool UNIT, bool CHAIN>
__global__ __launch_bounds__(kThreads, 2) void fwd_kernel(const RecArgs a) {
    constexpr int T = kFwd;
    using IO = Io<BF16, V>;
    using At = Column<BF16, V, T, CHAIN>;
    __shared__ float both[2][2][kW][64 * V], first[64 * V];
    __shared__ int taken[4];
    const At p(a);
    int k = 0, next = 1;
    if constexpr (CHAIN) {
        if (threadIdx.x == 0) {
            taken[0] = p.take(a, 0);
            taken[1] = p.take(a, 1);
        }
        __syncthreads();
        k = __builtin_amdgcn_readfirstlane(taken[0]);
        next = __builtin_amdgcn_readfirstlane(taken[1]);
    }
    typename IO::raw rx[T], rr[T], ri[GATE ? T : 1];
    // the loads of a tile, token by token (none behind the last tile)
    struct Source {
        typename IO::rsrc_t x, r, i;
        unsigned at;
    };
    auto source = [&](int tile) {
        const int64_t t0 = tile < a.ntile ? (int64_t)tile * At::kTile : 0;
        const int n = tile < a.ntile ? p.count(t0, p.len) : 0;
        return Source{IO::rows(a, a.x, p.row, t0, n), IO::rows(a, a.r, p.row, t0, n), IO::rows(a, GATE ? a.i : a.r, p.row, t0, n),
                      p.start()};
    };
    auto fetch = [&](Source &f, int t) {
        rr[t] = IO::load(f.r, f.at);
        if constexpr (GATE) ri[t] = IO::load(f.i, f.at);
        rx[t] = IO::load(f.x, f.at);
        f.at += p.bytes;
    };
    auto fetch_all = [&](int tile) {
        if (tile >= a.ntile) return;
        Source f = source(tile);
#pragma unroll
        for (int t = 0; t < T; ++t) fetch(f, t);
    };
    fetch_all(k);
    float ld2[V], h[V];
    bool mild = true;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ld2[v] = p.in ? a.ld[p.c + v] * 1.4426950408889634f : 0.f;
        h[v] = !CHAIN && p.in && a.h0 ? a.h0[(int64_t)p.row * a.C + p.c + v] : 0.f;
        mild = mild && ld2[v] >= kMild;
    }
    mild = __all(mild);
    int last = CHAIN ? -2 : -1;  // the tile behind which h is
    auto tile = [&](int turn, float(*maps)[kW][64 * V]) {
        int later = 0;
        if (CHAIN && threadIdx.x == 0) later = p.take(a, turn + 2);
        const int64_t t0 = (int64_t)k * At::kTile;
        const int n = p.count(t0, p.len);
        const bool whole = n == At::kTile;
        float sa[T][V], sb[T][V], A[V], B[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            B[v] = 0.f;
        }
        // The next tile is loaded behind the gates, and between them in a chain, where a workgroup waits for others: long
        // b2 L32768 of 2560 channels 340 us with the first, 300 with the second; prompt b8 L4096 of 4096, no chain, 206 and 214
        Source f{};
        if constexpr (CHAIN) f = source(next);
        auto gates = [&](auto easy) {
            constexpr bool MILD = decltype(easy)::value;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float x[V], r[V], i[V] = {};
                IO::unpack(rx[t], x);
                IO::unpack(rr[t], r);
                if constexpr (GATE) IO::unpack(ri[t], i);
                if constexpr (CHAIN) fetch(f, t);
                // (what is behind the length: x is 0, and with a decay of 1 the state stays)
                const bool valid = MILD || p.wave * T + t < n;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    step_map<BF16, GATE, UNIT, MILD>(x[v], r[v], i[v], valid ? ld2[v] : 0.f, sa[t][v], sb[t][v]);
                    B[v] = __builtin_fmaf(sa[t][v], B[v], sb[t][v]);
                    A[v] *= sa[t][v];
                }
            }
        };
        if (whole && mild) gates(std::true_type{});
        else gates(std::false_type{});
        if constexpr (!CHAIN) fetch_all(next);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            maps[0][p.wave][p.lane * V + v] = A[v];
            maps[1][p.wave][p.lane * V + v] = B[v];
        }
        if (CHAIN && threadIdx.x == 0) taken[2 + (turn & 1)] = later;
        __syncthreads();  // (two sides of maps: the next tile's are written while these are read)
        float hw[V];
        if constexpr (CHAIN) {
            later = __builtin_amdgcn_readfirstlane(taken[2 + (turn & 1)]);
            // The maps of the runs before this one, and of all. (The state behind the tile is always that of the joint map,
            // whoever forms it: the same bits)
            float PA[V], PB[V];
            auto fold = [&] {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    A[v] = 1.f;
                    B[v] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < kW; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (j == p.wave) {
                            PA[v] = A[v];
                            PB[v] = B[v];
                        }
                        B[v] = __builtin_fmaf(maps[0][j][p.lane * V + v], B[v], maps[1][j][p.lane * V + v]);
                        A[v] *= maps[0][j][p.lane * V + v];
                    }
            };
            // the first wave publishes, the last V look for the start, a channel a lane
            const bool look = k != last + 1;
            if (look && p.wave >= kW - V) {
                const int l = (p.wave - (kW - V)) * 64 + p.lane, c = p.c + l - p.lane * V;
                first[l] = chain(a, p.row, k, c, c < a.C, fold);
            } else {
                fold();
                if (p.wave == 0 && p.in && k + 1 < a.ntile)
#pragma unroll
                    for (int v = 0; v < V; ++v) give_map(a, p.row, k, p.c + v, A[v], B[v]);
            }
            if (look) {
                __syncthreads();
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = first[p.lane * V + v];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                hw[v] = __builtin_fmaf(PA[v], h[v], PB[v]);
                h[v] = __builtin_fmaf(A[v], h[v], B[v]);
                if (p.wave == 0 && p.in && k + 1 < a.ntile) give_end(a, p.row, k, p.c + v, h[v]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kW; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (j == p.wave) hw[v] = h[v];
                    h[v] = __builtin_fmaf(maps[0][j][p.lane * V + v], h[v], maps[1][j][p.lane * V + v]);
                }
        }
        if (a.hf && p.in && p.wave == 0 && k == a.ntile - 1)
#pragma unroll
            for (int v = 0; v < V; ++v) a.hf[(int64_t)p.row * a.C + p.c + v] = h[v];
        const int64_t at = t0 + p.wave * T;
        if (a.states && p.in && at % M3_REC_KEEP == 0 && at < a.L)
#pragma unroll
            for (int v = 0; v < V; ++v) a.states[((int64_t)p.row * a.nkeep + at / M3_REC_KEEP) * a.C + p.c + v] = hw[v];
        if (a.y) {
            const auto by = IO::rows(a, a.y, p.row, t0, p.count(t0, a.L));
            unsigned to = p.start();
#pragma unroll
            for (int t = 0; t < T; ++t, to += p.bytes) {
                float y[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    hw[v] = __builtin_fmaf(sa[t][v], hw[v], sb[t][v]);
                    y[v] = whole || p.wave * T + t < n ? hw[v] : 0.f;
                }
                IO::store(by, to, y);
            }
        }
        last = k;
        k = next;
        next = CHAIN ? later : k + 1;
    };
    for (int turn = 0; k < a.ntile; ++turn) tile(turn, both[turn & 1]);
}

// ---------------------------------------------------------------- gradients ---
// The chain runs from the last tile to the first: place k is tile ntile - 1 - k
template <bool BF16, int V, bool GATE, bool UNIT, bool CHAIN>
__global__ __launch_bounds__(kThreads, 2) void bwd_kernel(const RecArgs a) {
    constexpr int T = kBwd;
    using IO = Io<BF16, V>;
    using At = Column<BF16, V, T, CHAIN>;
    __shared__ float both[2][3][kW][64 * V], first[64 * V];
    __shared__ int taken[4];
    const At p(a);
    int k = 0, next = 1;
    if constexpr (CHAIN) {
        if (threadIdx.x == 0) {
            taken[0] = p.take(a, 0);
            taken[1] = p.take(a, 1);
        }
        __syncthreads();
        k = __builtin_amdgcn_readfirstlane(taken[0]);
        next = __builtin_amdgcn_readfirstlane(taken[1]);
    }
    typename IO::raw rx[T], rr[T], ri[GATE ? T : 1], rd[T];
    float kept[V] = {};
    auto fetch = [&](int place) {
        if (place >= a.ntile) return;
        const int64_t t0 = (int64_t)(a.ntile - 1 - place) * At::kTile;
        const int n = p.count(t0, p.len);
        const auto bx = IO::rows(a, a.x, p.row, t0, n), br = IO::rows(a, a.r, p.row, t0, n);
        const auto bi = IO::rows(a, GATE ? a.i : a.r, p.row, t0, n), bd = IO::rows(a, a.dy, p.row, t0, n);
        unsigned at = p.start();
#pragma unroll
        for (int t = 0; t < T; ++t, at += p.bytes) {
            rr[t] = IO::load(br, at);
            if constexpr (GATE) ri[t] = IO::load(bi, at);
            rx[t] = IO::load(bx, at);
            rd[t] = IO::load(bd, at);
        }
        if (p.in && a.nkeep)
#pragma unroll
            for (int v = 0; v < V; ++v) kept[v] = a.states[((int64_t)p.row * a.nkeep + a.ntile - 1 - place) * a.C + p.c + v];
    };
    fetch(k);
    float ld[V], ld2[V], G[V];
    bool mild = true;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ld[v] = p.in ? a.ld[p.c + v] : 0.f;
        ld2[v] = ld[v] * 1.4426950408889634f;
        G[v] = !CHAIN && p.in && a.dhf ? a.dhf[(int64_t)p.row * a.C + p.c + v] : 0.f;
        mild = mild && ld2[v] >= kMild;
    }
    mild = __all(mild);
    int last = CHAIN ? -2 : -1;
    auto tile = [&](int turn, float(*maps)[kW][64 * V]) {
        int later = 0;
        if (CHAIN && threadIdx.x == 0) later = p.take(a, turn + 2);
        const int64_t t0 = (int64_t)(a.ntile - 1 - k) * At::kTile;
        const int n = p.count(t0, p.len);
        const bool whole = n == At::kTile;
        // of a step: a, b; E's factors in dx, in di, in d(ld s) and from there in dr; s; dy
        float sa[T][V], sb[T][V], fx[T][V], fi[GATE ? T : 1][V], fl[T][V], fr[T][V], ss[T][V], dy[T][V];
        float A[V], B[V], D[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = kept[v];
            A[v] = 1.f;
            B[v] = D[v] = 0.f;
        }
        auto gates = [&](auto easy) {
            constexpr bool MILD = decltype(easy)::value;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                float x[V], r[V], i[V] = {};
                IO::unpack(rx[t], x);
                IO::unpack(rr[t], r);
                if constexpr (GATE) IO::unpack(ri[t], i);
                IO::unpack(rd[t], dy[t]);
                const bool valid = MILD || p.wave * T + t < n;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float q, s1, g = 1.f, g1 = 0.f;
                    const float s = sigmoid<BF16>(r[v], s1), l = valid ? ld2[v] * s : 0.f;
                    if constexpr (MILD) mild_decay(l, sa[t][v], q);
                    else decay(l, sa[t][v], q);
                    q *= 2.f - q;
                    if constexpr (GATE) g = sigmoid<BF16>(i[v], g1);
                    float m = 1.f, inv = 0.f;
                    if constexpr (!UNIT) {
                        // (below the smallest normal number the root counts as 0, and its slope too)
                        inv = q < 0x1p-126f ? 0.f : __builtin_amdgcn_rsqf(q);
                        m = q * inv;
                    }
                    const float b = g * x[v];
                    sb[t][v] = m * b;
                    fx[t][v] = m * g;
                    if constexpr (GATE) fi[t][v] = m * b * g1;
                    fl[t][v] = b * sa[t][v] * sa[t][v] * inv;
                    fr[t][v] = ld[v] * (s * s1);
                    ss[t][v] = s;
                    B[v] = __builtin_fmaf(sa[t][v], B[v], sb[t][v]);
                    A[v] *= sa[t][v];
                }
            }
        };
        if (whole && mild) gates(std::true_type{});
        else gates(std::false_type{});
        fetch(next);
#pragma unroll
        for (int t = T - 1; t >= 0; --t)
#pragma unroll
            for (int v = 0; v < V; ++v) D[v] = sa[t][v] * (dy[t][v] + D[v]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            maps[0][p.wave][p.lane * V + v] = A[v];
            maps[1][p.wave][p.lane * V + v] = B[v];
            maps[2][p.wave][p.lane * V + v] = D[v];
        }
        if (CHAIN && threadIdx.x == 0) taken[2 + (turn & 1)] = later;
        __syncthreads();
        // the state that this run starts from, and those before its tokens
        for (int j = 0; j < p.wave; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = __builtin_fmaf(maps[0][j][p.lane * V + v], h[v], maps[1][j][p.lane * V + v]);
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float left = sa[t][v] * h[v];
                fl[t][v] = left - fl[t][v];
                h[v] = left + sb[t][v];
            }
        if (!whole)  // (a state that is infinite or NaN has no part in what is behind the length)
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int v = 0; v < V; ++v) fl[t][v] = p.wave * T + t < n ? fl[t][v] : 0.f;
        if constexpr (CHAIN) {
            later = __builtin_amdgcn_readfirstlane(taken[2 + (turn & 1)]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A[v] = 1.f;
                D[v] = 0.f;
#pragma unroll
                for (int j = kW - 1; j >= 0; --j) {
                    A[v] *= maps[0][j][p.lane * V + v];
                    D[v] = __builtin_fmaf(maps[0][j][p.lane * V + v], D[v], maps[2][j][p.lane * V + v]);
                }
                if (p.wave == 0 && p.in && k + 1 < a.ntile) give_map(a, p.row, k, p.c + v, A[v], D[v]);
            }
            if (k != last + 1) {
                if (p.wave < V) {  // (a channel a lane)
                    const int c = p.c + (p.wave * 64 + p.lane) - p.lane * V;
                    first[p.wave * 64 + p.lane] = chain(a, p.row, k, c, c < a.C, [] {});
                }
                __syncthreads();
#pragma unroll
                for (int v = 0; v < V; ++v) G[v] = first[p.lane * V + v];
            }
        }
        float Gw[V];
        if constexpr (CHAIN) {
#pragma unroll
            for (int v = 0; v < V; ++v) Gw[v] = G[v];
            for (int j = kW - 1; j > p.wave; --j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    Gw[v] = __builtin_fmaf(maps[0][j][p.lane * V + v], Gw[v], maps[2][j][p.lane * V + v]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                G[v] = __builtin_fmaf(A[v], G[v], D[v]);
                if (p.wave == 0 && p.in && k + 1 < a.ntile) give_end(a, p.row, k, p.c + v, G[v]);
            }
        } else {
#pragma unroll
            for (int j = kW - 1; j >= 0; --j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (j == p.wave) Gw[v] = G[v];
                    G[v] = __builtin_fmaf(maps[0][j][p.lane * V + v], G[v], maps[2][j][p.lane * V + v]);
                }
        }
        if (a.dh0 && p.in && p.wave == 0 && k == a.ntile - 1)
#pragma unroll
            for (int v = 0; v < V; ++v) a.dh0[(int64_t)p.row * a.C + p.c + v] = G[v];
        const int rows = p.count(t0, a.L);
        const auto b1 = IO::rows(a, a.dx, p.row, t0, rows), b2 = IO::rows(a, a.dr, p.row, t0, rows);
        const auto b3 = IO::rows(a, GATE ? a.di : a.dr, p.row, t0, rows);
        float dl[V] = {};
        unsigned to = p.start() + (T - 1) * p.bytes;
#pragma unroll
        for (int t = T - 1; t >= 0; --t, to -= p.bytes) {
            float ox[V], orr[V], oi[V];
            const bool valid = whole || p.wave * T + t < n;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                // (behind the length: no gradient, and a decay of 1 passes G on)
                const float E = dy[t][v] + Gw[v], F = valid ? E : 0.f, d = F * fl[t][v];
                ox[v] = F * fx[t][v];
                orr[v] = d * fr[t][v];
                if constexpr (GATE) oi[v] = F * fi[t][v];
                dl[v] = __builtin_fmaf(d, ss[t][v], dl[v]);
                Gw[v] = sa[t][v] * E;
            }
            IO::store(b1, to, ox);
            IO::store(b2, to, orr);
            if constexpr (GATE) IO::store(b3, to, oi);
        }
        if (a.dpart) {
            __syncthreads();  // (the maps are read no more)
#pragma unroll
            for (int v = 0; v < V; ++v) maps[1][p.wave][p.lane * V + v] = dl[v];
            __syncthreads();
            if (p.wave == 0 && p.in)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    double d = 0.;
#pragma unroll
                    for (int j = 0; j < kW; ++j) d += maps[1][j][p.lane * V + v];
                    a.dpart[((int64_t)p.row * a.ntile + k) * a.C + p.c + v] = (float)d;
                }
        }
        last = k;
        k = next;
        next = CHAIN ? later : k + 1;
    };
    for (int turn = 0; k < a.ntile; ++turn) tile(turn, both[turn & 1]);
}

// dld[c]: the sums of all tiles, in a fixed order
constexpr int kRuns = 16;
__global__ __launch_bounds__(64 * kRuns) void decay_sums_kernel(const float *part, int64_t rows, int C, float *dld) {
    __shared__ double lds[kRuns][64];
    const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    double d = 0.;
    if (c < C)
        for (int64_t r = run; r < rows; r += kRuns) d += part[r * C + c];
    lds[run][lane] = d;
    __syncthreads();
    if (run == 0 && c < C) {
        for (int k = 1; k < kRuns; ++k) d += lds[k][lane];
        dld[c] = (float)d;
    }
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
            step_map<BF16, GATE, UNIT, false>(ld_io<BF16>(x, at + v), ld_io<BF16>(r, at + v), GATE ? ld_io<BF16>(i, at + v) : 0.f,
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

// one direction: channels a lane, tiles along and across, columns of all rows, workgroups a column (chained where
// there is more than one), bytes of the chain's words, of all of the chain
struct RecWay {
    int V;
    int64_t ntile, cols, columns, each;
    size_t words, chain;
};
struct RecPlan {
    int64_t nkeep;  // kept states of a row
    RecWay fwd, bwd;
    size_t states, dpart;  // bytes
};

m3_status rec_check(const m3_rec_shape *s) {
    if (!s) return M3_ERR_INVALID_ARG;
    if (s->batch < 0 || s->seqlen < 0 || s->channels < 1) return M3_ERR_INVALID_ARG;
    if (s->io_dtype != M3_F32 && s->io_dtype != M3_BF16) return M3_ERR_INVALID_ARG;
    if (s->flags & ~(uint32_t)M3_REC_UNSCALED) return M3_ERR_INVALID_ARG;
    if (s->channels > (1 << 20) || s->batch > (1LL << 31) || s->seqlen > (1LL << 40) ||
        (s->seqlen > 0 && s->batch > (1LL << 40) / s->seqlen))
        return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

m3_status way(const m3_rec_shape &s, int tile, RecWay *w) {
    *w = {};
    w->V = s.io_dtype == M3_BF16 && s.channels % 2 == 0 ? 2 : 1;
    w->ntile = s.seqlen ? ceil_div(s.seqlen, tile) : 1;
    w->cols = ceil_div(s.channels, 64 * w->V);
    w->columns = s.batch * w->cols;
    if (w->columns > kMaxGrid || w->columns * w->ntile > kMaxGrid) return M3_ERR_UNSUPPORTED;
    // enough workgroups a column that all of them fill the card once or a few times
    w->each = 1;
    double best = 0.;
    for (int64_t rounds = 1; rounds <= 4 && w->columns > 0; ++rounds) {
        const int64_t n = rounds * kSlots / w->columns, each = n < 1 ? 1 : (n < w->ntile ? n : w->ntile);
        const double full = (double)(w->columns * each) / (double)(ceil_div(w->columns * each, kSlots) * kSlots);
        if (full > best * 1.1) {
            best = full;
            w->each = each;
        }
    }
    w->words = w->each == 1 ? 0 : up((size_t)(s.batch * s.channels * w->ntile) * (sizeof(uint64_t) + sizeof(unsigned)));
    w->chain = w->each == 1 ? 0 : w->words + up((size_t)(s.batch * s.channels + w->columns) * sizeof(unsigned));
    return M3_OK;
}

m3_status rec_plan(const m3_rec_shape *s, RecPlan *p) {
    const m3_status st = rec_check(s);
    if (st != M3_OK) return st;
    if (s->batch > kMaxGrid || way(*s, kW * kFwd, &p->fwd) != M3_OK || way(*s, kW * kBwd, &p->bwd) != M3_OK)
        return M3_ERR_UNSUPPORTED;
    p->nkeep = ceil_div(s->seqlen, M3_REC_KEEP);
    p->states = up((size_t)(s->batch * p->nkeep * s->channels) * sizeof(float));
    p->dpart = up((size_t)(s->batch * p->bwd.ntile * s->channels) * sizeof(float));
    return M3_OK;
}

RecArgs rec_args(const m3_rec_shape &s, const m3_rec_io &io, const RecPlan &p) {
    RecArgs a{};
    a.x = io.x; a.r = io.decay_gate; a.i = io.input_gate; a.ld = io.log_decay; a.h0 = io.h0; a.lengths = io.lengths;
    a.L = s.seqlen; a.C = (int)s.channels; a.nkeep = (int)p.nkeep;
    return a;
}

// one direction's part of the arguments, and its chain in the workspace at `ws`, which starts from `from`
ChainStart set_way(RecArgs &a, const RecWay &w, int64_t batch, void *ws, const float *from) {
    a.ntile = (int)w.ntile;
    a.cols = (int)w.cols;
    a.columns = (unsigned)w.columns;
    a.turns = (int)ceil_div(w.ntile, w.each);
    if (w.each == 1) return {};
    const int64_t n = batch * w.ntile * a.C;
    a.maps = static_cast<uint64_t *>(ws);
    a.ends = reinterpret_cast<unsigned *>(a.maps + n);
    a.begins = reinterpret_cast<unsigned *>(static_cast<char *>(ws) + w.words);
    a.taken = a.begins + batch * a.C;
    return {static_cast<u32x4 *>(ws), (int64_t)(w.words / 16), a.begins, a.taken, from, batch * a.C, w.columns};
}
hipError_t start(const ChainStart &one, const ChainStart &two, hipStream_t s) {
    const int64_t n = one.nwords + two.nwords, g = ceil_div(n, 256 * 2);
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(chain_start_kernel, dim3((unsigned)(g < 2048 ? g : 2048)), dim3(256), 0, s, one, two);
    return hipGetLastError();
}

template <bool BF16, int V, bool GATE, bool UNIT>
hipError_t launch_fwd(const RecArgs &a, const RecWay &w, hipStream_t s) {
    const dim3 g((unsigned)(w.columns * w.each)), t(kThreads);
    if (w.each > 1) hipLaunchKernelGGL((fwd_kernel<BF16, V, GATE, UNIT, true>), g, t, 0, s, a);
    else hipLaunchKernelGGL((fwd_kernel<BF16, V, GATE, UNIT, false>), g, t, 0, s, a);
    return hipGetLastError();
}

template <bool BF16, int V, bool GATE, bool UNIT>
hipError_t launch_bwd(const RecArgs &a, const RecWay &w, hipStream_t s) {
    const dim3 g((unsigned)(w.columns * w.each)), t(kThreads);
    if (w.each > 1) hipLaunchKernelGGL((bwd_kernel<BF16, V, GATE, UNIT, true>), g, t, 0, s, a);
    else hipLaunchKernelGGL((bwd_kernel<BF16, V, GATE, UNIT, false>), g, t, 0, s, a);
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
#define M3_REC_PICK_V(f, BF, V, gate, unit, ...)                                            \
    (gate ? (unit ? f<BF, V, true, true>(__VA_ARGS__) : f<BF, V, true, false>(__VA_ARGS__)) \
          : (unit ? f<BF, V, false, true>(__VA_ARGS__) : f<BF, V, false, false>(__VA_ARGS__)))
#define M3_REC_PICK(f, s, gate, ...)                                                                             \
    ((s)->io_dtype != M3_BF16                                                                                    \
         ? M3_REC_PICK_V(f, false, 1, gate, ((s)->flags & M3_REC_UNSCALED) != 0, __VA_ARGS__)                    \
         : ((s)->channels % 2 == 0 ? M3_REC_PICK_V(f, true, 2, gate, ((s)->flags & M3_REC_UNSCALED) != 0, __VA_ARGS__) \
                                   : M3_REC_PICK_V(f, true, 1, gate, ((s)->flags & M3_REC_UNSCALED) != 0, __VA_ARGS__)))

hipError_t launch_fwd_any(const m3_rec_shape *s, bool gate, const RecArgs &a, const RecWay &w, hipStream_t hs) {
    return M3_REC_PICK(launch_fwd, s, gate, a, w, hs);
}
hipError_t launch_bwd_any(const m3_rec_shape *s, bool gate, const RecArgs &a, const RecWay &w, hipStream_t hs) {
    return M3_REC_PICK(launch_bwd, s, gate, a, w, hs);
}

}  // namespace
}  // namespace m3i

using namespace m3i;

extern "C" {

size_t m3_recurrence_workspace_bytes(const m3_rec_shape *shape) {
    RecPlan p;
    return rec_plan(shape, &p) == M3_OK ? p.fwd.chain : 0;
}

size_t m3_recurrence_bwd_workspace_bytes(const m3_rec_shape *shape, int states) {
    RecPlan p;
    return rec_plan(shape, &p) == M3_OK ? (states ? 0 : p.states + p.fwd.chain) + p.bwd.chain + p.dpart : 0;
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
    if (p.fwd.chain && (!workspace || ws_bytes < p.fwd.chain)) return M3_ERR_WORKSPACE_TOO_SMALL;
    void *ws = p.fwd.chain ? workspace : nullptr;
    if (clash({io->y, io->states, ws}, {io->x, io->decay_gate, io->input_gate, io->log_decay, io->h0, io->lengths, io->h_final}) ||
        clash({io->h_final}, {io->x, io->decay_gate, io->input_gate, io->log_decay, io->lengths}))
        return M3_ERR_INVALID_ARG;
    if (shape->batch == 0) return M3_OK;
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    RecArgs a = rec_args(*shape, *io, p);
    a.y = io->y; a.hf = io->h_final; a.states = io->states;
    hipError_t e = start(set_way(a, p.fwd, shape->batch, workspace, a.h0), {}, hs);
    if (e == hipSuccess) e = launch_fwd_any(shape, a.i != nullptr, a, p.fwd, hs);
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
    // the states, where they are formed here, and their chain; the gradients' chain; partial sums
    const size_t own_states = io->states ? 0 : p.states + p.fwd.chain, need = own_states + p.bwd.chain + p.dpart;
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
    a.dpart = gr->dlog_decay ? reinterpret_cast<float *>(at + own_states + p.bwd.chain) : nullptr;
    if (shape->batch > 0) {
        const bool first = !io->states && shape->seqlen > 0;
        RecArgs f = a;
        const ChainStart back = set_way(a, p.bwd, shape->batch, at + own_states, gr->dh_final);
        e = start(first ? set_way(f, p.fwd, shape->batch, at + p.states, a.h0) : ChainStart{}, back, hs);
        if (e == hipSuccess && first) e = launch_fwd_any(shape, a.i != nullptr, f, p.fwd, hs);
        a.dy = gr->dy; a.dhf = gr->dh_final; a.dx = gr->dx; a.dr = gr->ddecay_gate; a.di = gr->dinput_gate; a.dh0 = gr->dh0;
        if (e == hipSuccess) e = launch_bwd_any(shape, a.i != nullptr, a, p.bwd, hs);
    }
    if (e == hipSuccess && gr->dlog_decay) {
        hipLaunchKernelGGL(decay_sums_kernel, dim3((unsigned)ceil_div(shape->channels, 64)), dim3(64 * kRuns), 0, hs, a.dpart,
                           shape->batch * p.bwd.ntile, (int)shape->channels, gr->dlog_decay);
        e = hipGetLastError();
    }
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

m3_status m3_recurrence_step(const m3_rec_shape *shape, const m3_rec_step_io *io, void *stream) {
    if (!shape) return M3_ERR_INVALID_ARG;
    m3_rec_shape s = *shape;
    s.seqlen = 1;  // (not used)
    const m3_status st = rec_check(&s);
    if (st != M3_OK) return st;
    if (!io) return M3_ERR_INVALID_ARG;
    if (s.batch > 0 && (!io->x || !io->decay_gate || !io->log_decay || !io->h || !io->y)) return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->x, io->decay_gate, io->input_gate, io->log_decay, io->h, io->y};
    for (const void *q : ptrs)
        if (!al16(q)) return M3_ERR_MISALIGNED;
    if (clash({io->h, io->y}, {io->x, io->decay_gate, io->input_gate, io->log_decay})) return M3_ERR_INVALID_ARG;
    if (s.batch == 0) return M3_OK;
    const hipError_t e =
        M3_REC_PICK(launch_step, &s, io->input_gate != nullptr, s, *io, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

}  // extern "C"
