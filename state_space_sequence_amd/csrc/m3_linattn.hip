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
// with D the gradient of the state behind the chunk (si = su = scale, sr = 1). With
// the chunk's tokens taken last first the two differ in two exponents only
// (i + 1 - rev and nt - 1 - j + rev), and both masks keep j <= i. The gradients are three such passes over other tensors:
//   dq: forwards,  (q, k, v) = (dy, v, k), the state transposed
//   dk: backwards, (q, k, v) = (v, dy, q), the state transposed
//   dv: backwards, (q, k, v) = (k, q, dy)
// and d log_decay is sum_t scale dy_t . (U_t^T q_t) with U = dS / d log_decay,
// U_t = a (U_{t-1} + S_{t-1}), carried the same way by a forward pass of its own. Per chunk that is
//   sum_{j<i} (i - j) a^{i-j} (q_i . k_j)(dy_i . v_j) + <S, sum_i (i+1) a^{i+1} q_i dy_i^T> + <U, sum_i a^{i+1} q_i dy_i^T>
// whose first products are exact, and whose states enter in fp32: no operand but the weighted
// dy is split. Every weight stays local to its chunk, where sums of t (q.dq - k.dk)
// over a whole sequence would cancel.
//
// A workgroup of 4 waves owns one chain (batch, head), 64 of its values (columns of S) and one
// segment of the tokens. Wave w owns 16 columns: its part of S never leaves its
// registers. The accumulators of the update (keys down the rows) are, two row
// tiles at a time, the operand of the product with q: the update's rows are given to
// the keys so that a lane ends up with 8 consecutive ones. q, k and v lie in LDS as they are
// in memory, a row a token. The products that contract over tokens need k and v by
// columns: bf16 through the transposing LDS read (each lane of 16 names 4 consecutive elements of
// one of 4 rows and gets 4 rows of one column), fp32 element by element.
//
// bf16, b8 L4096 of 64 query heads on 8, 128 keys, 64 values: 333 us, 206 TFLOP/s of useful products (76 of a wave's 126
// products a chunk are those of the further parts of its operands), 2.8 TB/s; the bytes alone would take 157 us. No unit is
// full: vector issue takes 51% of the cycles, the LDS 50%, the matrix cores 41%, at 1.87 GHz; two waves a SIMD (registers:
// the state, a step's fragments, the next chunk) wait for each other. b2 L32768 of 24
// heads in ten segments: 414 us. Gradients of b8 L2048, 16 heads of 128 x 128: 417 us, of them d log_decay
// about 0.4, bound by the vector instructions of its splits. fp32 runs on the fp32 matrix cores in chunks of 32.
#include <math.h>

#include "m3_internal.h"
#include "m3_linattn.h"

namespace m3i {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kVT = 64;  // value columns of a workgroup
constexpr int kMaxDim = 256;
constexpr int64_t kMaxGrid = 0xffffff;  // workgroups along x: 2^32 threads

// kOut: outputs. kState, kStateU: segment states (and their derivatives) only. kDecay: d log_decay.
// kStateOnce: kState of keys and values that no other workgroup reads
enum Mode { kOut = 0, kState = 1, kStateU = 2, kDecay = 3, kStateOnce = 4 };

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
    Tensor dy;              // kDecay
    const float *dh_final;  // kDecay: [chains] or NULL
    double *part;           // kDecay: [H, b * nseg * nvt * nkt]
    int64_t b, L, nchunks, seg_chunks;
    int H, kd, vd, nseg, nvt;
    int nkt;  // kDecay: tiles of 64 keys, a workgroup each (d log_decay is a sum over keys and values); else 1
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
    // Parts of an operand that is no input (a state, a score, a weighted value): 3 of 8 bits hold all 24 of fp32. With two
    // parts of a state and of a score, 16 bits, 0.22% of the bf16 outputs land on the other side of a rounding
    // from the fp32 form's, with three 0.02%, what the order of fp32 sums gives; b8 L4096 takes 333 us instead of 297
    static constexpr int kParts = 3;
    static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // Two values as a sum of NP bf16 pairs: each part takes 8 of a value's bits, the remainders are exact
    template <int NP, typename F>
    static __device__ __forceinline__ void split2(float x, float y, const F &put) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const f32x2 v = {x, y};
            const unsigned w = __builtin_bit_cast(unsigned, __builtin_convertvector(v, bf16x2));
            put(n, w);
            if (n + 1 < NP) {
                x -= __uint_as_float(w << 16);
                y -= __uint_as_float(w & 0xffff0000u);
            }
        }
    }
    template <int NP>
    static __device__ __forceinline__ void parts(const float *x, frag *p) {
        u32x4 w[NP];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2<NP>(x[2 * e], x[2 * e + 1], [&](int n, unsigned u) { w[n][e] = u; });
#pragma unroll
        for (int n = 0; n < NP; ++n) p[n] = __builtin_bit_cast(frag, w[n]);
    }
    static __device__ __forceinline__ float value(frag f, int e) { return (float)f[e]; }
    // 4 values to 4 consecutive elements, in parts `plane` elements apart
    template <int NP>
    static __device__ __forceinline__ void store4(uint16_t *to, int plane, f32x4 x) {
        u32x2 w[NP];
#pragma unroll
        for (int e = 0; e < 2; ++e) split2<NP>(x[2 * e], x[2 * e + 1], [&](int n, unsigned u) { w[n][e] = u; });
#pragma unroll
        for (int n = 0; n < NP; ++n) *reinterpret_cast<u32x2 *>(to + n * plane) = w[n];
    }
};

template <>
struct Ops<float> {
    typedef f32x8 frag;
    typedef f32x8 pack;
    static constexpr int C = 32, kParts = 1;
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

// A chunk's valid rows of one tensor for one head are read by byte offsets from the first.
// With dims in multiples of 8 (VEC) the reads are buffer loads, whose bounds check gives zeros for what
// lies outside (rows before the first wrap around to offsets beyond 2^31; a chunk's rows
// span less, as H <= 65536) without a branch.
constexpr unsigned kOutside = 0x80000000u;

// 8 elements, packed; `cols` of them exist. ONCE: past the caches
template <typename E, bool VEC, bool ONCE = false>
__device__ __forceinline__ typename Ops<E>::pack load8(const char *p, unsigned bytes, unsigned at, int cols) {
    if constexpr (VEC) {
        constexpr int AUX = ONCE ? 2 : 0;  // (non-temporal)
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, (int)bytes, 0x00020000);
        if constexpr (sizeof(E) == 2) {
            return __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, AUX);
        } else {
            const f32x4 a = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, AUX));
            const f32x4 b = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at + 16, 0, AUX));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    } else {
        const int live = at < bytes ? cols : 0;
        const E *x = reinterpret_cast<const E *>(p + (live > 0 ? at : 0u));
        if constexpr (sizeof(E) == 2) {
            u32x4 w = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                unsigned lo = 0, hi = 0;
                if (2 * e < live) lo = x[2 * e];
                if (2 * e + 1 < live) hi = x[2 * e + 1];
                w[e] = lo | (hi << 16);
            }
            return w;
        } else {
            f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < live) v[e] = x[e];
            return v;
        }
    }
}

__device__ __forceinline__ u32x2 bf16_pack4(f32x4 x) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    const bf16x4 b = {(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};
    return __builtin_bit_cast(u32x2, b);
}

// LDS tiles [token][LD], in blocks of 8 elements (one lane's operand slots). Block b of row i lies at
// b ^ swap(i), so that the lanes that read one block of 16 rows, and those that read 4 blocks of
// 4 rows, spread over the 64 banks of 4 bytes. 16-byte reads are served to 16 lanes at a time, of two
// lane groups: rows 0-3 and 12-15 of one with rows 4-11 of the next, so the low bits of these rows' swaps
// have to stay apart when one block number is odd (0, 1 against 2, 3).
template <typename E, int LD>
__device__ __forceinline__ int swap_of(int row) {
    constexpr int NB = LD / 8;
    if constexpr (sizeof(E) == 2)
        return (NB >= 16 ? (row & 3) << 2 : ((row >> 1) & 1) << 2) | ((((row >> 2) ^ (row >> 3)) & 1) << 1) | ((row >> 3) & 1);
    else
        return NB >= 8 ? row & 7 : (row >> 1) & 3;
}
template <typename E>
__device__ __forceinline__ E *at_byte(E *tile, int byte) {
    return reinterpret_cast<E *>(reinterpret_cast<char *>(tile) + byte);
}
// Row fragment t, ks of a lane: row 16 t + lr, elements 32 ks + 8 lg .. + 7. base: for t = ks = 0, in bytes
template <typename E, int LD>
__device__ __forceinline__ int row_base(int lr, int lg) {
    return (lr * LD + ((lg ^ swap_of<E, LD>(lr)) << 3)) * (int)sizeof(E);
}
template <typename E, int LD>
__device__ __forceinline__ typename Ops<E>::frag row_frag(E *tile, int base, int t, int ks) {
    return *reinterpret_cast<const typename Ops<E>::frag *>(
        at_byte(tile + 128 * (ks >> 2) + 16 * LD * t, base ^ (32 * (ks & 3) * (int)sizeof(E))));
}
__device__ __forceinline__ bf16x8 transposed(uint16_t *p, uint16_t *q) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)q);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
// Column fragment t, ks of a lane: tokens 32 ks + 8 lg .. + 7 of key key_of(t, lr >> 2, lr & 3), where
// key_of gives rows 4 g + r of the two row tiles 2s, 2s + 1 the keys 32 s + 8 g + 0..7
__device__ __forceinline__ int key_of(int t, int g, int r) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1) + r; }
template <typename E, int LD>
__device__ __forceinline__ int col_base(int lr, int lg) {
    if constexpr (sizeof(E) == 2) {
        const int row = 8 * lg + (lr >> 2);
        return (row * LD + (((lr & 3) ^ swap_of<E, LD>(row)) << 3)) * 2;
    } else {
        return (8 * lg * LD + ((lr >> 2) << 3) + (lr & 3)) * 4;
    }
}
template <typename E, int LD>
__device__ __forceinline__ typename Ops<E>::frag col_frag(E *tile, int base, int t, int ks) {
    const int s = t >> 1, h = 4 * (t & 1);
    if constexpr (sizeof(E) == 2) {
        E *p = tile + 32 * ks * LD + h + 128 * (s >> 2);
        return transposed(at_byte(p, base ^ (64 * (s & 3))), at_byte(p + 4 * LD, base ^ (64 * (s & 3) + 32)));
    } else {
        f32x8 x;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = *at_byte(tile + e * LD + h + 64 * (s >> 1), base ^ (32 * (e ^ (4 * (s & 1)))));
        return x;
    }
}
// The same of value 16 w + lr, of a tile of 64 values
template <typename E>
__device__ __forceinline__ int val_base(int lr, int lg, int w) {
    if constexpr (sizeof(E) == 2) {
        const int row = 8 * lg + (lr >> 2);
        return (row * kVT + (((2 * w + ((lr >> 1) & 1)) ^ swap_of<E, kVT>(row)) << 3) + 4 * (lr & 1)) * 2;
    } else {
        return (8 * lg * kVT + ((2 * w + (lr >> 3)) << 3) + (lr & 7)) * 4;
    }
}
template <typename E>
__device__ __forceinline__ typename Ops<E>::frag val_frag(E *tile, int base, int ks) {
    if constexpr (sizeof(E) == 2) {
        E *p = tile + 32 * ks * kVT;
        return transposed(at_byte(p, base), at_byte(p + 4 * kVT, base ^ 32));
    } else {
        f32x8 x;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = *at_byte(tile + e * kVT, base ^ (32 * e));
        return x;
    }
}

// A value the compiler cannot see through: addresses formed from it are formed where they
// are used, not kept in registers across the loop
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// a^n to half a unit in the last place: a decay's rounding would otherwise add up over
// the chunks of a long sequence. A decay of 0 is e^-inf, and 0 * inf no number.
__device__ __forceinline__ double power(float log_decay, int64_t n) {
    return n == 0 ? 1.0 : exp((double)log_decay * (double)n);
}

// A workgroup's place in the work: consecutive ones (the value tiles of a chain, the
// heads of a group, which read the same tensors) go to one XCD and its L2
__device__ __forceinline__ unsigned xcd_order(unsigned id, unsigned total) {
    const unsigned q = total / 8, r = total % 8, x = id % 8;
    return x * q + (x < r ? x : r) + id / 8;
}

// a value that is the same in all lanes, in a scalar register
__device__ __forceinline__ float uniform(float x) {
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

__device__ __forceinline__ double uniform64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

// the passes of one launch (of the same key tiles): workgroups 0 .. ends[0] - 1 run the first, and so on
struct Passes {
    Args a[3];
    unsigned ends[3];
    int n;
};

template <typename E, int KD, int MODE, bool VEC>
__global__ __launch_bounds__(kThreads, KD == 256 ? 1 : 2) void linattn_kernel(const Passes passes) {
    // (each pass in the order of its own: see xcd_order)
    const int role = MODE != kOut || blockIdx.x < passes.ends[0] ? 0 : (blockIdx.x < passes.ends[1] ? 1 : 2);
    const unsigned begin = role ? passes.ends[role - 1] : 0u;
    Args a = passes.a[0];  // (indexed by a variable, the arguments would be copied to memory)
    if (role == 1) a = passes.a[1];
    if (role == 2) a = passes.a[2];
    typedef Ops<E> O;
    typedef typename O::frag frag;
    constexpr int C = O::C, KT = KD / 16, KS = KD / 32, JS = C / 32, IT = C / 16, ES = sizeof(E);
    constexpr bool kDec = MODE == kDecay, kOnce = MODE == kStateOnce,
                   kSt = MODE == kState || MODE == kStateU || kOnce, kU = kDec || MODE == kStateU;
    constexpr int NP = O::kParts;
    __shared__ __align__(16) E Qs[kSt ? 8 : C * KD];
    __shared__ __align__(16) E Ks[C * KD];
    __shared__ __align__(16) E Vs[C * kVT];
    __shared__ __align__(16) E As[MODE != kOut ? 8 : NP * C * C];
    __shared__ __align__(16) E Ds[kDec ? C * kVT : 8];  // dy
    __shared__ __align__(16) float wt[C], wu[kU ? C : 1], wd[kDec ? 2 : 1][kDec ? C : 1];
    __shared__ float pw[C + 1];  // a^n

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, lr = lane & 15, lg = lane >> 4;
    const unsigned id = xcd_order(blockIdx.x - begin, passes.ends[role] - begin);
    const unsigned tile = id % (unsigned)(a.nvt * a.nkt), rest = id / (unsigned)(a.nvt * a.nkt);
    const int vt = (int)tile / a.nkt, k0 = kDec ? (int)tile % a.nkt * KD : 0;  // the first key
    const int kdim = a.kd - k0;
    const unsigned chains = (unsigned)a.b * (unsigned)a.H;
    const int64_t chain = rest % chains;
    const int seg = (int)(rest / chains);
    const int64_t bi = (unsigned)chain / (unsigned)a.H;
    const int h = (int)((unsigned)chain % (unsigned)a.H), rv = a.rev ? 1 : 0;
    int64_t len = a.L;
    if (a.lengths) {
        const int64_t l = a.lengths[bi];
        len = l < 0 ? 0 : (l < a.L ? l : a.L);
    }
    const float ld = a.log_decay[h];
    const int64_t c_lo = seg * a.seg_chunks;
    const int64_t c_hi = c_lo + a.seg_chunks < a.nchunks ? c_lo + a.seg_chunks : a.nchunks;
    const int v0 = vt * kVT, col = v0 + 16 * wave + lr;  // this lane's value column
    const int64_t nstate = (int64_t)a.kd * a.vd;

    // the state: keys key_of(t, lg, r) of column col
    f32x4 S[KT], U[kU ? KT : 1];
    // (a stored state has up to 2^16 values: byte offsets from its first, and the buffer's bounds check for
    // keys and values that do not exist)
    const bool wide = a.sk == 1 && a.kd % 4 == 0;  // 4 keys at a time
    const auto state_at = [&](int c, int t, int r) {  // c: col
        const int n = k0 + key_of(t, lg, r);
        return n < a.kd && c < a.vd ? (unsigned)(n * a.sk + c * a.sv) * 4u : kOutside;
    };
    const auto state_rows = [&](const float *p, int64_t at) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(p) + at * nstate, 0, (int)(nstate * 4), 0x00020000);
    };
    const auto load_state = [&](f32x4 *to, const float *from, int64_t at) {
#pragma unroll
        for (int t = 0; t < KT; ++t) to[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (from == nullptr) return;
        const auto rsrc = state_rows(from, at);
        const int c = opaque(col);
        if (wide) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
                to[t] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, state_at(c, t, 0), 0, 0));
        } else {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    to[t][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, state_at(c, t, r), 0, 0));
        }
    };
    const auto store_state = [&](const f32x4 *from, float *to, int64_t at) {
        const auto rsrc = state_rows(to, at);
        const int c = opaque(col);
        if (wide) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, from[t]), rsrc, state_at(c, t, 0), 0, 0);
        } else {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(from[t][r]), rsrc, state_at(c, t, r), 0, 0);
        }
    };
    const int64_t in_at = a.seg_in ? chain * a.nseg + seg : chain;
    load_state(S, kSt ? nullptr : a.s_in, in_at);
    if constexpr (kU) load_state(U, kSt ? nullptr : a.u_in, in_at);

    if (tid <= C) pw[tid] = (float)power(ld, tid);
    __syncthreads();
    // Score tiles of this wave, (rows, columns) in 16s: of the 4 x 4 the 10 with j <= i are needed, and (0, 1) and
    // (2, 3) as zeros; three a wave, two of them in one row strip, so that no wave waits for another. fp32 has 2 x 2.
    constexpr int JW = IT == 4 ? 3 : 1;
    const int sa = IT == 4 ? (wave < 2 ? 3 : 4 - wave) : wave >> 1, sc_ = IT == 4 ? 2 * ((wave ^ (wave >> 1)) & 1) : sa;
    const int ta = IT == 4 ? (wave == 1 ? 2 : 0) : wave & 1, tc = IT == 4 ? (wave == 0 ? 0 : 4 - wave) : ta;
    const auto srow = [&](int t) { return t == 2 ? sc_ : sa; };
    const auto scol = [&](int t) { return t == 2 ? tc : ta + t; };
    float mask[kSt ? 1 : JW][4], rs[MODE != kOut ? 1 : IT];
    if constexpr (!kSt) {
#pragma unroll
        for (int t = 0; t < JW; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = 16 * srow(t) + lr - 16 * scol(t) - 4 * lg - r;
                mask[t][r] = n < 0 ? 0.f : a.si * pw[n < 0 ? 0 : n] * (kDec ? (float)n : 1.f);
            }
        if constexpr (MODE == kOut) {
#pragma unroll
            for (int it = 0; it < IT; ++it) rs[it] = a.sr * pw[16 * it + lr + 1 - rv];
        }
    }
    if constexpr (kDec) {
        if (tid < C) {
            wd[0][tid] = a.sr * pw[tid + 1];
            wd[1][tid] = a.sr * pw[tid + 1] * (float)(tid + 1);
        }
    }

    // Staging: 8 columns of a row a thread. Row i of a chunk is its token i, or nt - 1 - i backwards:
    // at (rv ? nt - 1 - i : i) strides from the first.
    constexpr int KN = C * (KD / 8) / kThreads, VN = C * (kVT / 8) / kThreads, QN = kSt ? 0 : KN;
    static_assert(C * (KD / 8) % kThreads == 0 && C * (kVT / 8) % kThreads == 0, "staging");
    constexpr int KR = kThreads / (KD / 8), VR = kThreads / (kVT / 8);  // rows of one pass
    typename O::pack kx[KN], vx[VN], qx[QN ? QN : 1], dx[kDec ? VN : 1];
    const int kn = 8 * (tid % (KD / 8)), ki = tid / (KD / 8), vn = 8 * (tid % (kVT / 8)), vi = tid / (kVT / 8);
    const unsigned kst = (unsigned)(a.k.heads * a.kd * ES), vst = (unsigned)(a.v.heads * a.vd * ES),
                   qst = kSt ? 0u : (unsigned)(a.q.heads * a.kd * ES), dst = kDec ? (unsigned)(a.dy.heads * a.vd * ES) : 0u;
    const auto first = [&](const Tensor &x, int head, int dim, unsigned stride) {
        return static_cast<const char *>(x.p) + bi * a.L * (int64_t)stride + (int64_t)head * dim * ES;
    };
    const char *kp = first(a.k, h / a.k.per, a.kd, kst) + k0 * ES, *vp = first(a.v, h / a.v.per, a.vd, vst),
               *qp = kSt ? nullptr : first(a.q, h / a.q.per, a.kd, qst) + k0 * ES,
               *dp = kDec ? first(a.dy, h / a.dy.per, a.vd, dst) : nullptr;
    const auto offset = [&](int i, unsigned stride, int n, int dim) {
        return n < dim ? (unsigned)(rv ? -1 - i : i) * stride + (unsigned)(n * ES) : kOutside;
    };
    const unsigned ko = offset(ki, kst, kn, kdim), vo = offset(vi, vst, v0 + vn, a.vd),
                   qo = kSt ? 0u : offset(ki, qst, kn, kdim), dof = kDec ? offset(vi, dst, v0 + vn, a.vd) : 0u;
    const auto tokens = [&](int64_t c) { return len - c * C >= C ? C : (len > c * C ? (int)(len - c * C) : 0); };
    const auto span = [&](int nt, unsigned stride, int dim) {
        return nt > 0 ? (unsigned)(nt - 1) * stride + (unsigned)(dim * ES) : 0u;
    };
    const auto down = [&](int nt, int rows, unsigned stride) { return (unsigned)(rv ? nt - rows : rows) * stride; };
    const auto fetch_k = [&](int nt, int u) {
        kx[u] = load8<E, VEC, kOnce>(kp, span(nt, kst, kdim), ko + down(nt, KR * u, kst), kdim - kn);
    };
    const auto fetch_v = [&](int nt, int u) {
        vx[u] = load8<E, VEC, kOnce>(vp, span(nt, vst, a.vd), vo + down(nt, VR * u, vst), a.vd - v0 - vn);
    };
    const auto fetch_q = [&](int nt, int u) {
        qx[u] = load8<E, VEC>(qp, span(nt, qst, kdim), qo + down(nt, KR * u, qst), kdim - kn);
    };
    const auto fetch_d = [&](int nt, int u) {
        if constexpr (kDec) dx[u] = load8<E, VEC>(dp, span(nt, dst, a.vd), dof + down(nt, VR * u, dst), a.vd - v0 - vn);
    };
    const auto put = [&](E *to, const typename O::pack &x) { *reinterpret_cast<typename O::pack *>(to) = x; };
    const auto k_at = [&](int u) { return (ki + KR * u) * KD + (((kn >> 3) ^ swap_of<E, KD>(ki + KR * u)) << 3); };
    const auto v_at = [&](int u) { return (vi + VR * u) * kVT + (((vn >> 3) ^ swap_of<E, kVT>(vi + VR * u)) << 3); };
    // The next chunk's tensors are loaded while this one is computed. Loads by single elements of
    // 128 keys leave no registers for that: there each piece is loaded and staged by itself.
    constexpr bool kAhead = VEC || (KD != 128 && !kDec) || ES == 4;
    const auto advance = [&](int64_t chunks) {
        kp += chunks * C * (int64_t)kst;
        vp += chunks * C * (int64_t)vst;
        if (!kSt) qp += chunks * C * (int64_t)qst;
        if (kDec) dp += chunks * C * (int64_t)dst;
    };
    const auto stage = [&](int nt) {
#pragma unroll
        for (int u = 0; u < KN; ++u) {
            if (!kAhead) {
                fetch_k(nt, u);
                __builtin_amdgcn_sched_barrier(0);
            }
            put(Ks + k_at(u), kx[u]);
        }
#pragma unroll
        for (int u = 0; u < VN; ++u) {
            if (!kAhead) {
                fetch_v(nt, u);
                __builtin_amdgcn_sched_barrier(0);
            }
            put(Vs + v_at(u), vx[u]);
            if constexpr (kDec) {
                if (!kAhead) {
                    fetch_d(nt, u);
                    __builtin_amdgcn_sched_barrier(0);
                }
                put(Ds + v_at(u), dx[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < QN; ++u) {
            if (!kAhead) {
                fetch_q(nt, u);
                __builtin_amdgcn_sched_barrier(0);
            }
            put(Qs + k_at(u), qx[u]);
        }
    };

    const int qb0 = row_base<E, KD>(lr, lg), ab0 = row_base<E, C>(lr, lg), cb0 = col_base<E, KD>(lr, lg),
              vb0 = val_base<E>(lr, lg, wave), rb0 = row_base<E, kVT>(lr, lg);
    const int p0 = v0 + 16 * wave + 4 * lg;  // the 4 values of this lane's outputs
    const unsigned oes = ES == 4 || a.o32 ? 4 : 2, ost = (unsigned)(a.H * a.vd) * oes;
    const int64_t ofirst = (bi * a.L * a.H + h) * (int64_t)a.vd;
    const auto row_of = [&](int i, int nt) { return rv ? nt - 1 - i : i; };
    const unsigned oo = (unsigned)row_of(lr, C) * ost + p0 * oes;
    double dsum = 0.0;

    // chunks that hold tokens; what lies behind the length is only filled with zeros
    const int64_t c_live = (len + C - 1) / C, c_end = c_hi < c_live ? c_hi : c_live;
    const int64_t nc = c_end > c_lo ? c_end - c_lo : 0;
    const int64_t c0 = rv ? c_end - 1 : c_lo;
    const int way = rv ? -1 : 1;
    if (nc > 0) advance(c0);
    if (kAhead && nc > 0) {
        const int nt = tokens(c0);
#pragma unroll
        for (int u = 0; u < KN; ++u) fetch_k(nt, u);
#pragma unroll
        for (int u = 0; u < VN; ++u) {
            fetch_v(nt, u);
            fetch_d(nt, u);
        }
#pragma unroll
        for (int u = 0; u < QN; ++u) fetch_q(nt, u);
    }
    char *op = MODE != kOut ? nullptr : static_cast<char *>(a.o) + ofirst * oes + (nc > 0 ? c0 : 0) * C * (int64_t)ost;
    // (formed here: in the loop the constants of exp would take registers of every step)
    const double p_full = uniform64(power(ld, C)), p_part = uniform64(power(ld, len % C));
    int nt_of = -1;                          // the tokens that these are for:
    double whole = 1.0, drift = 0.0;         // a^nt, nt a^nt, and the tables wt, wu
    float atn = 0.f;
    const auto stage_all = [&](int nt) {
        stage(nt);
        if (nt != nt_of) {
            nt_of = nt;
            if (tid < C) {
                const int n = nt - 1 - tid + rv;  // steps from this token to the state behind it
                wt[tid] = tid < nt ? a.su * pw[n] : 0.f;
                if constexpr (kU) wu[tid] = tid < nt ? a.su * pw[n] * (float)n : 0.f;
            }
            whole = nt == C ? p_full : p_part;
            atn = uniform((float)(whole * (double)nt));
        }
    };
    if (nc > 0) stage_all(tokens(c0));
    for (int64_t s = 0; s < nc; ++s) {
        const int64_t c = c0 + way * s;
        const int nt = tokens(c);
        __syncthreads();  // the chunk's tiles are there, the last one's scores have been read
        const bool more = s + 1 < nc;
        const int nt_next = more ? tokens(c + way) : 0;
        advance(way);  // (behind the last chunk nothing is valid, and nothing read)
        if (kSt && kAhead) {
#pragma unroll
            for (int u = 0; u < KN; ++u) fetch_k(nt_next, u);
        }
        const int qb = opaque(qb0), ab = opaque(ab0), cb = opaque(cb0), vb = opaque(vb0), rb = opaque(rb0);
        frag vf[JS];
        const auto read_v = [&]() {
#pragma unroll
            for (int ks = 0; ks < JS; ++ks) vf[ks] = val_frag<E>(Vs, vb, ks);
        };
        f32x4 acc[MODE == kOut ? IT : 1], sc[MODE == kOut ? JW : 1];
        float csum = 0.f;
        if constexpr (kSt) read_v();
        if constexpr (kDec) {
            // q.k and dy.v of this wave's tiles (rows j, column i)
            f32x4 qk[JW], dv[JW];
#pragma unroll
            for (int t = 0; t < JW; ++t) qk[t] = dv[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (kAhead) {
#pragma unroll
                    for (int u = 0; u < KN; ++u)
                        if (u % KS == ks) fetch_k(nt_next, u);
                }
#pragma unroll
                for (int t = 0; t < JW; ++t)
                    qk[t] = O::mfma(row_frag<E, KD>(Ks, qb, scol(t), ks), row_frag<E, KD>(Qs, qb, srow(t), ks), qk[t]);
                if (ks % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ks = 0; ks < kVT / 32; ++ks)
#pragma unroll
                for (int t = 0; t < JW; ++t)
                    dv[t] = O::mfma(row_frag<E, kVT>(Vs, rb, scol(t), ks), row_frag<E, kVT>(Ds, rb, srow(t), ks), dv[t]);
#pragma unroll
            for (int t = 0; t < JW; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) csum += mask[t][r] == 0.f ? 0.f : mask[t][r] * qk[t][r] * dv[t][r];
            __builtin_amdgcn_sched_barrier(0);
            // q^T (weighted dy), four key tiles at a time, against the states
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                frag wv[JS][NP];
#pragma unroll
                for (int ks = 0; ks < JS; ++ks) {
                    const frag df = val_frag<E>(Ds, vb, ks);
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = wd[n][32 * ks + 8 * lg + e] * O::value(df, e);
                    O::template parts<NP>(x, wv[ks]);
                }
#pragma unroll
                for (int t = 0; t < KT; t += 4) {
                    f32x4 g[4];
#pragma unroll
                    for (int d = 0; d < 4; ++d) g[d] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < JS; ++ks) {
                        frag kf[4];
#pragma unroll
                        for (int d = 0; d < 4; ++d) kf[d] = col_frag<E, KD>(Qs, cb, t + d, ks);
#pragma unroll
                        for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                            for (int d = 0; d < 4; ++d) g[d] = O::mfma(kf[d], wv[ks][p], g[d]);
                    }
#pragma unroll
                    for (int d = 0; d < 4; ++d)
#pragma unroll
                        for (int r = 0; r < 4; ++r) csum += (n ? S : U)[t + d][r] * g[d][r];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            dsum += (double)csum;
            read_v();
        }
        if constexpr (MODE == kOut) {
            // Scores, transposed (rows j, column i = this lane's token of the strip), and the carried
            // state's part of the outputs (rows are values, column i). A step's fragments are read, and
            // pieces of the next chunk's k loaded, while the step before is computed.
#pragma unroll
            for (int t = 0; t < JW; ++t) sc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int it = 0; it < IT; ++it) acc[it] = f32x4{0.f, 0.f, 0.f, 0.f};
            constexpr int QA = IT == 4 ? 2 : 1;
            frag qs[2][QA], kf[2][JW], qf[2][IT];
            const auto read = [&](int ks, int b) {
#pragma unroll
                for (int it = 0; it < IT; ++it) qf[b][it] = row_frag<E, KD>(Qs, qb, it, ks);
                qs[b][0] = row_frag<E, KD>(Qs, qb, sa, ks);
                if constexpr (QA == 2) qs[b][1] = row_frag<E, KD>(Qs, qb, sc_, ks);
#pragma unroll
                for (int t = 0; t < JW; ++t) kf[b][t] = row_frag<E, KD>(Ks, qb, scol(t), ks);
            };
            // the state's parts of a step, formed during the step before
            frag sp[2][NP];
            const auto split = [&](int ks, int b) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = S[2 * ks + (e >> 2)][e & 3];
                O::template parts<NP>(x, sp[b]);
            };
            if (kAhead) read(0, 0);
            split(0, 0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int b = kAhead ? ks & 1 : 0;
                if (!kAhead) read(ks, 0);
                else if (ks + 1 < KS) read(ks + 1, b ^ 1);
                if (kAhead) {
#pragma unroll
                    for (int u = 0; u < KN; ++u)
                        if (u % KS == ks) fetch_k(nt_next, u);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (ks + 1 < KS) split(ks + 1, (ks + 1) & 1);
#pragma unroll
                for (int n = NP - 1; n >= 0; --n)
#pragma unroll
                    for (int it = 0; it < IT; ++it) acc[it] = O::mfma(sp[ks & 1][n], qf[b][it], acc[it]);
#pragma unroll
                for (int t = 0; t < JW; ++t) sc[t] = O::mfma(kf[b][t], qs[b][t == 2 ? 1 : 0], sc[t]);
                __builtin_amdgcn_sched_barrier(0);
            }
            read_v();
        }
        // What is left of the scores and of the state's part of the outputs is done among the products of the update
        const auto put_scores = [&]() {
            if constexpr (MODE == kOut) {
#pragma unroll
                for (int t = 0; t < JW; ++t) {
                    const int jb = 2 * scol(t) + (lg >> 1);
                    f32x4 x;
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[r] = sc[t][r] * mask[t][r];
                    O::template store4<NP>(
                        As + (16 * srow(t) + lr) * C + ((jb ^ swap_of<E, C>(lr)) << 3) + 4 * (lg & 1), C * C, x);
                }
            }
        };
        const auto scale_rows = [&]() {
            if constexpr (MODE == kOut) {
#pragma unroll
                for (int it = 0; it < IT; ++it)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[it][r] *= rs[it];
            }
        };

        // the state behind the chunk
        {
            // A step: four key tiles and 32 tokens, whose fragments are read during the step before. U, which needs the
            // old S, goes first, then S.
            constexpr int TS = 4, NSTEP = KT / TS * JS;
            frag kf[2][TS];
            const auto read = [&](int step) {
#pragma unroll
                for (int d = 0; d < TS; ++d)
                    kf[kAhead ? step & 1 : 0][d] = col_frag<E, KD>(Ks, cb, TS * (step / JS) + d, step % JS);
            };
            // a^nt rounded so that the errors of the chunks cancel: of their product no more than one remains
            const float at = uniform((float)(whole + drift));
            drift = uniform64(drift + (whole - (double)at));
#pragma unroll
            for (int of_u = kU; of_u >= 0; --of_u) {
                f32x4 *const X = of_u ? U : S;
                frag wv[JS][NP];
                if (kAhead) read(0);
                const auto weigh = [&](int ks) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = (of_u ? wu : wt)[32 * ks + 8 * lg + e] * O::value(vf[ks], e);
                    O::template parts<NP>(x, wv[ks]);
                };
                weigh(0);
#pragma unroll
                for (int step = 0; step < NSTEP; ++step) {
                    const int t = TS * (step / JS), ks = step % JS;
                    if (!kAhead) read(step);
                    else if (step + 1 < NSTEP) read(step + 1);
                    if (kAhead && !of_u) {
#pragma unroll
                        for (int u = 0; u < VN; ++u)
                            if (u % NSTEP == step) {
                                fetch_v(nt_next, u);
                                fetch_d(nt_next, u);
                            }
#pragma unroll
                        for (int u = 0; u < QN; ++u)
                            if (u % NSTEP == step) fetch_q(nt_next, u);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    if (ks == 0) {
#pragma unroll
                        for (int d = 0; d < TS; ++d)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                X[t + d][r] = of_u ? at * X[t + d][r] + atn * S[t + d][r] : at * X[t + d][r];
                    }
#pragma unroll
                    for (int n = NP - 1; n >= 0; --n)
#pragma unroll
                        for (int d = 0; d < TS; ++d)
                            X[t + d] = O::mfma(kf[kAhead ? step & 1 : 0][d], wv[ks][n], X[t + d]);
                    if (step == 0 && JS == 2) weigh(1);
                    if (!of_u && step == (NSTEP > 1 ? 1 : 0)) put_scores();
                    if (!of_u && step == NSTEP - 1) scale_rows();
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        __syncthreads();  // the scores are there, the chunk's tiles have been read

        if constexpr (MODE == kOut) {
            // (the blocks of 32 tokens that lie behind a strip hold nothing for it)
#pragma unroll
            for (int ks = 0; ks < JS; ++ks) {
                frag af[NP][IT];
#pragma unroll
                for (int n = NP - 1; n >= 0; --n)
#pragma unroll
                    for (int it = 2 * ks; it < IT; ++it) af[n][it] = row_frag<E, C>(As + n * C * C, ab, it, ks);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = NP - 1; n >= 0; --n)
#pragma unroll
                    for (int it = 2 * ks; it < IT; ++it) acc[it] = O::mfma(vf[ks], af[n][it], acc[it]);
            }
        }
        if (more) stage_all(nt_next);
        if constexpr (MODE == kOut) {
            {
                const int rows = a.L - c * C < C ? (int)(a.L - c * C) : C;  // written: zeros behind the length
                if constexpr (VEC) {
                    // (rows behind the last lie outside the buffer, and are dropped)
                    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
                        op, 0, (int)((unsigned)(rows - 1) * ost + (unsigned)(a.vd * oes)), 0x00020000);
                    unsigned to[IT];
#pragma unroll
                    for (int it = 0; it < IT; ++it) to[it] = oo + (rv ? -16u : 16u) * it * ost;
                    if (nt < C) {
#pragma unroll
                        for (int it = 0; it < IT; ++it) {
                            const int i = 16 * it + lr;
                            to[it] = (unsigned)(i < nt ? row_of(i, nt) : i) * ost + (unsigned)(p0 * oes);
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[it][r] = i < nt ? acc[it][r] : 0.f;
                        }
                    }
                    if (p0 < a.vd) {
                        if (oes == 4) {
#pragma unroll
                            for (int it = 0; it < IT; ++it)
                                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[it]), rsrc, to[it], 0, 0);
                        } else {
#pragma unroll
                            for (int it = 0; it < IT; ++it)
                                __builtin_amdgcn_raw_buffer_store_b64(bf16_pack4(acc[it]), rsrc, to[it], 0, 0);
                        }
                    }
                } else {
#pragma unroll
                    for (int it = 0; it < IT; ++it) {
                        const int i = 16 * it + lr, row = i < nt ? row_of(i, nt) : i;
                        char *to = op + (int64_t)row * ost + p0 * oes;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float x = i < nt ? acc[it][r] : 0.f;
                            if (row < rows && p0 + r < a.vd) {
                                if (oes == 4) reinterpret_cast<float *>(to)[r] = x;
                                else reinterpret_cast<__bf16 *>(to)[r] = (__bf16)x;
                            }
                        }
                    }
                }
            }
            op += way * (int64_t)C * ost;
        }
    }

    if constexpr (MODE == kOut) {
        const int64_t from = (c_end > c_lo ? c_end : c_lo) * C, to = c_hi * C < a.L ? c_hi * C : a.L;
        constexpr int PV = VEC ? 8 : 1;  // values of one store
        for (int64_t e = tid; e < (to - from) * (kVT / PV); e += kThreads) {
            const int p = v0 + PV * (int)(e % (kVT / PV));
            char *at = static_cast<char *>(a.o) + (ofirst + (from + e / (kVT / PV)) * (int64_t)(a.H * a.vd) + p) * oes;
            if (p < a.vd) {
                if constexpr (VEC) {
                    *reinterpret_cast<u32x4 *>(at) = u32x4{0, 0, 0, 0};
                    if (oes == 4) reinterpret_cast<u32x4 *>(at)[1] = u32x4{0, 0, 0, 0};
                } else if (oes == 4) {
                    *reinterpret_cast<float *>(at) = 0.f;
                } else {
                    *reinterpret_cast<uint16_t *>(at) = 0;
                }
            }
        }
    }
    if constexpr (kSt) {
        store_state(S, a.s_out, chain * a.nseg + seg);
        if constexpr (kU) store_state(U, a.u_out, chain * a.nseg + seg);
    }
    const bool last = a.rev ? seg == 0 : seg == a.nseg - 1;
    if constexpr (MODE == kOut) {
        if (last && a.s_out) store_state(S, a.s_out, chain);
    }
    if constexpr (kDec) {
        if (last && a.dh_final) {
            load_state(S, a.dh_final, chain);
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) dsum += (double)U[t][r] * (double)S[t][r];
        }
        // sum over the workgroup, in a fixed order
        __shared__ double sums[kThreads];
        sums[tid] = dsum;
        __syncthreads();
        for (int n = kThreads / 2; n > 0; n >>= 1) {
            if (tid < n) sums[tid] += sums[tid + n];
            __syncthreads();
        }
        if (tid == 0) a.part[(((int64_t)h * a.b + bi) * a.nseg + seg) * (a.nvt * a.nkt) + tile] = sums[0];
    }
}

// Segment states into incoming states, in place: st[c][seg] <- the state before the
// segment (in the order of the sweep), from init [c] or zero. One thread a state element; the loads
// of 8 segments are in flight together.
struct ChainArgs {
    float *st, *ut;
    const float *init, *log_decay;
    const int *lengths;
    int64_t chains, nstate, L, seg_tokens;
    int H, nseg;
    bool rev;
};

__device__ __forceinline__ void chain_element(const ChainArgs &a, int64_t e) {
    const int64_t chain = e / a.nstate, i = e % a.nstate, bi = chain / a.H;
    int64_t len = a.L;
    if (a.lengths) {
        const int64_t l = a.lengths[bi];
        len = l < 0 ? 0 : (l < a.L ? l : a.L);
    }
    const float ld = a.log_decay[chain % a.H];
    const double whole = power(ld, a.seg_tokens);
    double s = a.init ? a.init[e] : 0.f, u = 0.0;
    constexpr int kAhead = 8;
    for (int k0 = 0; k0 < a.nseg; k0 += kAhead) {
        float own[kAhead], ou[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = k0 + j < a.nseg ? k0 + j : a.nseg - 1;
            const int64_t at = (chain * a.nseg + (a.rev ? a.nseg - 1 - k : k)) * a.nstate + i;
            own[j] = a.st[at];
            ou[j] = a.ut ? a.ut[at] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int k = k0 + j, seg = a.rev ? a.nseg - 1 - k : k;
            if (k >= a.nseg) break;
            int64_t n = len - seg * a.seg_tokens;
            n = n < 0 ? 0 : (n < a.seg_tokens ? n : a.seg_tokens);
            const double p = n == a.seg_tokens ? whole : power(ld, n);
            const int64_t at = (chain * a.nseg + seg) * a.nstate + i;
            a.st[at] = (float)s;
            if (a.ut) {
                a.ut[at] = (float)u;
                u = p * u + p * (double)n * s + ou[j];
            }
            s = p * s + own[j];
        }
    }
}

struct Chains {
    ChainArgs a[2];
    int n;
};

__global__ __launch_bounds__(kThreads) void linattn_chain_kernel(const Chains c) {
    const int64_t n = c.a[0].chains * c.a[0].nstate;
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < n * c.n; e += (int64_t)gridDim.x * kThreads) {
        if (e < n) chain_element(c.a[0], e);
        else chain_element(c.a[1], e - n);
    }
}

// out[row][g][d] = sum over the heads of group g of part[row][h][d], for dk and dv
struct Heads {
    const float *part[2];
    void *out[2];
    int64_t rows;
    int G, per, d[2];
};

template <bool BF16>
__global__ __launch_bounds__(kThreads) void linattn_heads_kernel(const Heads a) {
    const int64_t n0 = a.rows * a.G * a.d[0], n = n0 + a.rows * a.G * a.d[1];
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const bool v = i >= n0;
        const int64_t e = v ? i - n0 : i;
        const int d = v ? a.d[1] : a.d[0];
        const int64_t rg = e / d;
        const float *p = (v ? a.part[1] : a.part[0]) + rg * a.per * d + e % d;
        void *out = v ? a.out[1] : a.out[0];
        float s = 0.f;
        for (int k = 0; k < a.per; ++k) s += p[(int64_t)k * d];
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
hipError_t launch_dims(const Passes &p, hipStream_t s) {
    const dim3 g(p.ends[p.n - 1]), t(kThreads);
    int kd = 0;
    for (int i = 0; i < p.n; ++i) kd = p.a[i].kd > kd ? p.a[i].kd : kd;
    if constexpr (MODE == kDecay) hipLaunchKernelGGL((linattn_kernel<E, 64, MODE, VEC>), g, t, 0, s, p);
    else if (kd <= 64) hipLaunchKernelGGL((linattn_kernel<E, 64, MODE, VEC>), g, t, 0, s, p);
    else if (kd <= 128) hipLaunchKernelGGL((linattn_kernel<E, 128, MODE, VEC>), g, t, 0, s, p);
    else hipLaunchKernelGGL((linattn_kernel<E, 256, MODE, VEC>), g, t, 0, s, p);
    return hipGetLastError();
}

template <int MODE>
hipError_t launch_passes(Passes &p, bool bf16, hipStream_t s) {
    bool vec = true;
    int64_t end = 0;
    for (int i = 0; i < 3; ++i) {
        const Args &a = p.a[i];
        if (i < p.n) {
            end += a.b * a.H * a.nseg * a.nvt * a.nkt;
            vec = vec && a.kd % 8 == 0 && a.vd % 8 == 0;
        }
        p.ends[i] = (unsigned)end;
    }
    if (end == 0) return hipSuccess;
    constexpr int kSingle = MODE == kStateOnce ? kState : MODE;  // (loads by elements are all the same)
    if (bf16) return vec ? launch_dims<uint16_t, MODE, true>(p, s) : launch_dims<uint16_t, kSingle, false>(p, s);
    return vec ? launch_dims<float, MODE, true>(p, s) : launch_dims<float, kSingle, false>(p, s);
}

template <int MODE>
hipError_t launch_pass(const Args &a, bool bf16, hipStream_t s) {
    Passes p{};
    p.a[0] = a;
    p.n = 1;
    return launch_passes<MODE>(p, bf16, s);
}

struct LinPlan {
    int64_t nchunks, seg_chunks, chains;
    int nseg, C;
};

int tiles(int64_t d) { return (int)((d + kVT - 1) / kVT); }

// Key tiles of the kernels
int key_size(int64_t d) { return d <= 64 ? 64 : (d <= 128 ? 128 : 256); }

// Segments. A pass has a workgroup a chain and tile of values (the backward runs three passes at
// once), and a CU has room for two, or for one with 256 keys. Splitting reads k and v twice, about 1.45 times
// the work, and two workgroups of a CU run at 0.6 of the speed of one: two segments that fill the
// second place cost more than they bring (b4 L2048, 256 workgroups: 110 us in one piece, 138 in
// two), three or more pay (48 workgroups of L32768: 1487 us in one piece, 414 in ten). Segments have two
// chunks at least; below six chunks the two launches more cost as much as they save.
LinPlan make_lin_plan(const m3_shape &s, bool bwd) {
    LinPlan p{};
    p.C = s.io_dtype == M3_BF16 ? Ops<uint16_t>::C : Ops<float>::C;
    p.chains = s.batch * s.nheads;
    p.nchunks = (s.seqlen + p.C - 1) / p.C;
    int64_t n = s.nsegments;
    if (n == 0) {
        const int64_t have = p.chains * (bwd ? 2 * tiles(s.dstate) + tiles(s.headdim) : tiles(s.headdim));
        const bool one = key_size(s.dstate) == 256 || (bwd && key_size(s.headdim) == 256);
        n = have == 0 ? 1 : (one ? 256 : 512) / have;
        if (!one && n == 2) n = 1;
        if (n > p.nchunks / 2) n = p.nchunks / 2;
        if (p.nchunks < 6) n = 1;
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
    if (s->batch > (1LL << 31) || s->seqlen > (1LL << 31) || s->batch * s->nheads > kMaxGrid ||
        (s->seqlen > 0 && s->batch * s->nheads > (1LL << 40) / s->seqlen))
        return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

m3_status lin_plan(const m3_shape *s, bool bwd, LinPlan *p) {
    const m3_status st = lin_check(s, 0);
    if (st != M3_OK) return st;
    *p = make_lin_plan(*s, bwd);
    // one workgroup a chain, segment and tile of values and keys
    const int64_t wgs = p->chains * p->nseg;
    if (wgs * tiles(s->headdim) * tiles(s->dstate) > kMaxGrid || wgs * (2 * tiles(s->dstate) + tiles(s->headdim)) > kMaxGrid)
        return M3_ERR_UNSUPPORTED;
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
    w.part = up((size_t)p.chains * p.nseg * tiles(s.headdim) * tiles(s.dstate) * 8);
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
    a.nkt = 1;
    a.sk = swapped ? (int)vd : 1;
    a.sv = swapped ? 1 : (int)kd;
}

ChainArgs chain_args(const Args &a, const LinPlan &p, float *st, float *ut, const float *init) {
    ChainArgs c{};
    c.st = st; c.ut = ut; c.init = init; c.log_decay = a.log_decay; c.lengths = a.lengths;
    c.chains = p.chains; c.nstate = (int64_t)a.kd * a.vd; c.L = a.L; c.seg_tokens = p.seg_chunks * p.C;
    c.H = a.H; c.nseg = p.nseg; c.rev = a.rev;
    return c;
}

hipError_t chain_states(const Chains &c, hipStream_t s) {
    int64_t grid = (c.n * c.a[0].chains * c.a[0].nstate + kThreads - 1) / kThreads;
    if (grid > 65536) grid = 65536;
    hipLaunchKernelGGL(linattn_chain_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, c);
    return hipGetLastError();
}

hipError_t sum_heads(const Heads &h, bool bf16, hipStream_t s) {
    int64_t grid = (h.rows * h.G * (h.d[0] + h.d[1]) + kThreads - 1) / kThreads;
    if (grid == 0) return hipSuccess;
    if (grid > 65536) grid = 65536;
    if (bf16) hipLaunchKernelGGL((linattn_heads_kernel<true>), dim3((unsigned)grid), dim3(kThreads), 0, s, h);
    else hipLaunchKernelGGL((linattn_heads_kernel<false>), dim3((unsigned)grid), dim3(kThreads), 0, s, h);
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
    const float a = (float)power(log_decay[h], 1);
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
    // Rows of a thread: four (97 us for 8192 states of 64 x 128 in fp32; 99 with eight, 108 with two), or one
    // where the states are few, so that more of the card takes part
    const bool wide = a.b * a.H >= 1024;
    const int rows = RW * (wide ? 4 : 1);
    const dim3 grid((unsigned)(a.b * a.H), (unsigned)((a.P + rows - 1) / rows)), t(kThreads);
    if (wide)
        hipLaunchKernelGGL((linattn_step_kernel<E, T, LPR, 4, VEC>), grid, t, 0, s, io.q, io.k, io.v, io.log_decay, io.h,
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

// Each segment's own end states in one direction
hipError_t segment_states(Args a, bool bf16, float *st, float *ut, hipStream_t s) {
    a.s_in = nullptr; a.s_out = st; a.u_out = ut;
    if (ut) return launch_pass<kStateU>(a, bf16, s);
    // (heads or tiles of values that read the same rows find them in the caches; else these would only hold what the
    // outputs' pass reads long after: b2 L32768 of 24 heads 413 us, with ordinary loads 425;
    // b1 L65536 of 16 heads 275 and 287)
    return a.k.per == 1 && a.v.per == 1 && a.nvt == 1 ? launch_pass<kStateOnce>(a, bf16, s) : launch_pass<kState>(a, bf16, s);
}

}  // namespace
}  // namespace m3i

using namespace m3i;

extern "C" {

size_t m3_linattn_workspace_bytes(const m3_shape *shape) {
    LinPlan p;
    if (lin_plan(shape, false, &p) != M3_OK || p.nseg == 1) return 0;
    return up((size_t)p.chains * p.nseg * shape->headdim * shape->dstate * 4);
}

m3_status m3_linattn_fwd(const m3_shape *shape, const m3_linattn_io *io, void *workspace, size_t ws_bytes,
                         void *stream) {
    LinPlan p;
    const m3_status st = lin_plan(shape, false, &p);
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
    // (h_final may be h0: a state is read before its end is written)
    if (clash({io->y, io->h_final}, {io->q, io->k, io->v, io->log_decay, io->lengths, workspace}) ||
        clash({io->y}, {io->h0}) ||
        (need && clash({workspace}, {io->q, io->k, io->v, io->log_decay, io->lengths, io->h0})))
        return M3_ERR_INVALID_ARG;
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
        Chains c{};
        c.a[0] = chain_args(a, p, seg, nullptr, io->h0);
        c.n = 1;
        if (segment_states(a, bf16, seg, nullptr, hs) != hipSuccess || chain_states(c, hs) != hipSuccess)
            return M3_ERR_HIP;
        a.s_in = seg;
        a.seg_in = true;
    }
    a.o = io->y;
    a.s_out = io->h_final;
    return status(launch_pass<kOut>(a, bf16, hs));
}

size_t m3_linattn_bwd_workspace_bytes(const m3_shape *shape) {
    LinPlan p;
    return lin_plan(shape, true, &p) == M3_OK ? bwd_ws(*shape, p).total : 0;
}

m3_status m3_linattn_bwd(const m3_shape *shape, const m3_linattn_io *io, const m3_linattn_grads *gr, void *workspace,
                         size_t ws_bytes, void *stream) {
    LinPlan p;
    const m3_status st = lin_plan(shape, true, &p);
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
    if (clash({gr->dq, gr->dk, gr->dv, gr->dlog_decay, gr->dh0, w.total ? workspace : nullptr},
              {io->q, io->k, io->v, io->log_decay, io->h0, io->lengths, gr->dy, gr->dh_final}))
        return M3_ERR_INVALID_ARG;
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
            float *ut = gr->dlog_decay ? seg_u : nullptr;
            Chains c{};
            c.a[0] = chain_args(f, p, seg_s, ut, io->h0);
            c.a[1] = chain_args(r, p, seg_d, nullptr, gr->dh_final);
            c.n = 2;
            if (segment_states(f, bf16, seg_s, ut, hs) != hipSuccess ||
                segment_states(r, bf16, seg_d, nullptr, hs) != hipSuccess || chain_states(c, hs) != hipSuccess)
                return M3_ERR_HIP;
        }
        const float *s_in = split ? seg_s : io->h0, *d_in = split ? seg_d : gr->dh_final;
        f.seg_in = r.seg_in = split;
        Args dq = f;  // (dy, v, k), the state transposed
        set_dims(dq, s.headdim, s.dstate, true);
        dq.q = dy; dq.k = v; dq.v = k; dq.s_in = s_in; dq.o = gr->dq;
        Args dk = r;  // (v, dy, q), the state transposed
        set_dims(dk, s.headdim, s.dstate, true);
        dk.q = v; dk.k = dy; dk.v = q; dk.s_in = d_in;
        dk.o32 = per > 1; dk.o = per > 1 ? pk : gr->dk;
        Args dv = r;  // (k, q, dy)
        dv.s_in = d_in; dv.s_out = gr->dh0;
        dv.o32 = per > 1; dv.o = per > 1 ? pv : gr->dv;
        // all three at once where one kernel fits their keys (P of dq and dk, N of dv)
        // or, larger than some need, all workgroups of one launch run at the same time
        const int64_t wgs = p.chains * p.nseg * (2 * tiles(s.dstate) + tiles(s.headdim));
        const int kp = key_size(s.headdim), kn = key_size(s.dstate);
        Passes first{}, second{};
        first.a[0] = dq; first.a[1] = dk; first.a[2] = dv;
        first.n = kp == kn || wgs <= (kp == 256 || kn == 256 ? 256 : 512) ? 3 : 2;
        if ((e = launch_passes<kOut>(first, bf16, hs)) != hipSuccess) return M3_ERR_HIP;
        if (first.n == 2) {
            second.a[0] = dv;
            second.n = 1;
            if ((e = launch_passes<kOut>(second, bf16, hs)) != hipSuccess) return M3_ERR_HIP;
        }
        if (per > 1) {
            const Heads sums = {{pk, pv}, {gr->dk, gr->dv}, s.batch * s.seqlen, G, per, {(int)s.dstate, (int)s.headdim}};
            if ((e = sum_heads(sums, bf16, hs)) != hipSuccess) return M3_ERR_HIP;
        }
        if (gr->dlog_decay) {
            f.s_in = s_in; f.u_in = split ? seg_u : nullptr;
            f.nkt = tiles(s.dstate); f.dy = dy; f.dh_final = gr->dh_final; f.part = part;
            if ((e = launch_pass<kDecay>(f, bf16, hs)) != hipSuccess) return M3_ERR_HIP;
        }
    }
    if (gr->dlog_decay) {
        hipLaunchKernelGGL(linattn_decay_kernel, dim3((unsigned)H), dim3(kThreads), 0, hs, part, gr->dlog_decay,
                           s.batch * p.nseg * tiles(s.headdim) * tiles(s.dstate));
        e = hipGetLastError();
    }
    return status(e);
}

m3_status m3_linattn_step(const m3_shape *shape, const m3_linattn_step_io *io, void *stream) {
    if (!shape) return M3_ERR_INVALID_ARG;
    m3_shape s = *shape;
    s.seqlen = 1;
    s.nsegments = 0;  // (neither is used)
    const m3_status st = lin_check(&s, M3_FLAG_BF16_STATE);
    if (st != M3_OK) return st;
    if (!io || !isfinite(io->scale)) return M3_ERR_INVALID_ARG;
    if (s.batch == 0) return M3_OK;
    if (!io->q || !io->k || !io->v || !io->log_decay || !io->h || !io->y) return M3_ERR_INVALID_ARG;
    const void *ptrs[] = {io->q, io->k, io->v, io->log_decay, io->h, io->y};
    for (const void *x : ptrs)
        if (!al16(x)) return M3_ERR_MISALIGNED;
    if (clash({io->y, io->h}, {io->q, io->k, io->v, io->log_decay})) return M3_ERR_INVALID_ARG;
    const StepArgs a = {io, s.batch, (int)s.nheads, (int)(s.nheads / s.ngroups), (int)s.headdim, (int)s.dstate};
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const bool bs = (s.flags & M3_FLAG_BF16_STATE) != 0;
    if (s.io_dtype == M3_BF16)
        return status(bs ? launch_step<uint16_t, uint16_t>(a, hs) : launch_step<uint16_t, float>(a, hs));
    return status(bs ? launch_step<float, uint16_t>(a, hs) : launch_step<float, float>(a, hs));
}

}  // extern "C"
