/*
 * m3_rotary.h -- rotary positions: queries and keys turned by their positions,
 * for the linear attention of m3_linattn.h and any other attention.
 *
 * For every token with position pos, every head and every i < rotary/2, with
 * t = pos * freqs[i] and a pair (u, w) of the head's first `rotary` channels:
 *   (u', w') = scale * (u cos t - w sin t, u sin t + w cos t)
 * Pairs are channels (i, i + rotary/2), or (2i, 2i + 1) with M3_ROTARY_INTERLEAVED.
 * Channels from `rotary` on are copied as they are. With M3_ROTARY_BACKWARD t is
 * negated: the gradients of q and k from those of the outputs.
 *   q [b,L,H,D], k [b,L,G,D] io dtype (k NULL: none), q_out, k_out likewise
 *   freqs [rotary/2] fp32, radians a position, finite (scaling for long contexts is in
 *     them; `scale` is its factor on the magnitude)
 *   positions [b,L] int32: each token's; or offsets [b] int32: token t of row i is at
 *     offsets[i] + t; or neither: at t. (A single token a row: L = 1.)
 * t is formed and reduced in two fp64 numbers, so far positions keep their angle: cosine and sine are
 * off by at most 2^-22 where |t| <= 2^64. Each output is rounded once.
 * D: 1 to 1024; rotary even, 0 to D; H, G 1 to 4096, b * L * (H + G) * D <= 2^40 (else
 * M3_ERR_UNSUPPORTED). D in multiples of 8 in bf16, of 4 in fp32, load
 * fastest, with halves rotary in multiples of 16 or 8 too; half of each in bf16 comes next.
 *
 * Conventions as in m3.h: dense row-major tensors, 16-byte aligned pointers, the
 * caller owns every buffer, the stream is a hipStream_t of the current device
 * passed as void*, all arguments are checked on the host before any HIP call,
 * nothing is allocated, freed or synchronised, and every call can be captured into
 * a graph. The same call gives the same bits. q_out may be q itself and k_out k (then
 * the channels from `rotary` on are not touched); no other overlap with what is
 * written (a pointer given twice otherwise is M3_ERR_INVALID_ARG).
 */
#ifndef M3_ROTARY_H
#define M3_ROTARY_H

#include "m3.h"

#ifdef __cplusplus
extern "C" {
#endif

#define M3_ROTARY_INTERLEAVED 1
#define M3_ROTARY_BACKWARD 2

typedef struct {
    int64_t batch;    /* >= 0 */
    int64_t seqlen;   /* >= 0 */
    int64_t nheads;   /* >= 1: heads of q */
    int64_t ngroups;  /* >= 1: heads of k (not used without k) */
    int64_t headdim;  /* >= 1 */
    int64_t rotary;   /* even, 0 .. headdim */
    int32_t io_dtype; /* m3_dtype */
    uint32_t flags;
    float scale;      /* finite */
    int32_t reserved; /* 0 */
} m3_rotary_shape;

typedef struct {
    const void *q;            /* [b,L,H,D] io */
    const void *k;            /* [b,L,G,D] io or NULL */
    const float *freqs;       /* [rotary/2] */
    const int32_t *positions; /* [b,L] or NULL */
    const int32_t *offsets;   /* [b] or NULL; not both */
    void *q_out;              /* out [b,L,H,D] io */
    void *k_out;              /* out [b,L,G,D] io: required with k, else NULL */
} m3_rotary_io;

m3_status m3_rotary(const m3_rotary_shape *shape, const m3_rotary_io *io, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* M3_ROTARY_H */
