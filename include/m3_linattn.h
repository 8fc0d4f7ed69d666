/*
 * m3_linattn.h -- linear attention with a decay for each head, beside the
 * Mamba-3 mixer core of m3.h.
 *
 * For every batch row, with a_h = exp(log_decay[h]) and g = h / (H/G):
 *
 *   S_t = a_h S_{t-1} + v_t[g] k_t[g]^T          (state [P,N], S_{-1} = h0 or 0)
 *   y_t[h] = scale * S_t q_t[h]
 *
 * that is y_t = scale * sum_{j<=t} a_h^{t-j} (q_t . k_j) v_j (+ the initial
 * state's term). m3_linattn_fwd evaluates it for a prompt with the chunked
 * algorithm (masked products inside a chunk, a state carried between chunks),
 * m3_linattn_bwd gives the gradients, m3_linattn_step advances one token.
 *
 * Shapes use m3_shape: batch b, seqlen L, nheads H query heads, ngroups G key and
 * value heads (H % G == 0; head h reads h / (H/G)), headdim P values per head,
 * dstate N keys per head, io_dtype; rank must be 1, chunk and eps are not used.
 * N and P: 1 to 256, any value; multiples of 8 load fastest. H <= 65536, b * L * H <= 2^40,
 * and b * H, times the segments and the tiles of 64 values and keys, below 2^24 (else M3_ERR_UNSUPPORTED).
 *   q [b,L,H,N]   k [b,L,G,N]   v [b,L,G,P]   y [b,L,H,P]     io dtype
 *   log_decay [H] fp32: <= 0 (a decay of at most 1); -infinity is a decay of 0,
 *     a state that holds its last token only
 *   states [b,H,P,N] fp32 (the layout of m3.h's states)
 *   lengths [b] int32 or NULL: row i's tokens are 0 .. lengths[i]-1 (clamped to
 *     0 .. L). What the tensors hold behind them is not read; outputs and
 *     gradients there are written as 0, and the final state is the one after the
 *     last token (h0 for a length of 0)
 * bf16 inputs run on the bf16 matrix cores with what is computed in between
 * (states, weighted values, scores) split into three bf16 parts, which hold all
 * 24 bits of an fp32 value: nothing is rounded to fewer before the output is; fp32 inputs run
 * on the fp32 matrix cores. States and sums are fp32. The masked products of a
 * chunk (64 tokens, 32 in fp32) include zeros times later tokens: an infinity or
 * NaN in a token reaches the outputs of its whole chunk.
 *
 * Conventions as in m3.h: dense row-major tensors, 16-byte aligned pointers, the
 * caller owns every buffer and the workspace (contents need not be initialised
 * and are not kept; calls that may overlap need workspaces of their own), the
 * stream is a hipStream_t of the current device passed as void*, all arguments
 * are checked on the host before any HIP call, nothing is allocated, freed or
 * synchronised, and every call can be captured into a graph. Outputs and
 * the workspace may not overlap inputs or each other, but for the step's state, and
 * h_final, which may be h0 itself (a pointer given twice, one of the two for something
 * that is written, is M3_ERR_INVALID_ARG). Results do not
 * depend on timing: the same call gives the same bits.
 */
#ifndef M3_LINATTN_H
#define M3_LINATTN_H

#include "m3.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void *q;          /* [b,L,H,N] io */
    const void *k;          /* [b,L,G,N] io */
    const void *v;          /* [b,L,G,P] io */
    const float *log_decay; /* [H] */
    const float *h0;        /* [b,H,P,N] initial state or NULL (zero) */
    const int32_t *lengths; /* [b] or NULL (all L) */
    void *y;                /* out [b,L,H,P] io (not read or written by the backward) */
    float *h_final;         /* out [b,H,P,N] or NULL (likewise) */
    float scale;            /* finite */
} m3_linattn_io;

/* Gradients of <dy, y> + <dh_final, h_final>. dq, dk, dv have the io dtype of
 * their inputs, the others are fp32; all are fully overwritten. */
typedef struct {
    const void *dy;         /* [b,L,H,P] io */
    const float *dh_final;  /* [b,H,P,N] or NULL (zero) */
    void *dq;               /* [b,L,H,N] io */
    void *dk;               /* [b,L,G,N] io: summed over the heads that share it, in fp32 */
    void *dv;               /* [b,L,G,P] io: likewise */
    float *dlog_decay;      /* [H] or NULL (not wanted: a constant decay) */
    float *dh0;             /* [b,H,P,N] or NULL (not wanted) */
} m3_linattn_grads;

typedef struct {
    const void *q;          /* [b,H,N] io */
    const void *k;          /* [b,G,N] io */
    const void *v;          /* [b,G,P] io */
    const float *log_decay; /* [H] */
    void *h;                /* in/out [b,H,P,N] state: fp32, or bf16 with M3_FLAG_BF16_STATE
                               (updated in fp32, stored rounded to nearest even; y is
                               formed before that rounding) */
    void *y;                /* out [b,H,P] io */
    float scale;            /* finite */
} m3_linattn_step_io;

/* Prompt: y for every token and the final state. shape->nsegments: 0 picks the
 * sequence split, 1 none, k > 1 about k segments per sequence (each segment's own
 * end state first, then the states chained, then the outputs). shape->flags = 0. */
m3_status m3_linattn_fwd(const m3_shape *shape, const m3_linattn_io *io, void *workspace, size_t ws_bytes,
                         void *stream);

/* Bytes of device workspace m3_linattn_fwd needs (0 if none, or for a refused shape). */
size_t m3_linattn_workspace_bytes(const m3_shape *shape);

/* Gradients of m3_linattn_fwd for the same shape and io. Each is a linear
 * attention itself: dq of (dy, v, k) forwards, dk of (v, dy, q) and dv of
 * (k, q, dy) backwards in time. */
m3_status m3_linattn_bwd(const m3_shape *shape, const m3_linattn_io *io, const m3_linattn_grads *grads,
                         void *workspace, size_t ws_bytes, void *stream);

/* Bytes of device workspace m3_linattn_bwd needs. */
size_t m3_linattn_bwd_workspace_bytes(const m3_shape *shape);

/* One token: the state is updated in place, y written. seqlen and nsegments are
 * not used; shape->flags: 0 or M3_FLAG_BF16_STATE. */
m3_status m3_linattn_step(const m3_shape *shape, const m3_linattn_step_io *io, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* M3_LINATTN_H */
