/*
 * m3_recurrence.h -- gated linear recurrence, one state a channel, beside the
 * Mamba-3 mixer core of m3.h and the linear attention of m3_linattn.h.
 *
 * For every batch row and channel c, with s = sigmoid(decay_gate_t) and
 * g = sigmoid(input_gate_t) (1 without an input gate):
 *
 *   a_t = exp(log_decay[c] * s)
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) g x_t      (h_{-1} = h0 or 0)
 *   y_t = h_t
 *
 * With M3_REC_UNSCALED the factor sqrt(1 - a_t^2) is 1. m3_recurrence_fwd evaluates
 * a prompt (in tiles of 128 tokens, each joined to those before it by their decays
 * and end states), m3_recurrence_bwd gives the gradients, m3_recurrence_step advances one token.
 *
 *   x, decay_gate, input_gate, y [b,L,C]   io dtype
 *   log_decay [C] fp32: finite and <= 0
 *   h0, h_final [b,C] fp32
 *   lengths [b] int32 or NULL: row i's tokens are 0 .. lengths[i]-1 (clamped to
 *     0 .. L). What the tensors hold behind them is not read; outputs and
 *     gradients there are written as 0, and the final state is the one after the
 *     last token (h0 for a length of 0)
 *   states [b, ceil(L / M3_REC_KEEP), C] fp32: the state before every token whose
 *     index is a multiple of M3_REC_KEEP (behind a row's length: the last one). The
 *     forward writes it where it is given; the backward then need not run the
 *     recurrence over the sequence again first.
 * C: 1 to 2^20; even C load fastest in bf16. b * L <= 2^40, and b times the tiles of 64
 * channels times those of 64 tokens below 2^23 (else M3_ERR_UNSUPPORTED). States, gates and sums are fp32,
 * sums over tokens and rows fp64 beyond 8 terms, held in fp32 once for every 64 tokens; each output is rounded once. 1 - a_t
 * is formed without cancellation, so slow decays keep their input. Where
 * 1 - a_t^2 is 0 (a log_decay of 0), an input has no effect and no gradient.
 *
 * Conventions as in m3.h: dense row-major tensors, 16-byte aligned pointers, the
 * caller owns every buffer and the workspace (contents need not be initialised
 * and are not kept; calls that may overlap need workspaces of their own), the
 * stream is a hipStream_t of the current device passed as void*, all arguments
 * are checked on the host before any HIP call, nothing is allocated, freed or
 * synchronised, and every call can be captured into a graph. Outputs and the
 * workspace may not overlap inputs or each other, but for h_final, which may be h0
 * itself, and dh0, which may be dh_final (a pointer given twice otherwise, one of the
 * two for something that is written, is M3_ERR_INVALID_ARG). The same call gives the
 * same bits.
 */
#ifndef M3_RECURRENCE_H
#define M3_RECURRENCE_H

#include "m3.h"

#ifdef __cplusplus
extern "C" {
#endif

#define M3_REC_KEEP 64    /* tokens between two kept states */
#define M3_REC_UNSCALED 1 /* flags: no factor sqrt(1 - a^2) */

typedef struct {
    int64_t batch;     /* >= 0 */
    int64_t seqlen;    /* >= 0 */
    int64_t channels;  /* >= 1, up to 2^20 */
    int32_t io_dtype;  /* m3_dtype of x, gates, y and their gradients */
    uint32_t flags;    /* 0 or M3_REC_UNSCALED */
} m3_rec_shape;

typedef struct {
    const void *x;          /* [b,L,C] io */
    const void *decay_gate; /* [b,L,C] io */
    const void *input_gate; /* [b,L,C] io or NULL */
    const float *log_decay; /* [C] */
    const float *h0;        /* [b,C] initial state or NULL (zero); not read by a backward with states */
    const int32_t *lengths; /* [b] or NULL (all L) */
    void *y;                /* out [b,L,C] io (not read or written by the backward) */
    float *h_final;         /* out [b,C] or NULL (likewise) */
    float *states;          /* [b,ceil(L/M3_REC_KEEP),C] or NULL: out of the forward, input of the backward */
} m3_rec_io;

/* Gradients of <dy, y> + <dh_final, h_final>. */
typedef struct {
    const void *dy;        /* [b,L,C] io */
    const float *dh_final; /* [b,C] or NULL (zero) */
    void *dx;              /* out [b,L,C] io */
    void *ddecay_gate;     /* out [b,L,C] io */
    void *dinput_gate;     /* out [b,L,C] io: required with an input gate, else NULL */
    float *dlog_decay;     /* out [C] or NULL (not wanted) */
    float *dh0;            /* out [b,C] or NULL (not wanted) */
} m3_rec_grads;

typedef struct {
    const void *x;          /* [b,C] io */
    const void *decay_gate; /* [b,C] io */
    const void *input_gate; /* [b,C] io or NULL */
    const float *log_decay; /* [C] */
    float *h;               /* in/out [b,C] */
    void *y;                /* out [b,C] io */
} m3_rec_step_io;

m3_status m3_recurrence_fwd(const m3_rec_shape *shape, const m3_rec_io *io, void *workspace, size_t ws_bytes,
                            void *stream);
/* Bytes of device workspace m3_recurrence_fwd needs (0 if none, or for a refused shape). */
size_t m3_recurrence_workspace_bytes(const m3_rec_shape *shape);

m3_status m3_recurrence_bwd(const m3_rec_shape *shape, const m3_rec_io *io, const m3_rec_grads *grads, void *workspace,
                            size_t ws_bytes, void *stream);
/* Likewise of m3_recurrence_bwd; states: whether the call passes them. */
size_t m3_recurrence_bwd_workspace_bytes(const m3_rec_shape *shape, int states);

/* One token: the state is updated in place, y written. seqlen is not used. */
m3_status m3_recurrence_step(const m3_rec_shape *shape, const m3_rec_step_io *io, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* M3_RECURRENCE_H */
