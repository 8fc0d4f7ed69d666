/*
 * m3_norm.h -- group norm with an activation, channels last, beside the mixer
 * core of m3.h: the norm of every token's heads that follows a linear attention,
 * with its gate, or of a sequence as a whole.
 *
 * x is [rows, positions, channels], channels in `groups` equal groups. A group's mean
 * and variance are taken over its channels at all positions of a row:
 *   u = (x - mean) / sqrt(var + eps) * weight[c] + bias[c]     (var of the population)
 *   y = act(u), or u * act(z) where a gate z [rows, positions, channels] is given
 * With positions = 1 every row is a token by itself (rows = batch * length): no token
 * sees another, as a causal model needs. With positions = length a row is a sequence.
 *   lengths [rows] int32 or NULL: row i has lengths[i] positions (clamped to 0 ..
 *     positions). What lies behind them is not read into any result, and the
 *     outputs and gradients there are written as 0.
 *   weight, bias [channels] fp32 or NULL (ones, zeros). x, z, y: io dtype. Statistics and
 * sums are fp32 for at most 256 rows or positions, one after another, and fp64 beyond; each
 * output is rounded once.
 *
 * Conventions as in m3.h: dense row-major tensors, 16-byte aligned pointers, the
 * caller owns every buffer and the workspace (contents need not be initialised
 * and are not kept; calls that may overlap need workspaces of their own), the
 * stream is a hipStream_t of the current device passed as void*, all arguments
 * are checked on the host before any HIP call, nothing is allocated, freed or
 * synchronised, and every call can be captured into a graph. The same call gives
 * the same bits. y may be x or z itself, dx may be x or dy, dz may be z; no other overlap
 * with what is written, the workspace included (a pointer given twice otherwise is
 * M3_ERR_INVALID_ARG).
 */
#ifndef M3_NORM_H
#define M3_NORM_H

#include "m3.h"

#ifdef __cplusplus
extern "C" {
#endif

/* (the sigmoid is for the gate of m3_block_norm.h alone) */
typedef enum { M3_ACT_NONE = 0, M3_ACT_SILU = 1, M3_ACT_SIGMOID = 2 } m3_act;

typedef struct {
    int64_t rows;       /* >= 0 */
    int64_t positions;  /* >= 0 */
    int64_t channels;   /* >= 1, up to 2^20 */
    int64_t groups;     /* >= 1, divides channels */
    int32_t io_dtype;   /* m3_dtype of x, z, y, dy, dx, dz */
    int32_t activation; /* m3_act */
    float eps;          /* finite, >= 0 */
    uint32_t flags;     /* 0 */
} m3_norm_shape;

typedef struct {
    const void *x;          /* [rows,positions,channels] io */
    const void *z;          /* the same, or NULL (no gate) */
    const float *weight;    /* [channels] or NULL */
    const float *bias;      /* [channels] or NULL */
    const int32_t *lengths; /* [rows] or NULL */
    void *y;                /* out [rows,positions,channels] io (not used by the backward) */
} m3_norm_io;

typedef struct {
    const void *dy; /* [rows,positions,channels] io */
    void *dx;       /* out, io */
    void *dz;       /* out, io: required with a gate, else NULL */
    float *dweight; /* out [channels] or NULL (not wanted) */
    float *dbias;   /* out [channels] or NULL (not wanted) */
} m3_norm_grads;

m3_status m3_group_norm_fwd(const m3_norm_shape *shape, const m3_norm_io *io, void *workspace, size_t ws_bytes,
                            void *stream);
/* Bytes of device workspace m3_group_norm_fwd needs (0 if none, or for a refused
 * shape); lengths: whether the call passes them. */
size_t m3_group_norm_workspace_bytes(const m3_norm_shape *shape, int lengths);

/* Gradients of <dy, y>; the statistics are formed again from x. */
m3_status m3_group_norm_bwd(const m3_norm_shape *shape, const m3_norm_io *io, const m3_norm_grads *grads,
                            void *workspace, size_t ws_bytes, void *stream);
size_t m3_group_norm_bwd_workspace_bytes(const m3_norm_shape *shape, int lengths);

#ifdef __cplusplus
}
#endif
#endif /* M3_NORM_H */
