/*
 * m3_block_norm.h -- what stands between two blocks of a model, in one pass: the
 * norm behind a block, its gate and scale, the residual stream, and the norm
 * before the next block. Beside the group norm of m3_norm.h.
 *
 * For every row of `channels` values, x the block's output and r the residual stream:
 *   v = x / sqrt(mean(x^2) + eps) * post_weight[c]     (M3_BLOCK_POST_NORM, else v = x)
 *   R = residual_scale * r + scale[c] * act(z) * v     (no r: 0; no scale, no z: 1)
 *   y = R / sqrt(mean(R^2) + eps) * pre_weight[c]      (M3_BLOCK_PRE_NORM, else no y)
 * R is the stream behind the block, y the next block's input, formed from R before
 * R is rounded. m3_block_norm_bwd gives the gradients, from x, z and the stored R.
 *   x, z, y: io dtype. r, R: residual dtype, fp32 or that of x. Weights and scale
 *     [channels] fp32 or NULL (ones). Sums are fp32 within a row; those over rows
 *     fp32 for at most 256 rows, one after another, and fp64 beyond, held in fp32 once for
 *     every workgroup; each output is rounded once. A row of zeros with an eps of 0 gives NaN.
 * channels: 1 to 2^20; rows: up to 2^41 / max(channels, 64), up to 2^23 of over 8192 channels (more may be
 * M3_ERR_UNSUPPORTED). Rows of over 16384 channels (8192 with gradients) are read two or three times.
 *
 * Conventions as in m3.h: dense row-major tensors, 16-byte aligned pointers, the
 * caller owns every buffer and the workspace (contents need not be initialised
 * and are not kept; calls that may overlap need workspaces of their own), the
 * stream is a hipStream_t of the current device passed as void*, all arguments
 * are checked on the host before any HIP call, nothing is allocated, freed or
 * synchronised, and every call can be captured into a graph. The same call gives
 * the same bits. residual_out may be residual itself and y may be x or z; dx may be x or dy,
 * dz may be z, dresidual may be dresidual_out; no other overlap with what is written, the
 * workspace included (a pointer given twice otherwise is M3_ERR_INVALID_ARG).
 */
#ifndef M3_BLOCK_NORM_H
#define M3_BLOCK_NORM_H

#include "m3_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define M3_BLOCK_POST_NORM 1
#define M3_BLOCK_PRE_NORM 2

typedef struct {
    int64_t rows;           /* >= 0 */
    int64_t channels;       /* >= 1 */
    int32_t io_dtype;       /* m3_dtype of x, z, y, dy, dx, dz */
    int32_t residual_dtype; /* m3_dtype of r, R and their gradients: M3_F32 or io_dtype */
    int32_t activation;     /* m3_act of the gate: none, SiLU, sigmoid (not used without z) */
    float eps;              /* finite, >= 0 */
    float residual_scale;   /* finite */
    uint32_t flags;         /* M3_BLOCK_POST_NORM | M3_BLOCK_PRE_NORM */
} m3_block_norm_shape;

typedef struct {
    const void *x;            /* [rows,channels] io */
    const void *z;            /* the same, or NULL (no gate) */
    const void *residual;     /* [rows,channels] residual dtype, or NULL (0); not read by the backward */
    const float *post_weight; /* [channels] or NULL; NULL without M3_BLOCK_POST_NORM */
    const float *pre_weight;  /* [channels] or NULL; NULL without M3_BLOCK_PRE_NORM */
    const float *scale;       /* [channels] or NULL */
    void *residual_out;       /* [rows,channels] residual dtype: out of the forward (NULL with M3_BLOCK_PRE_NORM: not wanted),
                                 input of the backward */
    void *y;                  /* out [rows,channels] io: required with M3_BLOCK_PRE_NORM, else NULL (not used by the backward) */
} m3_block_norm_io;

/* Gradients of <dy, y> + <dresidual_out, R>. */
typedef struct {
    const void *dy;            /* [rows,channels] io: required with M3_BLOCK_PRE_NORM, else NULL */
    const void *dresidual_out; /* [rows,channels] residual dtype, or NULL (0); required without M3_BLOCK_PRE_NORM */
    void *dx;                  /* out, io */
    void *dz;                  /* out, io: required with a gate, else NULL */
    void *dresidual;           /* out, residual dtype, or NULL (not wanted) */
    float *dpost_weight;       /* out [channels] or NULL (not wanted) */
    float *dpre_weight;        /* likewise */
    float *dscale;             /* likewise */
} m3_block_norm_grads;

m3_status m3_block_norm_fwd(const m3_block_norm_shape *shape, const m3_block_norm_io *io, void *stream);

/* dpost_weight and dpre_weight need their norms. */
m3_status m3_block_norm_bwd(const m3_block_norm_shape *shape, const m3_block_norm_io *io,
                            const m3_block_norm_grads *grads, void *workspace, size_t ws_bytes, void *stream);
/* Bytes of device workspace m3_block_norm_bwd needs (0 for a refused shape); without a weight's gradient
 * it needs none up to 8192 channels. */
size_t m3_block_norm_bwd_workspace_bytes(const m3_block_norm_shape *shape);

#ifdef __cplusplus
}
#endif
#endif /* M3_BLOCK_NORM_H */
