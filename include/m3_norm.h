/*
 * m3_norm.h -- C ABI of libm3.so, third part: the joint between two blocks of a
 * hybrid stack on AMD MI355X (gfx950). A block's output is normed, gated, scaled
 * and added to the residual stream, and the stream's norm is the next block's
 * input: one pass over the rows, forward and backward.
 *
 * Conventions, ownership, streams and errors are those of m3.h: caller-owned
 * device buffers, no allocation, every argument checked before any HIP call,
 * asynchronous on `stream`, nothing throws.
 */
#ifndef M3_NORM_H
#define M3_NORM_H

#include "m3.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The gate's function a(g): g, g sigmoid(g), sigmoid(g). */
typedef enum m3_gate_fn { M3_GATE_IDENTITY = 0, M3_GATE_SILU = 1, M3_GATE_SIGMOID = 2 } m3_gate_fn;

/* Rows of tokens: row t at p + t * stride (elements), its `width` entries contiguous. */
typedef struct m3_lines {
    void* p;
    int64_t stride;
} m3_lines;

/*
 * With N(v; w) = v * w / sqrt(mean of v^2 over the row + eps):
 *   b = factor * scale * a(gate) * N(o; post_weight)     (without post_weight: o itself)
 *   h = x + b
 *   y = N(h; weight)
 * x and h are the residual stream, in stream_dtype; o, gate and y in io_dtype (of an fp32
 * stream bf16 or fp32, of a bf16 stream bf16). Vectors are fp32 [width]. All arithmetic is
 * fp32, y from h before its rounding; each output is rounded once. Sums of squares are
 * fp32: entries of h and of a normed o up to 2^60, whole rows of them too (beside an eps of 0 rows of
 * root mean square 2^-48 at least).
 */
typedef struct m3_joint {
    int64_t tokens;           /* rows, >= 0 */
    int32_t width;            /* 1 .. 8192 */
    int32_t stream_dtype;     /* m3_dtype */
    int32_t io_dtype;         /* m3_dtype */
    int32_t gate_fn;          /* m3_gate_fn, where a gate is given */
    float eps;                /* >= 0 */
    float factor;             /* finite; 1 without a fixed scale */
    const float* scale;       /* NULL: 1 */
    const float* post_weight; /* NULL: o is not normed */
    const float* weight;      /* NULL: there is no y */
} m3_joint;

/*
 * m3_residual_norm -- x, o, gate -> h, y.
 * o NULL: no branch (no gate, no h; scale, post_weight unused): y = N(x; weight). gate
 * NULL: 1. y is given exactly with weight, h exactly with o. h may be x itself and y may be o itself (or
 * x, without o), same strides and types; other overlaps are refused.
 */
m3_status m3_residual_norm(const m3_joint* joint, const m3_lines* x, const m3_lines* o, const m3_lines* gate,
                           const m3_lines* h, const m3_lines* y, void* stream);

/*
 * m3_residual_norm_backward -- the gradients at stream h (as stored), o, gate, from dh (NULL: 0)
 * and dy (given exactly with weight; one of the two is needed):
 *   dx = dh + (dN/dh)^T dy                                   stream_dtype
 *   d_o, d_gate = the gradients of <dx, b>                    io_dtype
 *   d_weight, d_post_weight, d_scale [width] = sums over the rows, fp32, in a fixed order (the same
 *   call gives the same bits); of no rows: 0
 * Any output may be NULL (one is needed); those of parts that are not given must be. dx is
 * not rounded before the branch's gradients are formed. dx may be dh itself; other overlaps
 * are refused.
 * workspace: m3_residual_norm_backward_workspace_size() bytes, 16-byte aligned (NULL when 0).
 */
m3_status m3_residual_norm_backward(const m3_joint* joint, const m3_lines* dh, const m3_lines* dy, const m3_lines* h,
                                    const m3_lines* o, const m3_lines* gate, const m3_lines* dx, const m3_lines* d_o,
                                    const m3_lines* d_gate, float* d_weight, float* d_post_weight, float* d_scale,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes that m3_residual_norm_backward needs where any of the three sums is asked for, else 0 (0 on
 * invalid sizes). Host only. */
size_t m3_residual_norm_backward_workspace_size(const m3_joint* joint, int32_t sums);

#ifdef __cplusplus
}
#endif
#endif /* M3_NORM_H */
