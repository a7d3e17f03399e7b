/*
 * zero_train.h -- training operators around the ZeRO optimizer step, on one
 * GPU (sm_103a).  Same library and conventions as zero.h: the caller owns all
 * memory, every call checks its arguments on the host and launches nothing if
 * they are invalid, work is asynchronous on `stream`, no exception crosses the
 * ABI, and no call allocates or keeps anything between calls.
 *
 * The optimizer step of zero.h reads 16-bit gradient rows and writes 16-bit
 * parameters.  The operators here read those parameters in the forward pass,
 * keep activations for the backward pass in 8 bits (the residual memory that
 * "ZeRO-R" is about) and write parameter gradients straight into a
 * contribution row (zero_grads_t):
 *   - the embedding lookup, and its gradient by sorted tokens;
 *   - the residual addition with the root-mean-square norm, whose backward
 *     pass reads an 8-bit checkpoint of the normalised rows;
 *   - 8-bit activation checkpoints of any matrix, and the weight gradient of a
 *     linear layer taken from one.
 * A matrix that crosses the end of a shard can be written into a row only where
 * the row's shards lie end to end: row_pitch equal to shard_elems (pad the flat
 * buffer until a shard is a multiple of row_align_elems).  Otherwise its gradient
 * needs a buffer of its own, to be copied into the row shard by shard.
 *
 * Conventions of this header:
 *   - All pointers of device data must be device (or managed) memory
 *     (ZERO_ERR_INVALID_ARG otherwise) that the current device can reach.
 *   - Arithmetic is in fp32 (products of 16-bit values on the tensor cores
 *     with fp32 sums); each 16-bit result is rounded once, to nearest even.
 *   - Every result is the same, bit for bit, in every run of the same call on
 *     the same device: no atomic operation decides an order of summation.
 *   - A parameter gradient is either stored (accumulate = 0) or added onto
 *     what its buffer holds (accumulate = 1: read, added in fp32, rounded),
 *     as over micro-batches or for a table shared with the output layer.
 *   - A call without rows (tokens) is legal: it writes no activation, and a
 *     stored parameter gradient is zero.
 *   - Outputs must not overlap inputs or each other, except where stated.
 *   - Workspaces: device memory of at least the size that the operator's
 *     ..._workspace function gives, 16-byte aligned, overwritten; calls that
 *     may run at the same time need workspaces of their own.
 *   - Work is programmatic dependent launches as in zero.h (ZERO_PDL).
 *   - stream NULL is the legacy default stream, as in zero.h.  It orders nothing
 *     with a non-blocking stream, such as another library's current one: pass
 *     the stream on which the inputs are made and the outputs are used.
 */
#ifndef ZERO_TRAIN_H
#define ZERO_TRAIN_H

#include "zero.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A row-major matrix of 16-bit elements: element (r, c) is base[r*pitch + c],
 * pitch >= cols.  Activations: base 16-byte aligned and pitch a multiple of 8
 * (ZERO_ERR_ALIGNMENT otherwise).  Parameters and their gradients lie anywhere
 * in a flat buffer: base 2-byte aligned, any pitch; they move faster where
 * base is 16-byte aligned and pitch a multiple of 8. */
typedef struct zero_mat {
    void* base;
    uint64_t rows;
    uint64_t cols;
    uint64_t pitch;    /* elements between the starts of consecutive rows */
    int32_t dtype;     /* zero_dtype_t */
} zero_mat_t;

/* Token numbers: `count` signed integers of `bytes` (4 or 8) bytes each, on a
 * boundary of their size, device memory.  A negative number is padding.  A
 * number >= the table's rows is treated as padding too and sets the call's
 * flag word. */
typedef struct zero_ids {
    const void* ids;
    uint64_t count;
    uint32_t bytes;
} zero_ids_t;

/* An 8-bit checkpoint of a [rows, cols] matrix.  Every block of
 * ZERO_ACT8_BLOCK consecutive elements of a row (the last block of a row may
 * be shorter) shares one scale byte s; its elements q stand for q * 2^(s-127).
 *   q      int8 [rows][q_pitch], 16-byte aligned, q_pitch >= cols a multiple of 16;
 *   scale  uint8 [rows][scale_pitch], scale_pitch >= ceil(cols / 32).
 * Writing a block with a = max |x|: k = s - 127 is the smallest integer with
 * a <= 127 * 2^k, kept within [-24, 9] (binary16 activations) or [-127, 121]
 * (bfloat16); q = x / 2^k rounded to nearest even, kept within [-127, 127].
 * Within those limits every value that a checkpoint stands for is finite and
 * exact in the activations' type, so reading one back rounds nothing.  A block
 * that holds an inf or NaN gets s = 255 and q = 0 and stands for NaN, so a
 * gradient computed from it is nonfinite and the optimizer step is skipped.
 * The elements of q between cols and q_pitch are neither read nor written. */
#define ZERO_ACT8_BLOCK 32u
typedef struct zero_act8 {
    int8_t* q;
    uint8_t* scale;
    uint64_t rows;
    uint64_t cols;
    uint64_t q_pitch;
    uint64_t scale_pitch;
} zero_act8_t;

/* ---- Embedding --------------------------------------------------------------- */

/* out[t] = scale * table[ids[t]] for every token t; a padding token's row is
 * zero.  table: a parameter matrix [vocab, dim] (a view into the gathered
 * buffer); out: an activation matrix [ids->count, dim] of the same type.
 * scale: finite.  *d_bad |= 1 if a number >= vocab was met (d_bad may be
 * NULL).  At most 2^31 - 1 tokens and table rows (ZERO_ERR_UNSUPPORTED).  A table
 * without columns is legal: the call does nothing then, and looks at no number. */
zero_status_t zero_embed_lookup(const zero_mat_t* table, const zero_ids_t* ids, float scale,
                                const zero_mat_t* out, uint32_t* d_bad, void* stream);

/* The lookup's gradient: d_table[v] = scale * sum of d_out[t] over the tokens
 * with ids[t] == v, in fp32 and in an order fixed by the ids alone, for every
 * row v of the table: rows of absent tokens are stored as zero
 * (accumulate = 0) or left untouched (accumulate = 1).  d_out: an activation
 * matrix [ids->count, dim]; d_table: a parameter gradient [vocab, dim] of the
 * same type.  The tokens are sorted by number within the call.  A table without
 * rows or columns is legal: the call does nothing then, and looks at no number. */
uint64_t zero_embed_grad_workspace(uint64_t tokens, uint64_t vocab, uint64_t dim);
zero_status_t zero_embed_grad(const zero_mat_t* d_out, const zero_ids_t* ids, float scale,
                              uint32_t accumulate, const zero_mat_t* d_table, void* workspace,
                              uint64_t workspace_bytes, uint32_t* d_bad, void* stream);

/* ---- Residual addition and root-mean-square norm -------------------------------- */

/* Most columns of a row that the norm accepts (ZERO_ERR_UNSUPPORTED above). */
#define ZERO_NORM_MAX_COLS 32768u

/* For every row:  s = x + residual (fp32; residual may be NULL);
 *     rstd = 1 / sqrt(mean(s^2) + eps);  xhat = s * rstd;
 *     h = s,  y = xhat * gain,  checkpoint = xhat in 8 bits.
 * x, residual, h, y: activation matrices of one shape and type; h and y may be
 * NULL (not wanted) and h may be x or residual itself (same base and pitch).
 * gain: 16-bit[cols] of that type, 2-byte aligned, or NULL for ones.
 * rstd: fp32[rows] or NULL.  checkpoint: [rows, cols] or NULL (serving).  At
 * least one output is needed.  eps > 0 and finite.  The norm is taken of the
 * unrounded sum s; its mean of squares is an fp32 sum. */
zero_status_t zero_norm_forward(const zero_mat_t* x, const zero_mat_t* residual,
                                const void* gain, float eps, const zero_mat_t* h,
                                const zero_mat_t* y, float* rstd, const zero_act8_t* checkpoint,
                                void* stream);

/* Backward of the above at the checkpoint's xhat:  u = gain * dy;
 *     dx = d_residual + rstd * (u - xhat * mean(u * xhat))
 *     d_gain = sum over rows of dy * xhat
 * dx is the gradient of s, so of x and of the residual alike.  d_residual, the
 * gradient that reaches h from the layers behind it, may be NULL; dx may be dy
 * or d_residual itself (same base and pitch).  d_gain: 16-bit[cols], 2-byte
 * aligned, stored or added; NULL if not wanted. */
uint64_t zero_norm_backward_workspace(uint64_t rows, uint64_t cols);
zero_status_t zero_norm_backward(const zero_mat_t* dy, const zero_act8_t* checkpoint,
                                 const float* rstd, const void* gain,
                                 const zero_mat_t* d_residual, const zero_mat_t* dx,
                                 void* d_gain, uint32_t accumulate, void* workspace,
                                 uint64_t workspace_bytes, void* stream);

/* ---- 8-bit activation checkpoints ------------------------------------------------ */

/* Writes the checkpoint of an activation matrix (same rows and cols). */
zero_status_t zero_act_pack(const zero_mat_t* x, const zero_act8_t* out, void* stream);

/* Reads a checkpoint back: out = the values it stands for, rounded to out's
 * type (exact for the type that it was written from). */
zero_status_t zero_act_unpack(const zero_act8_t* in, const zero_mat_t* out, void* stream);

/* Weight gradient of a linear layer y = X W^T whose input X = gain * xhat was
 * kept as the checkpoint of xhat:
 *     dw[o][i] = gain[i] * sum over tokens t of dy[t][o] * xhat[t][i].
 * dy: an activation matrix [tokens, outs]; x: the checkpoint [tokens, ins],
 * whose values are taken in dy's type; gain: 16-bit[ins] or NULL for ones (a
 * checkpoint that zero_act_pack wrote); dw: a parameter gradient [outs, ins]
 * of dy's type.  At most 2^30 tokens, 2^28 outs and ins (ZERO_ERR_UNSUPPORTED);
 * element offsets may pass 2^32.  The kernel's waits on its own copies and
 * products are bounded (4 s each, and 1 s for those still under way when it ends);
 * should one ever run out, the part of dw not finished is NaN, so that the
 * optimizer step skips the gradient. */
uint64_t zero_act_weight_grad_workspace(uint64_t tokens, uint64_t outs, uint64_t ins);
zero_status_t zero_act_weight_grad(const zero_mat_t* dy, const zero_act8_t* x, const void* gain,
                                   uint32_t accumulate, const zero_mat_t* dw, void* workspace,
                                   uint64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_TRAIN_H */
