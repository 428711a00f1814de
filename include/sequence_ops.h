/*
 * sequence_ops.h -- C ABI of the sequence operators of the MI355X (gfx950)
 * library: the causal convolution and the selective scan of a gated state
 * space block, and block-scaled fp8 matrix products.
 *
 * Conventions (as conv2d_nhwc.h where not stated otherwise):
 *   - The caller owns every buffer; the library allocates nothing.  Work is
 *     enqueued on `stream` (a hipStream_t, NULL = the null stream).
 *   - Status codes are those of conv2d_nhwc.h; every check runs before anything
 *     is enqueued, and on error no output byte is written.
 *     Sizes whose launches the device cannot take (2^32 threads along an axis:
 *     2^26 chunks of 16 channels of a scan, 2^32 values of dB, 2^28 blocks of
 *     an fp8 operand) are CONV2D_ERR_UNSUPPORTED among those checks.
 *   - Results are the same bits on every run: no atomics on values, every
 *     reduction in a fixed order.  Sums, states and gradients' partial sums
 *     are fp32 (of fp8 products see there); each output is rounded once, to
 *     nearest even.
 *   - Buffers need the alignment of their elements only, unless stated.
 *   - "rows" are tokens.  A tensor of rows has unit stride over its last
 *     axis; its strides between rows and between sequences are in elements.
 *   - Value pointers may be NULL only where stated.
 */
#ifndef SEQUENCE_OPS_H
#define SEQUENCE_OPS_H

#include <stddef.h>

#include "conv2d_nhwc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of the sequence operators beside CONV2D_DTYPE_F16 and _BF16. */
#define CONV2D_DTYPE_F32 3

/*
 * The sequences of a batch.  With seq_start NULL they are a dense batch
 * [seqs][len]; otherwise they lie packed, sequence s in rows
 * seq_start[s] .. seq_start[s+1]-1 of `tokens` rows (0 = first, tokens = last
 * value, not descending; empty sequences allowed).  seq_start is read on the
 * device: values outside 0..tokens are clamped, never followed.  Results of rows
 * that no sequence covers are unspecified, and all of them where starts descend.
 */
typedef struct seq_batch {
    const int *seq_start; /* device, [seqs + 1], or NULL */
    int seqs;             /* >= 1 */
    int len;              /* >= 0; dense batches only */
    long long tokens;     /* rows in all: seqs * len when dense; < 2^31 */
} seq_batch_t;

/* Strides of a tensor of rows, in elements; seq is read for dense batches only. */
typedef struct seq_stride {
    long long row, seq;
} seq_stride_t;

/*
 * Causal depthwise convolution over tokens, with bias and SiLU fused:
 *   pre[t][c] = bias[c] + sum_{k < w} weight[c][k] * x[t - (w-1) + k][c]
 *   y = pre * sigmoid(pre) if silu, else pre
 * where rows before a sequence's first are its initial_state [w-1][d] (oldest
 * first), or zero without one.
 *   x        rows of d elements, dtype, strides `x`
 *   weight   [d][w], bias [d] (NULL = zero); dtype
 *   initial_state, final_state  [seqs][w-1][d], dtype, or NULL.  final_state
 *            receives the last w-1 rows each sequence has seen.  They must not overlap.
 *   y        [tokens][d] dense, dtype; must not overlap x
 * dtype: CONV2D_DTYPE_F16, _BF16 or _F32; 2 <= w <= 4.
 */
typedef struct causal_conv_problem {
    seq_batch_t batch;
    int d, w;
    int silu; /* 0 or 1 */
    seq_stride_t x, dy;
} causal_conv_problem_t;

int causal_conv(const causal_conv_problem_t *prob, int dtype, const void *x, const void *weight,
                const void *bias, const void *initial_state, void *y, void *final_state, void *stream);

/*
 * Gradients of causal_conv for the output gradient dy (strides `dy`) and, if
 * given, that of final_state.
 *   dx [tokens][d]; dweight [d][w]; dbias [d] (NULL if not wanted);
 *   dinitial [seqs][w-1][d] (NULL if not wanted); all dtype, dense, overwritten.
 * The workspace (causal_conv_grad_workspace_size) holds fp32 partial sums of
 * dweight and dbias over runs of rows; it must be 16-byte aligned.
 */
int causal_conv_grad_workspace_size(const causal_conv_problem_t *prob, int dtype, size_t *bytes);
int causal_conv_grad(const causal_conv_problem_t *prob, int dtype, const void *dy, const void *x,
                     const void *weight, const void *bias, const void *initial_state,
                     const void *dfinal, void *dx, void *dweight, void *dbias, void *dinitial,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * causal_conv for one new token per request, on states that live in a pool:
 *   state [pool][w-1][d], dtype, updated in place; row r uses state slots[r]
 *   (int32, device; NULL = r).  Rows whose slot is outside 0..pool-1 (padding)
 *   give y = 0 and touch no state; no slot may appear twice.
 *   x [rows][d] with row stride x_row; y [rows][d] dense.
 */
typedef struct causal_conv_step_problem {
    int rows, pool;
    int d, w;
    int silu;
    long long x_row;
} causal_conv_step_problem_t;

int causal_conv_step(const causal_conv_step_problem_t *prob, int dtype, const void *x, void *state,
                     const void *weight, const void *bias, const int *slots, void *y, void *stream);

/*
 * Selective scan of a gated state space block, for channel c of group
 * g(c) = c / (d / groups) and state n:
 *   delta[t][c] = softplus(dt[t][c] + dt_bias[c])   (without softplus: the sum itself)
 *   h[t][c][n]  = exp(delta[t][c] * A[c][n]) * h[t-1][c][n] + delta[t][c] * x[t][c] * B[t][g][n]
 *   y[t][c]     = (sum_n h[t][c][n] * C[t][g][n] + D[c] * x[t][c]) * silu(z[t][c])
 * with h before a sequence's first token its initial_state, or zero without one.
 *   x, dt, z  rows of d elements; B, C rows of [groups][n] elements; dtype, with
 *             the strides below (b_group, c_group: between groups).  z may be NULL
 *             (no gate).
 *   A [d][n], D [d] (may be NULL: zero), dt_bias [d] (may be NULL: zero),
 *   initial_state and final_state [seqs][d][n] (may be NULL): fp32, dense.  The
 *             states must not overlap.
 *   y [tokens][d] dense, dtype; must not overlap the inputs.
 * Rates of A past 2e38 in size, infinite ones among them, count as 2e38: their
 * decays are 0 where delta > 0 and 1 where delta = 0.  Decays are also multiplied
 * over runs of tokens before they meet a state: for growing states (delta * A > 0)
 * results are NaN where such a product is infinite and the state is 0.
 * 1 <= n <= 64; groups divides d.  Row strides and d are below 2^24.
 * Long sequences are cut into chunks that run side by side, joined through the
 * workspace (selective_scan_workspace_size; 16-byte aligned; the size may be 0).
 */
typedef struct selective_scan_problem {
    seq_batch_t batch;
    int d, n, groups;
    int softplus; /* 0 or 1 */
    seq_stride_t x, dt, B, C, z, dy;
    long long b_group, c_group;
} selective_scan_problem_t;

int selective_scan_workspace_size(const selective_scan_problem_t *prob, int dtype, size_t *bytes);
int selective_scan(const selective_scan_problem_t *prob, int dtype, const void *x, const void *dt,
                   const float *A, const void *B, const void *C, const float *D, const void *z,
                   const float *dt_bias, const float *initial_state, void *y, float *final_state,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gradients of selective_scan for the output gradient dy (strides `dy`) and, if
 * given, that of final_state.  The forward pass's states are computed again.
 *   du, ddt, dz [tokens][d] (the gradients of x, dt and z; dz only with z) and
 *   dB, dC [tokens][groups][n]: dtype, dense; dA [d][n], dD [d] (NULL if not
 *   wanted), ddt_bias [d] (likewise), dinitial [seqs][d][n] (likewise): fp32.
 * All are overwritten; nothing may overlap an input.
 */
typedef struct selective_scan_grads {
    void *du, *ddt;
    float *dA;
    void *dB, *dC;
    float *dD;
    void *dz;
    float *ddt_bias, *dinitial;
} selective_scan_grads_t;

int selective_scan_grad_workspace_size(const selective_scan_problem_t *prob, int dtype, size_t *bytes);
int selective_scan_grad(const selective_scan_problem_t *prob, int dtype, const void *dy, const void *x,
                        const void *dt, const float *A, const void *B, const void *C, const float *D,
                        const void *z, const float *dt_bias, const float *initial_state,
                        const float *dfinal, const selective_scan_grads_t *grads, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * selective_scan for one new token per request, on fp32 states [pool][d][n]
 * updated in place; slots as for causal_conv_step.  The tensors' rows are
 * requests, with the strides given.
 */
typedef struct selective_scan_step_problem {
    int rows, pool;
    int d, n, groups;
    int softplus;
    long long x_row, dt_row, b_row, c_row, z_row, b_group, c_group;
} selective_scan_step_problem_t;

int selective_scan_step(const selective_scan_step_problem_t *prob, int dtype, const void *x, const void *dt,
                        const float *A, const void *B, const void *C, const float *D, const void *z,
                        const float *dt_bias, float *state, const int *slots, void *y, void *stream);

/*
 * Block-scaled fp8 products.  An fp8 operand is a matrix of e4m3 bytes (OCP
 * e4m3fn: 448 is the largest, no infinities) with an fp32 scale for every 128
 * values along the summed axis: of one row each, or (weights) of 128 rows
 * together.  Value [r][k] stands for q[r][k] * scale[r or r / 128][k / 128].
 *
 * fp8_quantize: x [m][k] (dtype, row stride x_row, in elements) to such an
 * operand.  The scale is the least power of two, at least 2^-126, that brings
 * the finite values of its block into e4m3's range, so that it costs no
 * accuracy; infinities and NaN become NaN and leave the others as they are.
 *   FP8_ROWS       q [m][q_pitch], scale [m][ceil(k/128)]
 *   FP8_TRANSPOSE  the operand is x's transpose: q [k][q_pitch], scale [k][ceil(m/128)]
 *   FP8_BLOCKS     q [m][q_pitch], scale [ceil(m/128)][ceil(k/128)]
 * q_pitch is a multiple of 16 and at least the operand's row length, less than
 * its whole blocks of 128 more; q is 16-byte aligned.  Bytes past a row's end
 * are set to zero.
 */
#define FP8_ROWS 0
#define FP8_TRANSPOSE 1
#define FP8_BLOCKS 2
int fp8_quantize(int form, int dtype, int m, int k, const void *x, long long x_row, void *q,
                 long long q_pitch, float *scale, void *stream);

/*
 * out[i][j] = sum_k a[i][k] a_scale[i][k/128] * b[j][k] b_scale[j or j/128][k/128],
 * rounded once to dtype (CONV2D_DTYPE_F16, _BF16 or _F32).
 * dtype _F32: products are exact and summed in fp32.  16-bit dtypes use the fp8
 * matrix unit at twice the rate, which cuts each of 8 neighbouring products of a
 * block at 2^-13 of the largest's power of two before it adds them; sums of such
 * groups, of blocks and of parts of k are fp32.  In norm the cut is 1.5e-5 of a
 * block's sum, below the result's own rounding (1.7e-3 bf16, 2e-4 fp16): on
 * normal data 1.5 of a hundred bf16 results, and 8 of fp16, round to a neighbour
 * of what fp32 sums give.  A 16-bit result of exact products is the _F32 one,
 * rounded.
 *   a [m][k] with pitch a_pitch, a_scale [m][ceil(k/128)]
 *   b [n][k] with pitch b_pitch, b_scale [n][ceil(k/128)], or with b_blocks = 1
 *     [ceil(n/128)][ceil(k/128)].  Scales are any fp32 values; a block's sum
 *     times either operand's has to stay in fp32's range.  Tiles all of whose scales are
 *     powers of two from 2^-62 to 2^62 take one walk along k, others three.
 *   out [m][n] dense; must not overlap the operands
 * a and b are 16-byte aligned, their pitches multiples of 16; bytes past a row's
 * end are read but have no influence.  The workspace (fp8_matmul_workspace_size;
 * 16-byte aligned; the size may be 0) holds partial sums over k.
 */
typedef struct fp8_matmul_problem {
    int m, n, k;
    int b_blocks; /* 0 or 1 */
    long long a_pitch, b_pitch;
} fp8_matmul_problem_t;

int fp8_matmul_workspace_size(const fp8_matmul_problem_t *prob, int dtype, size_t *bytes);
int fp8_matmul(const fp8_matmul_problem_t *prob, int dtype, const void *a, const float *a_scale,
               const void *b, const float *b_scale, void *out, void *workspace, size_t workspace_bytes,
               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SEQUENCE_OPS_H */
