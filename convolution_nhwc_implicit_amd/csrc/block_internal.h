// block_internal.h -- kernel arguments and launchers of a recurrent block's
// operators (layer norm, gated recurrence, 4-bit products), shared by the host
// side (block_api.cpp) and the kernels.  Not part of the ABI.
#pragma once

#include "seq_internal.h"

namespace cnv {

// ---- sums of partial sums (column_sums.hip) --------------------------------------
// partial [parts][outs][d] fp32 -> out[o][d] for each o, in type dtype; a NULL out is
// skipped.
struct ColumnSumArgs {
    const float *partial;
    int parts, outs, d;
    void *out[3];
    const float *over;  // where out[0] is a sum that is divided by over[c] (0 where that is 0)
};
hipError_t launch_column_sums(int dtype, const ColumnSumArgs &a, hipStream_t st);

// ---- layer norm (layer_norm.hip, layer_norm_grad.hip) -----------------------------
struct NormArgs {
    int rows, len, d;  // row = sequence * len + place; len = rows where one stride serves all
    float eps, count;  // count: d
    int param_f32;
    RowStride xs, rs, dys, dts;
    const void *x, *residual, *weight, *bias, *dy, *dtotal;
    void *y, *total, *dx;
    int per;         // rows of a part (gradient)
    int parts;
    float *partial;  // [parts][2][d]
    float *stats;    // [rows][4], for rows past the registers
    __device__ inline long long at(const RowStride &s, int row) const
    {
        if (len == rows) return (long long)row * s.row;
        const int q = row / len;
        return q * s.seq + (long long)(row - q * len) * s.row;
    }
};

// Lanes and vectors that hold a row: lanes * vecs * width elements.
struct NormShape {
    int lanes, vecs, width;
    bool held;  // whether a row fits the registers at all
};
NormShape layer_norm_shape(int dtype, int rows, int d);
NormShape layer_norm_grad_shape(int dtype, int d);
hipError_t launch_layer_norm(int dtype, const NormArgs &a, const NormShape &s, hipStream_t st);
hipError_t launch_layer_norm_grad(int dtype, const NormArgs &a, const NormShape &s, hipStream_t st);

// ---- gated recurrence (gated_recurrence.hip, gated_recurrence_grad.hip) -------------
// How a workgroup's lanes lie: `lanes` of a wave along channels, `vc` channels to each;
// a wave's other lanes, and the waves, take successive runs of tokens.
struct RecurShape {
    int lanes, vc;
    constexpr int channels() const { return lanes * vc; }
};
constexpr int kRecurChunkMost = 1 << 15;  // tokens of a chunk: their first-token bits lie in LDS
constexpr int kRecurStateSeqs = 256;   // sequences of a workgroup that writes the states of empty ones

struct RecurArgs {
    Seqs q;
    int d;
    int across;          // workgroups along channels
    int chunk, chunks;   // tokens of a chunk (whole segments), chunks in all
    int tail;            // chunks that no other follows
    int joined;          // chunks start inside sequences
    int per_seq;         // chunks of each sequence; 0: chunks run over all tokens
    RowStride xs, rs, is, zs, dys;
    const void *x, *r, *i, *z, *dy;
    const float *A, *r_bias, *i_bias, *initial, *dfinal;
    void *y;
    float *final_state, *dinitial;
    // workspace
    float *chunk_decay, *chunk_state;  // [chunks][d]: decay over a chunk (-1: cut inside), state it ends with from zero
    float *back_decay, *chunk_back;    // the same for the gradient that flows out of its first token
    float *seg_decay, *seg_state;      // [segments][d]: of the chunk's tokens before a segment
    float *partial;                    // [chunks][3][d]: sums of dL * L, dr, di
    void *dx, *dr, *di, *dz;
};
struct RecurStepArgs {
    int rows, pool, d;
    long long x_row, r_row, i_row, z_row;
    const void *x, *r, *i, *z;
    const float *A, *r_bias, *i_bias;
    float *state;
    const int *slots;
    void *y;
};
constexpr int kRecurRun = 4, kRecurWaves = 8;  // tokens of a lane's run, waves of a workgroup
constexpr int kRecurStepChannels = 4;  // channels of a thread of the single-token kernel
constexpr int recur_segment(const RecurShape &s) { return 64 / s.lanes * kRecurRun * kRecurWaves; }

hipError_t launch_recurrence(int dtype, const RecurArgs &a, const RecurShape &s, hipStream_t st);
hipError_t launch_recurrence_grad(int dtype, const RecurArgs &a, const RecurShape &s, hipStream_t st);
hipError_t launch_recurrence_step(int dtype, const RecurStepArgs &a, hipStream_t st);

// ---- 4-bit products (fp4.hip) ----------------------------------------------------
constexpr int kFp4Group = 32;  // values along the summed axis that share a scale

struct Fp4QuantArgs {
    int m, k, groups;
    long long x_row, q_pitch;
    const void *x;
    uint8_t *q, *scale;
};
struct Fp4MatmulArgs {
    int m, n, k, groups;
    long long x_row, w_pitch;
    const void *x;
    const uint8_t *w, *w_scale;
    void *out;
    int splits, per, tiles;  // Fp4Plan
    float *partial;   // [splits][m][n]
};
// Many rows of x: workgroups along k and the turns of 256 values of each.  splits 0: few
// rows, and workgroups of one or two tiles of 16 rows of w (two for more than 16 rows of x).
struct Fp4Plan {
    int splits, per, tiles;
    size_t bytes(int m, int n) const { return splits > 1 ? (size_t)splits * m * n * 4 : 0; }
};
Fp4Plan fp4_matmul_plan(int m, int n, int k, int dtype);
hipError_t launch_fp4_quantize(int dtype, const Fp4QuantArgs &a, hipStream_t st);
hipError_t launch_fp4_matmul(int dtype, const Fp4MatmulArgs &a, hipStream_t st);

}  // namespace cnv
