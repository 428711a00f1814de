// seq_internal.h -- kernel arguments and launchers of the sequence operators,
// shared by the host side (seq_api.cpp) and the kernels.  Not part of the ABI.
#pragma once

#include "seq_common.h"

namespace cnv {

// A launch's threads along x: the device counts them in 32 bits.
constexpr long long kMaxThreads = (1LL << 32) - 1;
constexpr bool fits(long long workgroups, int threads) { return workgroups <= kMaxThreads / threads; }

// ---- causal convolution (causal_conv.hip) -------------------------------------
constexpr int kConvUnroll = 4;    // rows whose loads are issued together
constexpr int kConvChannels = 4;  // channels per thread, where there are so many
constexpr int conv_channels(int d) { return d < kConvChannels ? 1 : kConvChannels; }

struct ConvArgs {
    Seqs q;
    int d, silu;
    int lanes;       // threads of a block along channels (a power of two, at most 64)
    int run;         // rows per thread
    int run_blocks;  // blocks along y that walk rows; the rest handle states
    RowStride xs, dys;
    const void *x, *weight, *bias, *initial, *dy, *dfinal;
    void *y;          // y, or dx in the gradient pass
    void *final_state, *dinitial;
    float *partial;   // [run_blocks][w+1][d]
    void *dweight, *dbias;
};

struct ConvStepArgs {
    int rows, pool, d, silu, lanes;
    long long x_row;
    const void *x, *weight, *bias;
    const int *slots;
    void *state, *y;
};

hipError_t launch_conv(int dtype, int w, const ConvArgs &a, dim3 grid, hipStream_t st);
hipError_t launch_conv_grad(int dtype, int w, const ConvArgs &a, dim3 grid, hipStream_t st);
hipError_t launch_conv_step(int dtype, int w, const ConvStepArgs &a, dim3 grid, hipStream_t st);

// ---- selective scan (selective_scan.hip, selective_scan_grad.hip) ----------------
constexpr int kScanWaveChannels = 16;  // channels of a wave, and of a workgroup of the forward pass
constexpr int kScanChannels = 64;      // channels of a workgroup of the gradient

struct ScanArgs {
    Seqs q;
    int d, n, groups, softplus;
    int blocks_per_group;  // workgroups along the channels of one group
    int chunk;             // tokens per chunk, a multiple of 16
    int chunks;            // chunks per sequence (dense)
    int slots;             // chunks in all; for packed sequences an upper bound
    RowStride xs, dts, bs, cs, zs, dys;
    long long b_group, c_group;  // strides between groups of B and C
    const void *x, *dt, *B, *C, *z, *dy;
    const float *A, *D, *dt_bias, *initial, *dfinal;
    void *y;               // y [tokens][d]
    float *final_state, *dinitial;
    // workspace: per chunk the state it ends with (from zero; then the state it starts
    // with), the sum of its steps, and the like for the gradient
    float *chunk_state;    // [slots][d][n]
    float *chunk_delta;    // [slots][d]
    float *chunk_back;     // [slots][d][n]
    float *check;          // [tokens/TS + slots + 1][d][n]: states before each step of TS tokens
    float *check_delta;    // [tokens/TS + slots + 1][d]: sums of steps before it
    float *part_A;         // [slots][d][n]
    float *part_D;         // [slots][d], and the same for dt_bias
    float *part_bias;
    float *part_B, *part_C; // [channel blocks][tokens][n]
    void *du, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *ddt_bias;
};

struct ScanStepArgs {
    int rows, pool, d, n, groups, softplus;
    long long x_row, dt_row, b_row, c_row, z_row, b_group, c_group;
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *dt_bias;
    const int *slots;
    float *state;
    void *y;
};

// Tokens a wave takes at once: as many as keep the loads of the next ones under
// way.  A run's decays and inputs take 128 registers for any n above 8; what is
// read ahead of B and C grows with n and spills past 16 states (3 to 19 registers
// up to 32, 55 to 88 up to 64): 4096 tokens of 2048 channels take 102 us with 16
// states, 265 with 32, 1270 with 64.
constexpr int scan_step_tokens(int n) { return n <= 16 ? 16 : n <= 32 ? 8 : 4; }
// The gradient keeps a step's decays and states in registers, TS * n/4 values of
// each: 64 registers of each would spill (16 tokens of 16 states: 1115 us for
// four sequences of 2048 with 2048 channels).
constexpr int scan_grad_step_tokens(int n) { return n <= 8 ? 16 : n <= 16 ? 8 : 4; }

// Rows a thread of the single-token kernel takes where there are many.
constexpr int scan_step_rows(int n) { return n > 16 ? 2 : 4; }

hipError_t launch_scan(int dtype, const ScanArgs &a, int waves, hipStream_t st);
hipError_t launch_scan_grad(int dtype, const ScanArgs &a, hipStream_t st);
hipError_t launch_scan_step(int dtype, const ScanStepArgs &a, hipStream_t st);

// ---- fp8 products (fp8_quantize.hip, fp8_matmul.hip) -------------------------------
constexpr int kFp8Block = 128;  // values along the summed axis that share a scale

struct Fp8QuantArgs {
    int m, k;
    long long x_row, q_pitch;
    const void *x;
    uint8_t *q;
    float *scale;
};

struct Fp8MatmulArgs {
    int m, n, k, kb;  // kb: blocks along k
    int b_blocks;
    long long a_pitch, b_pitch;
    const uint8_t *a, *b;
    const float *a_scale, *b_scale;
    void *out;
    int tiles_m, tiles_n;
    long long ldo;  // row stride of out
    int kb_split;  // blocks along k per workgroup
};

struct Fp8Plan {
    int shape, splits, per;  // tile shape; workgroups along k, and blocks of each
    bool narrow_m, narrow_n; // the rows of a, or of b, past whole tiles go to the narrow kernel
    bool all;                // everything does
};

hipError_t launch_fp8_quantize(int form, int dtype, const Fp8QuantArgs &a, hipStream_t st);
Fp8Plan fp8_matmul_plan(int m, int n, int k, int dtype);
bool fp8_matmul_fits(int m, int n, int k, const Fp8Plan &p);  // whether its launches fit
size_t fp8_matmul_bytes(int m, int n, const Fp8Plan &p);
hipError_t launch_fp8_matmul(int dtype, const Fp8MatmulArgs &a, const Fp8Plan &p, void *workspace, hipStream_t st);

}  // namespace cnv
