// column_sums.hip -- sums of partial sums over parts, in a fixed order.
//
// out[o][c] = sum_p partial[p][o][c].  A workgroup takes 32 columns, four to a lane; its
// 128 groups of eight lanes take every 128th part each, so that a part's row is read in
// lines of 128 bytes and few columns still have many loads under way, and are joined by
// shuffles and through LDS.  512 parts of 8192 columns: 5 us
// (8.4 with 64 columns and a group to a wave).
#include "block_internal.h"

namespace cnv {
namespace {

constexpr int kWaves = 16, kColumns = 32, kGroups = kWaves * 8;

template <class E>
__global__ __launch_bounds__(64 * kWaves) void column_sums_kernel(ColumnSumArgs a)
{
    __shared__ float part[kWaves][kColumns];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, col = lane % 8 * 4;
    const long long cols = (long long)a.outs * a.d, c = (long long)blockIdx.x * kColumns + col;
    const int have = c + 4 <= cols ? 4 : c < cols ? (int)(cols - c) : 0;
    float s[4] = {};
    if (have > 0) {
        const float *p = a.partial + c;
#pragma unroll 4
        for (int i = threadIdx.x / 8; i < a.parts; i += kGroups) {
            float v[4];
            load_vec<SF32, 4>(p + i * cols, have, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += v[k];
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 8; o < 64; o *= 2) s[k] += __shfl_xor(s[k], o);
        if (lane < 8) part[wave][col + k] = s[k];
    }
    __syncthreads();
    const long long at = (long long)blockIdx.x * kColumns + threadIdx.x;
    if (threadIdx.x >= kColumns || at >= cols) return;
    float sum = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += part[w][threadIdx.x];
    const int o = (int)(at / a.d), to = (int)(at - (long long)o * a.d);
    if (o == 0 && a.over) {
        const float d = a.over[to];
        sum = d == 0.0f ? 0.0f : sum / d;
    }
    if (a.out[o]) ((typename E::S *)a.out[o])[to] = E::from(sum);
}

}  // namespace

hipError_t launch_column_sums(int dtype, const ColumnSumArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)(((long long)a.outs * a.d + kColumns - 1) / kColumns));
    switch (dtype) {
        case CONV2D_DTYPE_F16: column_sums_kernel<SF16><<<grid, 64 * kWaves, 0, st>>>(a); break;
        case CONV2D_DTYPE_BF16: column_sums_kernel<SBF16><<<grid, 64 * kWaves, 0, st>>>(a); break;
        default: column_sums_kernel<SF32><<<grid, 64 * kWaves, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace cnv
