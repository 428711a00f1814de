// column_sums.hip -- sums of partial sums over parts, in a fixed order.
//
// out[o][c] = sum_p partial[p][o][c].  A workgroup takes 64 columns; its 16 waves take
// every 16th part each and are joined through LDS, so that few columns still have many
// loads under way.
#include "block_internal.h"

namespace cnv {
namespace {

constexpr int kWaves = 16;

template <class E>
__global__ __launch_bounds__(64 * kWaves) void column_sums_kernel(ColumnSumArgs a)
{
    __shared__ float part[kWaves][64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const long long cols = (long long)a.outs * a.d, c = (long long)blockIdx.x * 64 + lane;
    const float *p = a.partial + (c < cols ? c : cols - 1);
    float s = 0.0f;
    for (int i = wave; i < a.parts; i += kWaves) s += p[i * cols];
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || c >= cols) return;
    s = part[0][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += part[w][lane];
    const int o = (int)(c / a.d), col = (int)(c - (long long)o * a.d);
    if (o == 0 && a.over) {
        const float d = a.over[col];
        s = d == 0.0f ? 0.0f : s / d;
    }
    if (a.out[o]) ((typename E::S *)a.out[o])[col] = E::from(s);
}

}  // namespace

hipError_t launch_column_sums(int dtype, const ColumnSumArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)(((long long)a.outs * a.d + 63) / 64));
    switch (dtype) {
        case CONV2D_DTYPE_F16: column_sums_kernel<SF16><<<grid, 64 * kWaves, 0, st>>>(a); break;
        case CONV2D_DTYPE_BF16: column_sums_kernel<SBF16><<<grid, 64 * kWaves, 0, st>>>(a); break;
        default: column_sums_kernel<SF32><<<grid, 64 * kWaves, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace cnv
