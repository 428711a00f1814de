// norm_common.h -- a row of a layer norm in the registers of a group of lanes.
#pragma once

#include "block_internal.h"

namespace cnv {

template <int CTRL>
__device__ inline float norm_dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

__device__ inline float sum_of(uint32_t a, uint32_t b) { return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b); }

// The sum of v over the LANES lanes (16 or 64) around this one, the same bits in all of them.
template <int LANES>
__device__ inline float lanes_sum(float v)
{
    v += norm_dpp<0x128>(v);  // rotations of a row of 16 lanes by 8, 4, 2, 1
    v += norm_dpp<0x124>(v);
    v += norm_dpp<0x122>(v);
    v += norm_dpp<0x121>(v);
    if (LANES > 16) {  // rows change places with their neighbours, then the wave's halves
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        uint32_t u = __builtin_bit_cast(uint32_t, v);
        u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(u, u, false, false));
        u = __builtin_bit_cast(uint32_t, sum_of(r[0], r[1]));
        r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(u, u, false, false));
        v = sum_of(r[0], r[1]);
    }
    return v;
}

// Sums of K values over the LANES lanes that hold a row.  slot: LDS for LANES / 64
// waves, which nobody may still read from an earlier use.
template <int LANES, int K>
__device__ inline void row_sum(float (&v)[K], float *slot)
{
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_sum<(LANES < 64 ? LANES : 64)>(v[k]);
    if (LANES <= 64) return;
    constexpr int W = LANES / 64;
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) slot[wave * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float s = slot[k];
#pragma unroll
        for (int w = 1; w < W; ++w) s += slot[w * K + k];
        v[k] = s;
    }
}

// The columns of vector j of a lane: V from col[j] on.  Loads are whole vectors: one
// that would pass the row's end is moved back to end with it, and its first skip[j]
// elements belong to another lane (all V: the vector holds nothing).  d >= V.
template <int LANES, int N, int V>
struct Columns {
    int col[N], skip[N];
    __device__ inline Columns(int d)
    {
        const int lane = threadIdx.x % LANES;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * LANES + lane) * V;
            col[j] = c < d - V ? c : d - V;
            skip[j] = c - col[j] < V ? c - col[j] : V;
        }
    }
    __device__ inline bool mine(int j, int i) const { return i >= skip[j]; }
};

// weight or bias of a lane's columns
template <class E, int LANES, int N, int V>
__device__ inline void load_params(const void *p, int f32, float none, const Columns<LANES, N, V> &at, float (&out)[N][V])
{
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (!p) {
#pragma unroll
            for (int i = 0; i < V; ++i) out[j][i] = none;
        } else if (f32) {
            load_vec<SF32, V>((const float *)p + at.col[j], V, out[j]);
        } else {
            load_vec<E, V>((const typename E::S *)p + at.col[j], V, out[j]);
        }
    }
}

}  // namespace cnv
