// fp4.hip -- 4-bit operands: quantisation, and products of few rows with them.
//
//   out[i][j] = sum_k x[i][k] * e2m1(w[j][k]) * 2^(scale[j][k / 32] - 127)
//
// The product is bound by the weights' bytes.  They go from memory to the matrix unit in
// registers: a lane loads 16 bytes, one group of 32 values, of one row of w, and the
// conversion instruction turns two values at a time into bf16 with the group's scale
// applied, which is exact.  The matrix instruction sums over k in any order as long as
// both operands have the same, so x is loaded to match.  bf16 x is one operand; fp16
// x is the sum of two bf16 values and fp32 x of three, exactly, so that all products
// are exact and all sums fp32.  The waves of a workgroup take turns along k and are
// added through LDS in order.
#include "block_internal.h"

namespace cnv {
namespace {

// ---- quantisation ----------------------------------------------------------------
// four lanes to a group of 32 values, 8 each
template <class E>
__global__ __launch_bounds__(256) void fp4_quantize_kernel(Fp4QuantArgs a, long long groups)
{
    const long long b = (long long)blockIdx.x * 64 + threadIdx.x / 4;
    if (b >= groups) return;
    const long long row = b / a.groups, g = b - row * a.groups;
    const int part = threadIdx.x % 4;
    const long long c = g * kFp4Group + part * 8, have = a.k - c;
    float v[8];
    load_vec<E, 8>((const typename E::S *)a.x + row * a.x_row + c, have < 8 ? (int)have : 8, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
        top = top > u ? top : u;
    }
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
        const uint32_t o = __shfl_xor((int)top, d);
        top = top > o ? top : o;
    }
    // top = 1.f * 2^E and 6 = 1.5 * 2^2: 2^(E-2), or 2^(E-1) where 1.f > 1.5
    const int e0 = (int)(top >> 23) - 2 + ((top & 0x7fffffu) > 0x400000u ? 1 : 0);
    const bool finite = top < 0x7f800000u;
    const int e = !finite ? 255 : e0 < 0 ? 0 : e0;
    uint32_t codes = 0;
    if (finite)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = __builtin_amdgcn_ldexpf(fabsf(v[i]), 127 - e);
            // borders between neighbouring values go to the one with an even code
            uint32_t code = (s > 0.25f) + (s >= 0.75f) + (s > 1.25f) + (s >= 1.75f) + (s > 2.5f) + (s >= 3.5f) + (s > 5.0f);
            if (v[i] < 0.0f) code |= 8;
            codes |= code << (4 * i);
        }
    *(uint32_t *)(a.q + row * a.q_pitch + g * 16 + part * 4) = codes;
    if (part == 0) a.scale[b] = (uint8_t)e;
}

// ---- products --------------------------------------------------------------------
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// eight e2m1 values to bf16, times the power of two whose exponent field is scale's
__device__ inline bf16x8 weights8(uint32_t w, float scale)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <class E>
constexpr int kParts = 3;
template <>
constexpr int kParts<SBF16> = 1;
template <>
constexpr int kParts<SF16> = 2;

// The high half of v as bf16; what is left of v stays in v (0 where v is not finite).
__device__ inline uint32_t split(float &v)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const bool finite = (u & 0x7f800000u) != 0x7f800000u;
    const bool nan = v != v;
    v = finite ? v - __builtin_bit_cast(float, u & 0xffff0000u) : 0.0f;
    return nan ? 0x7fc0u : u >> 16;
}

// eight values of x at p, of which have are there, as kParts<E> operands
template <class E>
__device__ inline void load_x(const typename E::S *p, int have, bf16x8 (&out)[kParts<E>])
{
    if constexpr (kParts<E> == 1) {
        if (have >= 8) {
            out[0] = __builtin_bit_cast(bf16x8, *(const SVec<uint16_t, 8> *)p);
        } else {
            SVec<uint16_t, 8> v;
#pragma unroll
            for (int i = 0; i < 8; ++i) v.v[i] = i < have ? p[i] : 0;
            out[0] = __builtin_bit_cast(bf16x8, v);
        }
    } else {
        float v[8];
        load_vec<E, 8>(p, have, v);
#pragma unroll
        for (int s = 0; s < kParts<E>; ++s) {
            u32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = split(v[2 * i]), hi = split(v[2 * i + 1]);
                r[i] = lo | hi << 16;
            }
            out[s] = __builtin_bit_cast(bf16x8, r);
        }
    }
}

constexpr int kWaves = 8;

// MT tiles of 16 rows of x; 16 rows of w.
template <class E, int MT>
__global__ __launch_bounds__(64 * kWaves) void fp4_matmul_kernel(Fp4MatmulArgs a)
{
    __shared__ f32x4 part[kWaves][MT][64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, row = lane % 16, quarter = lane / 16;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * (16 * MT);
    const int nj = n0 + row < a.n ? n0 + row : a.n - 1;
    const uint8_t *w = a.w + (long long)nj * a.w_pitch, *sc = a.w_scale + (long long)nj * a.groups;
    const typename E::S *x[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int i = m0 + t * 16 + row;
        x[t] = (const typename E::S *)a.x + (long long)(i < a.m ? i : a.m - 1) * a.x_row;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    for (int g0 = wave * 4; g0 < a.groups; g0 += kWaves * 4) {
        // a lane past the last group takes it again, with zeros of x
        const int g = g0 + quarter, gc = g < a.groups ? g : a.groups - 1;
        const u32x4 q = *(const u32x4 *)(w + (long long)gc * 16);
        const float scale = __builtin_bit_cast(float, (uint32_t)sc[gc] << 23);
        const int have = g < a.groups ? a.k - g * kFp4Group : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x8 b = weights8(q[j], scale);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                bf16x8 xs[kParts<E>];
                load_x<E>(x[t] + (long long)gc * kFp4Group + j * 8, have - j * 8, xs);
#pragma unroll
                for (int s = kParts<E> - 1; s >= 0; --s) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs[s], b, acc[t], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    // a lane holds column `row` and rows 4 * quarter .. + 3 of a tile
    for (int t = wave; t < MT; t += kWaves) {
        f32x4 s = part[0][t][lane];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) s += part[v][t][lane];
        const int j = n0 + row;
        if (j < a.n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = m0 + t * 16 + quarter * 4 + r;
                if (i < a.m) ((typename E::S *)a.out)[(long long)i * a.n + j] = E::from(s[r]);
            }
    }
}

template <class E>
hipError_t launch_product(const Fp4MatmulArgs &a, hipStream_t st)
{
    const int tiles = (a.m + 15) / 16;
    const unsigned gx = (unsigned)((a.n + 15) / 16);
    if (tiles == 1) fp4_matmul_kernel<E, 1><<<dim3(gx, 1), 64 * kWaves, 0, st>>>(a);
    else if (tiles == 2) fp4_matmul_kernel<E, 2><<<dim3(gx, 1), 64 * kWaves, 0, st>>>(a);
    else fp4_matmul_kernel<E, 4><<<dim3(gx, (unsigned)((tiles + 3) / 4)), 64 * kWaves, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_quantize(int dtype, const Fp4QuantArgs &a, hipStream_t st)
{
    const long long groups = (long long)a.m * a.groups;
    const unsigned grid = (unsigned)((groups + 63) / 64);
    switch (dtype) {
        case CONV2D_DTYPE_F16: fp4_quantize_kernel<SF16><<<grid, 256, 0, st>>>(a, groups); break;
        case CONV2D_DTYPE_BF16: fp4_quantize_kernel<SBF16><<<grid, 256, 0, st>>>(a, groups); break;
        default: fp4_quantize_kernel<SF32><<<grid, 256, 0, st>>>(a, groups); break;
    }
    return hipGetLastError();
}

hipError_t launch_fp4_matmul(int dtype, const Fp4MatmulArgs &a, hipStream_t st)
{
    switch (dtype) {
        case CONV2D_DTYPE_F16: return launch_product<SF16>(a, st);
        case CONV2D_DTYPE_BF16: return launch_product<SBF16>(a, st);
        default: return launch_product<SF32>(a, st);
    }
}

}  // namespace cnv
