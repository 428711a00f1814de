// fp8_quantize.hip -- values to e4m3 with a power-of-two scale per block.
//
// One read of x and one write of q: bound by memory.  A block's scale needs its
// largest value first, so the block waits in registers (or, transposed, in LDS)
// between the two.  4057 x 4104 bf16 by rows: 11 us (4.6 TB/s); 8200 x 4104 by
// blocks of 128 x 128: 25 us (4.1 TB/s).
#include "seq_common.h"
#include "seq_internal.h"

namespace cnv {
namespace {

// |v| as ordered bits; infinities and NaN count as nothing
__device__ inline uint32_t finite_bits(float v)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

// The exponent field of the least power of two s >= 2^-126 with top <= 448 s.
// top = 1.f * 2^E and 448 = 1.75 * 2^8: s = 2^(E-8), or 2^(E-7) where 1.f > 1.75.
__device__ inline uint32_t scale_exponent(uint32_t top)
{
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < 1 ? 1u : (uint32_t)e;
}
__device__ inline float scale_value(uint32_t e) { return __builtin_bit_cast(float, e << 23); }
__device__ inline float scale_inverse(uint32_t e) { return __builtin_bit_cast(float, (254u - e) << 23); }

// four values times inv (a power of two: exact) to four e4m3 bytes, to nearest even
__device__ inline uint32_t pack4(float a, float b, float c, float d, float inv)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
}

// largest over a row of 16 lanes, in every lane
__device__ inline uint32_t row_max(uint32_t v)
{
    auto step = [&](auto ctrl) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, decltype(ctrl)::value, 0xf, 0xf, true);
        v = v > o ? v : o;
    };
    step(std::integral_constant<int, 0x128>{});  // rotations by 8, 4, 2, 1
    step(std::integral_constant<int, 0x124>{});
    step(std::integral_constant<int, 0x122>{});
    step(std::integral_constant<int, 0x121>{});
    return v;
}

// 8 bytes at column c of a row of q; bytes from k to the pitch are zero (their
// values were loaded as zero)
__device__ inline void store8(uint8_t *row, long long c, long long pitch, const float (&v)[8], float inv)
{
    if (c >= pitch) return;
    uint2 r;
    r.x = pack4(v[0], v[1], v[2], v[3], inv);
    r.y = pack4(v[4], v[5], v[6], v[7], inv);
    *(uint2 *)(row + c) = r;  // c and the pitch are multiples of 8
}

// 16 lanes to a block of one row, 8 values each.
template <class E>
__global__ __launch_bounds__(256) void quantize_rows_kernel(Fp8QuantArgs a, long long blocks, int kb)
{
    const long long b = (long long)blockIdx.x * 16 + threadIdx.x / 16;
    if (b >= blocks) return;
    const long long row = b / kb, block = b - row * kb, c = block * kFp8Block + threadIdx.x % 16 * 8;
    float v[8];
    const long long have = a.k - c;
    load_vec<E, 8>((const typename E::S *)a.x + row * a.x_row + c, have < 8 ? (int)have : 8, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = finite_bits(v[i]);
        top = top > u ? top : u;
    }
    const uint32_t e = scale_exponent(row_max(top));
    store8(a.q + row * a.q_pitch, c, a.q_pitch, v, scale_inverse(e));
    if (threadIdx.x % 16 == 0) a.scale[b] = scale_value(e);
}

// A workgroup to a block of 128 rows and 128 columns.
template <class E>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(Fp8QuantArgs a, int kb)
{
    const int bk = blockIdx.x, bm = blockIdx.y, tid = threadIdx.x;
    const long long c = (long long)bk * kFp8Block + tid % 16 * 8, r0 = (long long)bm * kFp8Block + tid / 16;
    const long long have = a.k - c;
    float v[8][8];
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const long long r = r0 + p * 16;
        load_vec<E, 8>((const typename E::S *)a.x + r * a.x_row + c, r < a.m ? (have < 8 ? (int)have : 8) : 0, v[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = finite_bits(v[p][i]);
            top = top > u ? top : u;
        }
    }
    top = row_max(top);
    __shared__ uint32_t tops[16];
    if (tid % 16 == 0) tops[tid / 16] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) top = top > tops[i] ? top : tops[i];
    const uint32_t e = scale_exponent(top);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const long long r = r0 + p * 16;
        if (r < a.m) store8(a.q + r * a.q_pitch, c, a.q_pitch, v[p], scale_inverse(e));
    }
    if (tid == 0) a.scale[(long long)bm * kb + bk] = scale_value(e);
}

// A workgroup to 128 rows and 64 columns of x: through LDS, then a quad of
// lanes to a column, 32 of its rows each.
template <class E>
__global__ __launch_bounds__(256) void quantize_transpose_kernel(Fp8QuantArgs a, int mb)
{
    // rows 65 apart, and each 32 rows 16 further: a wave reads 16 columns of 4
    // such parts, over all banks
    constexpr int kPitch = 65, kShift = 16;
    __shared__ float t[kFp8Block * kPitch + 4 * kShift];
    const int tid = threadIdx.x;
    const long long m0 = (long long)blockIdx.x * kFp8Block, c0 = (long long)blockIdx.y * 64;
    const int col = tid % 8 * 8;
    const long long have = a.k - (c0 + col);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int r = p * 32 + tid / 8;
        float v[8];
        const int n = m0 + r < a.m ? (have < 8 ? (int)have : 8) : 0;
        load_vec<E, 8>((const typename E::S *)a.x + (m0 + r) * a.x_row + c0 + col, n, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[r * kPitch + p * kShift + col + i] = v[i];
    }
    __syncthreads();
    const int part = tid % 4, cc = tid / 4;
    float v[32];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = t[(part * 32 + i) * kPitch + part * kShift + cc];
        const uint32_t u = finite_bits(v[i]);
        top = top > u ? top : u;
    }
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xb1, 0xf, 0xf, true);
    top = top > o ? top : o;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4e, 0xf, 0xf, true);
    top = top > o ? top : o;
    if (c0 + cc >= a.k) return;
    const uint32_t e = scale_exponent(top);
    const float inv = scale_inverse(e);
    uint8_t *row = a.q + (c0 + cc) * a.q_pitch;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long c = m0 + part * 32 + h * 16;
        if (c >= a.q_pitch) break;
        uint4 r;
        r.x = pack4(v[16 * h + 0], v[16 * h + 1], v[16 * h + 2], v[16 * h + 3], inv);
        r.y = pack4(v[16 * h + 4], v[16 * h + 5], v[16 * h + 6], v[16 * h + 7], inv);
        r.z = pack4(v[16 * h + 8], v[16 * h + 9], v[16 * h + 10], v[16 * h + 11], inv);
        r.w = pack4(v[16 * h + 12], v[16 * h + 13], v[16 * h + 14], v[16 * h + 15], inv);
        *(uint4 *)(row + c) = r;  // 16-byte aligned: so are q, its pitch and c
    }
    if (part == 0) a.scale[(c0 + cc) * mb + blockIdx.x] = scale_value(e);
}

}  // namespace

hipError_t launch_fp8_quantize(int form, int dtype, const Fp8QuantArgs &a, hipStream_t st)
{
    const int kb = (a.k + kFp8Block - 1) / kFp8Block, mb = (a.m + kFp8Block - 1) / kFp8Block;
    auto run = [&](auto e) {
        using E = decltype(e);
        if (form == FP8_ROWS) {
            const long long blocks = (long long)a.m * kb;
            quantize_rows_kernel<E><<<dim3((unsigned)((blocks + 15) / 16)), 256, 0, st>>>(a, blocks, kb);
        } else if (form == FP8_BLOCKS) {
            quantize_blocks_kernel<E><<<dim3((unsigned)kb, (unsigned)mb), 256, 0, st>>>(a, kb);
        } else {
            quantize_transpose_kernel<E><<<dim3((unsigned)mb, (unsigned)((a.k + 63) / 64)), 256, 0, st>>>(a, mb);
        }
        return hipGetLastError();
    };
    if (dtype == CONV2D_DTYPE_F16) return run(SF16{});
    if (dtype == CONV2D_DTYPE_BF16) return run(SBF16{});
    return run(SF32{});
}

}  // namespace cnv
