// fp8_matmul.hip -- products of block-scaled e4m3 operands.
//
//   out[i][j] = sum over blocks kb of a_scale[i][kb] b_scale[j][kb] * (sum over the block of a[i][k] b[j][k])
//
// A workgroup owns a tile of out and walks k a block of 128 at a time: the
// operands' rows go to LDS by direct loads, double buffered, and from there as
// 16x16x128 matrix instructions' fragments.  b is the instruction's first
// operand, so that a lane ends up with four neighbouring columns of a row of out.
#include <algorithm>

#include "seq_common.h"
#include "seq_internal.h"

namespace cnv {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two ways to multiply a block of 128 of 16 rows with 16 rows.  Both sum the
// values' products with fp32 accumulation, but the fp8 unit first aligns every
// 8 neighbouring products and cuts them at 2^-13 of the largest's power of two
// (measured; between those groups nothing is lost): about 1.5e-5 of a block's
// sum in norm, far below the rounding of a 16-bit result (1.7e-3 bf16, 2e-4
// fp16), but not below a float32 one's.  So 16-bit results use the fp8 unit
// (Fp8Unit), at twice the rate, and float32 results (Bf16Unit) convert the
// bytes to bf16, which holds every e4m3 value, for the bf16 unit, which is exact.
//
// `scaled` takes operands' scales 2^(s-127) into the product.
struct Fp8Unit {
    typedef i32x8 Frag;
    __device__ static inline Frag prepare(const i32x8 &raw, int) { return raw; }
    __device__ static inline f32x4 scaled(const Frag &a, const Frag &b, f32x4 c, int sa, int sb)
    {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
    }
    __device__ static inline f32x4 plain(const Frag &a, const Frag &b, f32x4 c) { return scaled(a, b, c, 127, 127); }
};

struct Bf16Unit {
    struct Frag {
        u32x4 v[4];
    };
    // 32 bytes to bf16 times 2^(s-127): exact for the scales the caller lets through
    __device__ static inline Frag prepare(const i32x8 &raw, int s)
    {
        const float scale = __builtin_bit_cast(float, (uint32_t)s << 23);
        Frag f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f.v[i / 2][i % 2 * 2] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[i], scale, false));
            f.v[i / 2][i % 2 * 2 + 1] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[i], scale, true));
        }
        return f;
    }
    __device__ static inline f32x4 plain(const Frag &a, const Frag &b, f32x4 c)
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) c = EBF16::mfma(a.v[q], b.v[q], c);
        return c;
    }
    __device__ static inline f32x4 scaled(const Frag &a, const Frag &b, f32x4 c, int, int) { return plain(a, b, c); }
};

__device__ inline int exponent_of(float s) { return (int)(__builtin_bit_cast(uint32_t, s) >> 23); }

// The exponent field of a scale that the units take as a power of two: 2^-62 to
// 2^62, so that scaled values stay normal bf16 numbers; any other gives -1.
__device__ inline int power_of_two(float s)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, s), e = u >> 23;  // the sign counts as exponent
    return (u & 0x7fffffu) == 0 && e >= 127 - 62 && e <= 127 + 62 ? (int)e : -1;
}

template <class E>
__device__ inline void store_out4(void *out, long long at, int have, const float (&v)[4])
{
    store_vec<E, 4>((typename E::S *)out + at, have, v);
}

// 128 rows of 128 bytes from row0 on, as 16-byte chunks; chunk c of row r lies
// at place c ^ (r & 7) of its row, so that 8 lanes reading one chunk column of
// 8 rows touch all banks.  A wave's load fills 8 rows.
template <int ROWS, int THREADS>
__device__ inline void stage_rows(const u32x4 &rsrc, uint32_t lds, uint32_t pitch, uint32_t k0, uint32_t kbytes)
{
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
    for (int i = 0; i < ROWS / 8 / (THREADS / 64); ++i) {
        const uint32_t r = (i * (THREADS / 64) + wave) * 8 + lane / 8;
        const uint32_t c = (lane % 8) ^ (r & 7);
        const uint32_t off = r * pitch + k0 + c * 16;
        dma16(rsrc, lds + (i * (THREADS / 64) + wave) * 1024, k0 + c * 16 < kbytes ? off : kBufOOBFar);
    }
}

// Clears the bytes past k of the last block's partly used chunk.
template <int ROWS, int THREADS>
__device__ inline void clear_tail(uint8_t *lds, uint32_t tail)
{
    const uint32_t c = tail / 16, keep = tail % 16;
    for (uint32_t r = threadIdx.x; r < ROWS; r += THREADS) {
        uint8_t *p = lds + r * 128 + ((c ^ (r & 7)) * 16);
        for (uint32_t i = keep; i < 16; ++i) p[i] = 0;
    }
}

__device__ inline i32x8 fragment(const uint8_t *lds, int row, int quarter)
{
    const uint8_t *p = lds + row * 128;
    const u32x4 lo = *(const u32x4 *)(p + ((quarter ^ (row & 7)) * 16));
    const u32x4 hi = *(const u32x4 *)(p + (((quarter + 4) ^ (row & 7)) * 16));
    i32x8 r;
    r[0] = lo.x; r[1] = lo.y; r[2] = lo.z; r[3] = lo.w;
    r[4] = hi.x; r[5] = hi.y; r[6] = hi.z; r[7] = hi.w;
    return r;
}

// The tile that a workgroup computes.  Workgroups go to the chip's 8 dies in
// turn; each die takes a run of neighbouring tiles, walked in strips of 8 tile
// rows, so that a die's second-level cache holds what its workgroups share.
__device__ inline void tile_of(const Fp8MatmulArgs &a, int *tm, int *tn)
{
    const int total = a.tiles_m * a.tiles_n, id = blockIdx.x, die = id % 8, at = id / 8;
    const int each = total / 8, more = total % 8;  // the first `more` dies have one tile more
    const int t = die * each + (die < more ? die : more) + at;
    constexpr int kStrip = 8;
    const int strip = t / (kStrip * a.tiles_n), r = t - strip * kStrip * a.tiles_n;
    const int rows = a.tiles_m - strip * kStrip < kStrip ? a.tiles_m - strip * kStrip : kStrip;
    *tm = strip * kStrip + r % rows;
    *tn = r / rows;
}

// SPLIT: the workgroup sums blocks blockIdx.y * kb_split on, and writes fp32
// partial sums [split][m][n].
template <class E, class UNIT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64, 2) void fp8_tile_kernel(Fp8MatmulArgs a)
{
    constexpr int THREADS = WM * WN * 64, MT = BM / WM / 16, NT = BN / WN / 16;
    static_assert(BM + BN <= THREADS, "a thread loads one scale");
    extern __shared__ __align__(16) uint8_t lds[];
    auto la = [&](int buf) { return lds + buf * BM * 128; };
    auto lb = [&](int buf) { return lds + 2 * BM * 128 + buf * BN * 128; };
    float *ls = (float *)(lds + 2 * (BM + BN) * 128);  // [2][BM + BN]: scales of a's rows, then b's
    int *odd = (int *)(ls + 2 * (BM + BN));              // [2]: some scale of the block is no power of two
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, quarter = lane / 16;
    const int wm = wave % WM, wn = wave / WM;
    int tile_m, tile_n;
    tile_of(a, &tile_m, &tile_n);
    const long long m0 = (long long)tile_m * BM, n0 = (long long)tile_n * BN;
    const int rows_a = a.m - m0 < BM ? (int)(a.m - m0) : BM, rows_b = a.n - n0 < BN ? (int)(a.n - n0) : BN;
    const int kb0 = blockIdx.y * a.kb_split, kb1 = kb0 + a.kb_split < a.kb ? kb0 + a.kb_split : a.kb;
    const uint32_t kbytes = (uint32_t)a.k, kceil = (kbytes + 15) / 16 * 16;
    // rows past the matrix lie past the buffers' ends and read as zero
    const u32x4 ra = make_buf_rsrc(a.a + m0 * a.a_pitch, (uint32_t)((rows_a - 1) * a.a_pitch) + kceil);
    const u32x4 rb = make_buf_rsrc(a.b + n0 * a.b_pitch, (uint32_t)((rows_b - 1) * a.b_pitch) + kceil);
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // this thread's row of scales; rows past the matrix get 1
    const float *scale_row = nullptr;
    if (tid < rows_a) scale_row = a.a_scale + (m0 + tid) * a.kb;
    else if (tid >= BM && tid - BM < rows_b) {
        const long long r = n0 + tid - BM;
        scale_row = a.b_scale + (a.b_blocks ? r / kFp8Block : r) * a.kb;
    }
    auto load_scale = [&](int kb) { return scale_row && kb < kb1 ? scale_row[kb] : 1.0f; };
    auto stage = [&](int kb, int buf) {
        stage_rows<BM, THREADS>(ra, lds_addr(la(buf)), (uint32_t)a.a_pitch, kb * 128u, kbytes);
        stage_rows<BN, THREADS>(rb, lds_addr(lb(buf)), (uint32_t)a.b_pitch, kb * 128u, kbytes);
    };
    // Scales of the next block go to LDS a step ahead; a thread whose scale is
    // no power of two says so beside them.
    auto put_scale = [&](int buf, float v) {
        if (tid < BM + BN) ls[buf * (BM + BN) + tid] = v;
        if (power_of_two(v) < 0) odd[buf] = 1;
    };
    float next_scale = 1.0f;
    if (tid < 2) odd[tid] = 0;
    __syncthreads();
    if (kb0 < kb1) {
        put_scale(0, load_scale(kb0));
        next_scale = load_scale(kb0 + 1);
        stage(kb0, 0);
    }
    const int ra0 = wm * MT * 16, rb0 = wn * NT * 16;
    // Block kb is in LDS for every wave, and the next one on its way.
    auto arrive = [&](int kb, int buf) {
        wait_vm_all();
        __syncthreads();
        if (kb + 1 == a.kb && kbytes % 16) {
            clear_tail<BM, THREADS>(la(buf), kbytes % 128);
            clear_tail<BN, THREADS>(lb(buf), kbytes % 128);
            __syncthreads();
        }
        if (kb + 1 < kb1) {
            put_scale(buf ^ 1, next_scale);
            stage(kb + 1, buf ^ 1);
            next_scale = load_scale(kb + 2);
        }
    };
    int kb = kb0;
    bool arrived = false;
    for (; kb < kb1; ++kb) {
        const int buf = (kb - kb0) & 1;
        arrive(kb, buf);
        arrived = true;
        if (__builtin_amdgcn_readfirstlane(odd[buf])) break;  // the same for every wave: nobody writes odd[buf] in this step
        const float *sa = ls + buf * (BM + BN), *sb = sa + BM;
        typename UNIT::Frag fb[NT];
        int eb[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            eb[j] = exponent_of(sb[rb0 + j * 16 + lane % 16]);
            fb[j] = UNIT::prepare(fragment(lb(buf), rb0 + j * 16 + lane % 16, quarter), eb[j]);
        }
        // a's next fragment is read while the unit works on this one; the
        // barriers keep the compiler from reading all of them first
        i32x8 raw = fragment(la(buf), ra0 + lane % 16, quarter);
        int ea = exponent_of(sa[ra0 + lane % 16]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const auto fa = UNIT::prepare(raw, ea);
            const int e = ea;
            if (i + 1 < MT) {
                raw = fragment(la(buf), ra0 + (i + 1) * 16 + lane % 16, quarter);
                ea = exponent_of(sa[ra0 + (i + 1) * 16 + lane % 16]);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = UNIT::scaled(fb[j], fa, acc[i][j], eb[j], e);
            __builtin_amdgcn_sched_barrier(0);
        }
        arrived = false;
    }
    // From the first block on with a scale that is no such power of two: the
    // block's sums first, then their scales in fp32.
    for (; kb < kb1; ++kb) {
        const int buf = (kb - kb0) & 1;
        if (!arrived) arrive(kb, buf);
        arrived = false;
        const float *sa = ls + buf * (BM + BN), *sb = sa + BM;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const auto fb = UNIT::prepare(fragment(lb(buf), rb0 + j * 16 + lane % 16, quarter), 127);
            const f32x4 vb = *(const f32x4 *)(sb + rb0 + j * 16 + quarter * 4);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const auto fa = UNIT::prepare(fragment(la(buf), ra0 + i * 16 + lane % 16, quarter), 127);
                const float va = sa[ra0 + i * 16 + lane % 16];
                const f32x4 p = UNIT::plain(fb, fa, f32x4{0, 0, 0, 0});
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e] * va, vb[e], acc[i][j][e]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    const long long at = (long long)blockIdx.y * a.m * a.n;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const long long r = m0 + (wm * MT + i) * 16 + lane % 16;
        if (r >= a.m) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const long long c = n0 + (wn * NT + j) * 16 + quarter * 4;
            const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            if (c < a.n) store_out4<E>(a.out, at + r * a.n + c, (int)(a.n - c < 4 ? a.n - c : 4), v);
        }
    }
}

// Adds the splits' partial sums in order.
template <class E>
__global__ __launch_bounds__(256) void fp8_sum_kernel(const float *part, int splits, long long total, void *out)
{
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= total) return;
    const int have = total - i < 4 ? (int)(total - i) : 4;
    float v[4] = {0, 0, 0, 0};
    for (int s = 0; s < splits; ++s) {
        float p[4];
        load_vec<SF32, 4>(part + s * total + i, have, p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += p[e];
    }
    store_out4<E>(out, i, have, v);
}

}  // namespace

// Tile and split.  A tile costs its area in matrix time plus what its shape
// loses (smaller tiles read the operands more often), rounds of tiles follow
// one another, and sums split over k pay for their partials.
Fp8Plan fp8_matmul_plan(int m, int n, int kb)
{
    struct Shape {
        int bm, bn, per_cu;
        double step;  // microseconds per block of 128 for a tile, per_cu tiles at a time
    };
    static const Shape shapes[] = {{256, 256, 1, 1.0}, {128, 128, 2, 0.62}};
    Fp8Plan best = {};
    double best_t = 1e30;
    for (int i = 0; i < 2; ++i) {
        const Shape &s = shapes[i];
        const long long tiles = (long long)((m + s.bm - 1) / s.bm) * ((n + s.bn - 1) / s.bn);
        for (int split = 1; split <= 32 && split <= std::max(kb, 1); ++split) {
            const int per = (kb + split - 1) / split;
            if (split > 1 && (per < 4 || (kb + per - 1) / per != split)) continue;
            const long long slots = 256 * s.per_cu, rounds = (tiles * split + slots - 1) / slots;
            double t = rounds * (per * s.step + 2.0);
            if (split > 1) t += 4.0 + (double)m * n * 4 * (2 * split + 1) / 4e6;
            if (t < best_t) {
                best_t = t;
                best = {i, split, per};
            }
        }
    }
    return best;
}

size_t fp8_matmul_bytes(int m, int n, const Fp8Plan &p) { return p.splits > 1 ? (size_t)p.splits * m * n * 4 : 0; }

template <class E, class UNIT>
static hipError_t launch_tiles(Fp8MatmulArgs a, const Fp8Plan &p, hipStream_t st)
{
    auto run = [&](auto bm, auto bn, auto wm, auto wn) {
        constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, WN = decltype(wn)::value;
        a.tiles_m = (a.m + BM - 1) / BM;
        a.tiles_n = (a.n + BN - 1) / BN;
        const int lds = 2 * (BM + BN) * (128 + 4) + 16;
        auto *kernel = fp8_tile_kernel<E, UNIT, BM, BN, WM, WN>;
        hipError_t r = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (r != hipSuccess) return r;
        const dim3 grid((unsigned)((long long)a.tiles_m * a.tiles_n), (unsigned)p.splits);
        kernel<<<grid, WM * WN * 64, lds, st>>>(a);
        return hipGetLastError();
    };
    using std::integral_constant;
    if (p.shape == 0)
        return run(integral_constant<int, 256>{}, integral_constant<int, 256>{}, integral_constant<int, 2>{}, integral_constant<int, 4>{});
    return run(integral_constant<int, 128>{}, integral_constant<int, 128>{}, integral_constant<int, 2>{}, integral_constant<int, 2>{});
}

hipError_t launch_fp8_matmul(int dtype, const Fp8MatmulArgs &args, const Fp8Plan &p, void *workspace, hipStream_t st)
{
    Fp8MatmulArgs a = args;
    a.kb_split = p.per;
    if (p.splits > 1) {
        a.out = workspace;
        hipError_t r = dtype == CONV2D_DTYPE_F32 ? launch_tiles<SF32, Bf16Unit>(a, p, st) : launch_tiles<SF32, Fp8Unit>(a, p, st);
        if (r != hipSuccess) return r;
        const long long total = (long long)a.m * a.n;
        const dim3 grid((unsigned)((total + 1023) / 1024));
        const float *part = (const float *)workspace;
        if (dtype == CONV2D_DTYPE_F16) fp8_sum_kernel<SF16><<<grid, 256, 0, st>>>(part, p.splits, total, args.out);
        else if (dtype == CONV2D_DTYPE_BF16) fp8_sum_kernel<SBF16><<<grid, 256, 0, st>>>(part, p.splits, total, args.out);
        else fp8_sum_kernel<SF32><<<grid, 256, 0, st>>>(part, p.splits, total, args.out);
        return hipGetLastError();
    }
    if (dtype == CONV2D_DTYPE_F16) return launch_tiles<SF16, Fp8Unit>(a, p, st);
    if (dtype == CONV2D_DTYPE_BF16) return launch_tiles<SBF16, Fp8Unit>(a, p, st);
    return launch_tiles<SF32, Bf16Unit>(a, p, st);
}

}  // namespace cnv
