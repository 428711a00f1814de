// fp8_matmul.hip -- products of block-scaled e4m3 operands.
//
//   out[i][j] = sum over blocks kb of a_scale[i][kb] b_scale[j][kb] * (sum over the block of a[i][k] b[j][k])
//
// A workgroup owns a tile of out and walks k a block of 128 at a time: the
// operands' rows go to LDS by direct loads, double buffered, and from there as
// 16x16x128 matrix instructions' fragments.  b is the instruction's first
// operand, so that a lane ends up with four neighbouring columns of a row of out.
// 4057 x 8200 x 4104: 153 us (1.8 PFLOP/s) where the matrix unit is busy for 57; the
// rest is waiting for blocks (64 KB each, one on its way) and writing results.
#include <algorithm>
#include <utility>

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
// `scaled` takes the operands' scales into the product, as bytes e of 2^(e-127),
// four to a register.
struct Fp8Unit {
    typedef i32x8 Frag;
    // A is the byte of the packed scales `s` that belongs to the fragment
    template <int A>
    __device__ static inline Frag prepare(const i32x8 &raw, int s) { return raw; }
    __device__ static inline Frag prepare_plain(const i32x8 &raw) { return raw; }
    template <int A, int B>
    __device__ static inline f32x4 scaled(const Frag &a, const Frag &b, f32x4 c, int sa, int sb)
    {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, A, sa, B, sb);
    }
    __device__ static inline f32x4 plain(const Frag &a, const Frag &b, f32x4 c) { return scaled<0, 0>(a, b, c, 127, 127); }
};

struct Bf16Unit {
    struct Frag {
        u32x4 v[4];
    };
    // 32 bytes to bf16 times scale (a power of two): exact for the scales the caller lets through
    __device__ static inline Frag convert(const i32x8 &raw, float scale)
    {
        Frag f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f.v[i / 2][i % 2 * 2] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[i], scale, false));
            f.v[i / 2][i % 2 * 2 + 1] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[i], scale, true));
        }
        return f;
    }
    template <int A>
    __device__ static inline Frag prepare(const i32x8 &raw, int s)
    {
        return convert(raw, __builtin_bit_cast(float, ((uint32_t)s >> (8 * A) & 255u) << 23));
    }
    __device__ static inline Frag prepare_plain(const i32x8 &raw) { return convert(raw, 1.0f); }
    __device__ static inline f32x4 plain(const Frag &a, const Frag &b, f32x4 c)
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) c = EBF16::mfma(a.v[q], b.v[q], c);
        return c;
    }
    template <int A, int B>
    __device__ static inline f32x4 scaled(const Frag &a, const Frag &b, f32x4 c, int, int) { return plain(a, b, c); }
};

// The exponent field of a scale that the units take as a power of two: 2^-62 to
// 2^62, so that scaled values stay normal bf16 numbers; any other gives -1.
__device__ inline int power_of_two(float s)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, s), e = u >> 23;  // the sign counts as exponent
    return (u & 0x7fffffu) == 0 && e >= 127 - 62 && e <= 127 + 62 ? (int)e : -1;
}

// f(0), f(1), .. with the index as a constant
template <class F, int... I>
__device__ inline void each(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ inline void each(F f)
{
    each(std::make_integer_sequence<int, N>{}, f);
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

// One tile of out (or with splits, its partial sum over blocks blockIdx.y *
// kb_split on, as fp32 [split][m][n]).
//
// Blocks of 128 follow one another without a gap in the matrix unit's work: two
// are in LDS or on their way; before the last two rows of fragments of a block a
// wave has read all of it, waits for the next block, and reads that one's first
// fragments while the unit works on the rest.  The loop's body is two blocks
// without a branch (branches made the compiler move products past the barrier
// and spill the sums); an odd last block has one of zeros after it.
//
// Scales are read two blocks at a time and kept in LDS as exponents, a byte each,
// so placed that a lane reads those of its four fragments' rows at once.  A tile
// one of whose scales is no power of two starts again on a path that multiplies
// each block's sum by its scales in fp32.
//
// Where k is no multiple of 16 the last chunk, whose bytes past k may hold
// anything, is left out of its block and comes first, as a block of its own.
template <class E, class UNIT, int BM, int BN, int WM, int WN>
struct Tile {
    static constexpr int THREADS = WM * WN * 64, MT = BM / WM / 16, NT = BN / WN / 16, ROWS = BM + BN;
    static constexpr int kLds = 2 * ROWS * 128 + 8 * THREADS;
    static_assert(ROWS <= THREADS, "a thread to a row's scales");
    static_assert(MT % 4 == 0 && NT == 4, "scales are packed by four fragments");
    const Fp8MatmulArgs &a;
    uint8_t *lds;
    int tid, lane, wave, quarter, lr, ra0, rb0;
    long long m0, n0;
    int rows_a, rows_b, kb0, kb1;  // blocks; kb0 - 1 stands for the last chunk where that is apart
    bool apart;
    uint32_t kbytes;  // where this workgroup's part of k ends
    u32x4 ra, rb;
    const float *scale_row;  // of this thread's row of a or b; past the matrix, of its last row

    __device__ inline Tile(const Fp8MatmulArgs &args, uint8_t *l) : a(args), lds(l)
    {
        tid = threadIdx.x;
        lane = tid % 64;
        wave = uniform(tid / 64);
        quarter = lane / 16;
        lr = lane % 16;
        int tile_m, tile_n;
        tile_of(a, &tile_m, &tile_n);
        m0 = (long long)tile_m * BM;
        n0 = (long long)tile_n * BN;
        ra0 = wave % WM * MT * 16;
        rb0 = wave / WM * NT * 16;
        rows_a = a.m - m0 < BM ? (int)(a.m - m0) : BM;
        rows_b = a.n - n0 < BN ? (int)(a.n - n0) : BN;
        kb0 = blockIdx.y * a.kb_split;
        kb1 = kb0 + a.kb_split < a.kb ? kb0 + a.kb_split : a.kb;
        kbytes = (uint32_t)(kb1 < a.kb ? kb1 * kFp8Block : a.k / 16 * 16);
        apart = kb1 == a.kb && a.k % 16;
        const uint32_t kceil = ((uint32_t)a.k + 15) / 16 * 16;
        // rows past the matrix lie past the buffers' ends and read as zero
        ra = make_buf_rsrc(a.a + m0 * a.a_pitch, (uint32_t)((rows_a - 1) * a.a_pitch) + kceil);
        rb = make_buf_rsrc(a.b + n0 * a.b_pitch, (uint32_t)((rows_b - 1) * a.b_pitch) + kceil);
        if (tid < BM) {
            scale_row = a.a_scale + (m0 + (tid < rows_a ? tid : rows_a - 1)) * a.kb;
        } else {
            const long long r = n0 + (tid - BM < rows_b ? tid - BM : rows_b - 1);
            scale_row = a.b_scale + (a.b_blocks ? r / kFp8Block : r) * a.kb;
        }
    }

    __device__ inline uint8_t *la(int buf) const { return lds + buf * BM * 128; }
    __device__ inline uint8_t *lb(int buf) const { return lds + 2 * BM * 128 + buf * BN * 128; }
    __device__ inline uint8_t *exps(int slot) const { return lds + 2 * ROWS * 128 + slot * THREADS; }
    __device__ inline i32x8 frag_a(int buf, int i) const { return fragment(la(buf), ra0 + i * 16 + lr, quarter); }
    __device__ inline i32x8 frag_b(int buf, int j) const { return fragment(lb(buf), rb0 + j * 16 + lr, quarter); }

    // Blocks past the end read as zeros.
    __device__ inline void stage(int kb, int buf) const
    {
        stage_rows<BM, THREADS>(ra, lds_addr(la(buf)), (uint32_t)a.a_pitch, kb * 128u, kbytes);
        stage_rows<BN, THREADS>(rb, lds_addr(lb(buf)), (uint32_t)a.b_pitch, kb * 128u, kbytes);
    }
    // Makes block kb visible to every wave, which has by then read all it needs
    // of block kb-1; that one's place then takes block kb+1.
    __device__ inline void arrive(int kb, int buf) const
    {
        wait_vm_all();
        __syncthreads();
        stage(kb + 1, buf ^ 1);
    }

    // The last chunk as block kb0 - 1, in place 0: a thread to a row.
    __device__ inline void stage_apart() const
    {
        if (tid >= ROWS) return;
        const int r = tid < BM ? tid : tid - BM;
        const uint8_t *p = tid < BM ? a.a + (m0 + r) * a.a_pitch : a.b + (n0 + r) * a.b_pitch;
        u32x4 v = {0, 0, 0, 0};
        if (r < (tid < BM ? rows_a : rows_b)) v = *(const u32x4 *)(p + a.k / 16 * 16);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int keep = a.k % 16 - d * 4;  // bytes of this word
            v[d] &= keep <= 0 ? 0u : keep >= 4 ? ~0u : (1u << (8 * keep)) - 1u;
        }
        u32x4 *row = (u32x4 *)((tid < BM ? la(0) : lb(0)) + r * 128);
#pragma unroll
        for (int c = 0; c < 8; ++c) row[c] = c == (r & 7) ? v : u32x4{0, 0, 0, 0};  // chunk 0 lies at place r & 7
    }
    __device__ inline int first() const { return kb0 - (apart ? 1 : 0); }
    __device__ inline void stage_first() const
    {
        if (apart) stage_apart();
        else stage(kb0, 0);
    }
    __device__ inline float scale_of(int kb) const { return scale_row[kb < kb0 || kb >= a.kb ? a.kb - 1 : kb]; }
    __device__ inline float2 load_scales(int kb) const { return float2{scale_of(kb), scale_of(kb + 1)}; }
    // Exponents of two blocks to slots slot and slot+1; 0 where there is none.
    __device__ inline void put_scales(int slot, float2 v) const
    {
        const int at = tid / 64 * 64 + tid % 16 * 4 + tid / 16 % 4, x = power_of_two(v.x), y = power_of_two(v.y);
        exps(slot)[at] = (uint8_t)(x < 0 ? 0 : x);
        exps(slot + 1)[at] = (uint8_t)(y < 0 ? 0 : y);
    }
    __device__ inline int exps_a(int slot, int i4) const { return *(const int *)(exps(slot) + ra0 + i4 * 64 + lr * 4); }
    __device__ inline int exps_b(int slot) const { return *(const int *)(exps(slot) + BM + rb0 + lr * 4); }

    // Whether all scales were powers of two and acc is the sum.
    __device__ inline bool scaled(f32x4 (&acc)[MT][NT]) const
    {
        // Slots 0, 1 and 2, 3 take turns: the pair after next is written while
        // one is at work and the next has been written.
        const int f = first();
        stage_first();
        put_scales(0, load_scales(f));
        float2 scales = load_scales(f + 2);
        arrive(f, 0);
        typename UNIT::Frag fb[NT];
        int eb = exps_b(0), ea[MT / 4];
        i32x8 raw;
        int ok = -1;  // bit 7 of each byte: every exponent so far was 64 or more
        each<NT>([&](auto j) { fb[j.value] = UNIT::template prepare<j.value>(frag_b(0, j.value), eb); });
#pragma unroll
        for (int i = 0; i < MT / 4; ++i) ea[i] = exps_a(0, i);
        raw = frag_a(0, 0);
        auto block = [&](int kb, auto odd, int pair) {
            constexpr int buf = decltype(odd)::value;
            // the next block's slot: the pair's second, or the other pair's first
            const int slot = buf == 0 ? pair + 1 : pair ^ 2;
            int nb = 0, na[MT / 4];
            ok &= eb | eb << 1;
#pragma unroll
            for (int i = 0; i < MT / 4; ++i) ok &= ea[i] | ea[i] << 1;
            each<MT>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                const auto fa = UNIT::template prepare<i % 4>(raw, ea[i / 4]);
                if (i + 1 < MT) raw = frag_a(buf, i + 1);
                if (i == MT - 2) {
                    if (buf == 0) put_scales(pair ^ 2, scales);
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    arrive(kb + 1, buf ^ 1);
                    // behind the block's loads: before them, arrive would wait for these
                    if (buf == 0) scales = load_scales(kb + 4);
                    nb = exps_b(slot);
#pragma unroll
                    for (int q = 0; q < MT / 4; ++q) na[q] = exps_a(slot, q);
                }
                if (i + 1 == MT) raw = frag_a(buf ^ 1, 0);
                each<NT>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    acc[i][j] = UNIT::template scaled<j, i % 4>(fb[j], fa, acc[i][j], eb, ea[i / 4]);
                    if (i + 1 == MT) fb[j] = UNIT::template prepare<j>(frag_b(buf ^ 1, j), nb);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            eb = nb;
#pragma unroll
            for (int i = 0; i < MT / 4; ++i) ea[i] = na[i];
        };
        for (int kb = f, pair = 0; kb < kb1; kb += 2, pair ^= 2) {
            block(kb, std::integral_constant<int, 0>{}, pair);
            block(kb + 1, std::integral_constant<int, 1>{}, pair);
        }
        wait_vm_all();  // blocks of zeros may still be on their way
        return !__syncthreads_or((ok & 0x80808080) != (int)0x80808080);
    }

    // Any scales: each block's sum times its rows' scales.  Half of a wave's
    // columns at a time: beside the other path's sums a whole tile's would spill.
    __device__ inline void general(int half) const
    {
        constexpr int NH = NT / 2;
        f32x4 acc[MT][NH];
        zero(acc);
        float *s = (float *)(lds + 2 * ROWS * 128);  // [2][THREADS]
        const int f = first();
        stage_first();
        for (int kb = f; kb < kb1; ++kb) {
            const int buf = (kb - f) & 1;
            s[buf * THREADS + tid] = scale_of(kb);
            arrive(kb, buf);
            const float *sa = s + buf * THREADS + ra0, *sb = s + buf * THREADS + BM + rb0 + half * NH * 16;
            typename UNIT::Frag fb[NH];
            f32x4 vb[NH];
#pragma unroll
            for (int j = 0; j < NH; ++j) {
                fb[j] = UNIT::prepare_plain(frag_b(buf, half * NH + j));
                vb[j] = *(const f32x4 *)(sb + j * 16 + quarter * 4);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const auto fa = UNIT::prepare_plain(frag_a(buf, i));
                const float va = sa[i * 16 + lr];
#pragma unroll
                for (int j = 0; j < NH; ++j) {
                    const f32x4 p = UNIT::plain(fb[j], fa, f32x4{0, 0, 0, 0});
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e] * va, vb[j][e], acc[i][j][e]);
                }
            }
        }
        wait_vm_all();
        __syncthreads();
        write(acc, half * NH * 16);
        __syncthreads();
    }

    template <int N>
    __device__ static inline void zero(f32x4 (&acc)[MT][N])
    {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    }

    // Out through LDS, 16 rows of a wave's columns at a time: a lane's four
    // neighbours alone would be written in pieces of 32 bytes.
    // N fragments of columns, from the wave's column `first` on.
    template <int N>
    __device__ inline void write(const f32x4 (&acc)[MT][N], int first) const
    {
        using S = typename E::S;
        constexpr int VEC = 16 / E::kBytes, COLS = N * 16, PER_ROW = COLS / VEC, PITCH = COLS * E::kBytes + 16;
        static_assert(64 % PER_ROW == 0 && WM * WN * 16 * PITCH <= 2 * ROWS * 128, "staging fits");
        uint8_t *mine = lds + wave * 16 * PITCH;
        const long long at = (long long)blockIdx.y * a.m * a.n;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                SVec<S, 4> r;
#pragma unroll
                for (int e = 0; e < 4; ++e) r.v[e] = E::from(acc[i][j][e]);
                __builtin_memcpy(__builtin_assume_aligned(mine + lr * PITCH + (j * 16 + quarter * 4) * E::kBytes, 4 * E::kBytes), &r, sizeof r);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int p = 0; p < 16 * PER_ROW / 64; ++p) {
                const int row = p * (64 / PER_ROW) + lane / PER_ROW, col = lane % PER_ROW * VEC;
                const SVec<S, VEC> v = __builtin_bit_cast(SVec<S, VEC>, *(const u32x4 *)(mine + row * PITCH + col * E::kBytes));
                const long long r = m0 + ra0 + i * 16 + row, c = n0 + rb0 + first + col;
                if (r >= a.m || c >= a.n) continue;
                S *o = (S *)a.out + at + r * a.ldo + c;
                if (c + VEC <= a.n) {
                    *(SVec<S, VEC> *)o = v;
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (c + e < a.n) o[e] = v.v[e];
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }
};

template <class E, class UNIT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64, 2) void fp8_tile_kernel(Fp8MatmulArgs a)
{
    typedef Tile<E, UNIT, BM, BN, WM, WN> T;
    extern __shared__ __align__(16) uint8_t lds[];
    const T t(a, lds);
    {
        f32x4 acc[T::MT][T::NT];
        T::zero(acc);
        if (t.kb0 >= t.kb1 || t.scaled(acc)) {
            t.write(acc, 0);
            return;
        }
    }
#pragma unroll 1
    for (int half = 0; half < 2; ++half) t.general(half);
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

// Products with few rows on one side ("small") stream the other side's rows
// ("big"): bound by its bytes.  A workgroup owns 16 big rows and up to 64 small
// ones (blockIdx.y), and its waves share the blocks of k, four (or two) of a wave's on their way at a time,
// straight to registers; their sums are added in order through LDS.  Scales are
// applied to each block's sum in fp32: there is time for it.
constexpr int kNarrow = 64;

struct NarrowArgs {
    const uint8_t *big, *small;
    const float *big_scale, *small_scale;
    long long big_pitch, small_pitch;
    int big_rows, small_rows, k, kb;
    int big_blocks, small_blocks;  // scales of 128 rows together
    int small_first;               // row of the small operand (within its matrix) that `small` starts at
    void *out;
    long long big_step, small_step;  // strides of out
};

template <class E, class UNIT, int MT, int BATCH>
__global__ __launch_bounds__(512) void fp8_narrow_kernel(NarrowArgs a)
{
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64), waves = blockDim.x / 64;
    const int lr = lane % 16, quarter = lane / 16;
    const int each_wave = (a.kb + waves - 1) / waves;
    const int kb0 = wave * each_wave, kb1 = kb0 + each_wave < a.kb ? kb0 + each_wave : a.kb;
    const long long b0 = (long long)blockIdx.x * 16;
    const int s0 = blockIdx.y * kNarrow, small_rows = a.small_rows - s0 < kNarrow ? a.small_rows - s0 : kNarrow;
    // rows past the matrix are its last row again; what they give is not written
    const long long brow = b0 + lr < a.big_rows ? b0 + lr : a.big_rows - 1;
    const uint8_t *pb = a.big + brow * a.big_pitch + quarter * 16;
    const float *sb = a.big_scale + (a.big_blocks ? brow / kFp8Block : brow) * a.kb;
    const uint8_t *ps[MT];
    const float *ss[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const long long r = s0 + (i * 16 + lr < small_rows ? i * 16 + lr : small_rows - 1);
        ps[i] = a.small + r * a.small_pitch + quarter * 16;
        ss[i] = a.small_scale + (a.small_blocks ? (a.small_first + r) / kFp8Block : a.small_first + r) * a.kb;
    }
    // 16 bytes at byte `at` of a row, those past k as zero
    auto chunk = [&](const uint8_t *p, int at) {
        u32x4 v = {0, 0, 0, 0};
        const int left = a.k - at - quarter * 16;
        if (left > 0) v = *(const u32x4 *)(p + at);
        if (left < 16) {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int keep = left - d * 4;
                v[d] &= keep <= 0 ? 0u : keep >= 4 ? ~0u : (1u << (8 * keep)) - 1u;
            }
        }
        return v;
    };
    struct Raw {
        u32x4 lo, hi;
    };
    auto load = [&](const uint8_t *p, int kb) { return Raw{chunk(p, kb * 128), chunk(p, kb * 128 + 64)}; };
    auto join = [](const Raw &r) {
        i32x8 f;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            f[d] = (int)r.lo[d];
            f[d + 4] = (int)r.hi[d];
        }
        return f;
    };
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0, 0, 0, 0};
    Raw big[BATCH], small[BATCH][MT];
    // lane (row, q) has the scales of block q of a batch; the others get them from it
    float vb, vs[MT];
    auto fetch = [&](int kb) {
        const int mine = kb + quarter;
        const bool have = quarter < BATCH && mine < kb1;
        vb = have ? sb[mine] : 0.0f;
#pragma unroll
        for (int i = 0; i < MT; ++i) vs[i] = have ? ss[i][mine] : 0.0f;
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
            if (kb + u < kb1) {
                big[u] = load(pb, kb + u);
#pragma unroll
                for (int i = 0; i < MT; ++i) small[u][i] = load(ps[i], kb + u);
            }
    };
    if (kb0 < kb1) fetch(kb0);
    for (int kb = kb0; kb < kb1; kb += BATCH) {
        Raw nb[BATCH], ns[BATCH][MT];
        const float cb = vb;
        float cs[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) cs[i] = vs[i];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            nb[u] = big[u];
#pragma unroll
            for (int i = 0; i < MT; ++i) ns[u][i] = small[u][i];
        }
        if (kb + BATCH < kb1) fetch(kb + BATCH);
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            if (kb + u >= kb1) break;
            const auto fb = UNIT::prepare_plain(join(nb[u]));
            f32x4 wb;
#pragma unroll
            for (int e = 0; e < 4; ++e) wb[e] = __shfl(cb, 16 * u + quarter * 4 + e);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const f32x4 p = UNIT::plain(fb, UNIT::prepare_plain(join(ns[u][i])), f32x4{0, 0, 0, 0});
                const float w = __shfl(cs[i], 16 * u + lr);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(p[e] * w, wb[e], acc[i][e]);
            }
        }
    }
    f32x4 *part = (f32x4 *)lds;  // [waves][MT][64]
#pragma unroll
    for (int i = 0; i < MT; ++i) part[(wave * MT + i) * 64 + lane] = acc[i];
    __syncthreads();
    for (int t = tid; t < MT * 64; t += blockDim.x) {
        f32x4 v = {0, 0, 0, 0};
        for (int w = 0; w < waves; ++w) {
            const f32x4 p = part[w * MT * 64 + t];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += p[e];
        }
        const int s = t / 64 * 16 + t % 16;
        const long long b = b0 + t % 64 / 16 * 4;
        if (s >= small_rows) continue;
        typename E::S *o = (typename E::S *)a.out + (s0 + s) * a.small_step;
        if (a.big_step == 1 && b + 4 <= a.big_rows) {
            const float r[4] = {v[0], v[1], v[2], v[3]};
            store_vec<E, 4>(o + b, 4, r);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (b + e < a.big_rows) o[(b + e) * a.big_step] = E::from(v[e]);
        }
    }
}

// Waves along k: where there are so many blocks at least two each, and no more
// than fill the chip.
int narrow_waves(long long workgroups, int kb)
{
    int waves = 4;
    if (workgroups * waves < 4096 && kb >= waves * 2) waves = 8;
    while (waves > 1 && waves > kb) waves /= 2;
    return waves;
}

template <class E, class UNIT>
hipError_t launch_narrow(const NarrowArgs &a, hipStream_t st)
{
    const int groups = (a.big_rows + 15) / 16, parts = (a.small_rows + kNarrow - 1) / kNarrow;
    const int mt = parts > 1 ? 4 : (a.small_rows + 15) / 16, waves = narrow_waves((long long)groups * parts, a.kb);
    auto run = [&](auto mtc, auto batch) {
        constexpr int MT = decltype(mtc)::value;
        fp8_narrow_kernel<E, UNIT, MT, decltype(batch)::value><<<dim3((unsigned)groups, (unsigned)parts), waves * 64, waves * MT * 1024, st>>>(a);
        return hipGetLastError();
    };
    using std::integral_constant;
    if (mt <= 1) return run(integral_constant<int, 1>{}, integral_constant<int, 4>{});
    if (mt == 2) return run(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    return run(integral_constant<int, 4>{}, integral_constant<int, 1>{});
}

// The small side's rows from `first` on.
template <class E, class UNIT>
hipError_t narrow_rows_of_a(const Fp8MatmulArgs &a, int first, int n, hipStream_t st)
{
    const NarrowArgs q = {a.b, a.a + first * a.a_pitch, a.b_scale, a.a_scale, a.b_pitch, a.a_pitch, n, a.m - first, a.k, a.kb,
                          a.b_blocks, 0, first, (typename E::S *)a.out + first * a.ldo, 1, a.ldo};
    return launch_narrow<E, UNIT>(q, st);
}
template <class E, class UNIT>
hipError_t narrow_rows_of_b(const Fp8MatmulArgs &a, int first, hipStream_t st)
{
    const NarrowArgs q = {a.a, a.b + first * a.b_pitch, a.a_scale, a.b_scale, a.a_pitch, a.b_pitch, a.m, a.n - first, a.k, a.kb,
                          0, a.b_blocks, first, (typename E::S *)a.out + first, a.ldo, 1};
    return launch_narrow<E, UNIT>(q, st);
}

struct TileCost {
    int bm, bn, threads, per_cu;
    double step16, step32;  // microseconds per block of 128 for per_cu tiles at a time: 16-bit results, float32
};
// Measured on 4096 x 8192 x 4096, normal data: 256 x 256 138-144 us, 128 x 128 165 us.
// On constant operands, which take less power: 121 and 140 (float32 results 128 x 128
// 214-220, 256 x 256 314: it spills); the steps below are from those.
static constexpr TileCost kTiles[] = {{256, 256, 512, 1, 1.95, 0}, {128, 128, 256, 2, 1.07, 1.7}};

double tiles_time(const TileCost &s, double step, long long m, long long n, int per, int splits)
{
    const long long tiles = (m + s.bm - 1) / s.bm * ((n + s.bn - 1) / s.bn), slots = 256 * s.per_cu;
    const long long rounds = (tiles * splits + slots - 1) / slots;
    // the last round's tiles have the compute units to themselves
    const long long last = tiles * splits - (rounds - 1) * slots;
    const double alone = s.per_cu > 1 && last <= 256 ? 0.65 : 1.0;
    return 6.0 + ((rounds - 1) + alone) * (per * step + 3.0);
}

}  // namespace

// How a product is cut.  Few rows on either side, or little work: the narrow kernel.  Else tiles
// of the shape that takes least time by the steps above, in whole rounds over the
// chip; with a few rows past whole tiles on either side left to the narrow kernel
// where that saves more than its pass over the other operand takes; and with k
// split where there are few tiles, for the partial sums' traffic.
Fp8Plan fp8_matmul_plan(int m, int n, int k, int dtype)
{
    const int kb = (k + kFp8Block - 1) / kFp8Block;
    Fp8Plan best = {};
    best.splits = 1;
    best.per = kb;
    if (m <= kNarrow || n <= kNarrow) {
        best.narrow_m = m <= kNarrow;
        best.narrow_n = !best.narrow_m;
        return best;
    }
    // Small products all through the narrow kernel, which needs no partial sums:
    // measured 3.5 us, and 1.8 us (float32 results, which convert 80 rows to bf16:
    // 4.5 us) a block of a wave's, three workgroups to a compute unit at a time.
    const long long groups = (n + 15LL) / 16 * ((m + kNarrow - 1LL) / kNarrow);
    const int waves = narrow_waves(groups, kb);
    double best_t = std::max(1.0, groups / 768.0) * (3.5 + (dtype == CONV2D_DTYPE_F32 ? 4.5 : 1.8) * ((kb + waves - 1) / waves));
    if ((m + kNarrow - 1LL) / kNarrow <= 65535) best.all = best.narrow_m = true;
    else best_t = 1e30;
    for (int shape = 0; shape < 2; ++shape) {
        const TileCost &s = kTiles[shape];
        const double step = dtype == CONV2D_DTYPE_F32 ? s.step32 : s.step16;
        if (step == 0) continue;
        for (int cut = 0; cut < 4; ++cut) {
            const int cm = cut & 1, cn = cut >> 1, rm = m % s.bm, rn = n % s.bn;
            if ((cm && (rm == 0 || rm > kNarrow || m < s.bm)) || (cn && (rn == 0 || rn > kNarrow || n < s.bn))) continue;
            const long long mm = m - (cm ? rm : 0), nn = n - (cn ? rn : 0);
            const double extra = (cm ? 4.0 + (double)nn * k / 3e6 : 0) + (cn ? 4.0 + (double)m * k / 3e6 : 0);
            for (int split = 1; split <= 32 && split <= std::max(kb, 1); ++split) {
                const int per = (kb + split - 1) / split;
                if (split > 1 && (per < 4 || (kb + per - 1) / per != split || cm || cn)) continue;
                double t = extra + tiles_time(s, step, mm, nn, per, split);
                if (split > 1) t += 3.0 + (double)m * n * 4 * (2 * split + 1) / 5e6;
                if (t < best_t) {
                    best_t = t;
                    best.all = false;
                    best.shape = shape;
                    best.splits = split;
                    best.per = per;
                    best.narrow_m = cm;
                    best.narrow_n = cn;
                }
            }
        }
    }
    return best;
}

bool fp8_matmul_fits(int m, int n, int k, const Fp8Plan &p)
{
    auto narrow = [&](long long big, long long small) {
        const long long groups = (big + 15) / 16, parts = (small + kNarrow - 1) / kNarrow;
        return parts <= 65535 && fits(groups, narrow_waves(groups * parts, (k + kFp8Block - 1) / kFp8Block) * 64);
    };
    if (p.all || (p.narrow_m && m <= kNarrow)) return narrow(n, m);
    if (p.narrow_n && n <= kNarrow) return narrow(m, n);
    const TileCost &s = kTiles[p.shape];
    const long long rm = p.narrow_m ? m % s.bm : 0, rn = p.narrow_n ? n % s.bn : 0;
    const long long tiles = (m - rm + s.bm - 1) / s.bm * ((n - rn + s.bn - 1) / s.bn);
    return fits(tiles, s.threads) && (p.splits == 1 || fits(((long long)m * n + 1023) / 1024, 256)) &&
           (!rm || narrow(n - rn, rm)) && (!rn || narrow(m, rn));
}

size_t fp8_matmul_bytes(int m, int n, const Fp8Plan &p) { return p.splits > 1 ? (size_t)p.splits * m * n * 4 : 0; }

template <class E, class UNIT>
static hipError_t launch_tiles(Fp8MatmulArgs a, const Fp8Plan &p, hipStream_t st)
{
    auto run = [&](auto bm, auto bn, auto wm, auto wn) {
        constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, WN = decltype(wn)::value;
        a.tiles_m = (a.m + BM - 1) / BM;
        a.tiles_n = (a.n + BN - 1) / BN;
        constexpr int lds = Tile<E, UNIT, BM, BN, WM, WN>::kLds;
        static_assert(kTiles[BM == 256 ? 0 : 1].bm == BM && kTiles[BM == 256 ? 0 : 1].threads == WM * WN * 64, "as fp8_matmul_fits counts");
        auto *kernel = fp8_tile_kernel<E, UNIT, BM, BN, WM, WN>;
        hipError_t r = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (r != hipSuccess) return r;
        const dim3 grid((unsigned)((long long)a.tiles_m * a.tiles_n), (unsigned)p.splits);
        kernel<<<grid, WM * WN * 64, lds, st>>>(a);
        return hipGetLastError();
    };
    using std::integral_constant;
    constexpr bool BIG = std::is_same<UNIT, Fp8Unit>::value;
    if constexpr (BIG)
        if (p.shape == 0)
            return run(integral_constant<int, 256>{}, integral_constant<int, 256>{}, integral_constant<int, 2>{}, integral_constant<int, 4>{});
    return run(integral_constant<int, 128>{}, integral_constant<int, 128>{}, integral_constant<int, 2>{}, integral_constant<int, 2>{});
}

template <class E, class UNIT>
static hipError_t launch_parts(Fp8MatmulArgs a, const Fp8Plan &p, hipStream_t st)
{
    if (p.all || (p.narrow_m && a.m <= kNarrow)) return narrow_rows_of_a<E, UNIT>(a, 0, a.n, st);
    if (p.narrow_n && a.n <= kNarrow) return narrow_rows_of_b<E, UNIT>(a, 0, st);
    const TileCost &s = kTiles[p.shape];
    const int mm = p.narrow_m ? a.m / s.bm * s.bm : a.m, nn = p.narrow_n ? a.n / s.bn * s.bn : a.n;
    if (mm < a.m) {
        const hipError_t r = narrow_rows_of_a<E, UNIT>(a, mm, nn, st);
        if (r != hipSuccess) return r;
    }
    if (nn < a.n) {
        const hipError_t r = narrow_rows_of_b<E, UNIT>(a, nn, st);
        if (r != hipSuccess) return r;
    }
    a.m = mm;
    a.n = nn;
    return launch_tiles<E, UNIT>(a, p, st);
}

hipError_t launch_fp8_matmul(int dtype, const Fp8MatmulArgs &args, const Fp8Plan &p, void *workspace, hipStream_t st)
{
    Fp8MatmulArgs a = args;
    a.kb_split = p.per;
    a.ldo = a.n;
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
    if (dtype == CONV2D_DTYPE_F16) return launch_parts<SF16, Fp8Unit>(a, p, st);
    if (dtype == CONV2D_DTYPE_BF16) return launch_parts<SBF16, Fp8Unit>(a, p, st);
    return launch_parts<SF32, Bf16Unit>(a, p, st);
}

}  // namespace cnv
