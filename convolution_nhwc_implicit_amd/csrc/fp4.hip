// fp4.hip -- 4-bit operands: quantisation, and products of few rows with them.
//
//   out[i][j] = sum_k x[i][k] * e2m1(w[j][k]) * 2^(scale[j][k / 32] - 127)
//
// The product is bound by the weights' bytes.  They go from memory to the matrix unit in
// registers: a lane loads 16 bytes, one group of 32 values, of one row of w, and the
// conversion instruction turns two values at a time into 16 bits with the group's scale
// applied, which is exact.  The matrix instruction sums over k in any order as long as
// both operands have the same, so x is loaded to match.  fp32 x is the sum of three bf16
// values, exactly, so that all products are exact and all sums fp32.  The waves of a
// workgroup take parts of k and are added through LDS in order.
//
// One row of x by 8192 x 4096 takes 7.2 us, a launch's latency and 18 MB (2.5 TB/s); by
// 32768 x 8192 41 us (3.5 TB/s, some 70 % of the copy's rate).  Waves that take 128 bytes
// of a row of w at a time in place of 64 change nothing (42.7 and 44.4 us).
#include <algorithm>
#include <type_traits>

#include "block_internal.h"

namespace cnv {
namespace {

// ---- quantisation ----------------------------------------------------------------
// four lanes to a group of 32 values, 8 each; 8192 x 4096 bf16 27 us (3.1 TB/s): weights are
// laid out once
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
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// How x meets the weights: bf16 and fp16 as they are (the weights in the same type), or
// as a sum of PARTS bf16 values.
struct AsBF16 {
    static constexpr int kParts = 1;
    static constexpr bool kF16 = false;
};
struct AsF16 {
    static constexpr int kParts = 1;
    static constexpr bool kF16 = true;
};
template <int PARTS>
struct AsParts {
    static constexpr int kParts = PARTS;
    static constexpr bool kF16 = false;
};

// Whether fp16 cannot hold e2m1 values with this scale, 0.5 * 2^-23 to 6 * 2^13.  The scale
// of a group of zeros, 2^-127, does not count: whatever it scales, times any fp16 value, is
// nothing to an fp16 sum.  A workgroup that meets such a scale walks all of k again with x in two
// parts: with one among the weights 1 x 8192 x 4096 takes 15 us for 8, 48 x 8200 x 4104 68 for 17.
__device__ inline bool too_wide(uint32_t e) { return e - 104u > 36u && e != 0; }

// eight e2m1 values in 16 bits, times the power of two whose exponent field is scale's
template <class How>
__device__ inline u32x4 weights8(uint32_t w, float scale)
{
    u32x4 r;
    if constexpr (How::kF16) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3));
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    }
    return r;
}

// Eight values of x as they lie in memory.
template <class E>
struct Eight {
    SVec<typename E::S, 8> v;
    __device__ inline void load(const typename E::S *p) { v = *(const SVec<typename E::S, 8> *)p; }
    // The 8 values that begin at c of a row of k, zeros past its end.  EIGHTS: k is a
    // multiple of 8, so that all or none are there.
    template <bool EIGHTS>
    __device__ inline void load(const typename E::S *row, int c, int k)
    {
        if (EIGHTS) {
            load(row + (c < k ? c : 0));
#pragma unroll
            for (int i = 0; i < 8; ++i) v.v[i] = c < k ? v.v[i] : (typename E::S)0;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const typename E::S e = row[c + i < k ? c + i : 0];
                v.v[i] = c + i < k ? e : (typename E::S)0;
            }
        }
    }
    // As a sum of bf16 values: the high half of a value, then that of what is left of it.
    template <class How>
    __device__ inline void parts(u32x4 (&out)[How::kParts]) const
    {
        if constexpr (How::kParts == 1) {
            out[0] = __builtin_bit_cast(u32x4, v);
        } else {
            uint32_t f[8], top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = __builtin_bit_cast(uint32_t, E::to(v.v[i]));
                const uint32_t size = f[i] & 0x7fffffffu;
                top = top > size ? top : size;
            }
            // an infinity is its own high half, and so is a NaN once it is a plain one
            const bool spoilt = __any(top >= 0x7f800000u);
#pragma unroll
            for (int s = 0; s < How::kParts; ++s) {
                if (spoilt)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t size = f[i] & 0x7fffffffu;
                        if (size > 0x7f800000u) f[i] = s == 0 ? 0x7fc00000u : 0u;
                        if (s > 0 && size == 0x7f800000u) f[i] = 0u;
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) out[s][i] = __builtin_amdgcn_perm(f[2 * i + 1], f[2 * i], 0x07060302u);
                if (s + 1 < How::kParts)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t high = f[i] & 0xffff0000u;
                        if (spoilt && (high & 0x7f800000u) == 0x7f800000u) continue;
                        f[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, f[i]) - __builtin_bit_cast(float, high));
                    }
            }
        }
    }
};

constexpr int kWaves = 8, kStep = 4;  // groups that the four lanes of a row load together
// Steps whose weights are under way together.
constexpr int steps_ahead(int mt, int nt) { return mt * nt == 1 ? 4 : 2; }

// Four groups of a row of w, one in each of the four lanes that share the row, to the
// same eight values of each group in each of them: registers and lanes change places.
__device__ inline void turn(u32x4 &q)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(q[i], q[i + 2], false, false));
        q[i] = r[0];
        q[i + 2] = r[1];
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(q[i], q[i + 1], false, false));
        q[i] = r[0];
        q[i + 1] = r[1];
    }
}

// The scales of groups g .. g + 3 of a row, a byte each; 1 past the last one.
__device__ inline uint32_t scales4(const uint8_t *sc, int g, int groups)
{
    if (groups < kStep) {
        uint32_t r = 0;
        for (int j = 0; j < kStep; ++j) r |= (g + j < groups ? (uint32_t)sc[g + j] : 127u) << (8 * j);
        return r;
    }
    const int from = g < groups - kStep ? g : groups - kStep, past = g - from;
    const uint32_t r = __builtin_bit_cast(uint32_t, *(const SVec<uint8_t, 4> *)(sc + from));
    return past >= kStep ? 0x7f7f7f7fu : past > 0 ? r >> (8 * past) | 0x7f7f7f7fu << (32 - 8 * past) : r;
}

// The wave's part of the sums for MT tiles of 16 rows of x and NT tiles of 16 rows of w,
// 128 values of k a step: matrix instruction j of a step takes its group j, 8 values to
// each of a row's four lanes, so that they read 64 bytes of x side by side.  Returns
// whether a scale lies outside what fp16 weights can hold (AsF16).
template <class E, class How, int MT, int NT>
__device__ inline bool fp4_wave(const Fp4MatmulArgs &a, int m0, int n0, f32x4 (&acc)[MT][NT])
{
    typedef typename E::S S;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), row = lane % 16, quarter = lane / 16;
    const uint8_t *w[NT], *sc[NT];
    const S *x[MT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int j = n0 + t * 16 + row, c = j < a.n ? j : a.n - 1;
        w[t] = a.w + (long long)c * a.w_pitch + quarter * 16;
        sc[t] = a.w_scale + (long long)c * a.groups;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int i = m0 + t * 16 + row;
        x[t] = (const S *)a.x + (long long)(i < a.m ? i : a.m - 1) * a.x_row + quarter * 8;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) acc[t][u] = f32x4{0, 0, 0, 0};
    bool wide = false;
    Eight<E> xv[MT][kStep];
    // matrix instructions of a step; refill(t, j): xv[t][j] has been used
    auto step_of = [&](u32x4 (&q)[NT], const uint32_t (&sb)[NT], auto refill) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < NT; ++u) turn(q[u]);
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
            u32x4 b[NT];
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const uint32_t e = sb[u] >> (8 * j) & 255u;
                if (How::kF16) wide = wide || too_wide(e);
                b[u] = weights8<How>(q[u][j], __builtin_bit_cast(float, e << 23));
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                u32x4 xs[How::kParts];
                xv[t][j].template parts<How>(xs);
                refill(t, j);
#pragma unroll
                for (int p = How::kParts - 1; p >= 0; --p)
#pragma unroll
                    for (int u = 0; u < NT; ++u) {
                        if constexpr (How::kF16) acc[t][u] = EF16::mfma(xs[p], b[u], acc[t][u]);
                        else acc[t][u] = EBF16::mfma(xs[p], b[u], acc[t][u]);
                    }
            }
        }
    };
    // whole steps to the waves in turn; what is left of k to the last one
    constexpr int kAhead = steps_ahead(MT, NT);
    const int steps = a.k / (kStep * kFp4Group), first = wave, last = steps;
    if (first < last) {
        u32x4 q[kAhead][NT];
        uint32_t sb[kAhead][NT];
        auto load_w = [&](int slot, int step) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                q[slot][u] = *(const u32x4 *)(w[u] + (long long)step * (kStep * 16));
                sb[slot][u] = __builtin_bit_cast(uint32_t, *(const SVec<uint8_t, 4> *)(sc[u] + (long long)step * kStep));
            }
        };
        auto load_x = [&](int t, int j, int step) { xv[t][j].load(x[t] + (long long)step * (kStep * kFp4Group) + j * kFp4Group); };
#pragma unroll
        for (int s = 0; s < kAhead; ++s) load_w(s, first + s * kWaves < last ? first + s * kWaves : first);
#pragma unroll
        for (int j = 0; j < kStep; ++j)
#pragma unroll
            for (int t = 0; t < MT; ++t) load_x(t, j, first);
        for (int s0 = first; s0 < last; s0 += kAhead * kWaves)
#pragma unroll
            for (int s = 0; s < kAhead; ++s) {
                const int step = s0 + s * kWaves;
                if (step < last) {
                    const int next = step + kWaves < last ? step + kWaves : step;
                    step_of(q[s], sb[s], [&](int t, int j) { load_x(t, j, next); });
                    if (step + kAhead * kWaves < last) load_w(s, step + kAhead * kWaves);
                }
            }
    }
    if (steps * kStep < a.groups && wave == kWaves - 1) {
        u32x4 q[NT];
        uint32_t sb[NT];
        // lanes past the last group take it again, with zeros of x
        const int g = steps * kStep, mine = g + quarter < a.groups ? g : a.groups - 1 - quarter;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            q[u] = *(const u32x4 *)(w[u] + (long long)mine * 16);
            sb[u] = scales4(sc[u], g, a.groups);
        }
        auto tail = [&](auto eights) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int j = 0; j < kStep; ++j)
                    xv[t][j].template load<decltype(eights)::value>(x[t] - quarter * 8, (g + j) * kFp4Group + quarter * 8, a.k);
        };
        if (a.k % 8 == 0) tail(std::true_type{});
        else tail(std::false_type{});
        step_of(q, sb, [](int, int) {});
    }
    return wide;
}

template <class E, int MT, int NT>
__global__ __launch_bounds__(64 * kWaves) void fp4_matmul_kernel(Fp4MatmulArgs a)
{
    __shared__ f32x4 part[kWaves][MT * NT][64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, row = lane % 16, quarter = lane / 16;
    const int n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
    f32x4 acc[MT][NT];
    if constexpr (std::is_same_v<E, SF16>) {
        // weights that fp16 cannot hold meet x in two bf16 parts instead
        if (__syncthreads_or(fp4_wave<E, AsF16, MT, NT>(a, m0, n0, acc))) fp4_wave<E, AsParts<2>, MT, NT>(a, m0, n0, acc);
    } else if constexpr (std::is_same_v<E, SBF16>) {
        fp4_wave<E, AsBF16, MT, NT>(a, m0, n0, acc);
    } else {
        fp4_wave<E, AsParts<3>, MT, NT>(a, m0, n0, acc);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) part[wave][t * NT + u][lane] = acc[t][u];
    __syncthreads();
    // a lane holds column `row` and rows 4 * quarter .. + 3 of a tile
    for (int t = wave; t < MT * NT; t += kWaves) {
        f32x4 s = part[0][t][lane];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) s += part[v][t][lane];
        const int j = n0 + t % NT * 16 + row;
        if (j < a.n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = m0 + t / NT * 16 + quarter * 4 + r;
                if (i < a.m) ((typename E::S *)a.out)[(long long)i * a.n + j] = E::from(s[r]);
            }
    }
}

// Many rows of x: they, not the weights, would be what a workgroup of 16 or 32 rows of w
// mostly reads.  Here four waves of 32 rows of w each share x, which goes through LDS
// 256 values of k a turn (twice: the next turn's is written while one is used; the one
// after that is under way), and workgroups split k, so that each reads a part of x only.
// 48 rows by 8200 x 4104, fp16: 14.6 us, of which the matrix unit needs 2.4 and the bytes
// 3.7: a workgroup has three or four turns, whose loads nothing covers at first.
constexpr int kManyWaves = 4, kManyTiles = 2, kManyRows = 16 * kManyTiles * kManyWaves;
constexpr int kManyPass = 64 * kManyWaves / 32;  // rows of x that the threads read together
constexpr int kTurn = 2 * kStep * kFp4Group;  // values of k
constexpr int kLine = kTurn * 2 + 16;         // bytes of a row of x in LDS: 16 more, to change banks from row to row

template <class E, class How, int MT>
__device__ inline bool fp4_many(const Fp4MatmulArgs &a, int m0, int n0, uint8_t *lds, f32x4 (&acc)[MT][kManyTiles])
{
    typedef typename E::S S;
    constexpr int kTile = MT * 16 * kLine, kAhead = 2, NT = kManyTiles, XT = MT * 16 / kManyPass;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), row = lane % 16, quarter = lane / 16;
    const uint8_t *w[NT], *sc[NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
        const int j = n0 + (wave * NT + u) * 16 + row, c = j < a.n ? j : a.n - 1;
        w[u] = a.w + (long long)c * a.w_pitch;
        sc[u] = a.w_scale + (long long)c * a.groups;
    }
    // a thread's part of a turn's x: 8 values of rows r0, r0 + kManyPass, ..
    const int part = threadIdx.x % 32 * 8, r0 = threadIdx.x / 32;
    const S *x[XT];
#pragma unroll
    for (int t = 0; t < XT; ++t) {
        const int i = m0 + t * kManyPass + r0;
        x[t] = (const S *)a.x + (long long)(i < a.m ? i : a.m - 1) * a.x_row + part;
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) acc[t][u] = f32x4{0, 0, 0, 0};
    bool wide = false;
    auto put_x = [&](int buf, const Eight<E> (&v)[XT]) __attribute__((always_inline)) {
        uint8_t *p = lds + buf * kTile + r0 * kLine + part * 2;
#pragma unroll
        for (int t = 0; t < XT; ++t) *(u32x4 *)(p + t * kManyPass * kLine) = __builtin_bit_cast(u32x4, v[t].v);
    };
    auto use = [&](int buf, const u32x4 (&q)[2][NT], const uint32_t (&es)[2][NT]) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 qs[NT];
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                qs[u] = q[h][u];
                turn(qs[u]);
            }
            const uint8_t *p = lds + buf * kTile + row * kLine + quarter * 16 + h * (kStep * 64);
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                u32x4 b[NT];
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    const uint32_t e = es[h][u] >> (8 * j) & 255u;
                    if (How::kF16) wide = wide || too_wide(e);
                    b[u] = weights8<How>(qs[u][j], __builtin_bit_cast(float, e << 23));
                }
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    Eight<E> v;
                    v.v = __builtin_bit_cast(decltype(v.v), *(const u32x4 *)(p + t * 16 * kLine + j * 64));
                    u32x4 xs[How::kParts];
                    v.template parts<How>(xs);
#pragma unroll
                    for (int i = How::kParts - 1; i >= 0; --i)
#pragma unroll
                        for (int u = 0; u < NT; ++u) {
                            if constexpr (How::kF16) acc[t][u] = EF16::mfma(xs[i], b[u], acc[t][u]);
                            else acc[t][u] = EBF16::mfma(xs[i], b[u], acc[t][u]);
                        }
                }
            }
        }
    };
    // this workgroup's whole turns, and what is left of k behind the last one's
    const int whole = a.k / kTurn, first = blockIdx.y * a.per, last = first + a.per < whole ? first + a.per : whole;
    const bool rest = (int)blockIdx.y == a.splits - 1 && whole * kTurn < a.k;
    Eight<E> xv[2][XT];
    u32x4 q[kAhead][2][NT];
    uint32_t sb[kAhead][2][NT];
    // of a turn past the last one: the last one's again
    auto load_x = [&](int slot, int k) __attribute__((always_inline)) {
        const long long c = (long long)(k < last ? k : last - 1) * kTurn;
#pragma unroll
        for (int t = 0; t < XT; ++t) xv[slot][t].load(x[t] + c);
    };
    auto load_w = [&](int slot, int k) __attribute__((always_inline)) {
        const int g = (k < last ? k : last - 1) * (2 * kStep);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                q[slot][h][u] = *(const u32x4 *)(w[u] + (long long)(g + h * kStep + quarter) * 16);
                sb[slot][h][u] = __builtin_bit_cast(uint32_t, *(const SVec<uint8_t, 4> *)(sc[u] + g + h * kStep));
            }
    };
    if (first < last) {
#pragma unroll
        for (int s = 0; s < kAhead; ++s) load_w(s, first + s);
        load_x(0, first);
        load_x(1, first + 1);
    }
    if (rest) {  // first, while the whole turns' values are on their way
        const int g = whole * (2 * kStep), end = a.groups - 1;
        Eight<E> v[XT];
        auto load_rest = [&](auto eights) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < XT; ++t) v[t].template load<decltype(eights)::value>(x[t] - part, whole * kTurn + part, a.k);
        };
        if (a.k % 8 == 0) load_rest(std::true_type{});
        else load_rest(std::false_type{});
        // lanes past the last group take it again, with zeros of x
        u32x4 tail[2][NT];
        uint32_t es[2][NT];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const int gl = g + h * kStep + quarter;
                tail[h][u] = *(const u32x4 *)(w[u] + (long long)(gl < end ? gl : end) * 16);
                es[h][u] = scales4(sc[u], g + h * kStep, a.groups);
            }
        put_x(1, v);
        __syncthreads();
        use(1, tail, es);
    }
    if (first < last) {
        put_x(0, xv[0]);
        __syncthreads();
        for (int s0 = first; s0 < last; s0 += kAhead)
#pragma unroll
            for (int s = 0; s < kAhead; ++s)
                if (s0 + s < last) {
                    load_x(s % 2, s0 + s + 2);
                    use(s % 2, q[s], sb[s]);
                    load_w(s, s0 + s + kAhead);
                    put_x((s + 1) % 2, xv[(s + 1) % 2]);
                    __syncthreads();
                }
    }
    return wide;
}

template <class E, int MT>
__global__ __launch_bounds__(64 * kManyWaves) void fp4_many_kernel(Fp4MatmulArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * MT * 16 * kLine];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, row = lane % 16, quarter = lane / 16;
    const int n0 = blockIdx.x * kManyRows, m0 = blockIdx.z * (16 * MT);
    f32x4 acc[MT][kManyTiles];
    if constexpr (std::is_same_v<E, SF16>) {
        // weights that fp16 cannot hold meet x in two bf16 parts instead
        if (__syncthreads_or(fp4_many<E, AsF16, MT>(a, m0, n0, lds, acc))) fp4_many<E, AsParts<2>, MT>(a, m0, n0, lds, acc);
    } else {
        fp4_many<E, AsBF16, MT>(a, m0, n0, lds, acc);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < kManyTiles; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = m0 + t * 16 + quarter * 4 + r, j = n0 + (wave * kManyTiles + u) * 16 + row;
                if (i < a.m && j < a.n) {
                    if (a.splits > 1) a.partial[((long long)blockIdx.y * a.m + i) * a.n + j] = acc[t][u][r];
                    else ((typename E::S *)a.out)[(long long)i * a.n + j] = E::from(acc[t][u][r]);
                }
            }
}

// the splits' sums in order, four values to a thread
template <class E>
__global__ __launch_bounds__(256) void fp4_sum_kernel(Fp4MatmulArgs a)
{
    const long long size = (long long)a.m * a.n, i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= size) return;
    const int have = size - i < 4 ? (int)(size - i) : 4;
    float s[4], v[4];
    load_vec<SF32, 4>(a.partial + i, have, s);
#pragma unroll 4
    for (int p = 1; p < a.splits; ++p) {
        load_vec<SF32, 4>(a.partial + p * size + i, have, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += v[k];
    }
    store_vec<E, 4>((typename E::S *)a.out + i, have, s);
}

template <class E>
hipError_t launch_product(const Fp4MatmulArgs &a, hipStream_t st)
{
    using std::integral_constant;
    const int tiles = (a.m + 15) / 16;
    if constexpr (!std::is_same_v<E, SF32>) {
        if (a.splits > 0) {
            auto go = [&](auto mt) {
                constexpr int MT = decltype(mt)::value;
                fp4_many_kernel<E, MT><<<dim3((unsigned)((a.n + kManyRows - 1) / kManyRows), (unsigned)a.splits, (unsigned)((tiles + MT - 1) / MT)),
                                         64 * kManyWaves, 0, st>>>(a);
            };
            if (tiles == 1) go(integral_constant<int, 1>{});
            else if (tiles == 2) go(integral_constant<int, 2>{});
            else if (tiles == 3) go(integral_constant<int, 3>{});
            else go(integral_constant<int, 4>{});
            if (hipError_t e = hipGetLastError()) return e;
            if (a.splits > 1) fp4_sum_kernel<E><<<(unsigned)(((long long)a.m * a.n + 1023) / 1024), 256, 0, st>>>(a);
            return hipGetLastError();
        }
    }
    auto go = [&](auto mt, auto nt) {
        constexpr int MT = decltype(mt)::value, NT = decltype(nt)::value;
        fp4_matmul_kernel<E, MT, NT><<<dim3((unsigned)((a.n + 16 * NT - 1) / (16 * NT)), (unsigned)((tiles + MT - 1) / MT)), 64 * kWaves, 0, st>>>(a);
    };
    if (a.tiles == 1 && tiles == 1) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else if (tiles == 1) go(integral_constant<int, 1>{}, integral_constant<int, 2>{});
    else if (tiles == 2) go(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    else if (tiles == 3) go(integral_constant<int, 3>{}, integral_constant<int, 2>{});
    else go(integral_constant<int, 4>{}, integral_constant<int, 2>{});
    return hipGetLastError();
}

}  // namespace

// Few rows of x: workgroups of all of k for 32 rows of w, or 16 where that would leave
// compute units without one (4 x 4096 x 4096 takes 5.8 us so and 7.5 with 32, 4 x 8192 x
// 4096 10.1 and 8.3).  They read x whole each, at some 45 bytes a nanosecond for every
// compute unit, which is what grows with the rows; past 4 us of that, 90000 values of x,
// for the workgroups that follow each other on one, k is split, which costs as much
// (16 x 8192 x 4096: 10.4 us, split 12.7; 48 rows 18.9 and 17.5; 4 x 32768 x 8192 45.7 and
// 40.4, 16 rows 64 and 42; 4 x 4096 x 14336 14.7 and 15.5, 16 rows 22 and 16).  It is split until every compute unit has a workgroup (with two, 17 instead of
// 14 us for 32 x 8192 x 4096), but into no less than two turns each.
Fp4Plan fp4_matmul_plan(int m, int n, int k, int dtype)
{
    Fp4Plan p = {0, 0, ((long long)n + 31) / 32 < 256 ? 1 : 2};
    const int wide = m <= 16 ? 16 * p.tiles : 32, rows = std::min(m, 64);
    const long long rounds = ((((long long)n + wide - 1) / wide) * ((m + 63) / 64) + 255) / 256;
    if (dtype == CONV2D_DTYPE_F32 || rounds * rows * k < 90000) return p;
    const long long blocks = ((long long)n + kManyRows - 1) / kManyRows * ((m + 63) / 64);
    const int whole = k / kTurn, splits = (int)std::max(1LL, std::min(256 / blocks, (long long)whole / 2));
    p.per = std::max(1, (whole + splits - 1) / splits);
    p.splits = std::max(1, (whole + p.per - 1) / p.per);
    return p;
}

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
