// scan_common.h -- what the forward and the gradient kernels of the selective
// scan share: the wave's layout, token loads, chunk lookup and cross-lane sums.
//
// Layout of a wave: 16 channels, 4 lanes each (lane = 4 * channel + part).
// Lane `part` holds NL neighbouring states of its channel, part*NL ..
// part*NL+NL-1 (n <= 4*NL; states past n have A = B = C = 0 and stay 0).  What
// belongs to a token and a channel but not to a state (step size, input, gate)
// is computed once: of every four tokens lane `part` takes token `part`, and
// the others read it through a quad broadcast.
#pragma once

#include "seq_internal.h"

namespace cnv {

template <int Q>
__device__ inline float quad_bcast(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), Q * 0x55, 0xf, 0xf, true));
}
template <int CTRL>
__device__ inline float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
constexpr int kQuadXor1 = 0xb1, kQuadXor2 = 0x4e, kRowRor4 = 0x124, kRowRor8 = 0x128;

// Sums over the four lanes of a quad of four values; lane q gets the sum of vq.
__device__ inline float quad_scatter_sum(float v0, float v1, float v2, float v3, bool odd, bool high)
{
    const float a = (odd ? v1 : v0) + dpp<kQuadXor1>(odd ? v0 : v1);
    const float b = (odd ? v3 : v2) + dpp<kQuadXor1>(odd ? v2 : v3);
    return (high ? b : a) + dpp<kQuadXor2>(high ? a : b);
}

// Sum over the quad of one value, in every lane.
__device__ inline float quad_sum(float v)
{
    v += dpp<kQuadXor1>(v);
    return v + dpp<kQuadXor2>(v);
}

// Sums of four values over the wave's 16 channels (lanes with the same
// lane % 4).  Row r of 16 lanes gets the sum of vr, in each of its quads.
__device__ inline float channel_sum4(float v0, float v1, float v2, float v3)
{
    // the builtins' two results, as values first: a bit cast of a vector's element reads element 0
    auto half = [](float a, float b) {
        const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b),
                                                        false, false);
        const unsigned u = r[0], v = r[1];
        return __builtin_bit_cast(float, u) + __builtin_bit_cast(float, v);
    };
    const float s01 = half(v0, v1), s23 = half(v2, v3);
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, s01), __builtin_bit_cast(unsigned, s23),
                                                    false, false);
    const unsigned lo = r[0], hi = r[1];
    float s = __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
    s += dpp<kRowRor4>(s);
    return s + dpp<kRowRor8>(s);
}

// The value, computed here whatever becomes of it: a choice by a flag of the
// call is then a select, where a branch would cut the code around it in pieces.
__device__ inline float here(float v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// log(1 + e^raw) = max(raw, 0) + log1p(e), e = e^-|raw| in (0, 1].  With
// w = e / (2 + e) <= 1/3, log1p(e) = 2 atanh(w) = 2 w (1 + w^2/3 + w^4/5 + ...):
// relative accuracy for every raw (1 + e would lose small e's bits); the first
// term left out is below 2^-27 of the sum.
__device__ inline float softplus_f32(float raw)
{
    const float e = __builtin_amdgcn_exp2f(-kLog2e * __builtin_fabsf(raw));
    const float w = e * __builtin_amdgcn_rcpf(2.0f + e), s = w * w;
    float p = 1.0f / 15.0f;
    p = __builtin_fmaf(p, s, 1.0f / 13.0f);
    p = __builtin_fmaf(p, s, 1.0f / 11.0f);
    p = __builtin_fmaf(p, s, 1.0f / 9.0f);
    p = __builtin_fmaf(p, s, 1.0f / 7.0f);
    p = __builtin_fmaf(p, s, 1.0f / 5.0f);
    p = __builtin_fmaf(p, s, 1.0f / 3.0f);
    p = __builtin_fmaf(p, s, 1.0f);
    const float r = __builtin_fmaf(2.0f * w, p, __builtin_fmaxf(raw, 0.0f));
    return raw != raw ? raw : r;  // the maximum above drops a NaN
}

// A rate as it is used: at most 2e38 in size, so that the decay exp(delta A) of
// an infinite one is still 0 (or infinite), but 1 for tokens that are not there
// (delta = 0), where 0 times infinity would spoil the state behind them.
__device__ inline float finite_rate(float A) { return A < -2e38f ? -2e38f : A > 2e38f ? 2e38f : A; }

// The chunk that a workgroup walks.
struct Chunk {
    int s;            // sequence
    bool first, last; // of its sequence
    int t0, t1;       // its rows
    bool valid;
};

// No more than there are in all (fewer than 2^25), which a sequence exceeds only
// if seq_start descends somewhere: sums over 64 sequences stay within 31 bits.
__device__ inline int chunks_of(const ScanArgs &a, int s)
{
    const long long len = a.q.end(s) - a.q.begin(s);
    const long long c = (len + a.chunk - 1) / a.chunk;
    return c < 1 ? 1 : c < a.slots ? (int)c : a.slots;  // an empty sequence still passes its state on
}

// Slot -> chunk.  Packed: sequences' chunks lie in order, 64 sequences looked
// at together, a lane each.
__device__ inline Chunk find_chunk(const ScanArgs &a, int slot)
{
    Chunk r;
    int c = 0, count = a.chunks;
    bool found = true;
    r.s = 0;
    if (!a.q.start) {
        r.s = slot / a.chunks;
        c = slot % a.chunks;
    } else {
        const int lane = threadIdx.x % 64;
        int base = 0;
        found = false;
        for (int s0 = 0; s0 < a.q.seqs && !found; s0 += 64) {
            const int mine = s0 + lane < a.q.seqs ? chunks_of(a, s0 + lane) : 0;
            int incl = mine;
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned long long past = __ballot(base + incl > slot);
            if (past) {
                const int at = __builtin_ctzll(past);
                r.s = s0 + at;
                count = __shfl(mine, at);
                c = slot - (base + __shfl(incl, at) - count);
                found = true;
            }
            base += __shfl(incl, 63);
        }
    }
    r.s = uniform(r.s);
    c = uniform(c);
    count = uniform(count);
    r.valid = found;
    r.first = c == 0;
    r.last = c == count - 1;
    const long long b = a.q.begin(r.s), e = a.q.end(r.s);
    long long t0 = b + (long long)c * a.chunk;
    t0 = t0 < b ? b : t0 > e ? e : t0;  // inside whatever seq_start says
    const long long t1 = t0 + a.chunk < e ? t0 + a.chunk : e;
    r.t0 = uniform((int)t0);
    r.t1 = found ? uniform((int)t1) : r.t0;
    return r;
}

// Where the state before the step at row t of a chunk is kept.  Neighbouring
// chunks' ranges do not meet: each has one entry more than the whole steps
// between its first row and the next chunk's.  Never past tokens/TS + slots.
template <int TS>
__device__ inline long long scan_keep_index(const Chunk &k, int slot, int t)
{
    return k.t0 / TS + slot + (t - k.t0) / TS;
}

// ---- buffers -----------------------------------------------------------------
// Tensors are read and written through buffer descriptors whose range ends with
// the rows of the step at hand: what lies past it (rows after the chunk, lanes
// without a channel or a state) reads as zero and is not written, without
// branches, and a lane needs one 32-bit offset per tensor.
constexpr uint32_t kNowhere = 0x80000000u;  // past every range

__device__ inline __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t bytes)
{
    const uint64_t v = (uint64_t)p;
    const uint64_t u = (uint64_t)(uint32_t)uniform((int)(uint32_t)v) | (uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32;
    return __builtin_amdgcn_make_buffer_rsrc((void *)u, 0, uniform((int)bytes), 0x00020000);
}
// A tensor of rows of `width` elements, walked a step at a time: the address of
// the step's first row stays in scalar registers.
template <class E>
struct Stream {
    uint64_t p;
    uint32_t row, width;  // bytes
    __device__ inline Stream(const void *base, long long at, long long r, int w)
        : p((uint64_t)base + at * E::kBytes), row((uint32_t)r * E::kBytes), width(base ? (uint32_t)w * E::kBytes : 0u)
    {
    }
    // the first `rows` rows from here; none where rows is below 1, or of no tensor
    __device__ inline __amdgpu_buffer_rsrc_t rows(int n) const
    {
        const uint32_t bytes = (uint32_t)(n - 1) * row + width;
        return buffer_of((const void *)p, n > 0 && width ? bytes : 0u);
    }
    __device__ inline void advance(int n) { p += (long long)n * row; }
};

template <class E>
__device__ inline typename E::S get(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    if constexpr (E::kBytes == 2) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    else return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}
template <class E>
__device__ inline void put(__amdgpu_buffer_rsrc_t r, uint32_t off, float v)
{
    if constexpr (E::kBytes == 2) __builtin_amdgcn_raw_buffer_store_b16(E::from(v), r, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, off, 0, 0);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// NL neighbouring fp32 at a byte offset (a multiple of 4).
template <int NL>
__device__ inline void get_run(__amdgpu_buffer_rsrc_t r, uint32_t off, float (&v)[NL])
{
    if constexpr (NL == 1) {
        v[0] = get<SF32>(r, off);
    } else if constexpr (NL == 2) {
        const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
        const uint32_t x = w[0], y = w[1];
        v[0] = __builtin_bit_cast(float, x);
        v[1] = __builtin_bit_cast(float, y);
    } else {
#pragma unroll
        for (int j = 0; j < NL; j += 4) {
            const f32x4 w = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 4 * j, 0, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j + e] = w[e];
        }
    }
}
template <int NL>
__device__ inline void put_run(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[NL])
{
    if constexpr (NL == 1) {
        put<SF32>(r, off, v[0]);
    } else if constexpr (NL == 2) {
        u32x2 w;
        w[0] = __builtin_bit_cast(uint32_t, v[0]);
        w[1] = __builtin_bit_cast(uint32_t, v[1]);
        __builtin_amdgcn_raw_buffer_store_b64(w, r, off, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < NL; j += 4) {
            const f32x4 w = {v[j], v[j + 1], v[j + 2], v[j + 3]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w), r, off + 4 * j, 0, 0);
        }
    }
}

// The channels of a workgroup and a lane.
struct Channels {
    int group, block;  // group of B and C, channel block over all groups
    int ch;            // this lane's channel, clamped to one that exists
    bool valid;        // whether it exists
    int part;          // lane % 4
    // `width` channels to a workgroup, 16 of them to wave `wave`
    __device__ inline Channels(const ScanArgs &a, int blk, int width, int wave)
    {
        const int dg = a.d / a.groups, lane = threadIdx.x % 64;
        block = blk;
        group = blk / a.blocks_per_group;
        const int c = (blk % a.blocks_per_group) * width + wave * 16 + lane / 4;
        valid = c < dg;
        ch = group * dg + (valid ? c : dg - 1);
        part = lane % 4;
    }
};

// A lane's place in a tensor of rows: token `part` of a step, its channel.
// Token 4*i + part lies i * four rows further.
template <class E>
struct TokenAt {
    uint32_t off, four;
    __device__ inline TokenAt(const Channels &c, long long row)
        : off(c.valid ? ((uint32_t)c.part * (uint32_t)row + (uint32_t)c.ch) * E::kBytes : kNowhere),
          four(4 * (uint32_t)row * E::kBytes)
    {
    }
    __device__ inline uint32_t operator[](int i) const { return off + i * four; }
};

// A lane's NL states in an array [..][d][n] of fp32: those of one entry.
template <int NL>
struct StateAt {
    uint32_t off;
    int n, part, d;
    __device__ inline StateAt(const ScanArgs &a, const Channels &c)
        : off(c.valid ? ((uint32_t)c.ch * (uint32_t)a.n + (uint32_t)c.part * NL) * 4 : kNowhere), n(a.n), part(c.part), d(a.d)
    {
    }
    __device__ inline __amdgpu_buffer_rsrc_t entry(const float *p, long long i) const
    {
        return buffer_of(p + i * d * n, (uint32_t)d * (uint32_t)n * 4);
    }
    __device__ inline void load(const float *p, long long i, float (&v)[NL]) const
    {
        const __amdgpu_buffer_rsrc_t r = entry(p, i);
        if (n == 4 * NL) {
            get_run<NL>(r, off, v);
        } else {
#pragma unroll
            for (int j = 0; j < NL; ++j) v[j] = get<SF32>(r, part * NL + j < n ? off + 4 * j : kNowhere);
        }
    }
    __device__ inline void store(float *p, long long i, const float (&v)[NL]) const
    {
        const __amdgpu_buffer_rsrc_t r = entry(p, i);
        if (n == 4 * NL) {
            put_run<NL>(r, off, v);
        } else {
#pragma unroll
            for (int j = 0; j < NL; ++j) put<SF32>(r, part * NL + j < n ? off + 4 * j : kNowhere, v[j]);
        }
    }
};

// A value per channel in an array [..][d], of entry i, read by every lane of
// the channel or written by its first.
__device__ inline float channel_load(const float *p, long long i, const ScanArgs &a, const Channels &c)
{
    return get<SF32>(buffer_of(p + i * a.d, (uint32_t)a.d * 4), c.valid ? (uint32_t)c.ch * 4 : kNowhere);
}
__device__ inline void channel_store(float *p, long long i, const ScanArgs &a, const Channels &c, float v)
{
    put<SF32>(buffer_of(p + i * a.d, (uint32_t)a.d * 4), c.valid && c.part == 0 ? (uint32_t)c.ch * 4 : kNowhere, v);
}

// B and C of a step as fp32 in LDS, [TS][4*NL].  Thread i of the workgroup
// takes value i (TS * 4*NL <= 256).
template <class E, int NL, int TS>
struct StageBC {
    static constexpr int kCount = TS * 4 * NL;
    static_assert(kCount <= 256, "a value per thread");
    typename E::S b, c;
    uint32_t boff, coff;
    Stream<E> sb, sc;
    __device__ inline StageBC(const ScanArgs &a, const Chunk &k, int group, int t)
        : sb(a.B, a.bs.at(a.q, k.s, t) + group * a.b_group, a.bs.row, a.n),
          sc(a.C, a.cs.at(a.q, k.s, t) + group * a.c_group, a.cs.row, a.n)
    {
        const uint32_t tok = threadIdx.x / (4 * NL), n = threadIdx.x % (4 * NL);
        const bool mine = threadIdx.x < kCount && (int)n < a.n;
        boff = mine ? tok * sb.row + n * E::kBytes : kNowhere;
        coff = mine ? tok * sc.row + n * E::kBytes : kNowhere;
    }
    __device__ inline void load(int rows, bool want_c)
    {
        b = get<E>(sb.rows(rows), boff);
        if (want_c) c = get<E>(sc.rows(rows), coff);
    }
    __device__ inline void advance(int n)
    {
        sb.advance(n);
        sc.advance(n);
    }
    __device__ inline void store(float *lb, float *lc) const
    {
        if (threadIdx.x < kCount) {
            lb[threadIdx.x] = E::to(b);
            if (lc) lc[threadIdx.x] = E::to(c);
        }
    }
};

// The lanes' NL values of four tokens, read from LDS ahead of their use.
template <int NL>
struct Four {
    float v[4][NL];
    __device__ inline void read(const float *p, int i, int part)
    {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < NL; ++j) v[q][j] = p[(4 * i + q) * 4 * NL + part * NL + j];
    }
};

// NL states of a lane at p, [n] of one channel; n may be short of 4*NL.
template <int NL>
__device__ inline void read_nl(const float *p, int n, int part, float (&v)[NL])
{
    if (n == 4 * NL) {
        const SVec<float, NL> r = *(const SVec<float, NL> *)(p + part * NL);
#pragma unroll
        for (int j = 0; j < NL; ++j) v[j] = r.v[j];
    } else {
#pragma unroll
        for (int j = 0; j < NL; ++j) v[j] = part * NL + j < n ? p[part * NL + j] : 0.0f;
    }
}
template <int NL>
__device__ inline void write_nl(float *p, int n, int part, const float (&v)[NL])
{
    if (n == 4 * NL) {
        SVec<float, NL> r;
#pragma unroll
        for (int j = 0; j < NL; ++j) r.v[j] = v[j];
        *(SVec<float, NL> *)(p + part * NL) = r;
    } else {
#pragma unroll
        for (int j = 0; j < NL; ++j)
            if (part * NL + j < n) p[part * NL + j] = v[j];
    }
}

// f(element type, NL as a constant) for the smallest NL with 4 * NL >= n
template <class F>
hipError_t scan_by_type(int dtype, int n, F f)
{
    auto states = [&](auto e) {
        if (n <= 4) return f(e, std::integral_constant<int, 1>{});
        if (n <= 8) return f(e, std::integral_constant<int, 2>{});
        if (n <= 16) return f(e, std::integral_constant<int, 4>{});
        if (n <= 32) return f(e, std::integral_constant<int, 8>{});
        return f(e, std::integral_constant<int, 16>{});
    };
    if (dtype == CONV2D_DTYPE_F16) return states(SF16{});
    if (dtype == CONV2D_DTYPE_BF16) return states(SBF16{});
    return states(SF32{});
}

}  // namespace cnv
