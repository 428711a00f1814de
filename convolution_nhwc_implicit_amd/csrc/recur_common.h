// recur_common.h -- the gated recurrence's gates, and where sequences begin in a chunk.
#pragma once

#include <type_traits>

#include "block_internal.h"

namespace cnv {

// A lane's channels' parameters, scaled for exponentials to the base 2: A times log2 e
// (clamped so that its product with a closed gate is 0; below the normal numbers, whose
// inverse the gradients take, 0), the biases times -log2 e.
template <int VC>
struct RecurChannels {
    float A[VC], rb[VC], ib[VC];
    __device__ inline RecurChannels(const float *A_, const float *r_bias, const float *i_bias, int c)
    {
        load_vec<SF32, VC>(A_ + c, VC, A);
#pragma unroll
        for (int v = 0; v < VC; ++v) rb[v] = ib[v] = 0.0f;
        if (r_bias) load_vec<SF32, VC>(r_bias + c, VC, rb);
        if (i_bias) load_vec<SF32, VC>(i_bias + c, VC, ib);
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            if (fabsf(A[v]) < 0x1p-126f) A[v] = 0.0f;
            A[v] = (A[v] < -2e38f ? -2e38f : A[v]) * kLog2e;
            rb[v] *= -kLog2e;
            ib[v] *= -kLog2e;
        }
    }
};
// sigmoid(v + b) for b scaled as above
__device__ inline float recur_gate(float v, float b)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(fmaf(v, -kLog2e, b)));
}
// and what it leaves of 1, to as many bits of its own: 1 / (1 + e) and e / (1 + e)
__device__ inline float recur_gate(float v, float b, float &rest)
{
    const float e = __builtin_amdgcn_exp2f(fmaf(v, -kLog2e, b)), g = __builtin_amdgcn_rcpf(1.0f + e);
    rest = __builtin_amdgcn_fmed3f(e * g, 0.0f, 1.0f);  // a number where e is infinite and g 0; what it meets is 0 with g
    asm("" : "+v"(rest));  // now: until it is used, e and g would take two registers
    return g;
}

// 1 - a^2 for a = 2^L, L <= 0.  Near 1 the difference would lose a's last bits: above L = -1/2,
// where a^2 is 1/2, a polynomial in L in its place, whose first coefficient is -2 ln 2 and the
// others a fit of (1 - 4^L) / L to the least relative error, 2^-25 as they are rounded.  With its
// operations it is off by 2^-22.9, the difference by up to 2^-22 for the exponential's last bit.
__device__ inline float one_minus_square(float L, float a)
{
    float p = fmaf(L, -0.0073865419f, -0.0413785987f);
    p = fmaf(L, p, -0.1535773128f);
    p = fmaf(L, p, -0.4439996779f);
    p = fmaf(L, p, -0.9609049559f);
    return L > -0.5f ? L * fmaf(L, p, -2.0f * kLn2) : fmaf(-a, a, 1.0f);
}

// The chunk of tokens that a workgroup walks, and which of its tokens begin a sequence:
// a bit each, and one for the token behind it.  The bits lie in LDS; every wave reads
// runs of them.
struct RecurChunk {
    static constexpr int kWords = kRecurChunkMost / 32 + 1;
    uint32_t *bits;
    long long c0;   // its first token
    int len;        // its tokens that sequences cover
    long long seq;  // its sequence, where chunks lie inside them (a.per_seq > 0)
    int before;     // the first chunk whose tokens may matter to this one's first state

    __device__ inline RecurChunk(const RecurArgs &a, uint32_t *bits_, int index) : bits(bits_), seq(0), before(0)
    {
        const Seqs &q = a.q;
        long long end = q.begin(q.seqs);
        if (a.per_seq) {
            seq = index / a.per_seq;
            before = (int)seq * a.per_seq;
            c0 = seq * q.len + (long long)(index - before) * a.chunk;
            end = (seq + 1) * q.len;
        } else {
            c0 = (long long)index * a.chunk;
        }
        const long long n = end - c0;
        len = n < 0 ? 0 : n < a.chunk ? (int)n : a.chunk;
    }
    // Sets the bits; all threads of the workgroup.  Holds barriers.
    __device__ inline void mark(const RecurArgs &a)
    {
        const Seqs &q = a.q;
        for (int w = threadIdx.x; w <= a.chunk / 32; w += blockDim.x) bits[w] = 0;
        __syncthreads();
        // the first sequence that may begin here; with few of them all are looked at
        int s = q.seqs > (int)blockDim.x && c0 < q.tokens ? q.find(c0) : 0;
        if (!q.start) s = q.len > 0 ? (int)(c0 / q.len) : q.seqs;
        for (s += threadIdx.x; s <= q.seqs; s += blockDim.x) {
            const long long at = q.begin(s) - c0;
            if (at > a.chunk) break;
            if (at >= 0) atomicOr(&bits[at / 32], 1u << (at % 32));
        }
        __syncthreads();
    }
    // The first token from `at` on, at > 0, that begins a sequence (or is behind the last one);
    // past the chunk if there is none.  Uniform.
    __device__ inline int next(int at, int chunk) const
    {
        const int lane = threadIdx.x % 64, words = chunk / 32 + 1;
        for (int w0 = at / 32; w0 < words; w0 += 64) {
            const int w = w0 + lane;
            uint32_t v = w < words ? bits[w] : 0u;
            if (w == at / 32) v &= ~0u << (at % 32);
            const unsigned long long some = __ballot(v != 0);
            if (some) {
                const int l = __builtin_ctzll(some);
                return uniform((w0 + l) * 32 + __builtin_ctz(__shfl(v, l)));
            }
        }
        return chunk + 1;
    }
    // The bits of T <= 16 tokens from c0 + at on (at is a multiple of T) and of the one behind them.
    template <int T>
    __device__ inline uint32_t run(int at) const
    {
        uint32_t v = bits[at / 32] >> (at % 32);
        if (at % 32 + T >= 32) v |= bits[at / 32 + 1] << (32 - at % 32);
        return v & ((2u << T) - 1);
    }
};

// Where a lane works: LC lanes of a wave lie along channels, VC neighbouring ones to each,
// and the wave's Q = 64 / LC groups of lanes take successive runs of T tokens.  The last
// lane's channels are moved back to end with the last one, where they overlap its
// neighbour's (both compute the same), so that every access is whole; d >= VC.
template <int VC, int LC, int T>
struct RecurPlace {
    static constexpr int Q = 64 / LC, kRun = T, kSpan = Q * T;  // tokens of a lane and of a wave
    int wave, q, c, slot;  // slot: of LC * VC channels in LDS
    bool mine;
    __device__ inline RecurPlace(int block, int d)
    {
        const int lane = threadIdx.x % 64;
        wave = uniform(threadIdx.x / 64);
        q = lane / LC;
        slot = lane % LC * VC;
        const int cx = block * (LC * VC) + slot;
        mine = cx < d;
        c = cx < d - VC ? cx : d - VC;
    }
};

// The span of a wave's tokens that begins `at` tokens behind c0; uniform.
struct RecurSpan {
    int at, tokens;  // tokens that are there
    template <class Place>
    __device__ inline RecurSpan(const RecurChunk &k, const Place &, int at_) : at(at_)
    {
        const int n = k.len - at;
        tokens = n < 0 ? 0 : n < Place::kSpan ? n : Place::kSpan;
    }
};
// A lane's run of T tokens in it.
template <int T>
struct RecurRun {
    int n;          // tokens that are there
    uint32_t f;     // which of them begin a sequence
    uint32_t last;  // which end one
    bool firsts, lasts;  // whether any lane's run has such tokens
    bool whole;     // whether all tokens of the span are there
    template <class Place>
    __device__ inline RecurRun(const RecurChunk &k, const Place &p, const RecurSpan &span)
    {
        n = span.tokens - p.q * T;
        n = n < 0 ? 0 : n > T ? T : n;
        const uint32_t v = n > 0 ? k.run<T>(span.at + p.q * T) : 0u, all = (1u << n) - 1;
        f = v & all;
        last = v >> 1 & all;
        if (n > 0 && n < T) last |= 1u << (n - 1);  // what is covered ends here
        firsts = __ballot(f != 0) != 0;
        lasts = __ballot(last != 0) != 0;
        whole = span.tokens == Place::kSpan;
    }
    // a run in the middle of a sequence
    __device__ inline RecurRun() : n(T), f(0), last(0), firsts(false), lasts(false), whole(true) {}
};

// Rows are read and written through buffer descriptors that begin with a span's first
// token and end with its last one that is there: tokens past it are not read (but where
// rows overlap) and not written, without branches, and a lane needs one 32-bit offset
// for a tensor.
constexpr uint32_t kRecurNowhere = 0xfffffff0u;  // past every range: at most 31 rows of 2^26 bytes and one's elements

__device__ inline __amdgpu_buffer_rsrc_t recur_buffer(const void *p, uint32_t bytes)
{
    const uint64_t v = (uint64_t)p;
    const uint64_t u = (uint64_t)(uint32_t)uniform((int)(uint32_t)v) | (uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32;
    return __builtin_amdgcn_make_buffer_rsrc((void *)u, 0, uniform((int)bytes), 0x00020000);
}

// v, in a scalar register and computed with here: offsets of a run's rows would
// otherwise be kept in a vector register each, for every tensor, all along the chunk.
__device__ inline uint32_t scalar_here(uint32_t v)
{
    asm volatile("" : "+s"(v));
    return v;
}

// VC neighbouring elements as they lie in memory.
template <class E, int VC>
struct RecurRaw {
    static constexpr int kBytes = E::kBytes * VC;
    uint32_t w;
    __device__ inline float operator[](int v) const
    {
        if constexpr (E::kBytes == 4) return __builtin_bit_cast(float, w);
        else return E::to((uint16_t)(v ? w >> 16 : w));
    }
    __device__ inline void load(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t more)
    {
        if constexpr (kBytes == 2) w = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, more, 0);
        else w = __builtin_amdgcn_raw_buffer_load_b32(r, off, more, 0);
    }
};
// two values rounded by one conversion
template <class E>
__device__ inline uint32_t recur_pack(float a, float b)
{
    if constexpr (std::is_same_v<E, SF16>) return Pack2<EF16>::cvt(f2v{a, b});
    else return Pack2<EBF16>::cvt(f2v{a, b});
}
template <class E, int VC>
__device__ inline void recur_store(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t more, const float (&v)[VC])
{
    if constexpr (E::kBytes == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[0]), r, off, more, 0);
    else if constexpr (VC == 1) __builtin_amdgcn_raw_buffer_store_b16(E::from(v[0]), r, off, more, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(recur_pack<E>(v[0], v[1]), r, off, more, 0);
}

// A tensor of rows: the lane's channels of the rows of a chunk.
template <class E, int VC>
struct RecurRows {
    const char *base;     // the chunk's first row; uniform
    uint32_t row, width;  // bytes
    uint32_t run;         // of the lane's channels and run in a span
    template <class Place>
    __device__ inline RecurRows(const void *p, const RowStride &s, const RecurArgs &a, const RecurChunk &k, const Place &at)
        : base((const char *)p + (a.per_seq ? k.seq * (s.seq - (long long)a.q.len * s.row) * E::kBytes : 0) + k.c0 * s.row * E::kBytes),
          row((uint32_t)s.row * E::kBytes), width((uint32_t)a.d * E::kBytes)
    {
        run = p ? (uint32_t)(at.q * Place::kRun) * row + (uint32_t)at.c * E::kBytes : kRecurNowhere;  // no tensor: zeros, at any row (its stride is 0)
    }
    __device__ inline __amdgpu_buffer_rsrc_t span(const RecurSpan &s) const
    {
        return recur_buffer(base + (long long)s.at * row, s.tokens > 0 ? (uint32_t)(s.tokens - 1) * row + width : 0u);
    }
    // Token j.  INSIDE: all of the span's tokens are there; the row's offset is then a scalar
    // operand of the load, which the range does not count.
    template <bool INSIDE>
    __device__ inline void load(__amdgpu_buffer_rsrc_t b, int j, RecurRaw<E, VC> &v) const
    {
        if (INSIDE) v.load(b, run, (uint32_t)j * row);
        else v.load(b, run + (uint32_t)j * scalar_here(row), 0);
    }
};
// A dense output of rows [tokens][d].
template <class E, int VC>
struct RecurOut {
    char *base;
    uint32_t row, run;
    template <class Place>
    __device__ inline RecurOut(void *p, const RecurArgs &a, const RecurChunk &k, const Place &at)
        : base((char *)p + k.c0 * a.d * E::kBytes), row((uint32_t)a.d * E::kBytes)
    {
        run = p && at.mine ? (uint32_t)(at.q * Place::kRun) * row + (uint32_t)at.c * E::kBytes : kRecurNowhere;
    }
    __device__ inline __amdgpu_buffer_rsrc_t span(const RecurSpan &s) const
    {
        return recur_buffer(base + (long long)s.at * row, (uint32_t)s.tokens * row);
    }
    template <bool INSIDE>
    __device__ inline void store(__amdgpu_buffer_rsrc_t b, int j, const float (&v)[VC]) const
    {
        if (INSIDE) {
            recur_store<E, VC>(b, run, (uint32_t)j * row, v);
        } else {
            const uint32_t off = run + (uint32_t)j * scalar_here(row);
            recur_store<E, VC>(b, run == kRecurNowhere ? run : off, 0, v);  // not round the 32 bits' end
        }
    }
};

// A piece of tokens as what it does to a state: decay * h + end, or just end where a
// sequence begins in it (decay -1), so that nothing before it, NaN or not, gets through.
__device__ inline float through(float decay, float end, float h) { return decay < 0.0f ? end : fmaf(decay, h, end); }
__device__ inline float joined_decay(float before, float decay) { return before < 0.0f || decay < 0.0f ? -1.0f : before * decay; }

template <int VC>
struct RecurPiece {
    float dec[VC], end[VC];
    __device__ inline void clear()
    {
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            dec[v] = 1.0f;
            end[v] = 0.0f;
        }
    }
    // this piece behind `p`.  INSIDE, here and below: no sequence begins in either
    template <bool INSIDE>
    __device__ inline void after(const RecurPiece &p)
    {
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            end[v] = INSIDE ? fmaf(dec[v], p.end[v], end[v]) : through(dec[v], end[v], p.end[v]);
            dec[v] = INSIDE ? dec[v] * p.dec[v] : joined_decay(p.dec[v], dec[v]);
        }
    }
    template <bool INSIDE>
    __device__ inline void carry(float (&h)[VC]) const
    {
#pragma unroll
        for (int v = 0; v < VC; ++v) h[v] = INSIDE ? fmaf(dec[v], h[v], end[v]) : through(dec[v], end[v], h[v]);
    }
    // the piece of the lane `by` lanes down (UP: up)
    template <bool UP>
    __device__ inline RecurPiece from(int by) const
    {
        RecurPiece p;
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            p.dec[v] = UP ? __shfl_down(dec[v], by) : __shfl_up(dec[v], by);
            p.end[v] = UP ? __shfl_down(end[v], by) : __shfl_up(end[v], by);
        }
        return p;
    }
    // An entry for every channel in LDS: decay and end side by side.
    __device__ inline void put(float2 *p) const
    {
#pragma unroll
        for (int v = 0; v < VC; ++v) p[v] = float2{dec[v], end[v]};
    }
    __device__ inline void get(const float2 *p)
    {
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            const float2 e = p[v];
            dec[v] = e.x;
            end[v] = e.y;
        }
    }
};

// Joins the pieces of a segment: those of a wave's lane groups by shuffles, the waves'
// through LDS, a barrier of the workgroup between put() and get().  BACK: what follows
// comes first.
template <int VC, int LC, int W, bool BACK, bool INSIDE>
struct RecurJoin {
    static constexpr int Q = 64 / LC;
    typedef float2 Lds[W][LC * VC];
    RecurPiece<VC> mine;
    int q, wave, slot;
    template <class Place>
    __device__ inline RecurJoin(const RecurPiece<VC> &p, const Place &at)
        : mine(p), q(BACK ? Q - 1 - at.q : at.q), wave(BACK ? W - 1 - at.wave : at.wave), slot(at.slot)
    {
    }
    __device__ inline void put(Lds &lds)
    {
#pragma unroll
        for (int s = 1; s < Q; s *= 2) {
            const RecurPiece<VC> p = mine.template from<BACK>(s * LC);
            if (q >= s) mine.template after<INSIDE>(p);
        }
        if (q == Q - 1) mine.put(&lds[wave][slot]);
    }
    // h, what the segment starts with, becomes what leaves it; before: what the lane's
    // own run starts with; total, if there is one, goes on with the segment.
    __device__ inline void get(const Lds &lds, float (&h)[VC], float (&before)[VC], RecurPiece<VC> *total) const
    {
#pragma unroll
        for (int v = 0; v < VC; ++v) before[v] = h[v];
#pragma unroll 4
        for (int w = 0; w < W; ++w) {  // four at a time: all of them would take too many registers
            RecurPiece<VC> p;
            p.get(&lds[w][slot]);
            p.template carry<INSIDE>(h);
            if (w < wave)
#pragma unroll
                for (int v = 0; v < VC; ++v) before[v] = h[v];
            if (total)
#pragma unroll
                for (int v = 0; v < VC; ++v) total->dec[v] = joined_decay(total->dec[v], p.dec[v]);
        }
        if (Q > 1) {
            const RecurPiece<VC> p = mine.template from<BACK>(LC);
            if (q > 0) p.template carry<INSIDE>(before);
        }
    }
};

// A lane's channels of an array [..][d] of fp32.
template <int VC>
__device__ inline void recur_get(const float *p, long long i, int d, int c, float (&v)[VC])
{
    load_vec<SF32, VC>(p + i * d + c, VC, v);
}
template <int VC>
__device__ inline void recur_put(float *p, long long i, int d, int c, const float (&v)[VC])
{
    store_vec<SF32, VC>(p + i * d + c, VC, v);
}

// Nothing comes in at tokens that are not there; how they decay does not matter, for
// nothing follows them.
template <int VC, int T>
__device__ inline void recur_cut(const RecurRun<T> &run, float (&in)[T][VC])
{
    if (!run.whole)
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int v = 0; v < VC; ++v) in[j][v] = j < run.n ? in[j][v] : 0.0f;
}

// The chunks from `first` up (or down, by `step`) to the one before `stop` as one piece
// each for the workgroup's waves, successive ones to a wave, so that their loads are all
// under way together; into lds, for recur_carried() behind a barrier.
template <int VC, int W, class Place, class Lds>
__device__ inline void recur_carry(const float *decay, const float *end, int first, int stop, int step, int d, const Place &at, Lds &lds)
{
    const int all = (stop - first) * step, per = (all + W - 1) / W;
    int left = all - at.wave * per;
    left = left < per ? left : per;
    RecurPiece<VC> mine;
    mine.clear();
    for (int k = first + at.wave * per * step; left > 0; left -= 4, k += 4 * step) {
        RecurPiece<VC> p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long chunk = k + (i < left ? i : left - 1) * step;
            recur_get<VC>(decay, chunk, d, at.c, p[i].dec);
            recur_get<VC>(end, chunk, d, at.c, p[i].end);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) {
                p[i].template after<false>(mine);
                mine = p[i];
            }
    }
    if (at.q == 0) mine.put(&lds[at.wave][at.slot]);
}
template <int VC, int W, class Place, class Lds>
__device__ inline void recur_carried(const Lds &lds, const Place &at, float (&h)[VC])
{
#pragma unroll 4
    for (int w = 0; w < W; ++w) {
        RecurPiece<VC> p;
        p.get(&lds[w][at.slot]);
        p.template carry<false>(h);
    }
}

// What a run does to a state, from its decays and inputs.
template <int VC, int T>
__device__ inline void recur_piece(uint32_t f, bool firsts, const float (&av)[T][VC], const float (&bv)[T][VC], RecurPiece<VC> &p)
{
    p.clear();
    if (!firsts) {
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                p.dec[v] *= av[j][v];
                p.end[v] = fmaf(av[j][v], p.end[v], bv[j][v]);
            }
    } else {
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const bool first = f >> j & 1;
                p.dec[v] = first || p.dec[v] < 0.0f ? -1.0f : p.dec[v] * av[j][v];
                p.end[v] = fmaf(av[j][v], first ? 0.0f : p.end[v], bv[j][v]);
            }
    }
}

// The same for the gradient that flows back through a run, from the decays and the
// gradients that come in at its tokens.
template <int VC, int T>
__device__ inline void recur_flow(uint32_t last, bool lasts, const float (&av)[T][VC], const float (&gv)[T][VC], RecurPiece<VC> &p)
{
    p.clear();
    if (!lasts) {
#pragma unroll
        for (int j = T - 1; j >= 0; --j)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                p.dec[v] *= av[j][v];
                p.end[v] = av[j][v] * (p.end[v] + gv[j][v]);
            }
    } else {
#pragma unroll
        for (int j = T - 1; j >= 0; --j)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const bool cut = last >> j & 1;
                p.dec[v] = cut || p.dec[v] < 0.0f ? -1.0f : p.dec[v] * av[j][v];
                p.end[v] = av[j][v] * ((cut ? 0.0f : p.end[v]) + gv[j][v]);
            }
    }
}

// Where sequences begin, every stride()th a lane: the wave finds a token's sequence among
// up to 64 of them without a load, among up to 4096 with one, where a search waits for a
// load each time it halves (2000 single tokens of 4096 channels with states take 81 us, by
// searches 170).
struct RecurStarts {
    int v;
    __device__ inline RecurStarts(const Seqs &q) : v(0)
    {
        if (q.start && stride(q) <= 64) v = start(q, threadIdx.x % 64 * stride(q));
    }
    static __device__ inline int stride(const Seqs &q) { return (q.seqs + 63) / 64; }
    static __device__ inline int start(const Seqs &q, int s) { return s < q.seqs ? (int)q.begin(s) : INT32_MAX; }
    // how many lanes' values are at most t, less one; not below 0 whatever they are
    static __device__ inline int last(int v, int t)
    {
        const int n = __builtin_popcountll(__ballot(v <= t));
        return n > 0 ? n - 1 : 0;
    }
    // The sequence of row t, whole waves at a time; t differs between a wave's groups of lanes.
    template <class Place>
    __device__ inline int find(const Seqs &q, const Place &at, long long t) const
    {
        const int step = (int)scalar_here(stride(q));
        if (!q.start || step > 64) return q.find(t);
        int s = 0;
#pragma unroll
        for (int g = 0; g < Place::Q; ++g) {
            const int tg = __builtin_amdgcn_readlane((int)t, g * (64 / Place::Q));
            int n = last(v, tg);
            if (step > 1) {
                const int lane = threadIdx.x % 64;
                n = n * step + last(lane < step ? start(q, n * step + lane) : INT32_MAX, tg);
            }
            s = at.q == g ? n : s;
        }
        return s < q.seqs ? s : q.seqs - 1;
    }
};

// Entries of p [seqs][d] for the tokens in `which` (from row t0 on): each goes to
// use(j, the entry).
template <int VC, int T, class Place, class F>
__device__ inline void recur_gather(const RecurArgs &a, const RecurStarts &starts, const float *p, uint32_t which, long long t0,
                                    const Place &at, F use)
{
#pragma unroll
    for (int j = 0; j < T; ++j)
        if (__ballot(which >> j & 1)) {
            const int s = starts.find(a.q, at, t0 + j);
            if (which >> j & 1) {
                float h[VC];
                recur_get<VC>(p, s, a.d, at.c, h);
                use(j, h);
            }
        }
}

// Writes the values of tokens in `which` to their sequences' entries of out [seqs][d].
template <int VC, int T, class Place>
__device__ inline void recur_scatter(const RecurArgs &a, const RecurStarts &starts, uint32_t which, long long t0, const Place &at,
                                     const float (&hv)[T][VC], float *out)
{
#pragma unroll
    for (int j = 0; j < T; ++j)
        if (__ballot(which >> j & 1)) {
            const int s = starts.find(a.q, at, t0 + j);
            if ((which >> j & 1) && at.mine) recur_put<VC>(out, s, a.d, at.c, hv[j]);
        }
}

// Blocks that read the same lines of memory (neighbouring channels of one chunk) go to
// one XCD, of which the workgroups are dealt out in turn: block -> chunk * across + channels.
__device__ inline int recur_block(int id, int blocks) { return id % 8 * ((blocks + 7) / 8) + id / 8; }

// f(channels of a lane, lanes along channels) for a shape
template <class E, class F>
hipError_t recur_by_shape(const RecurShape &s, F f)
{
    using std::integral_constant;
    constexpr int VC = E::kBytes == 2 ? 2 : 1;
    if (s.vc < VC) return f(integral_constant<int, 1>{}, integral_constant<int, 8>{});
    constexpr integral_constant<int, VC> vc{};
    switch (s.lanes) {
        case 8: return f(vc, integral_constant<int, 8>{});
        case 16: return f(vc, integral_constant<int, 16>{});
        case 32: return f(vc, integral_constant<int, 32>{});
        default: return f(vc, integral_constant<int, 64>{});
    }
}

}  // namespace cnv
