// recur_common.h -- the gated recurrence's gates, and where sequences begin in a chunk.
#pragma once

#include "block_internal.h"

namespace cnv {

// A channel's parameters; A is clamped so that its product with a closed gate is 0.
struct RecurChannel {
    float A, rb, ib;
    __device__ inline RecurChannel(const float *A_, const float *r_bias, const float *i_bias, int c)
        : A(A_[c] < -2e38f ? -2e38f : A_[c]), rb(r_bias ? r_bias[c] : 0.0f), ib(i_bias ? i_bias[c] : 0.0f) {}
};

// 1 - a^2 for a = exp(L), L <= 0.  Near 1 the difference would lose a's last bits: a
// series in -2L there (its first term left out is 2^-24 of the value at the border).
__device__ inline float one_minus_square(float L, float a)
{
    const float v = -2.0f * L;
    const float near = v * (1.0f - v * (0.5f - v * (1.0f / 6.0f - v * (1.0f / 24.0f))));
    return v < 0.0625f ? near : 1.0f - a * a;
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

    // all threads of the workgroup; ends with a barrier
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
    // The bits of T <= 16 tokens from c0 + at on (at is a multiple of T) and of the one behind them.
    template <int T>
    __device__ inline uint32_t run(int at) const
    {
        uint32_t v = bits[at / 32] >> (at % 32);
        if (at % 32 + T >= 32) v |= bits[at / 32 + 1] << (32 - at % 32);
        return uniform(v & ((2u << T) - 1));
    }
};

// A wave's run of T tokens of a chunk, from c0 + at on.
template <int T>
struct RecurRun {
    long long t0;  // its first row (a row of the chunk, if the run has no tokens)
    int n;         // its tokens
    uint32_t f;    // which of them begin a sequence
    uint32_t last; // which end one
    __device__ inline RecurRun(const RecurChunk &k, int at)
    {
        n = k.len - at;
        n = n < 0 ? 0 : n > T ? T : n;
        t0 = k.c0 + (n > 0 ? at : 0);
        const uint32_t v = n > 0 ? k.run<T>(at) : 0u, all = (1u << n) - 1;
        f = v & all;
        last = v >> 1 & all;
        if (n > 0 && n < T) last |= 1u << (n - 1);  // what is covered ends here
    }
    // the row that is read for token j: a row that is there
    __device__ inline int row(int j) const { return j < n ? j : n > 0 ? n - 1 : 0; }
};

// A tensor of rows: the lane's channel of rows of a chunk.
template <class E>
struct RecurRows {
    const char *base;    // the chunk's row 0 were it the batch's; uniform
    uint32_t row, lane;  // bytes
    __device__ inline RecurRows(const void *p, const RowStride &s, const RecurChunk &k, int len, bool per_seq, int c)
        : base((const char *)p + (per_seq ? k.seq * (s.seq - (long long)len * s.row) * E::kBytes : 0)),
          row((uint32_t)s.row * E::kBytes), lane((uint32_t)c * E::kBytes)
    {
    }
    template <int T>
    __device__ inline void load(const RecurRun<T> &run, typename E::S (&v)[T]) const
    {
        const char *p = base + run.t0 * row;
#pragma unroll
        for (int j = 0; j < T; ++j) v[j] = *(const typename E::S *)(p + (uint32_t)run.row(j) * row + lane);
    }
};

// A piece of tokens as what it does to a state: decay * h + end, or just end where a
// sequence begins in it (decay -1), so that nothing before it, NaN or not, gets through.
__device__ inline float through(float decay, float end, float h) { return decay < 0.0f ? end : fmaf(decay, h, end); }
__device__ inline float joined_decay(float before, float decay) { return before < 0.0f || decay < 0.0f ? -1.0f : before * decay; }

}  // namespace cnv
