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

// Which tokens of a chunk begin a sequence, a bit each, and one for the token behind
// it.  The bits lie in LDS; every wave reads runs of them.
struct FirstTokens {
    static constexpr int kWords = kRecurChunkMost / 32 + 1;
    uint32_t *bits;
    long long c0;       // the chunk's first token
    long long lo, hi;   // the tokens that sequences cover
    long long end;      // the chunk's last token that is covered, plus one

    // all threads of the workgroup; ends with a barrier
    __device__ inline FirstTokens(const Seqs &q, uint32_t *bits_, long long chunk, int index) : bits(bits_)
    {
        c0 = (long long)index * chunk;
        lo = q.begin(0);
        hi = q.begin(q.seqs);
        if (hi < lo) hi = lo;
        end = c0 + chunk < hi ? c0 + chunk : hi;
        for (int w = threadIdx.x; w <= chunk / 32; w += blockDim.x) bits[w] = 0;
        __syncthreads();
        // the first sequence that may begin here; with few of them all are looked at
        int s = q.seqs > (int)blockDim.x && c0 < q.tokens ? q.find(c0) : 0;
        if (!q.start) s = q.len > 0 ? (int)(c0 / q.len) : q.seqs;
        for (s += threadIdx.x; s <= q.seqs; s += blockDim.x) {
            const long long at = q.begin(s) - c0;
            if (at > chunk) break;
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

// Rows of a run: token t of the batch at t * row + (its sequence) * more.
struct RowWalk {
    long long row, more;
    __device__ inline RowWalk(const RowStride &s, const Seqs &q)
        : row(s.row), more(q.start || q.seqs == 1 ? 0 : s.seq - (long long)q.len * s.row) {}
    // element offset of token t, which is in sequence s
    __device__ inline long long at(long long t, long long s) const { return t * row + s * more; }
};

}  // namespace cnv
