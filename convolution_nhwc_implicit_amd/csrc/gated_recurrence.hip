// gated_recurrence.hip -- gated linear recurrence: forward pass and single tokens.
//
//   g = sigmoid(r + r_bias), u = sigmoid(i + i_bias), a = exp(A g)
//   h = a h + sqrt(1 - a^2) u x;  y = h silu(z)
//
// Lanes lie along channels.  A workgroup walks 64 channels of a chunk of tokens in
// segments; its waves take successive runs of a segment's tokens.  Each computes its
// run's decays and inputs, the product of the decays and the state it would end with
// from zero; these meet in LDS, every wave composes the state that its run starts with,
// and walks the run again in registers.  Where a sequence begins inside a run, product
// and state are cut off there (product -1), so that nothing of one sequence, infinities
// and NaN among it, reaches another: runs, segments and chunks need not know sequences.
// Chunks that begin inside a sequence get their state from a first pass over the chunks
// before them.
#include "recur_common.h"

namespace cnv {
namespace {

// ENDS: the first pass, which leaves only each chunk's decay and end state.
template <class E, bool ENDS>
__global__ __launch_bounds__(64 * kRecurWaves) void recur_kernel(RecurArgs a)
{
    constexpr int T = kRecurRun, W = kRecurWaves;
    __shared__ uint32_t bits[RecurChunk::kWords];
    __shared__ float ends[2][2][W][64];
    using S = typename E::S;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int cx = blockIdx.y * kRecurChannels + lane, c = cx < a.d ? cx : a.d - 1;
    const bool mine = cx < a.d;
    if (!ENDS && (int)blockIdx.x >= a.chunks) {  // final states of empty sequences
        const long long s0 = (long long)(blockIdx.x - a.chunks) * kRecurStateSeqs;
        for (long long s = s0 + wave; s < s0 + kRecurStateSeqs && s < a.q.seqs; s += W)
            if (mine && a.q.begin((int)s) == a.q.end((int)s))
                a.final_state[s * a.d + c] = a.initial ? a.initial[s * a.d + c] : 0.0f;
        return;
    }
    const RecurChunk chunk(a, bits, blockIdx.x);
    const RecurChannel ch(a.A, a.r_bias, a.i_bias, c);
    const RecurRows<E> xr(a.x, a.xs, chunk, a.q.len, a.per_seq, c), rr(a.r, a.rs, chunk, a.q.len, a.per_seq, c);
    const RecurRows<E> ir(a.i, a.is, chunk, a.q.len, a.per_seq, c), zr(a.z, a.zs, chunk, a.q.len, a.per_seq, c);
    const bool gate = !ENDS && a.z;

    float carry = 0.0f, total = 1.0f;
    if (!ENDS && a.joined)
        for (int k = chunk.before; k < (int)blockIdx.x; ++k)
            carry = through(a.chunk_decay[(long long)k * a.d + c], a.chunk_state[(long long)k * a.d + c], carry);

    // the next segment's values are under way while one is computed
    S xs[T], rs[T], is[T], zs[T];
    auto load = [&](const RecurRun<T> &run) {
        xr.load(run, xs);
        rr.load(run, rs);
        ir.load(run, is);
        if (gate) zr.load(run, zs);
    };
    if (chunk.len > 0) load(RecurRun<T>(chunk, wave * T));
    for (int at0 = 0, buf = 0; at0 < chunk.len; at0 += T * W, buf ^= 1) {
        const RecurRun<T> run(chunk, at0 + wave * T);
        float av[T], bv[T], zv[T];
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const float L = ch.A * sigmoid_f32(E::to(rs[j]) + ch.rb);
            av[j] = __builtin_amdgcn_exp2f(L * kLog2e);
            bv[j] = __builtin_amdgcn_sqrtf(one_minus_square(L, av[j])) * sigmoid_f32(E::to(is[j]) + ch.ib) * E::to(xs[j]);
            if (gate) {
                const float z = E::to(zs[j]);
                zv[j] = z * sigmoid_f32(z);
            }
        }
        load(RecurRun<T>(chunk, at0 + T * W + wave * T));
        if (run.n < T)
#pragma unroll
            for (int j = 0; j < T; ++j) {
                av[j] = j < run.n ? av[j] : 1.0f;
                bv[j] = j < run.n ? bv[j] : 0.0f;
            }
        // the state before token j where it is a sequence's first
        auto initial = [&](int j) {
            return a.initial ? a.initial[(long long)a.q.find(run.t0 + j) * a.d + c] : 0.0f;
        };
        float dec = 1.0f, end = 0.0f;
        if (run.f == 0) {
#pragma unroll
            for (int j = 0; j < T; ++j) {
                dec *= av[j];
                end = fmaf(av[j], end, bv[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < T; ++j) {
                if (run.f >> j & 1) {
                    dec = -1.0f;
                    end = initial(j);
                }
                dec = dec < 0.0f ? dec : dec * av[j];
                end = fmaf(av[j], end, bv[j]);
            }
        }
        ends[buf][0][wave][lane] = dec;
        ends[buf][1][wave][lane] = end;
        __syncthreads();
        float h = carry;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float d = ends[buf][0][w][lane], e = ends[buf][1][w][lane];
            carry = through(d, e, carry);
            if (w < wave) h = carry;
            if (ENDS) total = joined_decay(total, d);
        }
        if (ENDS) continue;
        S *y = (S *)a.y + run.t0 * a.d;
        if (run.n == T && run.f == 0 && (run.last == 0 || !a.final_state)) {
#pragma unroll
            for (int j = 0; j < T; ++j) {
                h = fmaf(av[j], h, bv[j]);
                if (mine) y[(uint32_t)(j * a.d) + (uint32_t)c] = E::from(gate ? h * zv[j] : h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < T; ++j) {
                if (j >= run.n) break;
                if (run.f >> j & 1) h = initial(j);
                h = fmaf(av[j], h, bv[j]);
                if (mine) y[(uint32_t)(j * a.d) + (uint32_t)c] = E::from(gate ? h * zv[j] : h);
                if (a.final_state && run.last >> j & 1) {
                    const int s = a.q.find(run.t0 + j);
                    if (mine) a.final_state[(long long)s * a.d + c] = h;
                }
            }
        }
    }
    if (ENDS && wave == 0 && mine) {
        a.chunk_decay[(long long)blockIdx.x * a.d + c] = total;
        a.chunk_state[(long long)blockIdx.x * a.d + c] = carry;
    }
}

// One token: a thread to a channel of a row.
template <class E>
__global__ __launch_bounds__(256) void recur_step_kernel(RecurStepArgs a)
{
    using S = typename E::S;
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= a.d) return;
    const long long row = blockIdx.x;
    const int slot = a.slots ? a.slots[row] : (int)row;
    S *y = (S *)a.y + row * a.d + c;
    if (slot < 0 || slot >= a.pool) {
        *y = E::from(0.0f);
        return;
    }
    const RecurChannel ch(a.A, a.r_bias, a.i_bias, c);
    float *state = a.state + (long long)slot * a.d + c;
    const float x = E::to(((const S *)a.x)[row * a.x_row + c]), r = E::to(((const S *)a.r)[row * a.r_row + c]);
    const float i = E::to(((const S *)a.i)[row * a.i_row + c]);
    const float L = ch.A * sigmoid_f32(r + ch.rb), dec = __builtin_amdgcn_exp2f(L * kLog2e);
    const float h = fmaf(dec, *state, __builtin_amdgcn_sqrtf(one_minus_square(L, dec)) * sigmoid_f32(i + ch.ib) * x);
    *state = h;
    float out = h;
    if (a.z) {
        const float z = E::to(((const S *)a.z)[row * a.z_row + c]);
        out = h * (z * sigmoid_f32(z));
    }
    *y = E::from(out);
}

template <class E>
hipError_t launch(const RecurArgs &a, hipStream_t st)
{
    const unsigned by = (unsigned)((a.d + kRecurChannels - 1) / kRecurChannels);
    if (a.joined && a.chunks > 1) {
        recur_kernel<E, true><<<dim3((unsigned)a.chunks - 1, by), 64 * kRecurWaves, 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const unsigned states = a.final_state ? (unsigned)((a.q.seqs + kRecurStateSeqs - 1) / kRecurStateSeqs) : 0;
    recur_kernel<E, false><<<dim3((unsigned)a.chunks + states, by), 64 * kRecurWaves, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_recurrence(int dtype, const RecurArgs &a, hipStream_t st)
{
    switch (dtype) {
        case CONV2D_DTYPE_F16: return launch<SF16>(a, st);
        case CONV2D_DTYPE_BF16: return launch<SBF16>(a, st);
        default: return launch<SF32>(a, st);
    }
}

hipError_t launch_recurrence_step(int dtype, const RecurStepArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)a.rows, (unsigned)((a.d + 255) / 256));
    switch (dtype) {
        case CONV2D_DTYPE_F16: recur_step_kernel<SF16><<<grid, 256, 0, st>>>(a); break;
        case CONV2D_DTYPE_BF16: recur_step_kernel<SBF16><<<grid, 256, 0, st>>>(a); break;
        default: recur_step_kernel<SF32><<<grid, 256, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace cnv
