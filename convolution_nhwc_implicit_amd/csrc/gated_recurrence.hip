// gated_recurrence.hip -- gated linear recurrence: forward pass and single tokens.
//
//   g = sigmoid(r + r_bias), u = sigmoid(i + i_bias), a = exp(A g) = 2^L
//   h = a h + sqrt(1 - a^2) u x;  y = h silu(z)
//
// A workgroup walks some channels of a chunk of tokens in segments; groups of its lanes
// take successive runs of a segment's tokens.  Each computes its run's decays and
// inputs, the product of the decays and the state it would end with from zero; these
// are joined by shuffles and through LDS, so that every lane has the state that its run
// starts with, and walks the run again in registers.  Where a sequence begins inside a
// run, product and state are cut off there (product -1), so that nothing of one sequence,
// infinities and NaN among it, reaches another: runs, segments and chunks need not know
// sequences.  Chunks that begin inside a sequence get their state from a first pass over
// the chunks before them, whose decays and states a chunk's waves compose.
//
// Bound by memory: 4 x 4096 tokens of 4096 bf16 channels, walked whole, 150 us (4.5 TB/s);
// one sequence of 8192, walked twice, 52 us (3.9 TB/s) for the chunks' ends and 63 (5.3
// TB/s) for the outputs.  Runs of 4 tokens: with 2 the batch takes 176 us and the long
// sequence 117 (with 4 both walks 102), with 8, whose values no longer fit the registers of
// four waves to a SIMD, 281 and 176.  Two channels to a lane: one load brings both.
#include "recur_common.h"

namespace cnv {
namespace {

// ENDS: the first pass, which leaves only each chunk's decay and end state.
// GATE: y is h silu(z).
template <class E, int VC, int LC, bool ENDS, bool GATE>
__global__ __launch_bounds__(64 * kRecurWaves, 4) void recur_kernel(RecurArgs a)
{
    constexpr int T = kRecurRun, W = kRecurWaves;
    typedef RecurPlace<VC, LC, T> Place;
    constexpr int kSegment = W * Place::kSpan;
    __shared__ uint32_t bits[RecurChunk::kWords];
    __shared__ float2 ends[2][W][LC * VC];
    typedef RecurRaw<E, VC> Raw;
    const int blocks = (a.chunks - (ENDS ? a.tail : 0)) * a.across, id = recur_block(blockIdx.x, blocks);
    if ((int)blockIdx.x >= (blocks + 7) / 8 * 8) {  // final states of empty sequences
        const int b = blockIdx.x - (blocks + 7) / 8 * 8;
        const Place at(b % a.across, a.d);
        const long long s0 = (long long)(b / a.across) * kRecurStateSeqs;
        for (long long s = s0 + at.wave; s < s0 + kRecurStateSeqs && s < a.q.seqs; s += W)
            if (at.mine && at.q == 0 && a.q.begin((int)s) == a.q.end((int)s)) {
                float h[VC] = {};
                if (a.initial) recur_get<VC>(a.initial, s, a.d, at.c, h);
                recur_put<VC>(a.final_state, s, a.d, at.c, h);
            }
        return;
    }
    if (id >= blocks) return;
    // the first pass leaves out the last chunk (of each sequence): nothing follows it
    int index = id / a.across;
    if (ENDS && a.per_seq) index += index / (a.per_seq - 1);
    const Place at(id % a.across, a.d);
    RecurChunk chunk(a, bits, index);
    const RecurStarts starts(a.q);
    const RecurChannels<VC> ch(a.A, a.r_bias, a.i_bias, at.c);
    const RecurRows<E, VC> xr(a.x, a.xs, a, chunk, at), rr(a.r, a.rs, a, chunk, at), ir(a.i, a.is, a, chunk, at), zr(a.z, a.zs, a, chunk, at);
    const RecurOut<E, VC> yr(a.y, a, chunk, at);

    // the next segment's values are under way while one is computed: a token's are asked
    // for as soon as its registers are free
    Raw xs[T], rs[T], is[T], zs[T];
    struct {
        __amdgpu_buffer_rsrc_t x, r, i, z;
    } next;
    auto aim = [&](const RecurSpan &span) {
        next.x = xr.span(span);
        next.r = rr.span(span);
        next.i = ir.span(span);
        if (GATE) next.z = zr.span(span);
    };
    auto load = [&](int j, auto inside) {
        constexpr bool INSIDE = decltype(inside)::value;
        rr.template load<INSIDE>(next.r, j, rs[j]);
        ir.template load<INSIDE>(next.i, j, is[j]);
        xr.template load<INSIDE>(next.x, j, xs[j]);
        if (GATE) zr.template load<INSIDE>(next.z, j, zs[j]);
    };
    const int lead = at.wave * Place::kSpan;
    aim(RecurSpan(chunk, at, lead));
#pragma unroll
    for (int j = 0; j < T; ++j) load(j, std::false_type{});

    if (!ENDS && a.joined) recur_carry<VC, W>(a.chunk_decay, a.chunk_state, chunk.before, index, 1, a.d, at, ends[1]);
    chunk.mark(a);
    float carry[VC] = {};
    RecurPiece<VC> total;
    total.clear();
    if (!ENDS && a.joined) recur_carried<VC, W>(ends[1], at, carry);  // the first segment uses ends[0]

    // INSIDE: this segment lies inside a sequence, and all of the next one's tokens are there
    auto segment = [&](int seg, auto inside) {
        constexpr bool INSIDE = decltype(inside)::value;
        const RecurSpan span(chunk, at, seg + lead);
        const RecurRun<T> run = INSIDE ? RecurRun<T>() : RecurRun<T>(chunk, at, span);
        aim(RecurSpan(chunk, at, seg + lead + kSegment));
        float av[T][VC], bv[T][VC], zv[T][VC];
#pragma unroll
        for (int j = 0; j < T; ++j) {
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const float L = ch.A[v] * recur_gate(rs[j][v], ch.rb[v]);
                av[j][v] = __builtin_amdgcn_exp2f(L);
                bv[j][v] = __builtin_amdgcn_sqrtf(one_minus_square(L, av[j][v])) * recur_gate(is[j][v], ch.ib[v]) * xs[j][v];
                if (GATE) {
                    const float z = zs[j][v];
                    zv[j][v] = z * sigmoid_f32(z);
                }
            }
            load(j, inside);
        }
        const long long t0 = chunk.c0 + seg + lead + at.q * T;
        if (!INSIDE) {
            recur_cut<VC, T>(run, bv);
            if (run.firsts && a.initial)  // what the initial states bring is an input of the first tokens
                recur_gather<VC, T>(a, starts, a.initial, run.f, t0, at, [&](int j, const float (&h)[VC]) {
#pragma unroll
                    for (int v = 0; v < VC; ++v) bv[j][v] = fmaf(av[j][v], h[v], bv[j][v]);
                });
        }
        RecurPiece<VC> p;
        recur_piece<VC, T>(run.f, run.firsts, av, bv, p);
        float h[VC];
        const int buf = seg / kSegment & 1;
        RecurJoin<VC, LC, W, false, INSIDE> join(p, at);
        join.put(ends[buf]);
        __syncthreads();
        join.get(ends[buf], carry, h, ENDS ? &total : nullptr);
        if (ENDS) return;
        const __amdgpu_buffer_rsrc_t y = yr.span(span);
#pragma unroll
        for (int j = 0; j < T; ++j) {
            float out[VC];
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                if (!INSIDE) h[v] = run.f >> j & 1 ? 0.0f : h[v];
                h[v] = fmaf(av[j][v], h[v], bv[j][v]);
                out[v] = GATE ? h[v] * zv[j][v] : h[v];
                if (!INSIDE) av[j][v] = h[v];
            }
            yr.template store<INSIDE>(y, j, out);
        }
        if (!INSIDE && run.lasts && a.final_state) recur_scatter<VC, T>(a, starts, run.last, t0, at, av, a.final_state);
    };
    for (int seg = 0, begin = 0; seg < chunk.len; seg += kSegment) {
        while (begin < seg) begin = chunk.next(seg, a.chunk);
        if (begin > seg + kSegment && seg + 2 * kSegment <= chunk.len) segment(seg, std::true_type{});
        else segment(seg, std::false_type{});
    }
    if (ENDS && at.wave == 0 && at.q == 0 && at.mine) {
        recur_put<VC>(a.chunk_decay, index, a.d, at.c, total.dec);
        recur_put<VC>(a.chunk_state, index, a.d, at.c, carry);
    }
}

// One token: a thread to VC channels of a row.  The last one's loads are moved back as
// above; states are updated in place, so it writes only the channels that are its own.
// 4 rows of 4096 channels take 4.8 us with the call, which is a launch's latency.
template <class E, int VC>
__global__ __launch_bounds__(256) void recur_step_kernel(RecurStepArgs a)
{
    using S = typename E::S;
    const int cx = (blockIdx.y * 256 + threadIdx.x) * VC, c = cx < a.d - VC ? cx : a.d - VC;
    if (cx >= a.d) return;
    const long long row = blockIdx.x;
    const int slot = a.slots ? a.slots[row] : (int)row;
    S *y = (S *)a.y + row * a.d + c;
    float out[VC] = {};
    if (slot < 0 || slot >= a.pool) {
        store_vec<E, VC>(y, VC, out);
        return;
    }
    const RecurChannels<VC> ch(a.A, a.r_bias, a.i_bias, c);
    float h[VC], x[VC], r[VC], i[VC], z[VC];
    load_vec<E, VC>((const S *)a.x + row * a.x_row + c, VC, x);
    load_vec<E, VC>((const S *)a.r + row * a.r_row + c, VC, r);
    load_vec<E, VC>((const S *)a.i + row * a.i_row + c, VC, i);
    if (a.z) load_vec<E, VC>((const S *)a.z + row * a.z_row + c, VC, z);
    recur_get<VC>(a.state, slot, a.d, c, h);
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        const float L = ch.A[v] * recur_gate(r[v], ch.rb[v]), dec = __builtin_amdgcn_exp2f(L);
        h[v] = fmaf(dec, h[v], __builtin_amdgcn_sqrtf(one_minus_square(L, dec)) * recur_gate(i[v], ch.ib[v]) * x[v]);
        out[v] = a.z ? h[v] * (z[v] * sigmoid_f32(z[v])) : h[v];
    }
    if (c == cx) {
        recur_put<VC>(a.state, slot, a.d, c, h);
        store_vec<E, VC>(y, VC, out);
    } else {
#pragma unroll
        for (int v = 1; v < VC; ++v)
            if (c + v >= cx) {
                a.state[(long long)slot * a.d + c + v] = h[v];
                y[v] = E::from(out[v]);
            }
    }
}

template <class E, int VC, int LC>
hipError_t launch_shape(const RecurArgs &a, hipStream_t st)
{
    if (a.joined) {
        const unsigned blocks = (unsigned)((a.chunks - a.tail) * a.across);
        recur_kernel<E, VC, LC, true, false><<<(blocks + 7) / 8 * 8, 64 * kRecurWaves, 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const unsigned blocks = (unsigned)(a.chunks * a.across), states = a.final_state ? (unsigned)((a.q.seqs + kRecurStateSeqs - 1) / kRecurStateSeqs) : 0;
    const unsigned grid = (blocks + 7) / 8 * 8 + states * a.across;
    if (a.z) recur_kernel<E, VC, LC, false, true><<<grid, 64 * kRecurWaves, 0, st>>>(a);
    else recur_kernel<E, VC, LC, false, false><<<grid, 64 * kRecurWaves, 0, st>>>(a);
    return hipGetLastError();
}
template <class E>
hipError_t launch(const RecurArgs &a, const RecurShape &s, hipStream_t st)
{
    return recur_by_shape<E>(s, [&](auto vc, auto lc) { return launch_shape<E, decltype(vc)::value, decltype(lc)::value>(a, st); });
}

}  // namespace

hipError_t launch_recurrence(int dtype, const RecurArgs &a, const RecurShape &s, hipStream_t st)
{
    switch (dtype) {
        case CONV2D_DTYPE_F16: return launch<SF16>(a, s, st);
        case CONV2D_DTYPE_BF16: return launch<SBF16>(a, s, st);
        default: return launch<SF32>(a, s, st);
    }
}

template <class E>
static hipError_t launch_step(const RecurStepArgs &a, hipStream_t st)
{
    constexpr int VC = kRecurStepChannels;
    if (a.d < VC) recur_step_kernel<E, 1><<<(unsigned)a.rows, 256, 0, st>>>(a);
    else recur_step_kernel<E, VC><<<dim3((unsigned)a.rows, (unsigned)((a.d + 256 * VC - 1) / (256 * VC))), 256, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_recurrence_step(int dtype, const RecurStepArgs &a, hipStream_t st)
{
    switch (dtype) {
        case CONV2D_DTYPE_F16: return launch_step<SF16>(a, st);
        case CONV2D_DTYPE_BF16: return launch_step<SBF16>(a, st);
        default: return launch_step<SF32>(a, st);
    }
}

}  // namespace cnv
