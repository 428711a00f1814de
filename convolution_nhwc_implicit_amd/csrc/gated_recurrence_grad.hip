// gated_recurrence_grad.hip -- gradients of the gated linear recurrence.
//
// With L = A g, b = sqrt(1 - a^2) u x, G = dy silu(z) and k the gradient of a state:
//   k = G + (what flows in from the next token);  flows on: a k
//   dx = k sqrt(1 - a^2) u;  di = k b (1 - u);  dz = dy h silu'(z)
//   dL = k (a h_before - a^2 / (1 - a^2) b);  dr = dL L (1 - g);  dA = sum dL g
// dL L is what is computed: L / (1 - a^2) goes to -1/2 with L, where the quotient alone has
// no bound; dA is the sum of dL L over A.  1 - g and 1 - u come from the gates' exponentials:
// as differences they would be off by 2^-24, whatever their size.
//
// Two walks over each chunk, in segments whose waves take successive runs as in the
// forward pass.  The first goes forwards and leaves, for every segment, what the
// chunk's tokens before it do to a state, and for the chunk what its tokens do to a
// state and to the gradient that flows back through it.  The second goes backwards: a
// segment's states come from what the first walk left, its gradients from behind.
//
// Bound by memory: 4 x 4096 tokens of 4096 bf16 channels 109 us (3.7 TB/s) for the first
// walk, which writes what the second one needs of a segment, and 262 us (4.6 TB/s) for the
// second, which holds some 200 registers: two waves to a SIMD.  Runs of 8 tokens spill
// (both walks 1127 us for 370); with 2 they take 493.
#include "recur_common.h"

namespace cnv {
namespace {

template <class E, int VC>
struct Tensors {
    RecurRows<E, VC> x, r, i, z, dy;
    template <class Place>
    __device__ inline Tensors(const RecurArgs &a, const RecurChunk &k, const Place &at)
        : x(a.x, a.xs, a, k, at), r(a.r, a.rs, a, k, at), i(a.i, a.is, a, k, at), z(a.z, a.zs, a, k, at), dy(a.dy, a.dys, a, k, at)
    {
    }
};

// The first walk.  BACK: sequences may go on in another chunk, which needs the
// gradient's flow through this one.
template <class E, int VC, int LC, bool BACK>
__global__ __launch_bounds__(64 * kRecurWaves) void recur_states_kernel(RecurArgs a)
{
    constexpr int T = kRecurRun, W = kRecurWaves;
    typedef RecurPlace<VC, LC, T> Place;
    constexpr int kSegment = W * Place::kSpan;
    __shared__ uint32_t bits[RecurChunk::kWords];
    __shared__ float2 ends[2][BACK ? 2 : 1][W][LC * VC];
    typedef RecurRaw<E, VC> Raw;
    const int blocks = a.chunks * a.across, id = recur_block(blockIdx.x, blocks);
    if (id >= blocks) return;
    const int index = id / a.across;
    const Place at(id % a.across, a.d);
    RecurChunk chunk(a, bits, index);
    const RecurStarts starts(a.q);
    const RecurChannels<VC> ch(a.A, a.r_bias, a.i_bias, at.c);
    const Tensors<E, VC> in(a, chunk, at);
    const bool gate = BACK && a.z;
    float state[VC] = {};
    RecurPiece<VC> total, back;
    total.clear();
    back.clear();
    const int lead = at.wave * Place::kSpan;
    Raw xs[T], rs[T], is[T], zs[T], ds[T];
    struct {
        __amdgpu_buffer_rsrc_t x, r, i, z, dy;
    } next;
    auto aim = [&](const RecurSpan &span) {
        next.x = in.x.span(span);
        next.r = in.r.span(span);
        next.i = in.i.span(span);
        if (BACK) {
            next.dy = in.dy.span(span);
            next.z = in.z.span(span);
        }
    };
    auto load = [&](int j, auto inside) {
        constexpr bool INSIDE = decltype(inside)::value;
        in.r.template load<INSIDE>(next.r, j, rs[j]);
        in.i.template load<INSIDE>(next.i, j, is[j]);
        in.x.template load<INSIDE>(next.x, j, xs[j]);
        if (BACK) {
            in.dy.template load<INSIDE>(next.dy, j, ds[j]);
            in.z.template load<INSIDE>(next.z, j, zs[j]);
        }
    };
    aim(RecurSpan(chunk, at, lead));
#pragma unroll
    for (int j = 0; j < T; ++j) load(j, std::false_type{});
    chunk.mark(a);
    // INSIDE: this segment lies inside a sequence, and all of the next one's tokens are there
    auto segment = [&](int seg, auto inside) {
        constexpr bool INSIDE = decltype(inside)::value;
        const int buf = seg / kSegment & 1;
        if (at.wave == 0 && at.q == 0 && at.mine) {
            const long long k = (long long)index * (a.chunk / kSegment) + seg / kSegment;
            recur_put<VC>(a.seg_decay, k, a.d, at.c, total.dec);
            recur_put<VC>(a.seg_state, k, a.d, at.c, state);
        }
        const RecurSpan span(chunk, at, seg + lead);
        const RecurRun<T> run = INSIDE ? RecurRun<T>() : RecurRun<T>(chunk, at, span);
        aim(RecurSpan(chunk, at, seg + lead + kSegment));
        float av[T][VC], bv[T][VC], gv[T][VC];
#pragma unroll
        for (int j = 0; j < T; ++j) {
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const float L = ch.A[v] * recur_gate(rs[j][v], ch.rb[v]);
                av[j][v] = __builtin_amdgcn_exp2f(L);
                bv[j][v] = __builtin_amdgcn_sqrtf(one_minus_square(L, av[j][v])) * recur_gate(is[j][v], ch.ib[v]) * xs[j][v];
                if (BACK) {
                    const float z = zs[j][v];
                    gv[j][v] = gate ? ds[j][v] * (z * sigmoid_f32(z)) : ds[j][v];
                }
            }
            load(j, inside);
        }
        if (!INSIDE) {
            recur_cut<VC, T>(run, bv);
            if (BACK) recur_cut<VC, T>(run, gv);
        }
        const long long t0 = chunk.c0 + seg + lead + at.q * T;
        if (!INSIDE && run.firsts && a.initial)
            recur_gather<VC, T>(a, starts, a.initial, run.f, t0, at, [&](int j, const float (&h)[VC]) {
#pragma unroll
                for (int v = 0; v < VC; ++v) bv[j][v] = fmaf(av[j][v], h[v], bv[j][v]);
            });
        RecurPiece<VC> p;
        recur_piece<VC, T>(run.f, run.firsts, av, bv, p);
        RecurJoin<VC, LC, W, false, INSIDE> join(p, at);
        join.put(ends[buf][0]);
        if constexpr (BACK) {
            if (!INSIDE && run.lasts && a.dfinal)
                recur_gather<VC, T>(a, starts, a.dfinal, run.last, t0, at, [&](int j, const float (&k)[VC]) {
#pragma unroll
                    for (int v = 0; v < VC; ++v) gv[j][v] += k[v];
                });
            RecurPiece<VC> flow;
            recur_flow<VC, T>(run.last, run.lasts, av, gv, flow);
            RecurJoin<VC, LC, W, true, INSIDE>(flow, at).put(ends[buf][1]);
        }
        __syncthreads();
        float h[VC];
        join.get(ends[buf][0], state, h, &total);
        if constexpr (BACK) {  // the segment's flow, behind the chunk's so far
#pragma unroll 4
            for (int w = W - 1; w >= 0; --w) {
                RecurPiece<VC> s;
                s.get(&ends[buf][1][w][at.slot]);
                back.template after<false>(s);
            }
        }
    };
    for (int seg = 0, begin = 0; seg < chunk.len; seg += kSegment) {
        while (begin < seg) begin = chunk.next(seg, a.chunk);
        if (begin > seg + kSegment && seg + 2 * kSegment <= chunk.len) segment(seg, std::true_type{});
        else segment(seg, std::false_type{});
    }
    if (BACK && at.wave == 0 && at.q == 0 && at.mine) {
        recur_put<VC>(a.chunk_decay, index, a.d, at.c, total.dec);
        recur_put<VC>(a.chunk_state, index, a.d, at.c, state);
        recur_put<VC>(a.back_decay, index, a.d, at.c, back.dec);
        recur_put<VC>(a.chunk_back, index, a.d, at.c, back.end);
    }
}

template <class E, int VC, int LC>
__global__ __launch_bounds__(64 * kRecurWaves) void recur_grad_kernel(RecurArgs a)
{
    constexpr int T = kRecurRun, W = kRecurWaves;
    typedef RecurPlace<VC, LC, T> Place;
    constexpr int kSegment = W * Place::kSpan;
    __shared__ uint32_t bits[RecurChunk::kWords];
    __shared__ float2 ends[2][2][W][LC * VC];
    typedef RecurRaw<E, VC> Raw;
    const int blocks = a.chunks * a.across, id = recur_block(blockIdx.x, blocks);
    if ((int)blockIdx.x >= (blocks + 7) / 8 * 8) {  // initial states of empty sequences
        const int b = blockIdx.x - (blocks + 7) / 8 * 8;
        const Place at(b % a.across, a.d);
        const long long s0 = (long long)(b / a.across) * kRecurStateSeqs;
        for (long long s = s0 + at.wave; s < s0 + kRecurStateSeqs && s < a.q.seqs; s += W)
            if (at.mine && at.q == 0 && a.q.begin((int)s) == a.q.end((int)s)) {
                float k[VC] = {};
                if (a.dfinal) recur_get<VC>(a.dfinal, s, a.d, at.c, k);
                recur_put<VC>(a.dinitial, s, a.d, at.c, k);
            }
        return;
    }
    if (id >= blocks) return;
    const int index = id / a.across;
    const Place at(id % a.across, a.d);
    RecurChunk chunk(a, bits, index);
    const RecurStarts starts(a.q);
    const RecurChannels<VC> ch(a.A, a.r_bias, a.i_bias, at.c);
    const Tensors<E, VC> in(a, chunk, at);
    const RecurOut<E, VC> dxr(a.dx, a, chunk, at), drr(a.dr, a, chunk, at), dir(a.di, a, chunk, at), dzr(a.dz, a, chunk, at);
    const bool gate = a.z;
    float dll[VC] = {}, drb[VC] = {}, dib[VC] = {};
    const int segs = (chunk.len + kSegment - 1) / kSegment;
    Raw xs[T], rs[T], is[T], zs[T], ds[T];
    struct {
        __amdgpu_buffer_rsrc_t x, r, i, z, dy;
    } next;
    auto aim = [&](const RecurSpan &span) {
        next.x = in.x.span(span);
        next.r = in.r.span(span);
        next.i = in.i.span(span);
        next.dy = in.dy.span(span);
        next.z = in.z.span(span);
    };
    auto load = [&](int j, auto inside) {
        constexpr bool INSIDE = decltype(inside)::value;
        in.r.template load<INSIDE>(next.r, j, rs[j]);
        in.i.template load<INSIDE>(next.i, j, is[j]);
        in.x.template load<INSIDE>(next.x, j, xs[j]);
        in.dy.template load<INSIDE>(next.dy, j, ds[j]);
        in.z.template load<INSIDE>(next.z, j, zs[j]);
    };
    const int lead = at.wave * Place::kSpan;
    aim(RecurSpan(chunk, at, (segs > 0 ? segs - 1 : 0) * kSegment + lead));
#pragma unroll
    for (int j = 0; j < T; ++j) load(j, std::false_type{});
    float start[VC] = {}, flow[VC] = {};  // the state the chunk starts with; the gradient that flows in behind it
    const int other = segs & 1;  // the last segment, which comes first, uses the other half of ends
    if (a.joined) {
        const int after = a.per_seq ? chunk.before + a.per_seq : a.chunks;
        recur_carry<VC, W>(a.chunk_decay, a.chunk_state, chunk.before, index, 1, a.d, at, ends[other][0]);
        recur_carry<VC, W>(a.back_decay, a.chunk_back, after - 1, index, -1, a.d, at, ends[other][1]);
    }
    chunk.mark(a);
    if (a.joined) {
        recur_carried<VC, W>(ends[other][0], at, start);
        recur_carried<VC, W>(ends[other][1], at, flow);
    }
    // INSIDE: this segment lies inside a sequence, and another one is before it
    auto segment = [&](int seg, auto inside) {
        constexpr bool INSIDE = decltype(inside)::value;
        const int buf = seg / kSegment & 1;
        const RecurSpan span(chunk, at, seg + lead);
        const RecurRun<T> run = INSIDE ? RecurRun<T>() : RecurRun<T>(chunk, at, span);
        const long long t0 = chunk.c0 + seg + lead + at.q * T, k0 = (long long)index * (a.chunk / kSegment) + seg / kSegment;
        RecurPiece<VC> until;  // the chunk before this segment
        recur_get<VC>(a.seg_decay, k0, a.d, at.c, until.dec);
        recur_get<VC>(a.seg_state, k0, a.d, at.c, until.end);
        aim(RecurSpan(chunk, at, seg > 0 ? seg + lead - kSegment : segs * kSegment));
        // su: sqrt(1 - a^2) u; rest, shut: 1 - g, 1 - u; hv: the inputs, then the states before the tokens; qv: dz by h
        float Lv[T][VC], av[T][VC], su[T][VC], rest[T][VC], shut[T][VC], hv[T][VC], gv[T][VC], qv[T][VC];
        Raw x[T];
#pragma unroll
        for (int j = 0; j < T; ++j) {
            x[j] = xs[j];
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                Lv[j][v] = ch.A[v] * recur_gate(rs[j][v], ch.rb[v], rest[j][v]);
                av[j][v] = __builtin_amdgcn_exp2f(Lv[j][v]);
                su[j][v] = __builtin_amdgcn_sqrtf(one_minus_square(Lv[j][v], av[j][v])) * recur_gate(is[j][v], ch.ib[v], shut[j][v]);
                hv[j][v] = su[j][v] * x[j][v];
                const float dy = ds[j][v];
                const float z = zs[j][v], s = sigmoid_f32(z);
                gv[j][v] = gate ? dy * (z * s) : dy;
                qv[j][v] = dy * (s * (1.0f + z * (1.0f - s)));
            }
            load(j, inside);
        }
        if (!INSIDE) {
            recur_cut<VC, T>(run, hv);
            recur_cut<VC, T>(run, gv);
        }
        if (!INSIDE && run.firsts && a.initial)
            recur_gather<VC, T>(a, starts, a.initial, run.f, t0, at, [&](int j, const float (&h)[VC]) {
#pragma unroll
                for (int v = 0; v < VC; ++v) hv[j][v] = fmaf(av[j][v], h[v], hv[j][v]);
            });
        if (!INSIDE && run.lasts && a.dfinal)
            recur_gather<VC, T>(a, starts, a.dfinal, run.last, t0, at, [&](int j, const float (&k)[VC]) {
#pragma unroll
                for (int v = 0; v < VC; ++v) gv[j][v] += k[v];
            });
        RecurPiece<VC> p;
        recur_piece<VC, T>(run.f, run.firsts, av, hv, p);
        RecurJoin<VC, LC, W, false, INSIDE> states(p, at);
        states.put(ends[buf][0]);
        recur_flow<VC, T>(run.last, run.lasts, av, gv, p);
        RecurJoin<VC, LC, W, true, INSIDE> flows(p, at);
        flows.put(ends[buf][1]);
        __syncthreads();
        float h[VC], k[VC], begin[VC];
#pragma unroll
        for (int v = 0; v < VC; ++v) begin[v] = start[v];
        until.template carry<false>(begin);
        states.get(ends[buf][0], begin, h, nullptr);
        flows.get(ends[buf][1], flow, k, nullptr);
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                if (!INSIDE) h[v] = run.f >> j & 1 ? 0.0f : h[v];
                const float b = hv[j][v];
                hv[j][v] = h[v];
                h[v] = fmaf(av[j][v], h[v], b);
            }
        if (!INSIDE && run.firsts && a.initial)
            recur_gather<VC, T>(a, starts, a.initial, run.f, t0, at, [&](int j, const float (&h0)[VC]) {
#pragma unroll
                for (int v = 0; v < VC; ++v) hv[j][v] = h0[v];
            });
        if (!INSIDE) recur_cut<VC, T>(run, hv);  // nothing times nothing for the sums, also behind a spoilt state
        const __amdgpu_buffer_rsrc_t dx = dxr.span(span), dr = drr.span(span), di = dir.span(span), dz = dzr.span(span);
#pragma unroll
        for (int j = T - 1; j >= 0; --j) {
            float ox[VC], orr[VC], oi[VC], oz[VC];
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const float L = Lv[j][v], dec = av[j][v], xx = x[j][v], b = su[j][v] * xx;
                // L / (1 - a^2) by an inverse that is finite where a is 1: it meets L and b there, which are 0
                const float ratio = L * __builtin_amdgcn_rcpf(fmaxf(one_minus_square(L, dec), 1.2e-38f));
                if (!INSIDE) k[v] = run.last >> j & 1 ? 0.0f : k[v];
                k[v] += gv[j][v];
                const float dl = kLn2 * k[v] * (L * dec * hv[j][v] - ratio * dec * (dec * b));  // dL * L; a first, which is 0 for the largest L
                orr[v] = dl * rest[j][v];
                oi[v] = k[v] * b * shut[j][v];
                ox[v] = k[v] * su[j][v];
                oz[v] = qv[j][v] * fmaf(dec, hv[j][v], b);
                dll[v] += dl;
                drb[v] += orr[v];
                dib[v] += oi[v];
                k[v] *= dec;
                gv[j][v] = k[v];
            }
            dxr.template store<INSIDE>(dx, j, ox);
            drr.template store<INSIDE>(dr, j, orr);
            dir.template store<INSIDE>(di, j, oi);
            dzr.template store<INSIDE>(dz, j, oz);
            __builtin_amdgcn_sched_barrier(0);  // a token's roots, worked out for all of them at once, would spill
        }
        if (!INSIDE && run.firsts && a.dinitial) recur_scatter<VC, T>(a, starts, run.f, t0, at, gv, a.dinitial);
    };
    for (int sg = segs - 1; sg >= 0; --sg) {
        // whether a sequence begins in it or right behind it, or tokens are missing
        const int seg = sg * kSegment;
        if (sg > 0 && seg + kSegment <= chunk.len && chunk.next(seg, a.chunk) > seg + kSegment) segment(seg, std::true_type{});
        else segment(seg, std::false_type{});
    }
    // the sums of a wave's groups, then the waves' in order
    __syncthreads();
    float *sums = (float *)ends;
    static_assert(sizeof(ends) >= sizeof(float) * W * 3 * LC * VC, "room for the sums");
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        float s[3] = {dll[v], drb[v], dib[v]};
#pragma unroll
        for (int i = 0; i < 3; ++i) {
#pragma unroll
            for (int o = LC; o < 64; o *= 2) s[i] += __shfl_xor(s[i], o);
            if (at.q == 0) sums[(at.wave * 3 + i) * LC * VC + at.slot + v] = s[i];
        }
    }
    __syncthreads();
    if (at.wave < 3 && at.q == 0 && at.mine) {
        float s[VC] = {};
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int v = 0; v < VC; ++v) s[v] += sums[(w * 3 + at.wave) * LC * VC + at.slot + v];
        recur_put<VC>(a.partial, (long long)index * 3 + at.wave, a.d, at.c, s);
    }
}

template <class E, int VC, int LC>
hipError_t launch_shape(const RecurArgs &a, hipStream_t st)
{
    const unsigned blocks = ((unsigned)(a.chunks * a.across) + 7) / 8 * 8, threads = 64 * kRecurWaves;
    if (blocks > 0) {
        if (a.joined) recur_states_kernel<E, VC, LC, true><<<blocks, threads, 0, st>>>(a);
        else recur_states_kernel<E, VC, LC, false><<<blocks, threads, 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const unsigned states = a.dinitial ? (unsigned)((a.q.seqs + kRecurStateSeqs - 1) / kRecurStateSeqs) * a.across : 0;
    if (blocks + states > 0) recur_grad_kernel<E, VC, LC><<<blocks + states, threads, 0, st>>>(a);
    return hipGetLastError();
}
template <class E>
hipError_t launch(const RecurArgs &a, const RecurShape &s, hipStream_t st)
{
    return recur_by_shape<E>(s, [&](auto vc, auto lc) { return launch_shape<E, decltype(vc)::value, decltype(lc)::value>(a, st); });
}

}  // namespace

hipError_t launch_recurrence_grad(int dtype, const RecurArgs &a, const RecurShape &s, hipStream_t st)
{
    switch (dtype) {
        case CONV2D_DTYPE_F16: return launch<SF16>(a, s, st);
        case CONV2D_DTYPE_BF16: return launch<SBF16>(a, s, st);
        default: return launch<SF32>(a, s, st);
    }
}

}  // namespace cnv
