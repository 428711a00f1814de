// gated_recurrence_grad.hip -- gradients of the gated linear recurrence.
//
// With L = A g, b = sqrt(1 - a^2) u x, G = dy silu(z) and k the gradient of a state:
//   k = G + (what flows in from the next token);  flows on: a k
//   dx = k sqrt(1 - a^2) u;  di = k b (1 - u);  dz = dy h silu'(z)
//   dL = k (a h_before - a^2 / sqrt(1 - a^2) u x);  dr = dL L (1 - g);  dA = sum dL g
// dL L is what is computed: L / sqrt(1 - a^2) goes to 0 with L, where the root's own
// derivative has no bound; dA is the sum of dL L over A.
//
// Two walks over each chunk, in segments whose waves take successive runs as in the
// forward pass.  The first goes forwards and leaves, for every segment, what the
// chunk's tokens before it do to a state, and for the chunk what its tokens do to a
// state and to the gradient that flows back through it.  The second goes backwards: a
// segment's states come from what the first walk left, its gradients from behind.
#include "recur_common.h"

namespace cnv {
namespace {

struct Token {
    float g, u, L, a, x;
    template <class E>
    __device__ static inline Token of(const RecurChannel &ch, E, float r, float i, float x)
    {
        Token k;
        k.g = sigmoid_f32(r + ch.rb);
        k.u = sigmoid_f32(i + ch.ib);
        k.L = ch.A * k.g;
        k.a = __builtin_amdgcn_exp2f(k.L * kLog2e);
        k.x = x;
        return k;
    }
};

// A run's values as they lie in memory.
template <class E, int T>
struct Loads {
    typename E::S x[T], r[T], i[T], z[T], dy[T];
};
template <class E>
struct Tensors {
    RecurRows<E> x, r, i, z, dy;
    bool gate;
    __device__ inline Tensors(const RecurArgs &a, const RecurChunk &k, int c)
        : x(a.x, a.xs, k, a.q.len, a.per_seq, c), r(a.r, a.rs, k, a.q.len, a.per_seq, c), i(a.i, a.is, k, a.q.len, a.per_seq, c),
          z(a.z, a.zs, k, a.q.len, a.per_seq, c), dy(a.dy, a.dys, k, a.q.len, a.per_seq, c), gate(a.z != nullptr)
    {
    }
    template <bool BACK, int T>
    __device__ inline void load(const RecurRun<T> &run, Loads<E, T> &v) const
    {
        x.load(run, v.x);
        r.load(run, v.r);
        i.load(run, v.i);
        if (BACK) {
            dy.load(run, v.dy);
            if (gate) z.load(run, v.z);
        }
    }
};

// What a run does to a state, and to the gradient that flows back through it.
struct Piece {
    float dec = 1.0f, end = 0.0f, bdec = 1.0f, flow = 0.0f;
};
template <int T>
__device__ inline void state_piece(const RecurArgs &a, const RecurRun<T> &run, int c, const float (&av)[T], const float (&bv)[T], Piece &p)
{
    if (run.f == 0) {
#pragma unroll
        for (int j = 0; j < T; ++j) {
            p.dec *= av[j];
            p.end = fmaf(av[j], p.end, bv[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < T; ++j) {
            if (run.f >> j & 1) {
                p.dec = -1.0f;
                p.end = a.initial ? a.initial[(long long)a.q.find(run.t0 + j) * a.d + c] : 0.0f;
            }
            p.dec = p.dec < 0.0f ? p.dec : p.dec * av[j];
            p.end = fmaf(av[j], p.end, bv[j]);
        }
    }
}
template <int T>
__device__ inline float final_gradient(const RecurArgs &a, const RecurRun<T> &run, int c, int j)
{
    return a.dfinal ? a.dfinal[(long long)a.q.find(run.t0 + j) * a.d + c] : 0.0f;
}
template <int T>
__device__ inline void flow_piece(const RecurArgs &a, const RecurRun<T> &run, int c, const float (&av)[T], const float (&G)[T], Piece &p)
{
    if (run.last == 0) {
#pragma unroll
        for (int j = T - 1; j >= 0; --j) {
            p.flow = av[j] * (p.flow + G[j]);
            p.bdec *= av[j];
        }
    } else {
#pragma unroll
        for (int j = T - 1; j >= 0; --j) {
            if (run.last >> j & 1) {
                p.bdec = -1.0f;
                p.flow = final_gradient(a, run, c, j);
            }
            p.flow = av[j] * (p.flow + G[j]);
            p.bdec = p.bdec < 0.0f ? p.bdec : p.bdec * av[j];
        }
    }
}
// tokens that are not there: nothing decays, nothing comes in
template <int T>
__device__ inline void cut_run(const RecurRun<T> &run, float (&av)[T], float (&in)[T])
{
    if (run.n < T)
#pragma unroll
        for (int j = 0; j < T; ++j) {
            av[j] = j < run.n ? av[j] : 1.0f;
            in[j] = j < run.n ? in[j] : 0.0f;
        }
}

// The first walk.  BACK: sequences may go on in another chunk, which needs the
// gradient's flow through this one.
template <class E, bool BACK>
__global__ __launch_bounds__(64 * kRecurGradWaves) void recur_states_kernel(RecurArgs a)
{
    constexpr int T = kRecurGradRun, W = kRecurGradWaves;
    __shared__ uint32_t bits[RecurChunk::kWords];
    __shared__ float ends[2][BACK ? 4 : 2][W][64];
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int cx = blockIdx.y * kRecurChannels + lane, c = cx < a.d ? cx : a.d - 1;
    const bool mine = cx < a.d;
    const RecurChunk chunk(a, bits, blockIdx.x);
    const RecurChannel ch(a.A, a.r_bias, a.i_bias, c);
    const Tensors<E> in(a, chunk, c);
    float decay = 1.0f, state = 0.0f, bdecay = 1.0f, flow = 0.0f;
    long long seg = (long long)blockIdx.x * (a.chunk / (T * W));
    Loads<E, T> v;
    if (chunk.len > 0) in.template load<BACK>(RecurRun<T>(chunk, wave * T), v);
    for (int at0 = 0, buf = 0; at0 < chunk.len; at0 += T * W, buf ^= 1, ++seg) {
        const RecurRun<T> run(chunk, at0 + wave * T);
        if (wave == 0 && mine) {
            a.seg_decay[seg * a.d + c] = decay;
            a.seg_state[seg * a.d + c] = state;
        }
        float av[T], bv[T], G[T];
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const Token k = Token::of(ch, E{}, E::to(v.r[j]), E::to(v.i[j]), E::to(v.x[j]));
            av[j] = k.a;
            bv[j] = __builtin_amdgcn_sqrtf(one_minus_square(k.L, k.a)) * k.u * k.x;
            if (BACK) {
                G[j] = E::to(v.dy[j]);
                if (in.gate) {
                    const float z = E::to(v.z[j]);
                    G[j] *= z * sigmoid_f32(z);
                }
            }
        }
        in.template load<BACK>(RecurRun<T>(chunk, at0 + T * W + wave * T), v);
        cut_run(run, av, bv);
        Piece p;
        state_piece(a, run, c, av, bv, p);
        if constexpr (BACK) {
            cut_run(run, av, G);
            flow_piece(a, run, c, av, G, p);
        }
        ends[buf][0][wave][lane] = p.dec;
        ends[buf][1][wave][lane] = p.end;
        if constexpr (BACK) {
            ends[buf][2][wave][lane] = p.bdec;
            ends[buf][3][wave][lane] = p.flow;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float d = ends[buf][0][w][lane];
            state = through(d, ends[buf][1][w][lane], state);
            decay = joined_decay(decay, d);
            if constexpr (BACK) {
                if (bdecay >= 0.0f) flow = fmaf(bdecay, ends[buf][3][w][lane], flow);
                bdecay = joined_decay(bdecay, ends[buf][2][w][lane]);
            }
        }
    }
    if (BACK && wave == 0 && mine) {
        const long long at = (long long)blockIdx.x * a.d + c;
        a.chunk_decay[at] = decay;
        a.chunk_state[at] = state;
        a.back_decay[at] = bdecay;
        a.chunk_back[at] = flow;
    }
}

template <class E>
__global__ __launch_bounds__(64 * kRecurGradWaves) void recur_grad_kernel(RecurArgs a)
{
    constexpr int T = kRecurGradRun, W = kRecurGradWaves;
    __shared__ uint32_t bits[RecurChunk::kWords];
    __shared__ float ends[2][4][W][64];
    using S = typename E::S;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int cx = blockIdx.y * kRecurChannels + lane, c = cx < a.d ? cx : a.d - 1;
    const bool mine = cx < a.d;
    if ((int)blockIdx.x >= a.chunks) {  // initial states of empty sequences
        const long long s0 = (long long)(blockIdx.x - a.chunks) * kRecurStateSeqs;
        for (long long s = s0 + wave; s < s0 + kRecurStateSeqs && s < a.q.seqs; s += W)
            if (mine && a.q.begin((int)s) == a.q.end((int)s))
                a.dinitial[s * a.d + c] = a.dfinal ? a.dfinal[s * a.d + c] : 0.0f;
        return;
    }
    const RecurChunk chunk(a, bits, blockIdx.x);
    const RecurChannel ch(a.A, a.r_bias, a.i_bias, c);
    const Tensors<E> in(a, chunk, c);
    float before = 0.0f, flow = 0.0f;  // the state the chunk starts with; the gradient that flows in behind it
    if (a.joined) {
        const int after = a.per_seq ? chunk.before + a.per_seq : a.chunks;
        for (int k = chunk.before; k < (int)blockIdx.x; ++k)
            before = through(a.chunk_decay[(long long)k * a.d + c], a.chunk_state[(long long)k * a.d + c], before);
        for (int k = after - 1; k > (int)blockIdx.x; --k)
            flow = through(a.back_decay[(long long)k * a.d + c], a.chunk_back[(long long)k * a.d + c], flow);
    }
    float dll = 0.0f, drb = 0.0f, dib = 0.0f;
    const int segs = (chunk.len + T * W - 1) / (T * W);
    Loads<E, T> v;
    if (segs > 0) in.template load<true>(RecurRun<T>(chunk, ((segs - 1) * W + wave) * T), v);
    for (int sg = segs - 1, buf = 0; sg >= 0; --sg, buf ^= 1) {
        const RecurRun<T> run(chunk, (sg * W + wave) * T);
        float xv[T], gv[T], uv[T], Lv[T], av[T], bv[T], wv[T], zv[T], dv[T], G[T];
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const Token k = Token::of(ch, E{}, E::to(v.r[j]), E::to(v.i[j]), E::to(v.x[j]));
            xv[j] = k.x;
            gv[j] = k.g;
            uv[j] = k.u;
            Lv[j] = k.L;
            av[j] = k.a;
            wv[j] = one_minus_square(k.L, k.a);
            bv[j] = __builtin_amdgcn_sqrtf(wv[j]) * k.u * k.x;
            dv[j] = E::to(v.dy[j]);
            zv[j] = 0.0f;
            G[j] = dv[j];
            if (in.gate) {
                zv[j] = E::to(v.z[j]);
                G[j] *= zv[j] * sigmoid_f32(zv[j]);
            }
        }
        if (sg > 0) in.template load<true>(RecurRun<T>(chunk, ((sg - 1) * W + wave) * T), v);
        cut_run(run, av, bv);
        cut_run(run, av, G);
        Piece p;
        state_piece(a, run, c, av, bv, p);
        flow_piece(a, run, c, av, G, p);
        ends[buf][0][wave][lane] = p.dec;
        ends[buf][1][wave][lane] = p.end;
        ends[buf][2][wave][lane] = p.bdec;
        ends[buf][3][wave][lane] = p.flow;
        __syncthreads();
        const long long seg = (long long)blockIdx.x * (a.chunk / (T * W)) + sg;
        float h = through(a.seg_decay[seg * a.d + c], a.seg_state[seg * a.d + c], before);
        float k = flow;
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (w < wave) h = through(ends[buf][0][w][lane], ends[buf][1][w][lane], h);
#pragma unroll
        for (int w = W - 1; w >= 0; --w) {
            flow = through(ends[buf][2][w][lane], ends[buf][3][w][lane], flow);
            if (w > wave) k = flow;
        }
        float hv[T];  // the states before each token
#pragma unroll
        for (int j = 0; j < T; ++j) {
            if (run.f >> j & 1) h = a.initial ? a.initial[(long long)a.q.find(run.t0 + j) * a.d + c] : 0.0f;
            hv[j] = h;
            h = fmaf(av[j], h, bv[j]);
        }
#pragma unroll
        for (int j = T - 1; j >= 0; --j) {
            if (j >= run.n) continue;
            if (run.last >> j & 1) k = final_gradient(a, run, c, j);
            const float root = __builtin_amdgcn_rsqf(fmaxf(wv[j], 1.2e-38f)), size = wv[j] * root;
            const float in_ = uv[j] * xv[j], hj = fmaf(av[j], hv[j], bv[j]);
            float dz = 0.0f;
            if (in.gate) {
                const float s = sigmoid_f32(zv[j]);
                dz = dv[j] * hj * (s * (1.0f + zv[j] * (1.0f - s)));
            }
            k += G[j];
            const float dl = k * (av[j] * hv[j] * Lv[j] - av[j] * av[j] * in_ * (Lv[j] * root));  // dL * L
            const float dr = dl * (1.0f - gv[j]), di = k * bv[j] * (1.0f - uv[j]);
            dll += dl;
            drb += dr;
            dib += di;
            if (mine) {
                const long long at = (run.t0 + j) * a.d + c;
                ((S *)a.dx)[at] = E::from(k * size * uv[j]);
                ((S *)a.dr)[at] = E::from(dr);
                ((S *)a.di)[at] = E::from(di);
                if (in.gate) ((S *)a.dz)[at] = E::from(dz);
            }
            k *= av[j];
            if ((run.f >> j & 1) && a.dinitial && mine) a.dinitial[(long long)a.q.find(run.t0 + j) * a.d + c] = k;
        }
    }
    // the waves' sums in order
    __syncthreads();
    float *sums = &ends[0][0][0][0];
    sums[(wave * 3 + 0) * 64 + lane] = dll;
    sums[(wave * 3 + 1) * 64 + lane] = drb;
    sums[(wave * 3 + 2) * 64 + lane] = dib;
    __syncthreads();
    if (wave < 3 && mine) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += sums[(w * 3 + wave) * 64 + lane];
        a.partial[((long long)blockIdx.x * 3 + wave) * a.d + c] = s;
    }
}

template <class E>
hipError_t launch(const RecurArgs &a, hipStream_t st)
{
    const unsigned by = (unsigned)((a.d + kRecurChannels - 1) / kRecurChannels);
    const dim3 grid((unsigned)a.chunks, by);
    if (a.chunks > 0) {
        if (a.joined) recur_states_kernel<E, true><<<grid, 64 * kRecurGradWaves, 0, st>>>(a);
        else recur_states_kernel<E, false><<<grid, 64 * kRecurGradWaves, 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const unsigned states = a.dinitial ? (unsigned)((a.q.seqs + kRecurStateSeqs - 1) / kRecurStateSeqs) : 0;
    if (a.chunks + states > 0) recur_grad_kernel<E><<<dim3((unsigned)a.chunks + states, by), 64 * kRecurGradWaves, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_recurrence_grad(int dtype, const RecurArgs &a, hipStream_t st)
{
    switch (dtype) {
        case CONV2D_DTYPE_F16: return launch<SF16>(a, st);
        case CONV2D_DTYPE_BF16: return launch<SBF16>(a, st);
        default: return launch<SF32>(a, st);
    }
}

}  // namespace cnv
