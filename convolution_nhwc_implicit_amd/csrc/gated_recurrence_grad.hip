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

__device__ inline float through(float decay, float state, float h) { return decay < 0.0f ? state : fmaf(decay, h, state); }
__device__ inline float joined_decay(float before, float decay) { return before < 0.0f || decay < 0.0f ? -1.0f : before * decay; }

// A wave's run of tokens in a segment.
template <int T>
struct Run {
    long long t0, s0;
    int n, skip;    // tokens that are there; of them, tokens before the first sequence
    uint32_t f;     // which begin a sequence (bit T: the one behind the run)
    uint32_t last;  // which end one
    __device__ inline Run(const RecurArgs &a, const FirstTokens &first, int at, int len)
    {
        t0 = first.c0 + at;
        n = len - at;
        n = n < 0 ? 0 : n > T ? T : n;
        skip = t0 < first.lo ? (first.lo - t0 < n ? (int)(first.lo - t0) : n) : 0;
        f = n > 0 ? first.run<T>(at) : 0u;
        last = f >> 1;
        if (n > 0 && t0 + n == first.hi) last |= 1u << (n - 1);
        last &= (1u << n) - 1;
        f &= (1u << n) - 1;
        s0 = a.q.start || n <= 0 ? 0 : t0 / a.q.len;
    }
    __device__ inline bool there(int j) const { return j < n && j >= skip; }
    // the row that stands for token j, and its sequence among dense ones
    __device__ inline long long token(int j) const { return t0 + (j < n ? j : n - 1); }
    __device__ inline long long seq(int j) const { return s0 + __builtin_popcount(f & ((2u << (j < n ? j : n - 1)) - 2)); }
};

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

// The first walk.  BACK: sequences may go on in another chunk, which needs the
// gradient's flow through this one.
template <class E, bool BACK>
__global__ __launch_bounds__(64 * kRecurGradWaves) void recur_states_kernel(RecurArgs a)
{
    constexpr int T = kRecurGradRun, W = kRecurGradWaves;
    __shared__ uint32_t bits[FirstTokens::kWords];
    __shared__ float ends[2][BACK ? 4 : 2][W][64];
    using S = typename E::S;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int cx = blockIdx.y * kRecurChannels + lane, c = cx < a.d ? cx : a.d - 1;
    const bool mine = cx < a.d;
    const FirstTokens first(a.q, bits, a.chunk, blockIdx.x);
    const RecurChannel ch(a.A, a.r_bias, a.i_bias, c);
    const RowWalk xw(a.xs, a.q), rw(a.rs, a.q), iw(a.is, a.q), zw(a.zs, a.q), dyw(a.dys, a.q);
    const S *xp = (const S *)a.x + c, *rp = (const S *)a.r + c, *ip = (const S *)a.i + c;
    const S *zp = (const S *)a.z + c, *dyp = (const S *)a.dy + c;
    float decay = 1.0f, state = 0.0f, bdecay = 1.0f, flow = 0.0f;
    const int len = (int)(first.end - first.c0);
    long long seg = (long long)blockIdx.x * (a.chunk / (T * W));
    for (int at0 = 0, buf = 0; at0 < len; at0 += T * W, buf ^= 1, ++seg) {
        const Run<T> run(a, first, at0 + wave * T, len);
        if (wave == 0 && mine) {
            a.seg_decay[seg * a.d + c] = decay;
            a.seg_state[seg * a.d + c] = state;
        }
        float dec = 1.0f, st = 0.0f, bdec = 1.0f, fl = 0.0f;
        if (run.n > 0) {
#pragma unroll
            for (int j = 0; j < T; ++j) {
                const long long t = run.token(j), s = run.seq(j);
                const float x = E::to(xp[xw.at(t, s)]), r = E::to(rp[rw.at(t, s)]), i = E::to(ip[iw.at(t, s)]);
                float G = 0.0f;
                if (BACK) {
                    G = E::to(dyp[dyw.at(t, s)]);
                    if (a.z) {
                        const float z = E::to(zp[zw.at(t, s)]);
                        G *= z * sigmoid_f32(z);
                    }
                }
                const Token k = Token::of(ch, E{}, r, i, x);
                if (run.there(j)) {
                    const float b = __builtin_amdgcn_sqrtf(one_minus_square(k.L, k.a)) * k.u * k.x;
                    if (run.f >> j & 1) {
                        dec = -1.0f;
                        st = a.initial ? a.initial[(long long)a.q.find(run.t0 + j) * a.d + c] : 0.0f;
                    }
                    dec = dec < 0.0f ? dec : dec * k.a;
                    st = fmaf(k.a, st, b);
                    if (BACK && bdec >= 0.0f) {
                        bdec *= k.a;
                        fl = fmaf(bdec, G, fl);
                        if (run.last >> j & 1) {
                            if (a.dfinal) fl = fmaf(bdec, a.dfinal[(long long)a.q.find(run.t0 + j) * a.d + c], fl);
                            bdec = -1.0f;
                        }
                    }
                }
            }
        }
        ends[buf][0][wave][lane] = dec;
        ends[buf][1][wave][lane] = st;
        if constexpr (BACK) {
            ends[buf][2][wave][lane] = bdec;
            ends[buf][3][wave][lane] = fl;
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
    __shared__ uint32_t bits[FirstTokens::kWords];
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
    const FirstTokens first(a.q, bits, a.chunk, blockIdx.x);
    const RecurChannel ch(a.A, a.r_bias, a.i_bias, c);
    const RowWalk xw(a.xs, a.q), rw(a.rs, a.q), iw(a.is, a.q), zw(a.zs, a.q), dyw(a.dys, a.q);
    const S *xp = (const S *)a.x + c, *rp = (const S *)a.r + c, *ip = (const S *)a.i + c;
    const S *zp = (const S *)a.z + c, *dyp = (const S *)a.dy + c;
    float before = 0.0f, flow = 0.0f;  // the state the chunk starts with; the gradient that flows in behind it
    if (a.joined) {
        for (int k = 0; k < (int)blockIdx.x; ++k)
            before = through(a.chunk_decay[(long long)k * a.d + c], a.chunk_state[(long long)k * a.d + c], before);
        for (int k = a.chunks - 1; k > (int)blockIdx.x; --k)
            flow = through(a.back_decay[(long long)k * a.d + c], a.chunk_back[(long long)k * a.d + c], flow);
    }
    float dll = 0.0f, drb = 0.0f, dib = 0.0f;
    const int len = (int)(first.end - first.c0), segs = len > 0 ? (len + T * W - 1) / (T * W) : 0;
    for (int sg = segs - 1, buf = 0; sg >= 0; --sg, buf ^= 1) {
        const Run<T> run(a, first, (sg * W + wave) * T, len);
        float xv[T], gv[T], uv[T], Lv[T], av[T], wv[T], zv[T], dv[T];
        float dec = 1.0f, st = 0.0f, bdec = 1.0f, fl = 0.0f;
        auto initial = [&](int j) {
            return a.initial ? a.initial[(long long)a.q.find(run.t0 + j) * a.d + c] : 0.0f;
        };
        auto dfinal = [&](int j) {
            return a.dfinal ? a.dfinal[(long long)a.q.find(run.t0 + j) * a.d + c] : 0.0f;
        };
        if (run.n > 0) {
#pragma unroll
            for (int j = 0; j < T; ++j) {
                const long long t = run.token(j), s = run.seq(j);
                const float x = E::to(xp[xw.at(t, s)]), r = E::to(rp[rw.at(t, s)]), i = E::to(ip[iw.at(t, s)]);
                dv[j] = E::to(dyp[dyw.at(t, s)]);
                zv[j] = a.z ? E::to(zp[zw.at(t, s)]) : 0.0f;
                const Token k = Token::of(ch, E{}, r, i, x);
                const bool there = run.there(j);
                xv[j] = there ? x : 0.0f;
                gv[j] = k.g;
                uv[j] = k.u;
                Lv[j] = k.L;
                av[j] = there ? k.a : 1.0f;
                wv[j] = there ? one_minus_square(k.L, k.a) : 0.0f;
                const float b = __builtin_amdgcn_sqrtf(wv[j]) * k.u * xv[j];
                if (there) {
                    if (run.f >> j & 1) {
                        dec = -1.0f;
                        st = initial(j);
                    }
                    dec = dec < 0.0f ? dec : dec * k.a;
                    st = fmaf(k.a, st, b);
                    if (bdec >= 0.0f) {
                        bdec *= k.a;
                        fl = fmaf(bdec, a.z ? dv[j] * (zv[j] * sigmoid_f32(zv[j])) : dv[j], fl);
                        if (run.last >> j & 1) {
                            fl = fmaf(bdec, dfinal(j), fl);
                            bdec = -1.0f;
                        }
                    }
                }
            }
        }
        ends[buf][0][wave][lane] = dec;
        ends[buf][1][wave][lane] = st;
        ends[buf][2][wave][lane] = bdec;
        ends[buf][3][wave][lane] = fl;
        __syncthreads();
        const long long seg = (long long)blockIdx.x * (a.chunk / (T * W)) + sg;
        float h = through(a.seg_decay[seg * a.d + c], a.seg_state[seg * a.d + c], before);
        float k = flow;
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (w < wave) h = through(ends[buf][0][w][lane], ends[buf][1][w][lane], h);
#pragma unroll
        for (int w = W - 1; w >= 0; --w) {
            const float d = ends[buf][2][w][lane], e = ends[buf][3][w][lane];
            if (w > wave) k = through(d, e, k);
            flow = through(d, e, flow);
        }
        float hv[T];  // the states before each token
#pragma unroll
        for (int j = 0; j < T; ++j) {
            if (run.there(j) && (run.f >> j & 1)) h = initial(j);
            hv[j] = h;
            if (run.there(j)) h = fmaf(av[j], h, __builtin_amdgcn_sqrtf(wv[j]) * uv[j] * xv[j]);
        }
#pragma unroll
        for (int j = T - 1; j >= 0; --j) {
            if (!run.there(j)) continue;
            if (run.last >> j & 1) k = dfinal(j);
            const float root = __builtin_amdgcn_rsqf(fmaxf(wv[j], 1.2e-38f)), size = wv[j] * root;
            const float in = uv[j] * xv[j], b = size * in, hj = fmaf(av[j], hv[j], b);
            float G = dv[j], dz = 0.0f;
            if (a.z) {
                const float s = sigmoid_f32(zv[j]);
                G *= zv[j] * s;
                dz = dv[j] * hj * (s * (1.0f + zv[j] * (1.0f - s)));
            }
            k += G;
            const float dl = k * (av[j] * hv[j] * Lv[j] - av[j] * av[j] * in * (Lv[j] * root));  // dL * L
            const float dr = dl * (1.0f - gv[j]), di = k * b * (1.0f - uv[j]);
            dll += dl;
            drb += dr;
            dib += di;
            if (mine) {
                const long long at = (run.t0 + j) * a.d + c;
                ((S *)a.dx)[at] = E::from(k * size * uv[j]);
                ((S *)a.dr)[at] = E::from(dr);
                ((S *)a.di)[at] = E::from(di);
                if (a.z) ((S *)a.dz)[at] = E::from(dz);
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
