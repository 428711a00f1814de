// causal_conv.hip -- causal depthwise convolution over tokens: forward,
// gradients, and the single-token step.
//
//   pre[t][c] = bias[c] + sum_k weight[c][k] * x[t-(w-1)+k][c],  y = silu(pre)
//
// Every pass is a handful of operations per element moved, so all of them are
// bound by memory.  A thread owns V neighbouring channels and a run of rows and
// walks down it with the last w-1 rows in registers, so that each row is read
// once but for the w-1 rows before a run.  Lanes lie along channels.
//
// 16384 rows of 4096 bf16 channels: forward 52 us (5.2 TB/s), gradients 92 us
// (4.4 TB/s) and 5 us for the sums of dweight and dbias; 5003 packed rows of 2731
// fp16 channels 18 us; 32 single tokens of 4096 channels 3.8 us.
#include "seq_common.h"
#include "seq_internal.h"

namespace cnv {
namespace {

__device__ inline float activate(float pre, int silu) { return silu ? pre * sigmoid_f32(pre) : pre; }

// d silu(v) / dv
__device__ inline float activate_grad(float pre, int silu)
{
    if (!silu) return 1.0f;
    const float s = sigmoid_f32(pre);
    return s * (1.0f + pre * (1.0f - s));
}

// A thread's channels and its part of the rows.  V channels from c on: the last
// thread's are moved back to end with the last channel, where they overlap its
// neighbour's (both compute the same values), so that every access is whole.
// WIDE: a wave's threads differ in channels only, and rows are scalars.
template <int V, bool WIDE>
struct Place {
    int cx, c, part, parts;
    bool mine;
    __device__ inline Place(const ConvArgs &a)
    {
        const int lanes = WIDE ? 64 : a.lanes;
        cx = threadIdx.x % lanes;
        part = WIDE ? uniform(threadIdx.x / 64) : threadIdx.x / lanes;
        parts = 256 / lanes;
        c = (blockIdx.y * lanes + cx) * V;
        mine = c < a.d;
        if (c > a.d - V) c = a.d - V;
    }
};

template <class E, int W, int V>
__device__ inline void load_taps(const void *weight, const void *b, int c, int have, float (&wt)[W][V], float (&bias)[V])
{
    float w[W * V];  // [V][W] as stored
    load_vec<E, W * V>((const typename E::S *)weight + (long long)c * W, have >= V ? W * V : have * W, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) wt[k][i] = w[i * W + k];
        bias[i] = 0.0f;
    }
    if (b) load_vec<E, V>((const typename E::S *)b + c, have, bias);
}

// Row p (counted from the sequence's first row, down to -(W-1)) of sequence s
// that begins at row t0 of the batch.
template <class E, int W, int V>
__device__ inline void load_row(const ConvArgs &a, int s, long long t0, long long p, int c, float (&out)[V])
{
    const typename E::S *x = (const typename E::S *)a.x, *init = (const typename E::S *)a.initial;
    if (p >= 0) {
        load_vec<E, V>(x + a.xs.at(a.q, s, t0 + p) + c, V, out);
    } else if (init) {
        load_vec<E, V>(init + ((long long)s * (W - 1) + (p + W - 1)) * a.d + c, V, out);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.0f;
    }
}

// The last W-1 rows that sequence s has seen, as stored (no arithmetic).
template <class E, int W, int V>
__device__ inline void write_state(const ConvArgs &a, int s, int c)
{
    const long long t0 = a.q.begin(s), len = a.q.end(s) - t0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        float v[V];
        load_row<E, W, V>(a, s, t0, len - (W - 1) + j, c, v);
        store_vec<E, V>((typename E::S *)a.final_state + ((long long)s * (W - 1) + j) * a.d + c, V, v);
    }
}

// Blocks below a.run_blocks walk runs of a.run rows; the ones past them copy
// the final states, a thread to a sequence and V channels.
template <class E, int W, int V, bool WIDE>
__global__ __launch_bounds__(256) void conv_kernel(ConvArgs a)
{
    const Place<V, WIDE> at(a);
    const int c = at.c, part = at.part, parts = at.parts;
    if (!at.mine) return;
    if (blockIdx.x >= a.run_blocks) {
        const long long s = (long long)(blockIdx.x - a.run_blocks) * parts + part;
        if (s < a.q.seqs) write_state<E, W, V>(a, (int)s, c);
        return;
    }
    long long t = ((long long)blockIdx.x * parts + part) * a.run;
    const long long stop = t + a.run < a.q.tokens ? t + a.run : a.q.tokens;
    if (t >= stop) return;
    float wt[W][V], bias[V];
    load_taps<E, W, V>(a.weight, a.bias, c, V, wt, bias);
    typename E::S *y = (typename E::S *)a.y;
    for (int s = a.q.find(t); s < a.q.seqs && t < stop; ++s) {
        const long long t0 = a.q.begin(s), e = a.q.end(s), last = e < stop ? e : stop;
        if (t < t0) t = t0;
        if (t >= last) continue;
        float win[W][V];  // rows t-(W-1) .. t
#pragma unroll
        for (int k = 0; k < W - 1; ++k) load_row<E, W, V>(a, s, t0, t - t0 - (W - 1) + k, c, win[k]);
        const typename E::S *x = (const typename E::S *)a.x + a.xs.at(a.q, s, t) + c;
        // four rows at a time, the next four under way; rows past the last are
        // the last again, and not used
        int left = (int)(last - t);
        SVec<typename E::S, V> next[kConvUnroll];
        auto fetch = [&]() {
#pragma unroll
            for (int u = 0; u < kConvUnroll; ++u) next[u] = *(const SVec<typename E::S, V> *)(x + (u < left ? u : left - 1) * a.xs.row);
        };
        fetch();
        typename E::S *out_row = y + t * a.d + c;
        for (; left > 0;) {
            SVec<typename E::S, V> in[kConvUnroll];
#pragma unroll
            for (int u = 0; u < kConvUnroll; ++u) in[u] = next[u];
            const int now = left;
            left -= kConvUnroll;
            x += kConvUnroll * a.xs.row;
            if (left > 0) fetch();
#pragma unroll
            for (int u = 0; u < kConvUnroll; ++u) {
                float out[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[W - 1][i] = E::to(in[u].v[i]);
                    float pre = bias[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) pre = __builtin_fmaf(wt[k][i], win[k][i], pre);
                    out[i] = activate(pre, a.silu);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) win[k][i] = win[k + 1][i];
                }
                if (u < now) store_vec<E, V>(out_row + u * a.d, V, out);
            }
            out_row += (long long)kConvUnroll * a.d;
        }
        t = last;
    }
}

// Gradients.  With g[t] = dy[t] * silu'(pre[t]):
//   dx[t]     = sum_k weight[k] * g[t + (W-1) - k]     (within the sequence)
//   dweight[k] = sum_t g[t] * x[t - (W-1) + k],  dbias = sum_t g[t]
// A run needs g of the W-1 rows after it too, which it recomputes; the sums
// cover its own rows only.  Each block adds its runs' sums in order in LDS and
// writes one partial [W+1][d]; conv_sum_kernel adds the partials in order.
template <class E, int W, int V, bool WIDE>
__global__ __launch_bounds__(256, 3) void conv_grad_kernel(ConvArgs a)
{
    const Place<V, WIDE> at(a);
    const int c = at.c, part = at.part, parts = at.parts, cx = at.cx;
    const typename E::S *dyp = (const typename E::S *)a.dy, *dfin = (const typename E::S *)a.dfinal;
    float wt[W][V], bias[V], sum[W + 1][V];
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[k][i] = 0.0f;
    if (at.mine) load_taps<E, W, V>(a.weight, a.bias, c, V, wt, bias);

    if (blockIdx.x >= a.run_blocks) {
        // dinitial: row i of the state is row i-(W-1) of the sequence, which
        // outputs t <= i read through tap i-t, and which the final state of a
        // short sequence still holds.
        const long long s = (long long)(blockIdx.x - a.run_blocks) * parts + part;
        if (!at.mine || s >= a.q.seqs) return;
        const long long t0 = a.q.begin((int)s), len = a.q.end((int)s) - t0;
        float g[W - 1][V];
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
#pragma unroll
            for (int i = 0; i < V; ++i) g[t][i] = 0.0f;
            if (t >= len) continue;
            float pre[V];
#pragma unroll
            for (int i = 0; i < V; ++i) pre[i] = bias[i];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                float r[V];
                load_row<E, W, V>(a, (int)s, t0, t - (W - 1) + k, c, r);
#pragma unroll
                for (int i = 0; i < V; ++i) pre[i] = __builtin_fmaf(wt[k][i], r[i], pre[i]);
            }
            load_vec<E, V>(dyp + a.dys.at(a.q, (int)s, t0 + t) + c, V, g[t]);
#pragma unroll
            for (int i = 0; i < V; ++i) g[t][i] *= activate_grad(pre[i], a.silu);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.0f;
            if (dfin && j >= len) load_vec<E, V>(dfin + (s * (W - 1) + (j - len)) * a.d + c, V, v);
#pragma unroll
            for (int t = 0; t <= j; ++t)
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = __builtin_fmaf(wt[j - t][i], g[t][i], v[i]);
            store_vec<E, V>((typename E::S *)a.dinitial + (s * (W - 1) + j) * a.d + c, V, v);
        }
        return;
    }

    long long t = ((long long)blockIdx.x * parts + part) * a.run;
    const long long stop = t + a.run < a.q.tokens ? t + a.run : a.q.tokens;
    if (at.mine && t < stop) {
        for (int s = a.q.find(t); s < a.q.seqs && t < stop; ++s) {
            const long long t0 = a.q.begin(s), e = a.q.end(s), last = e < stop ? e : stop;
            if (t < t0) t = t0;
            if (t >= last) continue;
            float win[W][V], g[W][V];  // x rows r-(W-1) .. r and g of the same rows
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                load_row<E, W, V>(a, s, t0, t - t0 - (W - 1) + k, c, win[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) g[k][i] = 0.0f;
            }
            const typename E::S *x = (const typename E::S *)a.x + a.xs.at(a.q, s, t) + c;
            const typename E::S *dy = dyp + a.dys.at(a.q, s, t) + c;
            typename E::S *dx = (typename E::S *)a.y + (t - (W - 1)) * a.d + c;  // of the row W-1 before
            // rows from here: of the run, of the sequence, and those whose g the
            // run's dx needs; past the sequence g is 0
            const int own = (int)(last - t), rest = (int)(e - t), halo = own + W - 1;
            SVec<typename E::S, V> next[kConvUnroll], gnext[kConvUnroll];
            auto fetch = [&](int r0) {
#pragma unroll
                for (int u = 0; u < kConvUnroll; ++u) {
                    const int r = r0 + u < rest ? u : rest - 1 - r0;
                    next[u] = *(const SVec<typename E::S, V> *)(x + r * a.xs.row);
                    gnext[u] = *(const SVec<typename E::S, V> *)(dy + r * a.dys.row);
                }
            };
            // Four rows from r0 on.  INNER: all the run's own, and dx of all of them is wanted.
            auto rows = [&](int r0, auto inner) {
                constexpr bool INNER = decltype(inner)::value;
                SVec<typename E::S, V> in[kConvUnroll], gin[kConvUnroll];
#pragma unroll
                for (int u = 0; u < kConvUnroll; ++u) {
                    in[u] = next[u];
                    gin[u] = gnext[u];
                }
                x += kConvUnroll * a.xs.row;
                dy += kConvUnroll * a.dys.row;
                if (r0 + kConvUnroll < rest && r0 + kConvUnroll < halo) fetch(r0 + kConvUnroll);
#pragma unroll
                for (int u = 0; u < kConvUnroll; ++u) {
                    const int r = r0 + u;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        win[W - 1][i] = E::to(in[u].v[i]);
                        float pre = bias[i];
#pragma unroll
                        for (int k = 0; k < W; ++k) pre = __builtin_fmaf(wt[k][i], win[k][i], pre);
                        g[W - 1][i] = E::to(gin[u].v[i]) * activate_grad(pre, a.silu);
                        if (!INNER) g[W - 1][i] = r < rest ? g[W - 1][i] : 0.0f;
                        if (INNER || r < own) {
#pragma unroll
                            for (int k = 0; k < W; ++k) sum[k][i] = __builtin_fmaf(g[W - 1][i], win[k][i], sum[k][i]);
                            sum[W][i] += g[W - 1][i];
                        }
                    }
                    // g now holds rows r-(W-1) .. r: dx of the first is complete
                    if (INNER || (r >= W - 1 && r < halo)) {
                        float v[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) v[i] = 0.0f;
                        const int o = r - (W - 1) - (rest - (W - 1));  // its row of the final state
                        if (dfin && o >= 0) load_vec<E, V>(dfin + ((long long)s * (W - 1) + o) * a.d + c, V, v);
#pragma unroll
                        for (int k = 0; k < W; ++k)
#pragma unroll
                            for (int i = 0; i < V; ++i) v[i] = __builtin_fmaf(wt[W - 1 - k][i], g[k][i], v[i]);
                        store_vec<E, V>(dx + (long long)u * a.d, V, v);
                    }
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            win[k][i] = win[k + 1][i];
                            g[k][i] = g[k + 1][i];
                        }
                }
                dx += (long long)kConvUnroll * a.d;
            };
            fetch(0);
            rows(0, std::false_type{});  // its first rows complete no row of the run
            int r0 = kConvUnroll;
            for (; r0 + kConvUnroll <= own; r0 += kConvUnroll) rows(r0, std::true_type{});
            for (; r0 < halo; r0 += kConvUnroll) rows(r0, std::false_type{});
            t = last;
        }
    }
    __shared__ float lds[256 * V];
    float *out = a.partial + (long long)blockIdx.x * (W + 1) * a.d;
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) lds[(part * V + i) * a.lanes + cx] = sum[k][i];
        __syncthreads();
        if (part == 0 && at.mine) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float v = 0.0f;
                for (int p = 0; p < parts; ++p) v += lds[(p * V + i) * a.lanes + cx];
                out[(long long)k * a.d + c + i] = v;
            }
        }
    }
}

// Adds the blocks' partials: 16 threads to a value, each an ascending strided
// share, the shares then in ascending order.  partial [blocks][W+1][d] ->
// dweight [d][W], dbias [d].
template <class E, int W>
__global__ __launch_bounds__(256) void conv_sum_kernel(const float *partial, int blocks, int d, void *dweight, void *dbias)
{
    const int lane = threadIdx.x % 16, share = threadIdx.x / 16;
    const long long total = (long long)(W + 1) * d, i = (long long)blockIdx.x * 16 + lane;
    __shared__ float lds[16][17];
    float v = 0.0f;
    if (i < total)
        for (int b = share; b < blocks; b += 16) v += partial[b * total + i];
    lds[share][lane] = v;
    __syncthreads();
    if (share == 0 && i < total) {
        v = 0.0f;
#pragma unroll
        for (int s = 0; s < 16; ++s) v += lds[s][lane];
        const int k = (int)(i / d), c = (int)(i % d);
        if (k < W) ((typename E::S *)dweight)[(long long)c * W + k] = E::from(v);
        else if (dbias) ((typename E::S *)dbias)[c] = E::from(v);
    }
}

// One token: the state's rows move up by one and x becomes the last.
template <class E, int W, int V>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepArgs a)
{
    const int cx = threadIdx.x % a.lanes, part = threadIdx.x / a.lanes, parts = 256 / a.lanes;
    const int c = (blockIdx.y * a.lanes + cx) * V;
    const long long r = (long long)blockIdx.x * parts + part;
    if (c >= a.d || r >= a.rows) return;
    const int have = a.d - c;
    const int slot = a.slots ? a.slots[r] : (int)r;
    typename E::S *y = (typename E::S *)a.y + r * a.d + c;
    float out[V];
    if (slot < 0 || slot >= a.pool) {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.0f;
        store_vec<E, V>(y, have, out);
        return;
    }
    typename E::S *state = (typename E::S *)a.state + (long long)slot * (W - 1) * a.d + c;
    float win[W][V], wt[W][V], bias[V];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_vec<E, V>(state + (long long)k * a.d, have, win[k]);
    load_vec<E, V>((const typename E::S *)a.x + r * a.x_row + c, have, win[W - 1]);
    load_taps<E, W, V>(a.weight, a.bias, c, have, wt, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float pre = bias[i];
#pragma unroll
        for (int k = 0; k < W; ++k) pre = __builtin_fmaf(wt[k][i], win[k][i], pre);
        out[i] = activate(pre, a.silu);
    }
    store_vec<E, V>(y, have, out);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_vec<E, V>(state + (long long)k * a.d, have, win[k + 1]);
}

// f(element type, W as a constant)
template <class F>
hipError_t by_type(int dtype, int w, F f)
{
    auto width = [&](auto e) {
        if (w == 2) return f(e, std::integral_constant<int, 2>{});
        if (w == 3) return f(e, std::integral_constant<int, 3>{});
        return f(e, std::integral_constant<int, 4>{});
    };
    if (dtype == CONV2D_DTYPE_F16) return width(SF16{});
    if (dtype == CONV2D_DTYPE_BF16) return width(SBF16{});
    return width(SF32{});
}

}  // namespace

// f(channels per thread, whether a wave's threads differ in channels only)
template <class F>
hipError_t by_width(const ConvArgs &a, F f)
{
    if (a.d < kConvChannels) return f(std::integral_constant<int, 1>{}, std::false_type{});
    if (a.lanes < 64) return f(std::integral_constant<int, kConvChannels>{}, std::false_type{});
    return f(std::integral_constant<int, kConvChannels>{}, std::true_type{});
}

hipError_t launch_conv(int dtype, int w, const ConvArgs &a, dim3 grid, hipStream_t st)
{
    return by_type(dtype, w, [&](auto e, auto wc) {
        return by_width(a, [&](auto v, auto wide) {
            conv_kernel<decltype(e), decltype(wc)::value, decltype(v)::value, decltype(wide)::value><<<grid, 256, 0, st>>>(a);
            return hipGetLastError();
        });
    });
}

hipError_t launch_conv_grad(int dtype, int w, const ConvArgs &a, dim3 grid, hipStream_t st)
{
    return by_type(dtype, w, [&](auto e, auto wc) {
        using E = decltype(e);
        constexpr int W = decltype(wc)::value;
        if (grid.x) {  // without rows and states only the sums remain: zeros
            const hipError_t r = by_width(a, [&](auto v, auto wide) {
                conv_grad_kernel<E, W, decltype(v)::value, decltype(wide)::value><<<grid, 256, 0, st>>>(a);
                return hipGetLastError();
            });
            if (r != hipSuccess) return r;
        }
        const long long total = (long long)(W + 1) * a.d;
        conv_sum_kernel<E, W><<<dim3((unsigned)((total + 15) / 16)), 256, 0, st>>>(a.partial, a.run_blocks, a.d,
                                                                                 a.dweight, a.dbias);
        return hipGetLastError();
    });
}

hipError_t launch_conv_step(int dtype, int w, const ConvStepArgs &a, dim3 grid, hipStream_t st)
{
    return by_type(dtype, w, [&](auto e, auto wc) {
        using E = decltype(e);
        conv_step_kernel<E, decltype(wc)::value, kConvChannels><<<grid, 256, 0, st>>>(a);
        return hipGetLastError();
    });
}

}  // namespace cnv
