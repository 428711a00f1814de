// layer_norm_grad.hip -- gradients of the layer norm.
//
//   xh = (x - mean) rstd;  g = dy weight
//   dx = rstd (g - mean(g) - xh mean(g xh)) + dtotal;  dweight = sum dy xh;  dbias = sum dy
//
// A group of lanes walks a run of rows, each held in registers as in the forward pass
// (whose statistics are computed again: the row is there), and keeps the sums for its
// columns of the weight's and the bias's gradients; they leave as one partial sum for
// each workgroup, and column_sums adds those.  Two sums over the lanes a row: the mean;
// then the squares around it, g, and g times the distance from the mean together.
//
// Bound by memory: 16384 rows of 4096 bf16, with dtotal, 115 us (4.8 TB/s with the
// partial sums) and 5 us for their sum.  The next row's loads ahead of the sums changed
// nothing; rows of two vectors a lane that are turned to fp32 at once spill with 1024
// lanes (4096 of 16384: 302 us with their sum, as they are 182).
#include "norm_common.h"

namespace cnv {
namespace {

// Keeps 16-bit values as they lie in memory past here: as fp32, which the compiler would
// keep them in rather than turn them again, rows of two vectors a lane take too many registers.
template <class Raw, int N>
__device__ inline void stay(Raw (&v)[N])
{
    if constexpr (N > 1 && sizeof(v[0].v[0]) == 2) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            u32x4 q = __builtin_bit_cast(u32x4, v[j]);
            asm volatile("" : "+v"(q));
            v[j] = __builtin_bit_cast(Raw, q);
        }
    }
}

template <class E, int LANES, int N, int V>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void norm_grad_kernel(NormArgs a)
{
    constexpr int BLOCK = LANES > 256 ? LANES : 256, GROUPS = BLOCK / LANES;
    __shared__ float slot[2][LANES > 64 ? 3 * (LANES / 64) : 1];
    const Columns<LANES, N, V> at(a.d);
    using S = typename E::S;
    float w[N][V], dw[N][V], db[N][V];
    load_params<E>(a.weight, a.param_f32, 1.0f, at, w);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.0f;
    const long long first = (long long)blockIdx.x * a.per, last = first + a.per < a.rows ? first + a.per : a.rows;
    for (long long row = first + threadIdx.x / LANES; row < last; row += GROUPS) {
        const S *x = (const S *)a.x + a.at(a.xs, (int)row), *dy = (const S *)a.dy + a.at(a.dys, (int)row);
        typedef SVec<S, V> Raw;
        Raw xv[N], gv[N], ev[N];
#pragma unroll
        for (int j = 0; j < N; ++j) xv[j] = *(const Raw *)(x + at.col[j]);
#pragma unroll
        for (int j = 0; j < N; ++j) gv[j] = *(const Raw *)(dy + at.col[j]);
        if (a.dtotal) {
            const S *dt = (const S *)a.dtotal + a.at(a.dts, (int)row);
#pragma unroll
            for (int j = 0; j < N; ++j) ev[j] = *(const Raw *)(dt + at.col[j]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) ev[j].v[i] = (S)0;
        }
        float s1[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) s1[0] += at.mine(j, i) ? E::to(xv[j].v[i]) : 0.0f;
        row_sum<LANES>(s1, slot[0]);
        const float mean = s1[0] / a.count;
        stay(xv);
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float t = E::to(xv[j].v[i]) - mean, gw = E::to(gv[j].v[i]) * w[j][i];
                s[0] += at.mine(j, i) ? t * t : 0.0f;
                s[1] += at.mine(j, i) ? gw : 0.0f;
                s[2] += at.mine(j, i) ? gw * t : 0.0f;
            }
        row_sum<LANES>(s, slot[1]);
        const float rstd = 1.0f / sqrtf(s[0] / a.count + a.eps);
        const float c1 = s[1] / a.count, c2 = s[2] / a.count * rstd * rstd;
        stay(xv);
        stay(gv);
        S *dx = (S *)a.dx + row * a.d;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float t = E::to(xv[j].v[i]) - mean, g = E::to(gv[j].v[i]);
                o[i] = rstd * (g * w[j][i] - c1 - t * c2) + E::to(ev[j].v[i]);
                dw[j][i] += g * (t * rstd);
                db[j][i] += g;
            }
            if (at.skip[j] < V) store_vec<E, V>(dx + at.col[j], V, o);
        }
    }
    // the groups' sums one after another
    float *out = a.partial + (long long)blockIdx.x * 2 * a.d;
    if constexpr (GROUPS > 1) {
        __shared__ float sums[LANES * N * V * 2];
        constexpr int C = LANES * N * V;
        const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
        for (int k = 0; k < GROUPS; ++k) {
            if (group == k)
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int c = (j * V + i) * LANES + lane;
                        dw[j][i] += k ? sums[c] : 0.0f;
                        db[j][i] += k ? sums[C + c] : 0.0f;
                        sums[c] = dw[j][i];
                        sums[C + c] = db[j][i];
                    }
            __syncthreads();
        }
        if (group < GROUPS - 1) return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (at.skip[j] < V) {
            store_vec<SF32, V>(out + at.col[j], V, dw[j]);
            store_vec<SF32, V>(out + a.d + at.col[j], V, db[j]);
        }
}

// Rows past the registers: their statistics first, a workgroup to a row; then columns,
// a thread to a column and a run of rows.
constexpr int kLongLanes = 1024;
template <class E>
__global__ __launch_bounds__(kLongLanes) void norm_stats_kernel(NormArgs a)
{
    __shared__ float slot[2][3 * (kLongLanes / 64)];
    const int row = blockIdx.x;
    using S = typename E::S;
    const S *x = (const S *)a.x + a.at(a.xs, row), *dy = (const S *)a.dy + a.at(a.dys, row);
    float s1[1] = {0.0f};
    for (int c = threadIdx.x; c < a.d; c += kLongLanes) s1[0] += E::to(x[c]);
    row_sum<kLongLanes>(s1, slot[0]);
    const float mean = s1[0] / a.count;
    float s[3] = {0.0f, 0.0f, 0.0f};
    for (int c = threadIdx.x; c < a.d; c += kLongLanes) {
        const float w = !a.weight ? 1.0f : a.param_f32 ? ((const float *)a.weight)[c] : E::to(((const S *)a.weight)[c]);
        const float t = E::to(x[c]) - mean, g = E::to(dy[c]) * w;
        s[0] += t * t;
        s[1] += g;
        s[2] += g * t;
    }
    row_sum<kLongLanes>(s, slot[1]);
    if (threadIdx.x > 0) return;
    const float rstd = 1.0f / sqrtf(s[0] / a.count + a.eps);
    float *out = a.stats + (long long)row * 4;
    out[0] = mean;
    out[1] = rstd;
    out[2] = s[1] / a.count;
    out[3] = s[2] / a.count * rstd * rstd;
}

template <class E>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs a)
{
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= a.d) return;
    using S = typename E::S;
    const float w = !a.weight ? 1.0f : a.param_f32 ? ((const float *)a.weight)[c] : E::to(((const S *)a.weight)[c]);
    const long long first = (long long)blockIdx.x * a.per, last = first + a.per < a.rows ? first + a.per : a.rows;
    float dw = 0.0f, db = 0.0f;
    for (long long row = first; row < last; ++row) {
        const float *st = a.stats + row * 4;
        const float rstd = st[1];
        const float t = E::to(((const S *)a.x)[a.at(a.xs, (int)row) + c]) - st[0];
        const float dy = E::to(((const S *)a.dy)[a.at(a.dys, (int)row) + c]);
        const float extra = a.dtotal ? E::to(((const S *)a.dtotal)[a.at(a.dts, (int)row) + c]) : 0.0f;
        ((S *)a.dx)[row * a.d + c] = E::from(rstd * (dy * w - st[2] - t * st[3]) + extra);
        dw += dy * (t * rstd);
        db += dy;
    }
    float *out = a.partial + (long long)blockIdx.x * 2 * a.d;
    out[c] = dw;
    out[a.d + c] = db;
}

template <class E, int V>
hipError_t launch(const NormArgs &a, const NormShape &s, hipStream_t st)
{
    if (!s.held) {
        norm_stats_kernel<E><<<(unsigned)a.rows, kLongLanes, 0, st>>>(a);
        norm_columns_kernel<E><<<dim3((unsigned)a.parts, (unsigned)((a.d + 255) / 256)), 256, 0, st>>>(a);
        return hipGetLastError();
    }
    auto go = [&](auto lanes, auto vecs, auto width) {
        constexpr int L = decltype(lanes)::value, N = decltype(vecs)::value, W = decltype(width)::value;
        norm_grad_kernel<E, L, N, W><<<(unsigned)a.parts, L > 256 ? L : 256, 0, st>>>(a);
    };
    using std::integral_constant;
    auto vecs = [&](auto lanes, auto width) {
        if (s.vecs == 1) go(lanes, integral_constant<int, 1>{}, width);
        else go(lanes, integral_constant<int, 2>{}, width);
    };
    constexpr integral_constant<int, V> width{};
    if (s.width == 1) go(integral_constant<int, 16>{}, integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else if (s.lanes == 16) vecs(integral_constant<int, 16>{}, width);
    else if (s.lanes == 64) vecs(integral_constant<int, 64>{}, width);
    else if (s.lanes == 256) vecs(integral_constant<int, 256>{}, width);
    else vecs(integral_constant<int, 1024>{}, width);
    return hipGetLastError();
}

}  // namespace

NormShape layer_norm_grad_shape(int dtype, int d)
{
    const int v = dtype == CONV2D_DTYPE_F32 ? 4 : 8;
    if (d < v) return {16, 1, 1, true};
    for (int n : {1, 2})
        if (d <= 16 * n * v) return {16, n, v, true};
    for (int lanes : {64, 256, 1024})
        for (int n : {1, 2})
            if (d <= lanes * n * v) return {lanes, n, v, true};
    return {kLongLanes, 1, 1, false};
}

hipError_t launch_layer_norm_grad(int dtype, const NormArgs &a, const NormShape &s, hipStream_t st)
{
    switch (dtype) {
        case CONV2D_DTYPE_F16: return launch<SF16, 8>(a, s, st);
        case CONV2D_DTYPE_BF16: return launch<SBF16, 8>(a, s, st);
        default: return launch<SF32, 4>(a, s, st);
    }
}

}  // namespace cnv
