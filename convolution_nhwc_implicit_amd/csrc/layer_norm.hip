// layer_norm.hip -- layer norm of rows, with the residual sum in front of it.
//
//   t = x + residual;  y = (t - mean) * rstd * weight + bias
//
// A group of lanes holds a row in registers: one read of the row, two sums over the
// lanes (the mean, then the squares around it, which loses nothing to cancellation),
// one write.  Bound by memory: 16384 rows of 4096 bf16 with residual 99 us (5.4 TB/s),
// 4057 of 2731 fp16, whose rows start anywhere, 20 us (4.4 TB/s); 32 rows 3.9 us.
#include "norm_common.h"

namespace cnv {
namespace {

template <class E, int LANES, int N, int V>
__global__ __launch_bounds__(LANES > 256 ? LANES : 256) void norm_kernel(NormArgs a)
{
    constexpr int BLOCK = LANES > 256 ? LANES : 256, GROUPS = BLOCK / LANES;
    __shared__ float slot[2][LANES > 64 ? LANES / 64 : 1];
    const Columns<LANES, N, V> at(a.d);
    const long long row = (long long)blockIdx.x * GROUPS + threadIdx.x / LANES;
    if (LANES <= 64 && row >= a.rows) return;
    using S = typename E::S;
    const S *x = (const S *)a.x + a.at(a.xs, (int)row), *res = (const S *)a.residual;
    float t[N][V];
#pragma unroll
    for (int j = 0; j < N; ++j) load_vec<E, V>(x + at.col[j], V, t[j]);
    if (res) {
        res += a.at(a.rs, (int)row);
        float u[N][V];
#pragma unroll
        for (int j = 0; j < N; ++j) load_vec<E, V>(res + at.col[j], V, u[j]);
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) t[j][i] += u[j][i];
    }
    float w[N][V], b[N][V];
    load_params<E>(a.weight, a.param_f32, 1.0f, at, w);
    load_params<E>(a.bias, a.param_f32, 0.0f, at, b);
    if (a.total) {
        S *total = (S *)a.total + row * a.d;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (at.skip[j] < V) store_vec<E, V>(total + at.col[j], V, t[j]);
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += at.mine(j, i) ? t[j][i] : 0.0f;
    row_sum<LANES>(s, slot[0]);
    const float mean = s[0] / a.count;
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            t[j][i] -= mean;
            s[0] += at.mine(j, i) ? t[j][i] * t[j][i] : 0.0f;
        }
    row_sum<LANES>(s, slot[1]);
    const float rstd = 1.0f / sqrtf(s[0] / a.count + a.eps);
    S *y = (S *)a.y + row * a.d;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = t[j][i] * rstd * w[j][i] + b[j][i];
        if (at.skip[j] < V) store_vec<E, V>(y + at.col[j], V, o);
    }
}

// Rows past the registers: a workgroup to a row, which is read three times.
constexpr int kLongLanes = 1024;
template <class E>
__global__ __launch_bounds__(kLongLanes) void norm_long_kernel(NormArgs a)
{
    __shared__ float slot[2][kLongLanes / 64];
    const long long row = blockIdx.x;
    using S = typename E::S;
    const S *x = (const S *)a.x + a.at(a.xs, (int)row);
    const S *res = a.residual ? (const S *)a.residual + a.at(a.rs, (int)row) : nullptr;
    auto value = [&](int c) { return E::to(x[c]) + (res ? E::to(res[c]) : 0.0f); };
    float s[1] = {0.0f};
    for (int c = threadIdx.x; c < a.d; c += kLongLanes) s[0] += value(c);
    row_sum<kLongLanes>(s, slot[0]);
    const float mean = s[0] / a.count;
    s[0] = 0.0f;
    for (int c = threadIdx.x; c < a.d; c += kLongLanes) {
        const float v = value(c) - mean;
        s[0] += v * v;
    }
    row_sum<kLongLanes>(s, slot[1]);
    const float rstd = 1.0f / sqrtf(s[0] / a.count + a.eps);
    auto param = [&](const void *p, int c, float none) {
        return !p ? none : a.param_f32 ? ((const float *)p)[c] : E::to(((const S *)p)[c]);
    };
    for (int c = threadIdx.x; c < a.d; c += kLongLanes) {
        const float t = value(c);
        if (a.total) ((S *)a.total)[row * a.d + c] = E::from(t);
        ((S *)a.y)[row * a.d + c] = E::from((t - mean) * rstd * param(a.weight, c, 1.0f) + param(a.bias, c, 0.0f));
    }
}

template <class E, int V>
hipError_t launch(const NormArgs &a, const NormShape &s, hipStream_t st)
{
    if (!s.held) {
        norm_long_kernel<E><<<(unsigned)a.rows, kLongLanes, 0, st>>>(a);
        return hipGetLastError();
    }
    auto go = [&](auto lanes, auto vecs, auto width) {
        constexpr int L = decltype(lanes)::value, N = decltype(vecs)::value, W = decltype(width)::value;
        constexpr int BLOCK = L > 256 ? L : 256, GROUPS = BLOCK / L;
        norm_kernel<E, L, N, W><<<(unsigned)((a.rows + (long long)GROUPS - 1) / GROUPS), BLOCK, 0, st>>>(a);
    };
    using std::integral_constant;
    auto vecs = [&](auto lanes, auto width) {
        switch (s.vecs) {
            case 1: go(lanes, integral_constant<int, 1>{}, width); break;
            case 2: go(lanes, integral_constant<int, 2>{}, width); break;
            default: go(lanes, integral_constant<int, 4>{}, width); break;
        }
    };
    constexpr integral_constant<int, V> width{};
    if (s.width == 1) go(integral_constant<int, 16>{}, integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else if (s.lanes == 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{}, width);
    else if (s.lanes == 64) vecs(integral_constant<int, 64>{}, width);
    else if (s.lanes == 256) vecs(integral_constant<int, 256>{}, width);
    else vecs(integral_constant<int, 1024>{}, width);
    return hipGetLastError();
}

}  // namespace

NormShape layer_norm_shape(int dtype, int rows, int d)
{
    const int v = dtype == CONV2D_DTYPE_F32 ? 4 : 8;
    if (d < v) return {16, 1, 1, true};
    if (d <= 16 * v) return {16, 1, v, true};
    for (int lanes : {64, 256, 1024})
        for (int n : {1, 2, 4})
            if (d <= lanes * n * v) return {lanes, n, v, true};
    return {kLongLanes, 1, 1, false};
}

hipError_t launch_layer_norm(int dtype, const NormArgs &a, const NormShape &s, hipStream_t st)
{
    switch (dtype) {
        case CONV2D_DTYPE_F16: return launch<SF16, 8>(a, s, st);
        case CONV2D_DTYPE_BF16: return launch<SBF16, 8>(a, s, st);
        default: return launch<SF32, 4>(a, s, st);
    }
}

}  // namespace cnv
