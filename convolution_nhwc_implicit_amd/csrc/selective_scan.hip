// selective_scan.hip -- the selective scan forward, and its single-token step.
//
//   delta = softplus(dt + dt_bias)
//   h[t][c][n] = exp(delta[t][c] A[c][n]) h[t-1][c][n] + delta[t][c] x[t][c] B[t][g(c)][n]
//   y[t][c] = (sum_n h[t][c][n] C[t][g(c)][n] + D[c] x[t][c]) silu(z[t][c])
//
// States stay in fp32 registers; only inputs and outputs cross memory.  Every
// (t, c, n) costs one exp2 (8 cycles of a wave64) and four plain operations (4
// each), which outweighs the bytes: the kernels are bound by the vector units.
#include "scan_common.h"

namespace cnv {
namespace {

// One chunk of one sequence for 64 channels.  LOCAL: from a zero state, only
// the state the chunk ends with and the sum of its steps are written (the
// decay over a chunk is exp(A * that sum)), for scan_join_kernel.
template <class E, int NL, bool LOCAL>
__global__ __launch_bounds__(256) void scan_kernel(ScanArgs a)
{
    constexpr int TS = scan_step_tokens(4 * NL), G = TS / 4;
    using S = typename E::S;
    const int slot = blockIdx.x;
    const Chunk k = find_chunk(a, slot);
    if (!k.valid || (LOCAL && k.last)) return;
    const Channels c(a, blockIdx.y);
    const StateAt<NL> at(a, c);
    const int part = c.part;
    const bool odd = part & 1, high = part & 2, gated = !LOCAL && a.z;

    float A2[NL], h[NL];
    at.load(a.A, 0, A2);
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        A2[j] *= kLog2e;
        h[j] = 0.0f;
    }
    if (!LOCAL) {
        if (a.chunk_state) at.load(a.chunk_state, slot, h);
        else if (a.initial) at.load(a.initial, k.s, h);
    }
    const float bias = a.dt_bias ? channel_load(a.dt_bias, 0, a, c) : 0.0f;
    const float D = !LOCAL && a.D ? channel_load(a.D, 0, a, c) : 0.0f;
    float sum_delta = 0.0f;

    __shared__ float lb[2][TS * 4 * NL], lc[2][TS * 4 * NL];
    const TokenAt<E> ax(c, a.xs.row), adt(c, a.dts.row), az(c, gated ? a.zs.row : 0), ay(c, a.d);
    S x[G], dt[G], z[G];
    StageBC<E, NL, TS> bc(a);
    auto fetch = [&](int t) {
        const int rows = k.t1 - t < TS ? k.t1 - t : TS;
        const auto bx = rows_of<E>(a.x, a.xs.at(a.q, k.s, t), rows, a.xs.row, a.d);
        const auto bdt = rows_of<E>(a.dt, a.dts.at(a.q, k.s, t), rows, a.dts.row, a.d);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            x[i] = get<E>(bx, ax[i]);
            dt[i] = get<E>(bdt, adt[i]);
        }
        if (gated) {
            const auto bz = rows_of<E>(a.z, a.zs.at(a.q, k.s, t), rows, a.zs.row, a.d);
#pragma unroll
            for (int i = 0; i < G; ++i) z[i] = get<E>(bz, az[i]);
        }
        bc.load(a, k, c.group, t, !LOCAL);
    };
    if (k.t0 < k.t1) fetch(k.t0);
    int buf = 0;
    for (int t = k.t0; t < k.t1; t += TS, buf ^= 1) {
        const int rem = k.t1 - t;
        float delta[G], dx[G], xv[G], zv[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const bool valid = c.valid && 4 * i + part < rem;
            const float raw = E::to(dt[i]) + bias;
            xv[i] = E::to(x[i]);
            delta[i] = a.softplus ? softplus_f32(raw) : raw;
            delta[i] = valid ? delta[i] : 0.0f;  // a token that is not there leaves the state as it is
            dx[i] = delta[i] * xv[i];
            if (LOCAL) sum_delta += delta[i];
            zv[i] = gated ? E::to(z[i]) : 0.0f;
        }
        bc.store(lb[buf], LOCAL ? nullptr : lc[buf]);
        if (rem > TS) fetch(t + TS);
        __syncthreads();
        const auto by = rows_of<E>(a.y, (long long)t * a.d, rem < TS ? rem : TS, a.d, a.d);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            float acc[4];
            auto token = [&](auto qc) {
                constexpr int Q = decltype(qc)::value;
                const float *pb = &lb[buf][(4 * i + Q) * 4 * NL + part * NL], *pc = &lc[buf][(4 * i + Q) * 4 * NL + part * NL];
                const float dq = quad_bcast<Q>(delta[i]), dxq = quad_bcast<Q>(dx[i]);
                float v = 0.0f;
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(dq * A2[j]), h[j], dxq * pb[j]);
                    if (!LOCAL) v = __builtin_fmaf(h[j], pc[j], v);
                }
                acc[Q] = v;
            };
            token(std::integral_constant<int, 0>{});
            token(std::integral_constant<int, 1>{});
            token(std::integral_constant<int, 2>{});
            token(std::integral_constant<int, 3>{});
            if (!LOCAL) {
                float v = __builtin_fmaf(D, xv[i], quad_scatter_sum(acc[0], acc[1], acc[2], acc[3], odd, high));
                if (gated) v *= zv[i] * sigmoid_f32(zv[i]);
                put<E>(by, ay[i], v);
            }
        }
    }
    if (LOCAL) {
        at.store(a.chunk_state, slot, h);
        channel_store(a.chunk_delta, slot, a, c, quad_sum(sum_delta));
    } else if (a.final_state && k.last) {
        at.store(a.final_state, k.s, h);
    }
}

// Turns the chunks' own end states into the states they start with, one thread
// to a (sequence, channel, state).  With chunk_back the gradient's carries are
// joined the same way from the last chunk back: what a chunk hands back from
// its own tokens becomes what it gets from the chunks after it.
__global__ __launch_bounds__(256) void scan_join_kernel(ScanArgs a)
{
    const int s = blockIdx.x;
    int first = 0, count = a.chunks;
    if (!a.q.start) {
        first = s * a.chunks;
    } else {
        const int lane = threadIdx.x % 64;
        for (int s0 = 0; s0 < s; s0 += 64) {
            int v = s0 + lane < s ? chunks_of(a, s0 + lane) : 0;
            for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
            first += v;
        }
        first = __builtin_amdgcn_readfirstlane(first);
        count = chunks_of(a, s);
    }
    if (count > a.slots - first) count = a.slots - first;  // only if seq_start descends somewhere
    const long long i = (long long)blockIdx.y * 256 + threadIdx.x, per = (long long)a.d * a.n;
    if (i >= per) return;
    const long long ch = i / a.n;
    const float A2 = a.A[i] * kLog2e;
    float h = a.initial ? a.initial[s * per + i] : 0.0f;
    for (int c = 0; c < count; ++c) {
        float *p = a.chunk_state + (first + c) * per + i;
        const float own = *p;
        *p = h;
        if (c + 1 < count) h = __builtin_fmaf(__builtin_amdgcn_exp2f(A2 * a.chunk_delta[(long long)(first + c) * a.d + ch]), h, own);
    }
    if (!a.chunk_back) return;
    float b = a.dfinal ? a.dfinal[s * per + i] : 0.0f;
    for (int c = count - 1; c >= 0; --c) {
        float *p = a.chunk_back + (first + c) * per + i;
        const float own = *p;
        *p = b;
        b = __builtin_fmaf(__builtin_amdgcn_exp2f(A2 * a.chunk_delta[(long long)(first + c) * a.d + ch]), b, own);
    }
    if (a.dinitial) a.dinitial[s * per + i] = b;
}

// One token per row on pooled states: 4 lanes to a channel as above, R rows to a
// thread.  Bound by the states' bytes; what the rows share is loaded once, and
// all rows' loads are under way together.
template <class E, int NL, int R>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanStepArgs a)
{
    using S = typename E::S;
    const int part = threadIdx.x % 4, ch = blockIdx.y * 64 + threadIdx.x / 4;
    const int r0 = blockIdx.x * R;
    if (ch >= a.d) return;
    const int group = ch / (a.d / a.groups), first = part * NL, have = a.n - first;
    float A2[NL], h[R][NL], B[R][NL], C[R][NL];
    S x[R], dt[R], z[R];
    float *state[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const long long r = r0 + u < a.rows ? r0 + u : a.rows - 1;
        const int slot = a.slots ? a.slots[r] : (int)r;
        const bool mine = slot >= 0 && slot < a.pool && r0 + u < a.rows;
        state[u] = mine ? a.state + ((long long)slot * a.d + ch) * a.n : nullptr;
        x[u] = ((const S *)a.x)[r * a.x_row + ch];
        dt[u] = ((const S *)a.dt)[r * a.dt_row + ch];
        z[u] = a.z ? ((const S *)a.z)[r * a.z_row + ch] : (S)0;
        load_vec<E, NL>((const S *)a.B + r * a.b_row + group * a.b_group + first, have, B[u]);
        load_vec<E, NL>((const S *)a.C + r * a.c_row + group * a.c_group + first, have, C[u]);
        if (mine) read_nl<NL>(state[u], a.n, part, h[u]);
    }
    read_nl<NL>(a.A + (long long)ch * a.n, a.n, part, A2);
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.0f, D = a.D ? a.D[ch] : 0.0f;
#pragma unroll
    for (int j = 0; j < NL; ++j) A2[j] *= kLog2e;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        if (r0 + u >= a.rows) break;
        S *y = (S *)a.y + (long long)(r0 + u) * a.d + ch;
        if (!state[u]) {
            if (part == 0) *y = E::from(0.0f);
            continue;
        }
        const float xv = E::to(x[u]), raw = E::to(dt[u]) + bias;
        const float delta = a.softplus ? softplus_f32(raw) : raw, dx = delta * xv;
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            h[u][j] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A2[j]), h[u][j], dx * B[u][j]);
            v = __builtin_fmaf(h[u][j], C[u][j], v);
        }
        write_nl<NL>(state[u], a.n, part, h[u]);
        v = __builtin_fmaf(D, xv, quad_sum(v));
        if (a.z) {
            const float zv = E::to(z[u]);
            v *= zv * sigmoid_f32(zv);
        }
        if (part == 0) *y = E::from(v);
    }
}

}  // namespace

void launch_scan_join(const ScanArgs &a, hipStream_t st)
{
    const long long per = (long long)a.d * a.n;
    scan_join_kernel<<<dim3((unsigned)a.q.seqs, (unsigned)((per + 255) / 256)), 256, 0, st>>>(a);
}

hipError_t launch_scan(int dtype, const ScanArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)a.slots, (unsigned)(a.blocks_per_group * a.groups));
    return scan_by_type(dtype, a.n, [&](auto e, auto nl) {
        using E = decltype(e);
        constexpr int NL = decltype(nl)::value;
        if (a.chunk_state) {
            scan_kernel<E, NL, true><<<grid, 256, 0, st>>>(a);
            launch_scan_join(a, st);
        }
        scan_kernel<E, NL, false><<<grid, 256, 0, st>>>(a);
        return hipGetLastError();
    });
}

hipError_t launch_scan_step(int dtype, const ScanStepArgs &a, hipStream_t st)
{
    const int blocks = (a.d + 63) / 64;
    return scan_by_type(dtype, a.n, [&](auto e, auto nl) {
        using E = decltype(e);
        constexpr int NL = decltype(nl)::value, R = NL > 4 ? 2 : 4;
        // few rows: one each, over as many compute units
        if ((long long)a.rows * blocks < 4096) scan_step_kernel<E, NL, 1><<<dim3((unsigned)a.rows, (unsigned)blocks), 256, 0, st>>>(a);
        else scan_step_kernel<E, NL, R><<<dim3((unsigned)((a.rows + R - 1) / R), (unsigned)blocks), 256, 0, st>>>(a);
        return hipGetLastError();
    });
}

}  // namespace cnv
