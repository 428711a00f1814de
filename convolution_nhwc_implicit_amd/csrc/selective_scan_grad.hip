// selective_scan_grad.hip -- gradients of the selective scan.
//
// With the output gradient through the gate g[t] = dy[t] silu(z[t]) and
// a[t] = exp(delta[t] A), the states' gradients run backwards,
//   dh[t] = g[t] C[t] + a[t+1] dh[t+1],
// and give, with k[t] = a[t] dh[t] (what goes on to token t-1),
//   dC[t] = sum_c g[t] h[t]                 dB[t] = sum_c delta[t] x[t] dh[t]
//   inner[t] = sum_n dh[t] B[t]             du[t] = delta[t] inner[t] + D g[t]
//   ddelta[t] = x[t] inner[t] + sum_n k[t] h[t-1] A
//   dA = sum_t k[t] h[t-1] delta[t]         dD = sum_t g[t] x[t]
//   ddt = ddelta softplus'(dt + dt_bias)    dz = dy y_before_gate silu'(z)
// where c runs over the channels of a group.
//
// Three kernels.  The first walks each chunk forwards and keeps the state before
// every step of TS tokens; where sequences are cut into chunks it starts them
// from zero, and adds up what the chunk's own tokens hand back to the tokens
// before it, sum_t (a[0] .. a[t]) g[t] C[t], so that scan_join_kernel can give
// every chunk both its first state and its last carry.  The second walks each
// chunk backwards, a step at a time: the step's states and decays are computed
// again from the kept state into registers (TS * NL values of each), so that the
// backward walk needs no further exponential.  The last adds up the partial sums
// of dA, dB, dC, dD and ddt_bias in a fixed order.
//
// Bound by the vector units at two waves a SIMD: on 4 x 2048 tokens, 2048 channels,
// 16 states the first walk takes 117 us (1540 of their cycles per 8 tokens of a
// wave), the backward walk 269 us (3472), the sums 10 us.
#include "scan_common.h"

namespace cnv {

void launch_scan_join(const ScanArgs &a, hipStream_t st);

namespace {

// What a step's tokens read, as stored, from row t on.
template <class E, int TS>
struct Tokens {
    static constexpr int G = TS / 4;
    typename E::S x[G], dt[G], z[G], dy[G];
    TokenAt<E> ax, adt, az, ady;
    Stream<E> sx, sdt, sz, sdy;
    __device__ inline Tokens(const ScanArgs &a, const Channels &c, const Chunk &k, int t)
        : ax(c, a.xs.row), adt(c, a.dts.row), az(c, a.z ? a.zs.row : 0), ady(c, a.dys.row),
          sx(a.x, a.xs.at(a.q, k.s, t), a.xs.row, a.d), sdt(a.dt, a.dts.at(a.q, k.s, t), a.dts.row, a.d),
          sz(a.z, a.zs.at(a.q, k.s, t), a.zs.row, a.d), sdy(a.dy, a.dys.at(a.q, k.s, t), a.dys.row, a.d)
    {
    }
    // without z its rows read as zero
    __device__ inline void fetch(int rows, bool grad)
    {
        const auto bx = sx.rows(rows), bdt = sdt.rows(rows), bdy = sdy.rows(rows), bz = sz.rows(rows);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            x[i] = get<E>(bx, ax[i]);
            dt[i] = get<E>(bdt, adt[i]);
            if (grad) dy[i] = get<E>(bdy, ady[i]);
            if (grad) z[i] = get<E>(bz, az[i]);
        }
    }
    __device__ inline void advance(int n)
    {
        sx.advance(n);
        sdt.advance(n);
        sz.advance(n);
        sdy.advance(n);
    }
};

template <class E, int NL, bool CARRY>
__global__ __launch_bounds__(256) void scan_keep_kernel(ScanArgs a)
{
    constexpr int TS = scan_grad_step_tokens(4 * NL), G = TS / 4;
    const int slot = blockIdx.x;
    const Chunk k = find_chunk(a, slot);
    if (!k.valid) return;
    const Channels c(a, blockIdx.y, kScanChannels, threadIdx.x / 64);
    const StateAt<NL> at(a, c);
    const int part = c.part;
    float A2[NL], h[NL], P[NL], back[NL];
    at.load(a.A, 0, A2);
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        A2[j] = finite_rate(A2[j]) * kLog2e;
        h[j] = back[j] = 0.0f;
        P[j] = 1.0f;
    }
    if (!CARRY && a.initial) at.load(a.initial, k.s, h);
    const float bias = a.dt_bias ? channel_load(a.dt_bias, 0, a, c) : 0.0f;
    float sum_delta = 0.0f;

    __shared__ float lb[2][TS * 4 * NL], lc[2][TS * 4 * NL];
    Tokens<E, TS> in(a, c, k, k.t0);
    StageBC<E, NL, TS> bc(a, k, c.group, k.t0);
    auto fetch = [&](int rem) {
        const int rows = rem < TS ? rem : TS;
        in.fetch(rows, CARRY);
        bc.load(rows, CARRY);
        in.advance(TS);
        bc.advance(TS);
    };
    fetch(k.t1 - k.t0);
    const long long keep = scan_keep_index<TS>(k, slot, k.t0);
    float *check = a.check + keep * a.d * a.n, *check_delta = a.check_delta + keep * a.d;
    int buf = 0;
    for (int rem = k.t1 - k.t0; rem > 0; rem -= TS, buf ^= 1) {
        float delta[G], dx[G], g[G], step_delta = 0.0f;
        at.store(check, 0, h);
        check += (long long)a.d * a.n;
        if (CARRY) {
            channel_store(check_delta, 0, a, c, sum_delta);
            check_delta += a.d;
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const bool valid = c.valid && 4 * i + part < rem;
            const float raw = E::to(in.dt[i]) + bias, soft = here(softplus_f32(raw));
            delta[i] = a.softplus ? soft : raw;
            delta[i] = valid ? delta[i] : 0.0f;
            dx[i] = valid ? delta[i] * E::to(in.x[i]) : 0.0f;
            step_delta += delta[i];
            g[i] = 0.0f;
            if (CARRY) {
                const float z = E::to(in.z[i]), dy = E::to(in.dy[i]), through = here(dy * (z * sigmoid_f32(z)));
                g[i] = a.z ? through : dy;
                g[i] = valid ? g[i] : 0.0f;  // an expanded tensor's rows (stride 0) all lie in range
            }
        }
        if (CARRY) sum_delta += quad_sum(step_delta);
        bc.store(lb[buf], CARRY ? lc[buf] : nullptr);
        fetch(rem - TS);
        __syncthreads();
        Four<NL> nb, nc;
        nb.read(lb[buf], 0, part);
        if (CARRY) nc.read(lc[buf], 0, part);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const Four<NL> B = nb, C = nc;
            if (i + 1 < G) {
                nb.read(lb[buf], i + 1, part);
                if (CARRY) nc.read(lc[buf], i + 1, part);
            }
            __builtin_amdgcn_sched_barrier(0);
            auto token = [&](auto qc) {
                constexpr int Q = decltype(qc)::value;
                const float dq = quad_bcast<Q>(delta[i]), dxq = quad_bcast<Q>(dx[i]), gq = quad_bcast<Q>(g[i]);
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    const float e = __builtin_amdgcn_exp2f(dq * A2[j]);
                    h[j] = __builtin_fmaf(e, h[j], dxq * B.v[Q][j]);
                    if (CARRY) {
                        P[j] *= e;
                        back[j] = __builtin_fmaf(P[j], gq * C.v[Q][j], back[j]);
                    }
                }
            };
            token(std::integral_constant<int, 0>{});
            token(std::integral_constant<int, 1>{});
            token(std::integral_constant<int, 2>{});
            token(std::integral_constant<int, 3>{});
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (CARRY) {
        at.store(a.chunk_state, slot, h);
        at.store(a.chunk_back, slot, back);
        channel_store(a.chunk_delta, slot, a, c, sum_delta);
    }
}

template <class E, int NL>
__global__ __launch_bounds__(256, NL > 8 ? 1 : 2) void scan_back_kernel(ScanArgs a)
{
    constexpr int TS = scan_grad_step_tokens(4 * NL), G = TS / 4, N4 = 4 * NL;
    const int slot = blockIdx.x, tid = threadIdx.x;
    const Chunk k = find_chunk(a, slot);
    const Channels c(a, blockIdx.y, kScanChannels, threadIdx.x / 64);
    const StateAt<NL> at(a, c);
    const int part = c.part, row = tid % 64 / 16, wave = tid / 64;
    const bool odd = part & 1, high = part & 2;
    float A[NL], carry[NL], H0[NL], dA[NL], sum_D = 0.0f, sum_bias = 0.0f;
    at.load(a.A, 0, A);
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        A[j] = finite_rate(A[j]);
        dA[j] = carry[j] = H0[j] = 0.0f;
    }
    const bool joined = a.chunk_state != nullptr;
    if (k.valid) {
        if (joined) {
            at.load(a.chunk_back, slot, carry);
            at.load(a.chunk_state, slot, H0);
        } else if (a.dfinal) {
            at.load(a.dfinal, k.s, carry);
        }
    }
    const float bias = a.dt_bias ? channel_load(a.dt_bias, 0, a, c) : 0.0f;
    const float D = a.D ? channel_load(a.D, 0, a, c) : 0.0f;

    __shared__ float lb[TS * N4], lc[TS * N4];
    __shared__ float sb[4][TS * N4], sc[4][TS * N4];  // the waves' sums of dB and dC
    const int len = k.t1 - k.t0, last = k.t0 + (len > 0 ? (len - 1) / TS * TS : 0);  // the last step, perhaps short
    Tokens<E, TS> in(a, c, k, last);
    StageBC<E, NL, TS> bc(a, k, c.group, last);
    const TokenAt<E> ao(c, a.d);
    // where the step's rows lie in du, ddt and dz, and in part_B and part_C
    long long out = (long long)last * a.d * E::kBytes, part_out = ((long long)c.block * a.q.tokens + last) * a.n * 4;
    // this thread's value of a step's dB and dC
    const uint32_t sum_off = tid < TS * N4 && tid % N4 < a.n ? (uint32_t)(tid / N4 * a.n + tid % N4) * 4 : kNowhere;
    const long long keep = scan_keep_index<TS>(k, slot, last);
    const float *check = a.check + keep * a.d * a.n, *check_delta = a.check_delta + keep * a.d;
    float kept[NL], kept_delta = 0.0f;
    auto fetch = [&](int rows) {
        in.fetch(rows, true);
        bc.load(rows, true);
        at.load(check, 0, kept);
        if (joined) kept_delta = channel_load(check_delta, 0, a, c);
        in.advance(-TS);
        bc.advance(-TS);
        check -= (long long)a.d * a.n;
        check_delta -= a.d;
    };
    if (len > 0) fetch(k.t1 - last);
    int rem = k.t1 - last;
    for (int left = (len + TS - 1) / TS; left > 0; --left, rem = TS) {
        float delta[G], dx[G], xv[G], g[G], dyv[G], zv[G], sig_raw[G], h0[NL];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const bool valid = c.valid && 4 * i + part < rem;
            const float raw = E::to(in.dt[i]) + bias;
            const float soft = here(softplus_f32(raw)), sig = here(sigmoid_f32(raw));
            xv[i] = E::to(in.x[i]);
            delta[i] = a.softplus ? soft : raw;
            sig_raw[i] = a.softplus ? sig : 1.0f;
            sig_raw[i] = valid ? sig_raw[i] : 0.0f;  // so that ddt, whose sum is ddt_bias, is 0 where there is no token
            delta[i] = valid ? delta[i] : 0.0f;
            dx[i] = valid ? delta[i] * xv[i] : 0.0f;
            dyv[i] = E::to(in.dy[i]);
            zv[i] = E::to(in.z[i]);
            const float through = here(dyv[i] * (zv[i] * sigmoid_f32(zv[i])));
            g[i] = a.z ? through : dyv[i];
            g[i] = valid ? g[i] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            h0[j] = kept[j];
            if (joined) h0[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(kept_delta * (A[j] * kLog2e)), H0[j], h0[j]);
        }
        bc.store(lb, lc);
        if (left > 1) fetch(TS);
        __syncthreads();

        float e[TS][NL], h[TS][NL], ys[G];
        Four<NL> nb, nc;
        nb.read(lb, 0, part);
        nc.read(lc, 0, part);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const Four<NL> B = nb, C = nc;
            // the next group's, or for the walk back the last one's again
            if (i + 1 < G) {
                nb.read(lb, i + 1, part);
                nc.read(lc, i + 1, part);
            }
            __builtin_amdgcn_sched_barrier(0);
            float acc[4];
            auto token = [&](auto qc) {
                constexpr int Q = decltype(qc)::value;
                const int u = 4 * i + Q;
                const float dq = quad_bcast<Q>(delta[i]), dxq = quad_bcast<Q>(dx[i]);
                float v = 0.0f;
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    e[u][j] = __builtin_amdgcn_exp2f(dq * (A[j] * kLog2e));
                    h[u][j] = __builtin_fmaf(e[u][j], u ? h[u - 1][j] : h0[j], dxq * B.v[Q][j]);
                    v = __builtin_fmaf(h[u][j], C.v[Q][j], v);
                }
                acc[Q] = v;
            };
            token(std::integral_constant<int, 0>{});
            token(std::integral_constant<int, 1>{});
            token(std::integral_constant<int, 2>{});
            token(std::integral_constant<int, 3>{});
            ys[i] = quad_scatter_sum(acc[0], acc[1], acc[2], acc[3], odd, high);
            __builtin_amdgcn_sched_barrier(0);
        }
        const uint32_t out_bytes = (uint32_t)(rem * a.d) * E::kBytes;
        const auto bdu = buffer_of((char *)a.du + out, out_bytes), bddt = buffer_of((char *)a.ddt + out, out_bytes);
        const auto bdz = buffer_of((char *)a.dz + out, a.z ? out_bytes : 0);  // without z nothing is written
        out -= (long long)TS * a.d * E::kBytes;
#pragma unroll
        for (int i = G - 1; i >= 0; --i) {
            const Four<NL> B = nb, C = nc;  // of group i: the last group's are still there
            float inner[4], along[4], vb[NL][4], vc[NL][4];
            auto token = [&](auto qc) {
                constexpr int Q = decltype(qc)::value;
                const int u = 4 * i + Q;
                const float dq = quad_bcast<Q>(delta[i]), dxq = quad_bcast<Q>(dx[i]), gq = quad_bcast<Q>(g[i]);
                inner[Q] = along[Q] = 0.0f;
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    const float dh = __builtin_fmaf(gq, C.v[Q][j], carry[j]);
                    vc[j][Q] = gq * h[u][j];
                    vb[j][Q] = dxq * dh;
                    inner[Q] = __builtin_fmaf(dh, B.v[Q][j], inner[Q]);
                    carry[j] = dh * e[u][j];
                    const float b = carry[j] * (u ? h[u - 1][j] : h0[j]);
                    along[Q] = __builtin_fmaf(b, A[j], along[Q]);
                    dA[j] = __builtin_fmaf(b, dq, dA[j]);
                }
            };
            token(std::integral_constant<int, 3>{});
            token(std::integral_constant<int, 2>{});
            token(std::integral_constant<int, 1>{});
            token(std::integral_constant<int, 0>{});
            __builtin_amdgcn_sched_barrier(0);
            if (i > 0) {
                nb.read(lb, i - 1, part);
                nc.read(lc, i - 1, part);
            }
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const float tb = channel_sum4(vb[j][0], vb[j][1], vb[j][2], vb[j][3]);
                const float tc = channel_sum4(vc[j][0], vc[j][1], vc[j][2], vc[j][3]);
                // the four quads of a row write the same value to the same place
                sb[wave][(4 * i + row) * N4 + part * NL + j] = tb;
                sc[wave][(4 * i + row) * N4 + part * NL + j] = tc;
            }
            const float in_sum = quad_scatter_sum(inner[0], inner[1], inner[2], inner[3], odd, high);
            const float al_sum = quad_scatter_sum(along[0], along[1], along[2], along[3], odd, high);
            const float draw = __builtin_fmaf(xv[i], in_sum, al_sum) * sig_raw[i];
            sum_D = __builtin_fmaf(g[i], xv[i], sum_D);
            sum_bias += draw;
            put<E>(bdu, ao[i], __builtin_fmaf(delta[i], in_sum, D * g[i]));
            put<E>(bddt, ao[i], draw);
            const float sg = sigmoid_f32(zv[i]), yv = __builtin_fmaf(D, xv[i], ys[i]);
            put<E>(bdz, ao[i], dyv[i] * yv * (sg * (1.0f + zv[i] * (1.0f - sg))));
        }
        __syncthreads();
        if (tid < TS * N4) {
            const uint32_t bytes = (uint32_t)(rem * a.n) * 4;
            put<SF32>(buffer_of((char *)a.part_B + part_out, bytes), sum_off, (sb[0][tid] + sb[1][tid]) + (sb[2][tid] + sb[3][tid]));
            put<SF32>(buffer_of((char *)a.part_C + part_out, bytes), sum_off, (sc[0][tid] + sc[1][tid]) + (sc[2][tid] + sc[3][tid]));
        }
        part_out -= (long long)TS * a.n * 4;
    }
    // a slot that no chunk uses adds nothing
    at.store(a.part_A, slot, dA);
    channel_store(a.part_D, slot, a, c, quad_sum(sum_D));
    channel_store(a.part_bias, slot, a, c, quad_sum(sum_bias));
    if (!joined && a.dinitial && k.valid) at.store(a.dinitial, k.s, carry);
}

// Adds the partial sums in ascending order.  Blocks: first dB and dC, a thread
// to a value; then dA, dD and ddt_bias.
template <class E>
__global__ __launch_bounds__(256) void scan_sum_kernel(ScanArgs a, unsigned bc_blocks)
{
    using S = typename E::S;
    if (blockIdx.x < bc_blocks) {
        const long long i = (long long)blockIdx.x * 256 + threadIdx.x, per = a.q.tokens * a.n;
        if (i >= per * a.groups) return;
        const int n = (int)(i % a.n), grp = (int)(i / a.n % a.groups);
        const long long t = i / ((long long)a.n * a.groups);
        float b = 0.0f, c = 0.0f;
        const long long o = (long long)grp * a.blocks_per_group * per + t * a.n + n;
#pragma unroll 8
        for (int k = 0; k < a.blocks_per_group; ++k) {
            b += a.part_B[o + k * per];
            c += a.part_C[o + k * per];
        }
        ((S *)a.dB)[i] = E::from(b);
        ((S *)a.dC)[i] = E::from(c);
        return;
    }
    long long i = (long long)(blockIdx.x - bc_blocks) * 256 + threadIdx.x;
    const long long dn = (long long)a.d * a.n;
    const float *p;
    float *out;
    long long per = a.d;
    if (i < dn) {
        p = a.part_A;
        out = a.dA;
        per = dn;
    } else if ((i -= dn) < a.d) {
        p = a.part_D;
        out = a.dD;
    } else {
        i -= a.d;
        p = a.part_bias;
        out = a.ddt_bias;
    }
    if (i >= per || !out) return;
    float v = 0.0f;
#pragma unroll 8
    for (int s = 0; s < a.slots; ++s) v += p[s * per + i];
    out[i] = v;
}

}  // namespace

hipError_t launch_scan_grad(int dtype, const ScanArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)a.slots, (unsigned)(a.blocks_per_group * a.groups));
    return scan_by_type(dtype, a.n, [&](auto e, auto nl) {
        using E = decltype(e);
        constexpr int NL = decltype(nl)::value;
        if (a.chunk_state) {
            scan_keep_kernel<E, NL, true><<<grid, 256, 0, st>>>(a);
            launch_scan_join(a, st);
        } else {
            scan_keep_kernel<E, NL, false><<<grid, 256, 0, st>>>(a);
        }
        scan_back_kernel<E, NL><<<grid, 256, 0, st>>>(a);
        const unsigned bc = (unsigned)((a.q.tokens * a.groups * a.n + 255) / 256);
        const unsigned rest = (unsigned)(((long long)a.d * (a.n + 2) + 255) / 256);
        scan_sum_kernel<E><<<dim3(bc + rest), 256, 0, st>>>(a, bc);
        return hipGetLastError();
    });
}

}  // namespace cnv
