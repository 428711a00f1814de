// selective_scan.hip -- the selective scan forward, and its single-token step.
//
//   delta = softplus(dt + dt_bias)
//   h[t][c][n] = exp(delta[t][c] A[c][n]) h[t-1][c][n] + delta[t][c] x[t][c] B[t][g(c)][n]
//   y[t][c] = (sum_n h[t][c][n] C[t][g(c)][n] + D[c] x[t][c]) silu(z[t][c])
//
// States stay in fp32 registers; only inputs and outputs cross memory.  Every
// (t, c, n) costs one exp2 (8 cycles of a wave64) and at least four plain
// operations (4 each), which outweighs the bytes: bound by the vector units.
//
// The recurrence is linear in the state, so a workgroup's waves take successive
// runs of TS tokens of the same 16 channels at once.  A wave scans its run from a
// zero state, keeping each token's decay and input in registers; then the runs'
// ends are joined through LDS (a run's decay is exp(A * the sum of its steps)),
// and the wave scans again from its true first state, which takes no further
// exponential.  One exponential and six plain operations a state, against two and
// seven where sequences are cut into chunks that are walked twice: 220 against
// 278 us for 8192 tokens, 4096 channels, 16 states (47 cycles of the vector units
// per 64 states, used to 70 %).
#include "scan_common.h"

namespace cnv {
namespace {

// A wave's B and C of TS tokens as fp32 in LDS, [TS][4*NL] each: lanes take
// neighbouring values, value k of a lane 64/(4*NL) tokens further each.
template <class E, int NL, int TS>
struct WaveBC {
    static constexpr int kCount = TS * 4 * NL, kEach = (kCount + 63) / 64, kTokens = 64 / (4 * NL);
    typename E::S b[kEach], c[kEach];
    uint32_t boff, coff;
    Stream<E> sb, sc;
    __device__ inline WaveBC(const ScanArgs &a, const Chunk &q, int group, long long t)
        : sb(a.B, a.bs.at(a.q, q.s, t) + group * a.b_group, a.bs.row, a.n),
          sc(a.C, a.cs.at(a.q, q.s, t) + group * a.c_group, a.cs.row, a.n)
    {
        const uint32_t lane = threadIdx.x % 64, tok = lane / (4 * NL), n = lane % (4 * NL);
        const bool mine = (int)n < a.n;
        boff = mine ? tok * sb.row + n * E::kBytes : kNowhere;
        coff = mine ? tok * sc.row + n * E::kBytes : kNowhere;
    }
    __device__ inline void load(int rows, bool want_c)
    {
        const auto rb = sb.rows(rows), rc = sc.rows(rows);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            b[k] = get<E>(rb, boff + k * kTokens * sb.row);
            if (want_c) c[k] = get<E>(rc, coff + k * kTokens * sc.row);
        }
    }
    __device__ inline void store(float *lb, float *lc, bool want_c) const
    {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x % 64 + 64 * k;
            lb[i] = E::to(b[k]);
            if (want_c) lc[i] = E::to(c[k]);
        }
    }
};

// One chunk of one sequence for 16 channels.  LOCAL: from a zero state, only the
// state the chunk ends with and the sum of its steps are written, for
// scan_join_kernel.
template <class E, int NL, int waves, bool LOCAL>
__global__ __launch_bounds__(waves * 64, 2) void scan_kernel(ScanArgs a)
{
    constexpr int TS = scan_step_tokens(4 * NL), G = TS / 4;
    using S = typename E::S;
    // Each die takes a run of channel blocks, all their chunks (sequences differ
    // in length); four neighbouring blocks of a chunk, which share lines of
    // memory, follow one another.
    const int blocks = a.blocks_per_group * a.groups, total = a.slots * blocks, per_die = (total + 7) / 8;
    const int id = blockIdx.x % 8 * per_die + blockIdx.x / 8;
    if (id >= total) return;
    const int four = id / (4 * a.slots), wide = blocks - 4 * four < 4 ? blocks - 4 * four : 4, at4 = id - 4 * four * a.slots;
    const int slot = at4 / wide, block = 4 * four + at4 % wide;
    const Chunk k = find_chunk(a, slot);
    if (!k.valid || (LOCAL && k.last)) return;
    const int wave = uniform(threadIdx.x / 64), lane = threadIdx.x % 64;
    const Channels c(a, block, kScanWaveChannels, 0);
    const StateAt<NL> at(a, c);
    const int part = c.part;
    const bool odd = part & 1, high = part & 2, gated = !LOCAL && a.z;

    float A2[NL], first[NL];  // first: the state before the waves' next runs
    at.load(a.A, 0, A2);
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        A2[j] = finite_rate(A2[j]) * kLog2e;
        first[j] = 0.0f;
    }
    if (!LOCAL) {
        if (a.chunk_state) at.load(a.chunk_state, slot, first);
        else if (a.initial) at.load(a.initial, k.s, first);
    }
    const float bias = a.dt_bias ? channel_load(a.dt_bias, 0, a, c) : 0.0f;
    const float D = !LOCAL && a.D ? channel_load(a.D, 0, a, c) : 0.0f;
    float sum_delta = 0.0f;

    extern __shared__ __align__(16) float shared[];
    // the runs' decays and ends, double buffered: [2][waves][2][64][NL]; then the waves' B and C
    constexpr int kEnds = waves * 2 * 64 * NL;
    float *lb = shared + 2 * kEnds + wave * 2 * WaveBC<E, NL, TS>::kEach * 64, *lc = lb + WaveBC<E, NL, TS>::kEach * 64;

    const TokenAt<E> ax(c, a.xs.row), adt(c, a.dts.row), az(c, gated ? a.zs.row : 0), ay(c, a.d);
    // Rows are counted down from the chunk's length: k.t0 + .. may pass 31 bits behind the last row.
    const long long start = (long long)k.t0 + wave * TS;
    Stream<E> sx(a.x, a.xs.at(a.q, k.s, start), a.xs.row, a.d), sdt(a.dt, a.dts.at(a.q, k.s, start), a.dts.row, a.d);
    Stream<E> sz(gated ? a.z : nullptr, a.zs.at(a.q, k.s, start), a.zs.row, a.d), sy(a.y, start * a.d, a.d, a.d);
    S x[G], dt[G], z[G];
    WaveBC<E, NL, TS> bc(a, k, c.group, start);
    // rows past the chunk read as zero, and a whole run past it takes no memory
    auto fetch = [&](int rem) {
        const int rows = rem < TS ? rem : TS;
        const auto bx = sx.rows(rows), bdt = sdt.rows(rows), bz = sz.rows(rows);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            x[i] = get<E>(bx, ax[i]);
            dt[i] = get<E>(bdt, adt[i]);
            if (!LOCAL) z[i] = get<E>(bz, az[i]);
        }
        bc.load(rows, !LOCAL);
        sx.advance(waves * TS);
        sdt.advance(waves * TS);
        sz.advance(waves * TS);
        bc.sb.advance(waves * TS);
        bc.sc.advance(waves * TS);
    };
    const int len = k.t1 - k.t0;
    fetch(len - wave * TS);
    int buf = 0;
    for (int left = len; left > 0; left -= waves * TS, buf ^= 1) {
        const int rem = left - wave * TS;  // may be below 1: then no token is valid
        float delta[G], dx[G], xv[G], zv[G], run_delta = 0.0f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const bool valid = c.valid && 4 * i + part < rem;
            const float raw = E::to(dt[i]) + bias, soft = here(softplus_f32(raw));
            xv[i] = E::to(x[i]);
            delta[i] = a.softplus ? soft : raw;
            delta[i] = valid ? delta[i] : 0.0f;  // a token that is not there leaves the state as it is
            dx[i] = valid ? delta[i] * xv[i] : 0.0f;
            run_delta += delta[i];
            zv[i] = LOCAL ? 0.0f : E::to(z[i]);
        }
        bc.store(lb, lc, !LOCAL);
        fetch(rem - waves * TS);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        run_delta = quad_sum(run_delta);

        // the run from a zero state
        float e[TS][NL], in[TS][NL], h[NL];
#pragma unroll
        for (int j = 0; j < NL; ++j) h[j] = 0.0f;
        Four<NL> ahead;
        ahead.read(lb, 0, part);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const Four<NL> B = ahead;
            if (i + 1 < G) ahead.read(lb, i + 1, part);
            else if (!LOCAL) ahead.read(lc, 0, part);
            __builtin_amdgcn_sched_barrier(0);
            auto token = [&](auto qc) {
                constexpr int Q = decltype(qc)::value;
                const int u = 4 * i + Q;
                const float dq = quad_bcast<Q>(delta[i]), dxq = quad_bcast<Q>(dx[i]);
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    e[u][j] = __builtin_amdgcn_exp2f(dq * A2[j]);
                    in[u][j] = dxq * B.v[Q][j];
                    h[j] = __builtin_fmaf(e[u][j], h[j], in[u][j]);
                }
            };
            token(std::integral_constant<int, 0>{});
            token(std::integral_constant<int, 1>{});
            token(std::integral_constant<int, 2>{});
            token(std::integral_constant<int, 3>{});
            __builtin_amdgcn_sched_barrier(0);
        }
        // the runs' ends, and from them every run's first state
        float *mine = shared + buf * kEnds + wave * 2 * 64 * NL + lane * NL;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            mine[j] = __builtin_amdgcn_exp2f(run_delta * A2[j]);
            mine[64 * NL + j] = h[j];
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < waves; ++w) {
            const float *p = shared + buf * kEnds + w * 2 * 64 * NL + lane * NL;
            if (w == wave) {
                // one wave in `waves` takes this: a branch, not a select for each value
#pragma unroll
                for (int j = 0; j < NL; ++j) asm volatile("v_mov_b32 %0, %1" : "=v"(h[j]) : "v"(first[j]));
            }
#pragma unroll
            for (int j = 0; j < NL; ++j) first[j] = __builtin_fmaf(p[j], first[j], p[64 * NL + j]);
        }
        if (LOCAL) {
            sum_delta += run_delta;
            continue;
        }
        // and the run from it
        const auto by = sy.rows(rem < TS ? rem : TS);
        sy.advance(waves * TS);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const Four<NL> C = ahead;
            if (i + 1 < G) ahead.read(lc, i + 1, part);
            __builtin_amdgcn_sched_barrier(0);
            float acc[4];
            auto token = [&](auto qc) {
                constexpr int Q = decltype(qc)::value;
                const int u = 4 * i + Q;
                float v = 0.0f;
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    h[j] = __builtin_fmaf(e[u][j], h[j], in[u][j]);
                    v = __builtin_fmaf(h[j], C.v[Q][j], v);
                }
                acc[Q] = v;
            };
            token(std::integral_constant<int, 0>{});
            token(std::integral_constant<int, 1>{});
            token(std::integral_constant<int, 2>{});
            token(std::integral_constant<int, 3>{});
            const float v = __builtin_fmaf(D, xv[i], quad_scatter_sum(acc[0], acc[1], acc[2], acc[3], odd, high));
            const float w = here(v * (zv[i] * sigmoid_f32(zv[i])));
            put<E>(by, ay[i], gated ? w : v);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    if (LOCAL) {
        if (wave == 0) at.store(a.chunk_state, slot, first);
        // the waves' sums of steps, in order
        __syncthreads();
        shared[wave * 64 + lane] = sum_delta;
        __syncthreads();
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += shared[w * 64 + lane];
        if (wave == 0) channel_store(a.chunk_delta, slot, a, c, v);
    } else if (a.final_state && k.last && wave == 0) {
        at.store(a.final_state, k.s, first);
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
            first = first + v < a.slots ? first + v : a.slots;
        }
        first = __builtin_amdgcn_readfirstlane(first);
        count = chunks_of(a, s);
    }
    if (count > a.slots - first) count = a.slots - first;  // only if seq_start descends somewhere
    const long long i = (long long)blockIdx.y * 256 + threadIdx.x, per = (long long)a.d * a.n;
    if (i >= per) return;
    const long long ch = i / a.n;
    const float A2 = finite_rate(a.A[i]) * kLog2e;
    // Eight chunks' values are loaded together: one after the other, each would
    // wait for memory.
    constexpr int AHEAD = 8;
    float own[AHEAD], decay[AHEAD];
    auto fetch = [&](const float *from, int c0, int dir) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int c = c0 + dir * u;
            if (c < 0 || c >= count) continue;
            own[u] = from[(first + c) * per + i];
            decay[u] = a.chunk_delta[(long long)(first + c) * a.d + ch];
        }
    };
    float h = a.initial ? a.initial[s * per + i] : 0.0f;
    for (int c0 = 0; c0 < count; c0 += AHEAD) {
        fetch(a.chunk_state, c0, 1);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (c0 + u >= count) break;
            a.chunk_state[(first + c0 + u) * per + i] = h;
            h = __builtin_fmaf(__builtin_amdgcn_exp2f(A2 * decay[u]), h, own[u]);  // after the last chunk not used
        }
    }
    if (!a.chunk_back) return;
    float b = a.dfinal ? a.dfinal[s * per + i] : 0.0f;
    for (int c0 = count - 1; c0 >= 0; c0 -= AHEAD) {
        fetch(a.chunk_back, c0, -1);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (c0 - u < 0) break;
            a.chunk_back[(first + c0 - u) * per + i] = b;
            b = __builtin_fmaf(__builtin_amdgcn_exp2f(A2 * decay[u]), b, own[u]);
        }
    }
    if (a.dinitial) a.dinitial[s * per + i] = b;
}

// One token per row on pooled states: 4 lanes to a channel as above, R rows to a
// thread.  Bound by the states' bytes; what the rows share is loaded once, and
// all rows' loads are under way together: 256 rows x 5120 x 16 51 us (one row to
// a thread: 62).
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
    for (int j = 0; j < NL; ++j) A2[j] = finite_rate(A2[j]) * kLog2e;
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

hipError_t launch_scan(int dtype, const ScanArgs &a, int waves, hipStream_t st)
{
    const long long total = (long long)a.slots * a.blocks_per_group * a.groups;
    const dim3 grid((unsigned)((total + 7) / 8 * 8));
    return scan_by_type(dtype, a.n, [&](auto e, auto nl) {
        using E = decltype(e);
        constexpr int NL = decltype(nl)::value, TS = scan_step_tokens(4 * NL);
        auto run = [&](auto wc) {
            constexpr int W = decltype(wc)::value, lds = W * (4 * NL * 64 + 2 * WaveBC<E, NL, TS>::kEach * 64) * 4;
            auto launch = [&](auto *kernel) {
                if (lds > 64 << 10) {
                    const hipError_t r = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
                    if (r != hipSuccess) return r;
                }
                kernel<<<grid, W * 64, lds, st>>>(a);
                return hipGetLastError();
            };
            if (a.chunk_state) {
                const hipError_t r = launch(scan_kernel<E, NL, W, true>);
                if (r != hipSuccess) return r;
                launch_scan_join(a, st);
            }
            return launch(scan_kernel<E, NL, W, false>);
        };
        if (waves == 1) return run(std::integral_constant<int, 1>{});
        if (waves == 2) return run(std::integral_constant<int, 2>{});
        if (waves == 4) return run(std::integral_constant<int, 4>{});
        return run(std::integral_constant<int, 8>{});
    });
}

hipError_t launch_scan_step(int dtype, const ScanStepArgs &a, hipStream_t st)
{
    const int blocks = (a.d + 63) / 64;
    return scan_by_type(dtype, a.n, [&](auto e, auto nl) {
        using E = decltype(e);
        constexpr int NL = decltype(nl)::value, R = scan_step_rows(4 * NL);
        // few rows: one each, over as many compute units
        if ((long long)a.rows * blocks < 4096) scan_step_kernel<E, NL, 1><<<dim3((unsigned)a.rows, (unsigned)blocks), 256, 0, st>>>(a);
        else scan_step_kernel<E, NL, R><<<dim3((unsigned)((a.rows + R - 1) / R), (unsigned)blocks), 256, 0, st>>>(a);
        return hipGetLastError();
    });
}

}  // namespace cnv
