// seq_api.cpp -- the C ABI of the sequence operators: argument checks,
// workspace layout, launch shapes.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "seq_internal.h"

using namespace cnv;

namespace {

constexpr long long kMaxRows = (1LL << 31) - 1;
constexpr long long kMaxStride = (1LL << 24) - 1;  // 16 rows of it in bytes fit 31 bits
constexpr long long kMaxGridY = 65535;
constexpr int kCUs = 256;  // MI355X

bool float_type(int dtype) { return dtype == CONV2D_DTYPE_F16 || dtype == CONV2D_DTYPE_BF16 || dtype == CONV2D_DTYPE_F32; }
int bytes_of(int dtype) { return dtype == CONV2D_DTYPE_F32 ? 4 : 2; }
bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t up(size_t v) { return (v + 255) / 256 * 256; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
int status(hipError_t e) { return e == hipSuccess ? CONV2D_OK : CONV2D_ERR_DEVICE; }

int check_batch(const seq_batch_t &b)
{
    if (b.seqs < 1 || b.len < 0 || b.tokens < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!b.seq_start && b.tokens != (long long)b.seqs * b.len) return CONV2D_ERR_INVALID_ARGUMENT;
    if (b.tokens > kMaxRows || b.seqs > (1 << 24)) return CONV2D_ERR_UNSUPPORTED;
    return aligned(b.seq_start, 4) ? CONV2D_OK : CONV2D_ERR_UNSUPPORTED;
}

Seqs seqs_of(const seq_batch_t &b) { return Seqs{b.seq_start, b.seqs, b.len, b.tokens}; }
RowStride stride_of(const seq_stride_t &s) { return RowStride{s.row, s.seq}; }

bool all_aligned(size_t a, std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if (!aligned(p, a)) return false;
    return true;
}

int lanes_for(int d, int v)
{
    int lanes = 1;
    while (lanes < 64 && (long long)lanes * v < d) lanes *= 2;
    return lanes;
}

// ---- causal convolution -------------------------------------------------------
int check_conv(const causal_conv_problem_t *p, int dtype, bool grad)
{
    if (!p) return CONV2D_ERR_INVALID_ARGUMENT;
    const int r = check_batch(p->batch);
    if (r != CONV2D_OK) return r;
    if (p->d < 1 || p->w < 1 || (p->silu != 0 && p->silu != 1)) return CONV2D_ERR_INVALID_ARGUMENT;
    if (p->x.row < 0 || p->x.seq < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    if (grad && (p->dy.row < 0 || p->dy.seq < 0)) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || p->w < 2 || p->w > 4 || p->d > kMaxStride) return CONV2D_ERR_UNSUPPORTED;
    return CONV2D_OK;
}

struct ConvPlan {
    int lanes, run, run_blocks, state_blocks;
};

// Rows per thread: long runs read fewer rows twice (and leave fewer partial
// sums), short ones fill the chip.  About 16 waves to a CU before runs grow.
ConvPlan conv_plan(const causal_conv_problem_t *p, int v, int most, bool states)
{
    ConvPlan c;
    c.lanes = lanes_for(p->d, v);
    const long long vecs = ceil_div(p->d, v), parts = 256 / c.lanes;
    long long run = kConvUnroll;
    while (run < most && p->batch.tokens / run * vecs > (long long)kCUs * 16 * 64) run *= 2;
    c.run = (int)run;
    c.run_blocks = (int)ceil_div(ceil_div(p->batch.tokens, run), parts);
    c.state_blocks = states ? (int)ceil_div(p->batch.seqs, parts) : 0;
    return c;
}
constexpr int kConvMostRows = 32, kConvGradMostRows = 64;

bool conv_fits(const ConvPlan &c, int d, int v)
{
    return ceil_div(d, c.lanes * v) <= kMaxGridY && fits((long long)c.run_blocks + c.state_blocks, 256);
}

int conv_grad_plan(const causal_conv_problem_t *p, int dtype, bool states, ConvPlan *c, size_t *ws)
{
    *c = conv_plan(p, conv_channels(p->d), kConvGradMostRows, states);
    *ws = up((size_t)c->run_blocks * (p->w + 1) * p->d * 4);
    return CONV2D_OK;
}

// ---- selective scan --------------------------------------------------------------
int check_stride(const seq_stride_t &s)
{
    if (s.row < 0 || s.seq < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    return s.row > kMaxStride ? CONV2D_ERR_UNSUPPORTED : CONV2D_OK;
}

int check_scan_sizes(int d, int n, int groups, int softplus, int dtype)
{
    if (d < 1 || n < 1 || groups < 1 || d % groups || (softplus != 0 && softplus != 1)) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || n > 64 || d > kMaxStride || (long long)d * n > kMaxGridY * 256) return CONV2D_ERR_UNSUPPORTED;
    return CONV2D_OK;
}

int check_scan(const selective_scan_problem_t *p, int dtype, bool grad)
{
    if (!p) return CONV2D_ERR_INVALID_ARGUMENT;
    int r = check_batch(p->batch);
    if (r == CONV2D_OK) r = check_scan_sizes(p->d, p->n, p->groups, p->softplus, dtype);
    for (const seq_stride_t *s : {&p->x, &p->dt, &p->B, &p->C, &p->z})
        if (r == CONV2D_OK) r = check_stride(*s);
    if (r == CONV2D_OK && grad) r = check_stride(p->dy);
    if (r == CONV2D_OK && (p->b_group < 0 || p->c_group < 0)) r = CONV2D_ERR_INVALID_ARGUMENT;
    if (r == CONV2D_OK && ceil_div(p->d / p->groups, kScanWaveChannels) * p->groups > kMaxGridY) r = CONV2D_ERR_UNSUPPORTED;
    return r;
}

struct ScanPlan {
    int blocks_per_group, chunk, chunks, slots, waves;
    bool joined;  // sequences are cut into more than one chunk
    size_t state, delta, check, check_delta, part_B;  // bytes
};

// How many waves of a forward workgroup take runs of a walk of `len` tokens: as
// many as it has runs, and no more than give each SIMD two waves.
int scan_waves(long long walks, long long len, int ts)
{
    int w = 8;
    while (w > 1 && (w / 2 * ts >= len || walks * (w / 2) >= 2 * 4 * kCUs)) w /= 2;
    return w;
}

// Microseconds of a forward pass with sequences cut into chunks of `chunk` tokens
// (walked twice and joined) or, if longest <= chunk, not cut.  A segment (waves *
// ts tokens) was measured at 2.8 us where workgroups have the compute units to
// themselves, 3.7 us at two waves per SIMD; chunks add a shorter first walk,
// launches, and the join's batches of eight.
double scan_time(double blocks, const seq_batch_t &b, long long longest, long long chunk, int ts, double weight)
{
    const bool cut = longest > chunk;
    const double pieces = cut ? (double)b.tokens / chunk + (b.seq_start ? 0.5 * b.seqs : 0) : b.seqs, walks = blocks * pieces;
    const long long len = cut ? chunk : longest;
    const int w = scan_waves((long long)walks, len, ts);
    const double segment = weight * (walks * w > 4 * kCUs ? 3.7 : 2.8), slots = 2.0 * 4 * kCUs / w;
    const double alone = (double)ceil_div(len, (long long)w * ts), all = (double)b.tokens / (w * ts) * blocks / slots;
    const double walk = std::max(alone, all) * segment;
    return cut ? 1.65 * walk + 10 + 0.8 * (double)ceil_div(ceil_div(longest, chunk), 8) : walk;
}

// The same for the gradient: a step of ts tokens of both walks 3.9 us for up to a
// workgroup to a compute unit, 6.6 us for two, in rounds.
double scan_grad_time(double blocks, const seq_batch_t &b, long long longest, long long chunk, int ts, double weight)
{
    const bool cut = longest > chunk;
    const double pieces = cut ? (double)b.tokens / chunk + (b.seq_start ? 0.5 * b.seqs : 0) : b.seqs;
    const long long walks = std::max(1LL, (long long)(blocks * pieces)), rest = walks % (2 * kCUs);
    const double round = (double)(walks / (2 * kCUs)) * 6.6 + (rest == 0 ? 0 : rest <= kCUs ? 3.9 : 6.6);
    return (double)ceil_div(std::min(longest, chunk), ts) * round * weight +
           (cut ? 5 + 1.6 * (double)ceil_div(ceil_div(longest, chunk), 8) : 0);
}

// Tokens per chunk: what the estimates above say takes least time.  The lengths
// of packed sequences are on the device: the longest is taken as twice the mean.
void scan_plan(const selective_scan_problem_t *p, bool grad, ScanPlan *s)
{
    const seq_batch_t &b = p->batch;
    const int ts = grad ? scan_grad_step_tokens(p->n) : scan_step_tokens(p->n);
    const int nl = p->n <= 4 ? 1 : p->n <= 8 ? 2 : p->n <= 16 ? 4 : p->n <= 32 ? 8 : 16;
    const double weight = std::max(0.6, (double)nl * ts / (grad ? 32 : 64));
    s->blocks_per_group = (int)ceil_div(p->d / p->groups, grad ? kScanChannels : kScanWaveChannels);
    const long long blocks = (long long)s->blocks_per_group * p->groups;
    const long long whole = std::max<long long>(ceil_div(b.seq_start ? b.tokens : b.len, 16) * 16, 16);
    const long long longest = b.seq_start ? std::max(1LL, std::min(b.tokens, 2 * ceil_div(b.tokens, b.seqs))) : std::max(1, b.len);
    auto time = [&](long long c) {
        return grad ? scan_grad_time((double)blocks, b, longest, c, ts, weight) : scan_time((double)blocks, b, longest, c, ts, weight);
    };
    long long chunk = whole;
    double best = time(whole);
    for (long long c = grad ? 16 : 4 * ts; c < whole; c += std::max<long long>(16, c / 4 / 16 * 16)) {
        const double t = time(c);
        if (t < best && b.tokens / c + b.seqs < (1 << 24)) {
            best = t;
            chunk = c;
        }
    }
    s->chunk = (int)std::min<long long>(chunk, 1 << 30);
    s->waves = scan_waves(blocks * (longest > chunk ? b.tokens / chunk + 1 : b.seqs), std::min(longest, chunk), ts);
    s->chunks = std::max(1, (int)ceil_div(b.len, s->chunk));
    s->joined = whole > s->chunk;
    s->slots = b.seq_start ? (int)(b.tokens / s->chunk) + b.seqs : s->chunks * b.seqs;
    const size_t dn = (size_t)p->d * p->n * 4, d = (size_t)p->d * 4;
    s->state = up(s->slots * dn);
    s->delta = up(s->slots * d);
    s->check = s->check_delta = s->part_B = 0;
    if (grad) {
        const long long steps = b.tokens / ts + s->slots + 1;  // scan_keep_index
        s->check = up(steps * dn);
        s->check_delta = up(steps * d);
        s->part_B = up((size_t)blocks * b.tokens * p->n * 4);
    }
}

// Whether the launches of a pass fit, and the sums of their counts 31 bits.
bool scan_fits(const selective_scan_problem_t *p, const ScanPlan &s, bool grad)
{
    if (s.joined && !fits(p->batch.seqs, 256)) return false;
    if (!grad) return fits(ceil_div((long long)s.slots * s.blocks_per_group * p->groups, 8) * 8, s.waves * 64);
    const long long tokens = p->batch.tokens, bc = (long long)p->groups * p->n;  // scan_sum_kernel, a thread to a value
    return fits(s.slots, 256) && tokens <= kMaxThreads / bc &&
           fits(ceil_div(tokens * bc, 256) + ceil_div((long long)p->d * (p->n + 2), 256), 256);
}

size_t scan_bytes(const ScanPlan &s, bool grad)
{
    if (!grad) return s.joined ? s.state + s.delta : 0;
    return (s.joined ? 2 * s.state + s.delta + s.check_delta : 0) + s.check + s.state + 2 * s.delta + 2 * s.part_B;
}

ScanArgs scan_args(const selective_scan_problem_t *p, const ScanPlan &s)
{
    ScanArgs a = {};
    a.q = seqs_of(p->batch);
    a.d = p->d;
    a.n = p->n;
    a.groups = p->groups;
    a.softplus = p->softplus;
    a.blocks_per_group = s.blocks_per_group;
    a.chunk = s.chunk;
    a.chunks = s.chunks;
    a.slots = s.slots;
    a.xs = stride_of(p->x);
    a.dts = stride_of(p->dt);
    a.bs = stride_of(p->B);
    a.cs = stride_of(p->C);
    a.zs = stride_of(p->z);
    a.dys = stride_of(p->dy);
    a.b_group = p->b_group;
    a.c_group = p->c_group;
    return a;
}

struct Carver {
    char *p;
    float *take(size_t bytes)
    {
        float *r = (float *)p;
        p += bytes;
        return r;
    }
};

}  // namespace

extern "C" {

int causal_conv(const causal_conv_problem_t *prob, int dtype, const void *x, const void *weight,
                const void *bias, const void *initial_state, void *y, void *final_state, void *stream)
{
    const int r = check_conv(prob, dtype, false);
    if (r != CONV2D_OK) return r;
    const bool rows = prob->batch.tokens > 0;
    if (!weight || (rows && (!x || !y))) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {x, weight, bias, initial_state, y, final_state})) return CONV2D_ERR_UNSUPPORTED;
    const int v = conv_channels(prob->d);
    const ConvPlan c = conv_plan(prob, v, kConvMostRows, final_state != nullptr);
    if (!conv_fits(c, prob->d, v)) return CONV2D_ERR_UNSUPPORTED;
    if (c.run_blocks + c.state_blocks == 0) return CONV2D_OK;
    ConvArgs a = {};
    a.q = seqs_of(prob->batch);
    a.d = prob->d;
    a.silu = prob->silu;
    a.lanes = c.lanes;
    a.run = c.run;
    a.run_blocks = c.run_blocks;
    a.xs = stride_of(prob->x);
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.initial = initial_state;
    a.y = y;
    a.final_state = final_state;
    return status(launch_conv(dtype, prob->w, a,
                              dim3((unsigned)(c.run_blocks + c.state_blocks), (unsigned)ceil_div(prob->d, c.lanes * v)),
                              (hipStream_t)stream));
}

int causal_conv_grad_workspace_size(const causal_conv_problem_t *prob, int dtype, size_t *bytes)
{
    const int r = check_conv(prob, dtype, true);
    if (r != CONV2D_OK) return r;
    if (!bytes) return CONV2D_ERR_INVALID_ARGUMENT;
    ConvPlan c;
    return conv_grad_plan(prob, dtype, false, &c, bytes);
}

int causal_conv_grad(const causal_conv_problem_t *prob, int dtype, const void *dy, const void *x,
                     const void *weight, const void *bias, const void *initial_state,
                     const void *dfinal, void *dx, void *dweight, void *dbias, void *dinitial,
                     void *workspace, size_t workspace_bytes, void *stream)
{
    const int r = check_conv(prob, dtype, true);
    if (r != CONV2D_OK) return r;
    const bool rows = prob->batch.tokens > 0;
    if (!weight || !dweight || (rows && (!x || !dy || !dx))) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {dy, x, weight, bias, initial_state, dfinal, dx, dweight, dbias, dinitial}) ||
        !aligned(workspace, 16))
        return CONV2D_ERR_UNSUPPORTED;
    ConvPlan c;
    size_t need;
    conv_grad_plan(prob, dtype, dinitial != nullptr, &c, &need);
    const int v = conv_channels(prob->d);
    if (!conv_fits(c, prob->d, v)) return CONV2D_ERR_UNSUPPORTED;
    if (need && !workspace) return CONV2D_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    ConvArgs a = {};
    a.q = seqs_of(prob->batch);
    a.d = prob->d;
    a.silu = prob->silu;
    a.lanes = c.lanes;
    a.run = c.run;
    a.run_blocks = c.run_blocks;
    a.xs = stride_of(prob->x);
    a.dys = stride_of(prob->dy);
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.initial = initial_state;
    a.dy = dy;
    a.dfinal = dfinal;
    a.y = dx;
    a.dinitial = dinitial;
    a.partial = (float *)workspace;
    a.dweight = dweight;
    a.dbias = dbias;
    return status(launch_conv_grad(dtype, prob->w, a,
                                   dim3((unsigned)(c.run_blocks + c.state_blocks), (unsigned)ceil_div(prob->d, c.lanes * v)),
                                   (hipStream_t)stream));
}

int causal_conv_step(const causal_conv_step_problem_t *prob, int dtype, const void *x, void *state,
                     const void *weight, const void *bias, const int *slots, void *y, void *stream)
{
    if (!prob || prob->rows < 0 || prob->pool < 0 || prob->d < 1 || prob->w < 1 || prob->x_row < 0 ||
        (prob->silu != 0 && prob->silu != 1))
        return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || prob->w < 2 || prob->w > 4 || prob->d > kMaxStride) return CONV2D_ERR_UNSUPPORTED;
    if (prob->rows == 0) return CONV2D_OK;
    if (!x || !weight || !y || (prob->pool > 0 && !state)) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {x, state, weight, bias, y}) || !aligned(slots, 4)) return CONV2D_ERR_UNSUPPORTED;
    const int v = kConvChannels, lanes = lanes_for(prob->d, v);
    if (ceil_div(prob->d, lanes * v) > kMaxGridY || !fits(ceil_div(prob->rows, 256 / lanes), 256)) return CONV2D_ERR_UNSUPPORTED;
    ConvStepArgs a = {prob->rows, prob->pool, prob->d, prob->silu, lanes, prob->x_row, x, weight, bias, slots, state, y};
    return status(launch_conv_step(dtype, prob->w, a,
                                   dim3((unsigned)ceil_div(prob->rows, 256 / lanes), (unsigned)ceil_div(prob->d, lanes * v)),
                                   (hipStream_t)stream));
}

int selective_scan_workspace_size(const selective_scan_problem_t *prob, int dtype, size_t *bytes)
{
    const int r = check_scan(prob, dtype, false);
    if (r != CONV2D_OK) return r;
    if (!bytes) return CONV2D_ERR_INVALID_ARGUMENT;
    ScanPlan s;
    scan_plan(prob, false, &s);
    if (!scan_fits(prob, s, false)) return CONV2D_ERR_UNSUPPORTED;
    *bytes = scan_bytes(s, false);
    return CONV2D_OK;
}

int selective_scan(const selective_scan_problem_t *prob, int dtype, const void *x, const void *dt,
                   const float *A, const void *B, const void *C, const float *D, const void *z,
                   const float *dt_bias, const float *initial_state, void *y, float *final_state,
                   void *workspace, size_t workspace_bytes, void *stream)
{
    const int r = check_scan(prob, dtype, false);
    if (r != CONV2D_OK) return r;
    const bool rows = prob->batch.tokens > 0;
    if (!A || (rows && (!x || !dt || !B || !C || !y))) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {x, dt, B, C, z, y}) ||
        !all_aligned(4, {A, D, dt_bias, initial_state, final_state}) || !aligned(workspace, 16))
        return CONV2D_ERR_UNSUPPORTED;
    ScanPlan s;
    scan_plan(prob, false, &s);
    if (!scan_fits(prob, s, false)) return CONV2D_ERR_UNSUPPORTED;
    const size_t need = scan_bytes(s, false);
    if (need && !workspace) return CONV2D_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    if (!rows && !final_state) return CONV2D_OK;
    ScanArgs a = scan_args(prob, s);
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.B = B;
    a.C = C;
    a.D = D;
    a.z = z;
    a.dt_bias = dt_bias;
    a.initial = initial_state;
    a.y = y;
    a.final_state = final_state;
    if (s.joined) {
        Carver w{(char *)workspace};
        a.chunk_state = w.take(s.state);
        a.chunk_delta = w.take(s.delta);
    }
    return status(launch_scan(dtype, a, s.waves, (hipStream_t)stream));
}

int selective_scan_grad_workspace_size(const selective_scan_problem_t *prob, int dtype, size_t *bytes)
{
    const int r = check_scan(prob, dtype, true);
    if (r != CONV2D_OK) return r;
    if (!bytes) return CONV2D_ERR_INVALID_ARGUMENT;
    ScanPlan s;
    scan_plan(prob, true, &s);
    if (!scan_fits(prob, s, true)) return CONV2D_ERR_UNSUPPORTED;
    *bytes = scan_bytes(s, true);
    return CONV2D_OK;
}

int selective_scan_grad(const selective_scan_problem_t *prob, int dtype, const void *dy, const void *x,
                        const void *dt, const float *A, const void *B, const void *C, const float *D,
                        const void *z, const float *dt_bias, const float *initial_state,
                        const float *dfinal, const selective_scan_grads_t *g, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    const int r = check_scan(prob, dtype, true);
    if (r != CONV2D_OK) return r;
    const bool rows = prob->batch.tokens > 0;
    if (!A || !g || !g->dA || !workspace) return CONV2D_ERR_INVALID_ARGUMENT;
    if (rows && (!dy || !x || !dt || !B || !C || !g->du || !g->ddt || !g->dB || !g->dC || (z && !g->dz)))
        return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {dy, x, dt, B, C, z, g->du, g->ddt, g->dB, g->dC, g->dz}) ||
        !all_aligned(4, {A, D, dt_bias, initial_state, dfinal, g->dA, g->dD, g->ddt_bias, g->dinitial}) ||
        !aligned(workspace, 16))
        return CONV2D_ERR_UNSUPPORTED;
    ScanPlan s;
    scan_plan(prob, true, &s);
    if (!scan_fits(prob, s, true)) return CONV2D_ERR_UNSUPPORTED;
    if (workspace_bytes < scan_bytes(s, true)) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    ScanArgs a = scan_args(prob, s);
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.B = B;
    a.C = C;
    a.D = D;
    a.z = z;
    a.dy = dy;
    a.dt_bias = dt_bias;
    a.initial = initial_state;
    a.dfinal = dfinal;
    a.du = g->du;
    a.ddt = g->ddt;
    a.dA = g->dA;
    a.dB = g->dB;
    a.dC = g->dC;
    a.dD = g->dD;
    a.dz = g->dz;
    a.ddt_bias = g->ddt_bias;
    a.dinitial = g->dinitial;
    Carver w{(char *)workspace};
    a.check = w.take(s.check);
    a.part_A = w.take(s.state);
    a.part_D = w.take(s.delta);
    a.part_bias = w.take(s.delta);
    a.part_B = w.take(s.part_B);
    a.part_C = w.take(s.part_B);
    if (s.joined) {
        a.chunk_state = w.take(s.state);
        a.chunk_back = w.take(s.state);
        a.chunk_delta = w.take(s.delta);
        a.check_delta = w.take(s.check_delta);
    }
    return status(launch_scan_grad(dtype, a, (hipStream_t)stream));
}

int selective_scan_step(const selective_scan_step_problem_t *p, int dtype, const void *x, const void *dt,
                        const float *A, const void *B, const void *C, const float *D, const void *z,
                        const float *dt_bias, float *state, const int *slots, void *y, void *stream)
{
    if (!p || p->rows < 0 || p->pool < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    for (long long v : {p->x_row, p->dt_row, p->b_row, p->c_row, p->z_row, p->b_group, p->c_group})
        if (v < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    const int r = check_scan_sizes(p->d, p->n, p->groups, p->softplus, dtype);
    if (r != CONV2D_OK) return r;
    if (p->rows == 0) return CONV2D_OK;
    if (!x || !dt || !A || !B || !C || !y || (p->pool > 0 && !state)) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {x, dt, B, C, z, y}) || !all_aligned(4, {A, D, dt_bias, state, slots}))
        return CONV2D_ERR_UNSUPPORTED;
    if (ceil_div(p->d, 64) > kMaxGridY || !fits(ceil_div(p->rows, scan_step_rows(p->n)), 256)) return CONV2D_ERR_UNSUPPORTED;
    ScanStepArgs a = {p->rows, p->pool, p->d, p->n, p->groups, p->softplus, p->x_row, p->dt_row, p->b_row, p->c_row,
                      p->z_row, p->b_group, p->c_group, x, dt, B, C, z, A, D, dt_bias, slots, state, y};
    return status(launch_scan_step(dtype, a, (hipStream_t)stream));
}

int fp8_quantize(int form, int dtype, int m, int k, const void *x, long long x_row, void *q, long long q_pitch,
                 float *scale, void *stream)
{
    if (form != FP8_ROWS && form != FP8_TRANSPOSE && form != FP8_BLOCKS) return CONV2D_ERR_INVALID_ARGUMENT;
    if (m < 0 || k < 0 || x_row < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    const long long len = form == FP8_TRANSPOSE ? m : k;
    if (q_pitch < len || q_pitch > ceil_div(len, kFp8Block) * kFp8Block) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || q_pitch % 16) return CONV2D_ERR_UNSUPPORTED;
    if (m == 0 || k == 0) return CONV2D_OK;
    if (!x || !q || !scale) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!aligned(x, bytes_of(dtype)) || !aligned(q, 16) || !aligned(scale, 4)) return CONV2D_ERR_UNSUPPORTED;
    const long long kb = ceil_div(k, kFp8Block), mb = ceil_div(m, kFp8Block);
    if (form == FP8_ROWS && !fits(ceil_div(kb * m, 16), 256)) return CONV2D_ERR_UNSUPPORTED;
    if (form == FP8_TRANSPOSE && (ceil_div(k, 64) > kMaxGridY || !fits(mb, 256))) return CONV2D_ERR_UNSUPPORTED;
    if (form == FP8_BLOCKS && (mb > kMaxGridY || !fits(kb, 256))) return CONV2D_ERR_UNSUPPORTED;
    const Fp8QuantArgs a = {m, k, x_row, q_pitch, x, (uint8_t *)q, scale};
    return status(launch_fp8_quantize(form, dtype, a, (hipStream_t)stream));
}

static int check_matmul(const fp8_matmul_problem_t *p, int dtype)
{
    if (!p || p->m < 0 || p->n < 0 || p->k < 0 || (p->b_blocks != 0 && p->b_blocks != 1) || p->a_pitch < p->k ||
        p->b_pitch < p->k)
        return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || p->a_pitch % 16 || p->b_pitch % 16) return CONV2D_ERR_UNSUPPORTED;
    // a tile's rows are read through 32-bit offsets
    if (p->a_pitch > (1LL << 22) || p->b_pitch > (1LL << 22)) return CONV2D_ERR_UNSUPPORTED;
    return CONV2D_OK;
}

int fp8_matmul_workspace_size(const fp8_matmul_problem_t *prob, int dtype, size_t *bytes)
{
    const int r = check_matmul(prob, dtype);
    if (r != CONV2D_OK) return r;
    if (!bytes) return CONV2D_ERR_INVALID_ARGUMENT;
    size_t need = 0;
    if (prob->m > 0 && prob->n > 0) {
        const Fp8Plan plan = fp8_matmul_plan(prob->m, prob->n, prob->k, dtype);
        if (!fp8_matmul_fits(prob->m, prob->n, prob->k, plan)) return CONV2D_ERR_UNSUPPORTED;
        need = fp8_matmul_bytes(prob->m, prob->n, plan);
    }
    *bytes = need;
    return CONV2D_OK;
}

int fp8_matmul(const fp8_matmul_problem_t *prob, int dtype, const void *a, const float *a_scale,
               const void *b, const float *b_scale, void *out, void *workspace, size_t workspace_bytes,
               void *stream)
{
    const int r = check_matmul(prob, dtype);
    if (r != CONV2D_OK) return r;
    if (prob->m == 0 || prob->n == 0) return CONV2D_OK;
    if (!out || (prob->k > 0 && (!a || !a_scale || !b || !b_scale))) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!aligned(a, 16) || !aligned(b, 16) || !all_aligned(4, {a_scale, b_scale}) || !aligned(out, bytes_of(dtype)) ||
        !aligned(workspace, 16))
        return CONV2D_ERR_UNSUPPORTED;
    const Fp8Plan plan = fp8_matmul_plan(prob->m, prob->n, prob->k, dtype);
    if (!fp8_matmul_fits(prob->m, prob->n, prob->k, plan)) return CONV2D_ERR_UNSUPPORTED;
    const size_t need = fp8_matmul_bytes(prob->m, prob->n, plan);
    if (need && !workspace) return CONV2D_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    Fp8MatmulArgs m = {};
    m.m = prob->m;
    m.n = prob->n;
    m.k = prob->k;
    m.kb = (int)ceil_div(prob->k, kFp8Block);
    m.b_blocks = prob->b_blocks;
    m.a_pitch = prob->a_pitch;
    m.b_pitch = prob->b_pitch;
    m.a = (const uint8_t *)a;
    m.b = (const uint8_t *)b;
    m.a_scale = a_scale;
    m.b_scale = b_scale;
    m.out = out;
    return status(launch_fp8_matmul(dtype, m, plan, workspace, (hipStream_t)stream));
}

}  // extern "C"
