// block_api.cpp -- the C ABI of a recurrent block's operators (gated recurrence, layer
// norm, 4-bit products): argument checks, workspace layout, launch shapes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <numeric>

#include "block_internal.h"
#include "seq_checks.h"

using namespace cnv;

namespace {

// ---- gated recurrence --------------------------------------------------------------
int check_recurrence(const gated_recurrence_problem_t *p, int dtype, bool grad)
{
    if (!p) return CONV2D_ERR_INVALID_ARGUMENT;
    int r = check_batch(p->batch);
    if (r != CONV2D_OK) return r;
    if (p->d < 1) return CONV2D_ERR_INVALID_ARGUMENT;
    for (const seq_stride_t *s : {&p->x, &p->r, &p->i, &p->z})
        if (r == CONV2D_OK) r = check_stride(*s);
    if (r == CONV2D_OK && grad) r = check_stride(p->dy);
    if (r != CONV2D_OK) return r;
    if (!float_type(dtype) || p->d > kMaxStride) return CONV2D_ERR_UNSUPPORTED;
    return CONV2D_OK;
}

struct RecurPlan {
    RecurShape shape;
    int across, chunk, chunks, joined, per_seq;
    size_t per_chunk, per_segment;  // bytes of a value for each of them and channel
};

// Whether one stride reaches all rows of a batch.  Of sequences of one token it is that
// between sequences: such an axis's own stride means nothing, and callers give any.
bool single_tokens(const seq_batch_t &b) { return !b.seq_start && b.seqs > 1 && b.len == 1; }
bool one_stride(const seq_batch_t &b, const seq_stride_t &s)
{
    return b.seq_start || b.seqs == 1 || (single_tokens(b) ? s.seq <= kMaxStride : s.seq == b.len * s.row);
}

// Sequences are walked whole where that alone gives every compute unit a workgroup, for
// chunks are read twice; else they are cut so that each unit has as many workgroups as
// it holds: two in the forward pass, one in the gradient's.  (8192 tokens of 4096 bf16
// channels: forward 102 us with two, 114 with one; gradients 230 with one, 228 with two, but
// of 3001 packed tokens of 1999 channels with states 58 and 62.)  Whole sequences give a
// workgroup 128 bytes of a row (with 64 and twice the workgroups 4 x 4096 x 4096 takes 188 us
// instead of 150, its gradients 457 instead of 370), cut ones, which can make up for it by
// shorter chunks, 256: the 8192 tokens take 102 us, with 128 bytes 119.
// Chunks run over all tokens, sequences' borders inside them, unless a dense batch's
// sequences lie apart.
RecurPlan recur_plan(const gated_recurrence_problem_t *p, int dtype, bool grad)
{
    const seq_batch_t &b = p->batch;
    bool flat = one_stride(b, p->x) && one_stride(b, p->r) && one_stride(b, p->i) && one_stride(b, p->z);
    if (grad) flat = flat && one_stride(b, p->dy);
    RecurPlan r;
    r.shape = {32, dtype != CONV2D_DTYPE_F32 ? 2 : 1};
    if (p->d < r.shape.vc) r.shape = {8, 1};
    // sequences that are walked whole; all tokens together where their lengths are on the device
    const long long walks = b.seq_start ? 1 : b.seqs;
    while (r.shape.lanes > 8 && p->d <= r.shape.channels() / 2) r.shape.lanes /= 2;
    const bool cut = ceil_div(p->d, r.shape.channels()) * walks < kCUs;
    if (cut && p->d > r.shape.channels()) r.shape.lanes *= 2;
    const int segment = recur_segment(r.shape);
    const long long across = ceil_div(p->d, r.shape.channels());
    long long chunk = b.tokens;
    if (!cut && !b.seq_start && b.len >= segment && b.len % segment) flat = false;
    // sequences that whole segments hold, a few together where they are short
    const long long whole = b.seq_start || b.len < 1 ? 0 : std::lcm((long long)b.len, (long long)segment);
    if (!cut && !flat) chunk = b.len;
    else if (!cut && whole > 0 && whole <= kRecurChunkMost && across * ceil_div(b.tokens, whole) >= kCUs)
        chunk = whole * std::max(1LL, 256 / whole);
    else if (cut || !b.seq_start) chunk = ceil_div(b.tokens, ceil_div(grad ? kCUs : 2 * kCUs, across));
    chunk = std::min(std::max(1LL, ceil_div(std::min(chunk, flat ? b.tokens : b.len), segment)) * segment, (long long)kRecurChunkMost);
    r.across = (int)across;
    r.chunk = (int)chunk;
    r.per_seq = flat ? 0 : (int)ceil_div(b.len, chunk);
    r.chunks = flat ? (int)ceil_div(b.tokens, chunk) : r.per_seq * b.seqs;
    r.joined = flat ? r.chunks > 1 && (b.seq_start || chunk % b.len != 0) : r.per_seq > 1;
    r.per_chunk = up((size_t)r.chunks * p->d * 4);
    r.per_segment = up((size_t)r.chunks * (chunk / segment) * p->d * 4);
    return r;
}
size_t recur_bytes(const RecurPlan &r) { return r.joined ? 2 * r.per_chunk : 0; }
size_t recur_grad_bytes(const gated_recurrence_problem_t *p, const RecurPlan &r)
{
    return up((size_t)r.chunks * 3 * p->d * 4) + 2 * r.per_segment + (r.joined ? 4 * r.per_chunk : 0);
}
bool recur_fits(const gated_recurrence_problem_t *p, const RecurPlan &r)
{
    return fits((r.chunks + ceil_div(p->batch.seqs, kRecurStateSeqs)) * r.across + 8, 64 * kRecurWaves);
}

RecurArgs recur_args(const gated_recurrence_problem_t *p, const RecurPlan &r, const void *z)
{
    RecurArgs a = {};
    a.q = seqs_of(p->batch);
    a.d = p->d;
    a.chunk = r.chunk;
    a.chunks = r.chunks;
    a.across = r.across;
    a.tail = r.per_seq ? p->batch.seqs : 1;
    a.joined = r.joined;
    a.per_seq = r.per_seq;
    a.xs = stride_of(p->x);
    a.rs = stride_of(p->r);
    a.is = stride_of(p->i);
    a.z = z;
    if (z) a.zs = stride_of(p->z);  // else 0: the kernels mark an absent tensor by an offset, which a row's would carry round
    a.dys = stride_of(p->dy);
    if (!r.per_seq && single_tokens(p->batch))
        for (RowStride *s : {&a.xs, &a.rs, &a.is, &a.zs, &a.dys}) s->row = s->seq;
    return a;
}

// ---- layer norm --------------------------------------------------------------------
int check_norm(const layer_norm_problem_t *p, int dtype, int param_dtype)
{
    if (!p || p->seqs < 0 || p->len < 0 || p->d < 1 || !(p->eps >= 0.0f)) return CONV2D_ERR_INVALID_ARGUMENT;
    for (const seq_stride_t *s : {&p->x, &p->residual, &p->dy, &p->dtotal})
        if (s->row < 0 || s->seq < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(p->eps)) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || (param_dtype != dtype && param_dtype != CONV2D_DTYPE_F32)) return CONV2D_ERR_UNSUPPORTED;
    return p->d > kMaxStride || (long long)p->seqs * p->len > kMaxRows ? CONV2D_ERR_UNSUPPORTED : CONV2D_OK;
}

// Whether a launch with each row in a shape's lanes fits.
bool norm_fits(const NormShape &s, long long rows) { return fits(ceil_div(rows * s.lanes, 256), 256); }

NormArgs norm_args(const layer_norm_problem_t *p, int param_dtype)
{
    NormArgs a = {};
    a.rows = p->seqs * p->len;
    a.len = p->len;
    a.d = p->d;
    a.eps = p->eps;
    a.count = (float)p->d;
    a.param_f32 = param_dtype == CONV2D_DTYPE_F32;
    a.xs = stride_of(p->x);
    a.rs = stride_of(p->residual);
    a.dys = stride_of(p->dy);
    a.dts = stride_of(p->dtotal);
    return a;
}

struct NormGradPlan {
    NormShape shape;
    int per, parts;
    size_t partial, stats;
};
// Parts of rows, each with a partial sum of both parameters' gradients, which is written
// and read: as many as a compute unit holds workgroups.  Of 1024 lanes one (8192 rows of
// 8192: 135 us, with two 146), of 256 and less four where a lane has one vector (16384 of
// 2048: 56 us, with two 72), else two (16384 of 4096: 122 us, with four 131).
NormGradPlan norm_grad_plan(const layer_norm_problem_t *p, int dtype)
{
    NormGradPlan r;
    r.shape = layer_norm_grad_shape(dtype, p->d);
    const long long rows = (long long)p->seqs * p->len;
    const int groups = r.shape.held ? std::max(1, 256 / r.shape.lanes) : 1;
    r.per = (int)(ceil_div(ceil_div(std::max(rows, 1LL), (r.shape.lanes > 256 ? 1 : r.shape.vecs == 1 ? 4 : 2) * kCUs), groups) * groups);
    r.parts = (int)ceil_div(rows, r.per);
    r.partial = up((size_t)r.parts * 2 * p->d * 4);
    r.stats = r.shape.held ? 0 : up((size_t)rows * 16);
    return r;
}

}  // namespace

extern "C" {

int gated_recurrence_workspace_size(const gated_recurrence_problem_t *prob, int dtype, size_t *bytes)
{
    const int r = check_recurrence(prob, dtype, false);
    if (r != CONV2D_OK) return r;
    if (!bytes) return CONV2D_ERR_INVALID_ARGUMENT;
    const RecurPlan plan = recur_plan(prob, dtype, false);
    if (!recur_fits(prob, plan)) return CONV2D_ERR_UNSUPPORTED;
    *bytes = recur_bytes(plan);
    return CONV2D_OK;
}

int gated_recurrence(const gated_recurrence_problem_t *prob, int dtype, const void *x, const void *r, const void *i,
                     const float *A, const void *z, const float *r_bias, const float *i_bias, const float *initial_state,
                     void *y, float *final_state, void *workspace, size_t workspace_bytes, void *stream)
{
    const int e = check_recurrence(prob, dtype, false);
    if (e != CONV2D_OK) return e;
    const bool rows = prob->batch.tokens > 0;
    if (!A || (rows && (!x || !r || !i || !y))) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {x, r, i, z, y}) || !all_aligned(4, {A, r_bias, i_bias, initial_state, final_state}) ||
        !aligned(workspace, 16))
        return CONV2D_ERR_UNSUPPORTED;
    const RecurPlan plan = recur_plan(prob, dtype, false);
    if (!recur_fits(prob, plan)) return CONV2D_ERR_UNSUPPORTED;
    const size_t need = recur_bytes(plan);
    if (need && !workspace) return CONV2D_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    if (!rows && !final_state) return CONV2D_OK;
    RecurArgs a = recur_args(prob, plan, z);
    a.x = x;
    a.r = r;
    a.i = i;
    a.A = A;
    a.r_bias = r_bias;
    a.i_bias = i_bias;
    a.initial = initial_state;
    a.y = y;
    a.final_state = final_state;
    if (plan.joined) {
        Carver w{(char *)workspace};
        a.chunk_decay = w.take(plan.per_chunk);
        a.chunk_state = w.take(plan.per_chunk);
    }
    return status(launch_recurrence(dtype, a, plan.shape, (hipStream_t)stream));
}

int gated_recurrence_grad_workspace_size(const gated_recurrence_problem_t *prob, int dtype, size_t *bytes)
{
    const int r = check_recurrence(prob, dtype, true);
    if (r != CONV2D_OK) return r;
    if (!bytes) return CONV2D_ERR_INVALID_ARGUMENT;
    const RecurPlan plan = recur_plan(prob, dtype, true);
    if (!recur_fits(prob, plan)) return CONV2D_ERR_UNSUPPORTED;
    *bytes = recur_grad_bytes(prob, plan);
    return CONV2D_OK;
}

int gated_recurrence_grad(const gated_recurrence_problem_t *prob, int dtype, const void *dy, const void *x, const void *r,
                          const void *i, const float *A, const void *z, const float *r_bias, const float *i_bias,
                          const float *initial_state, const float *dfinal, const gated_recurrence_grads_t *g,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    const int e = check_recurrence(prob, dtype, true);
    if (e != CONV2D_OK) return e;
    const bool rows = prob->batch.tokens > 0;
    if (!A || !g || !g->dA) return CONV2D_ERR_INVALID_ARGUMENT;
    if (rows && (!dy || !x || !r || !i || !g->dx || !g->dr || !g->di || (z && !g->dz))) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {dy, x, r, i, z, g->dx, g->dr, g->di, g->dz}) ||
        !all_aligned(4, {A, r_bias, i_bias, initial_state, dfinal, g->dA, g->dr_bias, g->di_bias, g->dinitial}) ||
        !aligned(workspace, 16))
        return CONV2D_ERR_UNSUPPORTED;
    const RecurPlan plan = recur_plan(prob, dtype, true);
    if (!recur_fits(prob, plan)) return CONV2D_ERR_UNSUPPORTED;
    const size_t need = recur_grad_bytes(prob, plan);
    if (need && !workspace) return CONV2D_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    RecurArgs a = recur_args(prob, plan, z);
    a.x = x;
    a.r = r;
    a.i = i;
    a.dy = dy;
    a.A = A;
    a.r_bias = r_bias;
    a.i_bias = i_bias;
    a.initial = initial_state;
    a.dfinal = dfinal;
    a.dinitial = g->dinitial;
    a.dx = g->dx;
    a.dr = g->dr;
    a.di = g->di;
    a.dz = z ? g->dz : nullptr;
    Carver w{(char *)workspace};
    a.partial = w.take(up((size_t)plan.chunks * 3 * prob->d * 4));
    a.seg_decay = w.take(plan.per_segment);
    a.seg_state = w.take(plan.per_segment);
    if (plan.joined) {
        a.chunk_decay = w.take(plan.per_chunk);
        a.chunk_state = w.take(plan.per_chunk);
        a.back_decay = w.take(plan.per_chunk);
        a.chunk_back = w.take(plan.per_chunk);
    }
    if (hipError_t h = launch_recurrence_grad(dtype, a, plan.shape, (hipStream_t)stream)) return status(h);
    const ColumnSumArgs s = {a.partial, plan.chunks, 3, prob->d, {g->dA, g->dr_bias, g->di_bias}, A};
    return status(launch_column_sums(CONV2D_DTYPE_F32, s, (hipStream_t)stream));
}

int gated_recurrence_step(const gated_recurrence_step_problem_t *p, int dtype, const void *x, const void *r, const void *i,
                          const float *A, const void *z, const float *r_bias, const float *i_bias, float *state,
                          const int *slots, void *y, void *stream)
{
    if (!p || p->rows < 0 || p->pool < 0 || p->d < 1) return CONV2D_ERR_INVALID_ARGUMENT;
    for (long long v : {p->x_row, p->r_row, p->i_row, p->z_row})
        if (v < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || p->d > kMaxStride) return CONV2D_ERR_UNSUPPORTED;
    if (p->rows == 0) return CONV2D_OK;
    if (!x || !r || !i || !A || !y || (p->pool > 0 && !state)) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {x, r, i, z, y}) || !all_aligned(4, {A, r_bias, i_bias, state, slots}))
        return CONV2D_ERR_UNSUPPORTED;
    if (ceil_div(p->d, 256 * kRecurStepChannels) > kMaxGridY || !fits(p->rows, 256)) return CONV2D_ERR_UNSUPPORTED;
    const RecurStepArgs a = {p->rows, p->pool, p->d, p->x_row, p->r_row, p->i_row, p->z_row, x, r, i, z, A, r_bias, i_bias,
                             state, slots, y};
    return status(launch_recurrence_step(dtype, a, (hipStream_t)stream));
}

int layer_norm(const layer_norm_problem_t *prob, int dtype, int param_dtype, const void *x, const void *residual,
               const void *weight, const void *bias, void *y, void *total, void *stream)
{
    const int e = check_norm(prob, dtype, param_dtype);
    if (e != CONV2D_OK) return e;
    NormArgs a = norm_args(prob, param_dtype);
    if (a.rows == 0) return CONV2D_OK;
    if (!x || !y) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {x, residual, y, total}) || !all_aligned(bytes_of(param_dtype), {weight, bias}))
        return CONV2D_ERR_UNSUPPORTED;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.total = total;
    const NormShape shape = layer_norm_shape(dtype, a.rows, a.d);
    if (!norm_fits(shape, a.rows)) return CONV2D_ERR_UNSUPPORTED;
    return status(launch_layer_norm(dtype, a, shape, (hipStream_t)stream));
}

int layer_norm_grad_workspace_size(const layer_norm_problem_t *prob, int dtype, size_t *bytes)
{
    const int e = check_norm(prob, dtype, CONV2D_DTYPE_F32);
    if (e != CONV2D_OK) return e;
    if (!bytes) return CONV2D_ERR_INVALID_ARGUMENT;
    const NormGradPlan plan = norm_grad_plan(prob, dtype);
    if (!norm_fits(plan.shape, (long long)prob->seqs * prob->len)) return CONV2D_ERR_UNSUPPORTED;
    *bytes = plan.partial + plan.stats;
    return CONV2D_OK;
}

int layer_norm_grad(const layer_norm_problem_t *prob, int dtype, int param_dtype, const void *dy, const void *x,
                    const void *weight, const void *dtotal, void *dx, void *dweight, void *dbias, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    const int e = check_norm(prob, dtype, param_dtype);
    if (e != CONV2D_OK) return e;
    NormArgs a = norm_args(prob, param_dtype);
    if (a.rows > 0 && (!dy || !x || !dx)) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {dy, x, dtotal, dx}) || !all_aligned(bytes_of(param_dtype), {weight, dweight, dbias}) ||
        !aligned(workspace, 16))
        return CONV2D_ERR_UNSUPPORTED;
    const NormGradPlan plan = norm_grad_plan(prob, dtype);
    if (!norm_fits(plan.shape, a.rows)) return CONV2D_ERR_UNSUPPORTED;
    const size_t need = plan.partial + plan.stats;
    if (need && !workspace) return CONV2D_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    a.dy = dy;
    a.x = x;
    a.weight = weight;
    a.dtotal = dtotal;
    a.dx = dx;
    a.per = plan.per;
    a.parts = plan.parts;
    Carver w{(char *)workspace};
    a.partial = w.take(plan.partial);
    a.stats = w.take(plan.stats);
    if (a.rows > 0)
        if (hipError_t h = launch_layer_norm_grad(dtype, a, plan.shape, (hipStream_t)stream)) return status(h);
    if (!dweight && !dbias) return CONV2D_OK;
    const ColumnSumArgs s = {a.partial, plan.parts, 2, prob->d, {dweight, dbias, nullptr}, nullptr};
    return status(launch_column_sums(param_dtype, s, (hipStream_t)stream));
}

int fp4_quantize(int dtype, int m, int k, const void *x, long long x_row, void *q, long long q_pitch, void *scale,
                 void *stream)
{
    if (m < 0 || k < 0 || x_row < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    const long long groups = ceil_div(k, kFp4Group);
    if (q_pitch < groups * 16) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || q_pitch % 16) return CONV2D_ERR_UNSUPPORTED;
    if (m == 0 || k == 0) return CONV2D_OK;
    if (!x || !q || !scale) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!aligned(x, bytes_of(dtype)) || !aligned(q, 16)) return CONV2D_ERR_UNSUPPORTED;
    if (!fits(ceil_div(groups * m, 64), 256)) return CONV2D_ERR_UNSUPPORTED;
    const Fp4QuantArgs a = {m, k, (int)groups, x_row, q_pitch, x, (uint8_t *)q, (uint8_t *)scale};
    return status(launch_fp4_quantize(dtype, a, (hipStream_t)stream));
}

static int check_fp4(const fp4_matmul_problem_t *p, int dtype)
{
    if (!p || p->m < 0 || p->n < 0 || p->k < 0 || p->x_row < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    if (p->w_pitch < ceil_div(p->k, kFp4Group) * 16) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!float_type(dtype) || p->w_pitch % 16) return CONV2D_ERR_UNSUPPORTED;
    // workgroups of up to 512 threads along n and 64 rows along m; the sums' a value to a thread
    if (ceil_div(p->m, 64) > kMaxGridY || !fits(ceil_div(p->n, 16), 512) || !fits(ceil_div((long long)p->m * p->n, 1024), 256))
        return CONV2D_ERR_UNSUPPORTED;
    return CONV2D_OK;
}

int fp4_matmul_workspace_size(const fp4_matmul_problem_t *prob, int dtype, size_t *bytes)
{
    const int r = check_fp4(prob, dtype);
    if (r != CONV2D_OK) return r;
    if (!bytes) return CONV2D_ERR_INVALID_ARGUMENT;
    *bytes = up(fp4_matmul_plan(prob->m, prob->n, prob->k, dtype).bytes(prob->m, prob->n));
    return CONV2D_OK;
}

int fp4_matmul(const fp4_matmul_problem_t *p, int dtype, const void *x, const void *w, const void *w_scale, void *out,
               void *workspace, size_t workspace_bytes, void *stream)
{
    const int r = check_fp4(p, dtype);
    if (r != CONV2D_OK) return r;
    if (p->m == 0 || p->n == 0) return CONV2D_OK;
    if (!out || (p->k > 0 && (!x || !w || !w_scale))) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!all_aligned(bytes_of(dtype), {x, out}) || !aligned(w, 16) || !aligned(workspace, 16)) return CONV2D_ERR_UNSUPPORTED;
    const Fp4Plan plan = fp4_matmul_plan(p->m, p->n, p->k, dtype);
    const size_t need = up(plan.bytes(p->m, p->n));
    if (need && !workspace) return CONV2D_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return CONV2D_ERR_WORKSPACE_TOO_SMALL;
    const Fp4MatmulArgs a = {p->m, p->n, p->k, (int)ceil_div(p->k, kFp4Group), p->x_row, p->w_pitch, x, (const uint8_t *)w,
                             (const uint8_t *)w_scale, out, plan.splits, plan.per, plan.tiles, (float *)workspace};
    return status(launch_fp4_matmul(dtype, a, (hipStream_t)stream));
}

}  // extern "C"
