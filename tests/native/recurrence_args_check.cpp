// What the gated recurrence's C entry points hand to their kernels: block_api.cpp with
// launchers that only keep their arguments.  Prints "ok" or what is wrong.
#include <stdio.h>

#include "block_internal.h"

namespace cnv {
static RecurArgs seen;
static int launches;
hipError_t launch_recurrence(int, const RecurArgs &a, const RecurShape &, hipStream_t)
{
    seen = a;
    ++launches;
    return hipSuccess;
}
hipError_t launch_recurrence_grad(int dtype, const RecurArgs &a, const RecurShape &s, hipStream_t st) { return launch_recurrence(dtype, a, s, st); }
hipError_t launch_recurrence_step(int, const RecurStepArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_column_sums(int, const ColumnSumArgs &, hipStream_t) { return hipSuccess; }
NormShape layer_norm_shape(int, int, int) { return {}; }
NormShape layer_norm_grad_shape(int, int) { return {}; }
hipError_t launch_layer_norm(int, const NormArgs &, const NormShape &, hipStream_t) { return hipSuccess; }
hipError_t launch_layer_norm_grad(int, const NormArgs &, const NormShape &, hipStream_t) { return hipSuccess; }
Fp4Plan fp4_matmul_plan(int, int, int, int) { return {}; }
hipError_t launch_fp4_quantize(int, const Fp4QuantArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_fp4_matmul(int, const Fp4MatmulArgs &, hipStream_t) { return hipSuccess; }
}  // namespace cnv

using namespace cnv;

static void *const at = (void *)(1 << 20);  // never followed
static int bad;
static void expect(bool good, const char *what, int seqs, int len)
{
    if (good) return;
    ++bad;
    printf("%s (%d sequences of %d)\n", what, seqs, len);
}

int main()
{
    const int d = 64;
    for (int seqs : {1, 3, 40})
        for (int len : {2, 50, 20000}) {
            const seq_stride_t s = {d, (long long)len * d};
            gated_recurrence_problem_t p = {{nullptr, seqs, len, (long long)seqs * len}, d, s, s, s, s, s};
            float *f = (float *)at;
            gated_recurrence_grads_t g = {at, at, at, f, at, f, f, f};
            for (const void *z : {(const void *)nullptr, (const void *)at}) {
                launches = 0;
                const int r = gated_recurrence(&p, CONV2D_DTYPE_BF16, at, at, at, f, z, f, f, f, at, f, at, (size_t)1 << 40, nullptr);
                expect(r == CONV2D_OK && launches == 1, "the forward pass is refused", seqs, len);
                expect(seen.z == z && seen.zs.row == (z ? d : 0) && seen.zs.seq == (z ? s.seq : 0), "strides of z, forward pass", seqs, len);
                launches = 0;
                const int e = gated_recurrence_grad(&p, CONV2D_DTYPE_BF16, at, at, at, at, f, z, f, f, f, f, &g, at, (size_t)1 << 40, nullptr);
                expect(e == CONV2D_OK && launches == 1, "the gradient is refused", seqs, len);
                expect(seen.z == z && seen.zs.row == (z ? d : 0) && seen.zs.seq == (z ? s.seq : 0), "strides of z, gradient", seqs, len);
                expect(!seen.dz == !z, "a gradient for z, just where z is there", seqs, len);
                expect(seen.xs.row == d && seen.rs.row == d && seen.is.row == d && seen.dys.row == d, "strides", seqs, len);
            }
        }
    // sequences of one token: rows like any others, whatever the stride over the tokens' axis is called
    for (int seqs : {2, 100, 1024, 150000})
        for (long long row : {0LL, 4096LL, 8192LL}) {
            const seq_stride_t s = {row, 4096}, half = {row, 8192};
            gated_recurrence_problem_t p = {{nullptr, seqs, 1, seqs}, 4096, s, half, half, s, s};
            float *f = (float *)at;
            gated_recurrence_grads_t g = {at, at, at, f, at, f, f, f};
            for (bool grad : {false, true}) {
                const int r = grad ? gated_recurrence_grad(&p, CONV2D_DTYPE_BF16, at, at, at, at, f, at, f, f, f, f, &g, at, (size_t)1 << 40, nullptr)
                                   : gated_recurrence(&p, CONV2D_DTYPE_BF16, at, at, at, f, at, f, f, f, at, f, at, (size_t)1 << 40, nullptr);
                expect(r == CONV2D_OK, "one-token sequences are refused", seqs, 1);
                expect(!seen.per_seq && seen.xs.row == 4096 && seen.rs.row == 8192 && seen.is.row == 8192 && seen.zs.row == 4096 &&
                       (!grad || seen.dys.row == 4096), "one-token sequences lie apart", seqs, 1);
            }
        }
    // but for strides that no row may have
    {
        const seq_stride_t s = {0, 64}, far = {0, 1LL << 25};
        gated_recurrence_problem_t p = {{nullptr, 9, 1, 9}, 64, far, s, s, s, s};
        const int r = gated_recurrence(&p, CONV2D_DTYPE_BF16, at, at, at, (float *)at, at, nullptr, nullptr, nullptr, at, nullptr, at, (size_t)1 << 40, nullptr);
        expect(r == CONV2D_OK && seen.per_seq == 1 && seen.xs.seq == 1LL << 25 && seen.xs.row == 0, "one-token sequences far apart", 9, 1);
    }
    if (!bad) printf("ok\n");
    return bad != 0;
}
