"""Where the gated recurrence's fp32 arithmetic could lose bits that its 64-bit form has: decays near 1, gates near 1.

U = 2^-24 is an fp32 rounding; the exponential, reciprocal and root instructions are off by a step, 2 U at most.
Sequences are of one token, so that no term cancels another."""
import pytest
import torch

import block_ref as R
import convolution_nhwc_implicit_amd as nn

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF = float("inf")


def call(fn, *args, **kw):
    n = args[0].shape[0]
    return fn(*(t.to(DEV) for t in args), seq_start=torch.arange(n + 1, dtype=torch.int32, device=DEV),
              **{k: v if v is None else v.to(DEV) for k, v in kw.items()})


@pytest.mark.parametrize("lo,hi", [(-60.0, -20.0), (-20.0, -4.0), (-4.0, -3.0), (-3.0, -2.0), (-2.0, -1.0), (-1.0, 0.0), (0.0, 2.0)], ids=str)
def test_inputs_scale_of_all_decays(lo, hi):
    """sqrt(1 - a^2) itself, as the state that open gates and an input of 1 leave, for decays A = -2^lo .. -2^hi; and as the
    factor of the input's gradient.

    L = A log2 e is off by 2 U relative, 1 - a^2 by no more for it. As a series it is off by a U of the fit and 2 for its last
    operations, the root of that by half and 2 U more: 5 U. As a difference, where a^2 is at most 1/2: a is off by a step of
    U, a^2 by 1.5 U, the difference, a half at least, by 3 U for that, 2 U for L and U of its own: 6 U, the root 5 U again. A
    product and the result round by one more each."""
    d = 4096
    A = -torch.exp2(torch.linspace(lo, hi, d))
    open_ = torch.full((1, d), INF)
    one = torch.ones(1, d)
    y = call(nn.gated_recurrence, one, open_, open_, A).double().cpu()[0]
    dx = call(nn.gated_recurrence_grad, one, one, open_, open_, A)["dx"].double().cpu()[0]
    want = torch.sqrt(-torch.expm1(2 * A.double()))
    assert float(((y - want) / want).abs().max()) <= 7 * R.U
    assert float(((dx - want) / want).abs().max()) <= 7 * R.U
