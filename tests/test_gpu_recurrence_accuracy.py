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


@pytest.mark.parametrize("typ", [F16, BF16, F32], ids=str)
def test_gradients_of_open_and_shut_gates(typ):
    """dr and di of gates near 0 and 1, relative to themselves: a gate times its complement, both of which a sigmoid has
    to all its bits. One term each, in which no sum cancels:
      dr = -k a^2 / s u x A g (1 - g),  di = k s x u (1 - u)
    A sigmoid or a complement is off by (8 + 4 |v|) U relative, a^2 / s by 32 U and (8 + 4 |r|) |L| U, ten products by U
    each; below fp32's normal numbers nothing is left (a complement of 2^-126 times terms of at most 2^6)."""
    g = torch.Generator().manual_seed(3)
    v = torch.tensor([-INF, -100.0, -20.0, -8.0, -1.0, 0.0, 1.0, 4.0, 8.0, 12.0, 16.0, 20.0, 60.0, 100.0, INF])
    r, i = torch.cartesian_prod(v, v).t()
    d = 12
    A = -torch.exp2(torch.linspace(-8, 1, d))
    r, i = (t[:, None].expand(-1, d).to(typ).contiguous() for t in (r, i))
    x, dy = (torch.randn(r.shape, generator=g).to(typ) for _ in range(2))
    got = call(nn.gated_recurrence_grad, dy, x, r, i, A)
    xd, dyd, rd, id_, Ad = (t.double() for t in (x, dy, r, i, A))
    gate, take = torch.sigmoid(rd), torch.sigmoid(id_)
    gate[gate < 2.0 ** -126] = 0  # as documented: their root, some 2^-72, is gone with them
    L = Ad * gate
    s = torch.sqrt(-torch.expm1(2 * L))
    want = dict(dr=-dyd * torch.exp(2 * L) / s.clamp_min(1e-300) * take * xd * L * torch.sigmoid(-rd),
                di=dyd * s * xd * take * torch.sigmoid(-id_))
    vr, vi = (t.abs().clamp_max(128) for t in (rd, id_))  # infinite gates are exact
    count = 64 + 12 * vr + 8 * vi + (8 + 4 * vr) * L.abs()
    for k, w in want.items():
        tol = (count * R.U + R.half_step(typ)) * w.abs() + 2.0 ** -120 + torch.finfo(typ).smallest_normal * torch.finfo(typ).eps
        off = (got[k].double().cpu() - w).abs()
        assert bool((off <= tol).all()), (k, float((off / tol).max()))
    assert not got["dr"][(r == INF).to(DEV)].any() and not got["di"][(i == INF).to(DEV)].any()


def test_bias_gradients_of_open_gates_vanish():
    """Fully open gates: 4000 tokens leave nothing in the biases' gradients, and nothing of one sign at 30."""
    g = torch.Generator().manual_seed(4)
    t, d = 4000, 70
    x, dy = (torch.randn(t, d, generator=g).to(DEV) for _ in range(2))
    A, b = -torch.rand(d, generator=g).to(DEV) - 0.01, torch.zeros(d, device=DEV)
    for v, most in ((INF, 0.0), (100.0, 0.0), (30.0, t * 2.0 ** -40)):
        gate = torch.full_like(x, v)
        k = nn.gated_recurrence_grad(dy, x, gate, gate, A, r_bias=b, i_bias=b)
        # sums of t terms of a few times e^-30 = 2^-43.3 each; e^-100 is below the normal numbers
        assert float(k["dr_bias"].abs().max()) <= most + 2.0 ** -110 and float(k["di_bias"].abs().max()) <= most + 2.0 ** -110
