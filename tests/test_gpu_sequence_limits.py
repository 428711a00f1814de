"""Sequence operators at the ends of their accepted sizes: token numbers up to the last that 31 bits hold."""
import pytest
import torch

import convolution_nhwc_implicit_amd as nn
import sequence_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def test_scan_to_the_last_token():
    """2^31 - 1 tokens of one channel: the loop's count may not pass 31 bits behind the last one.  The end against
    the 64-bit form from 1000 tokens back, of which exp(-250) would be left."""
    T, far, cut = 2 ** 31 - 1, 1000, 500
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(1, T, 1, generator=g, device=DEV, dtype=BF16)
    one = torch.ones(1, 1, 1, device=DEV, dtype=BF16)
    dt, BC = (0.5 * one).expand(1, T, 1), one.unsqueeze(-1).expand(1, T, 1, 1)
    y, final = nn.selective_scan(x, dt, -torch.ones(1, 1, device=DEV), BC, BC, return_state=True)
    end, out = x[0, T - far:].double().cpu(), y[0, T - cut:].double().cpu()
    o = torch.ones(far, 1, 1, dtype=torch.float64)
    want, fin, mag, worst = R.scan(end, 0.5 * o[:, 0], -o[:1, 0], o, o, None, None, None, False, [far])
    tol = R.half_step(BF16) * want.abs() + R.U * (worst + 24) * mag
    assert ((out - want[far - cut:]).abs() <= tol[far - cut:]).all()
    assert abs(float(final) - float(fin)) <= R.U * (worst + 24) * float(mag[-1])


def test_descending_starts_stay_in_bounds():
    """Starts that go up and down between 0 and 2^20 in 2^15 sequences: their chunks, counted together, pass 31 bits.
    What they give is not specified, but they may reach nothing outside the buffers, so a batch after them is right."""
    T, seqs, d = 2 ** 20, 2 ** 15, 1
    g = torch.Generator(device=DEV).manual_seed(4)
    x, dt = torch.randn(T, d, generator=g, device=DEV), torch.rand(T, d, generator=g, device=DEV)
    B, C = (torch.randn(T, 1, 1, generator=g, device=DEV) for _ in range(2))
    A = -torch.ones(d, 1, device=DEV)
    rising = torch.arange(seqs + 1, device=DEV, dtype=torch.int32) * (T // seqs)
    descending = (torch.arange(seqs + 1, device=DEV) % 2 * T).to(torch.int32)

    def run(start):
        return [v for v in nn.selective_scan_grad(x, x, dt, A, B, C, seq_start=start).values() if v is not None]

    want = run(rising)
    run(descending)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, run(rising)))


def test_scan_grad_past_31_bits():
    """Gradients of [5][40000][11264], 2.25e9 elements: the last sequence's as by itself.  Chunks may lie otherwise, so
    within half a step of each and the fp32 roundings: with |values| below 6.4 and decays of at most exp(-0.97) a token
    no sum of terms is above 1700, nor rounded more often than 90 times (2^-24 each)."""
    L, d, n = 40000, 11264, 4
    g = torch.Generator(device=DEV).manual_seed(5)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=BF16)

    x, dy, B, C = randn(5, L, d), randn(5, L, d), randn(5, L, 1, n), randn(5, L, 1, n)
    dt = torch.full((1, 1, d), 0.5, dtype=BF16, device=DEV).expand(5, L, d)
    A = -1 - torch.rand(d, n, generator=g, device=DEV)
    whole = nn.selective_scan_grad(dy, x, dt, A, B, C, softplus=True)
    last = nn.selective_scan_grad(dy[4:], x[4:], dt[4:], A, B[4:], C[4:], softplus=True)
    for k in ("du", "ddt"):
        for lo in (0, L // 2, L - 64):
            a, b = whole[k][4, lo:lo + 64].float(), last[k][0, lo:lo + 64].float()
            assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -6).all(), (k, lo)
    # sums over the channels: as often again rounded, and half a step
    for k in ("dB", "dC"):
        a, b = whole[k][4].float(), last[k][0].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -6 * d ** 0.5).all(), k


@pytest.mark.parametrize("packed", [False, True])
def test_infinite_rates(packed):
    """A of minus infinity forgets the state at every token, also where a chunk ends inside a step: h = delta x B."""
    L, d, n = 300, 20, 16
    g = torch.Generator(device=DEV).manual_seed(6)
    lead = (2 * L + 3,) if packed else (2, L)
    start = torch.tensor([0, L, 2 * L + 3], dtype=torch.int32, device=DEV) if packed else None
    x, dt, dy = (torch.randn(*lead, d, generator=g, device=DEV) for _ in range(3))
    B, C = (torch.randn(*lead, 1, n, generator=g, device=DEV) for _ in range(2))
    A = -torch.rand(d, n, generator=g, device=DEV)
    A[:, 3] = -float("inf")
    A[5] = -float("inf")
    dfinal = torch.randn(2, d, n, generator=g, device=DEV)
    kw = dict(softplus=True, seq_start=start)
    y, final = nn.selective_scan(x, dt, A, B, C, return_state=True, **kw)
    got = nn.selective_scan_grad(dy, x, dt, A, B, C, dfinal_state=dfinal, **kw)
    assert y.isfinite().all() and all(v.isfinite().all() for v in got.values() if v is not None)
    ends = [L - 1, 2 * L + 2] if packed else None
    xe, de, Be = ((t[ends] if packed else t[:, -1]) for t in (x, torch.nn.functional.softplus(dt.double()), B))
    want = (de * xe).unsqueeze(-1) * Be.double()
    bound = 16 * R.U * want.abs() + 1e-30  # the step size's roundings and two products
    for c, k in ((slice(None), 3), (5, slice(None))):
        assert ((final.double() - want).abs() <= bound)[:, c, k].all()
    # no such rate takes part in what lies beside it
    A2 = A.clone()
    A2[:, 3] = -2e38
    A2[5] = -2e38
    y2, final2 = nn.selective_scan(x, dt, A2, B, C, return_state=True, **kw)
    assert torch.equal(y, y2) and torch.equal(final, final2)
    state, pool = torch.randn(4, d, n, generator=g, device=DEV), (x[:4] if packed else x[0, :4])
    t = [v[:4] if packed else v[0, :4] for v in (dt, B, C)]
    other = state.clone()
    assert torch.equal(nn.selective_scan_step(pool, t[0], A, t[1], t[2], state, softplus=True),
                       nn.selective_scan_step(pool, t[0], A2, t[1], t[2], other, softplus=True))
    assert torch.equal(state, other)
