"""Edges of the sequence operators: elements past 2^31, infinities and NaN that must stay in their sequences, rows and
channels, expanded tensors, and starts that no batch has."""
import pytest
import torch

import convolution_nhwc_implicit_amd as nn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def randn(g, *shape, scale=1.0, dtype=F32):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


@pytest.fixture
def g():
    return torch.Generator(device=DEV).manual_seed(31)


def test_conv_past_31_bits(g):
    """[3][90000][8192]: 2.2e9 elements.  The last sequence, and its gradients, as by itself."""
    x = randn(g, 3, 90000, 8192, dtype=BF16)
    w, b = randn(g, 8192, 4, dtype=BF16), randn(g, 8192, dtype=BF16)
    y, s = nn.causal_conv(x, w, b, silu=True, return_state=True)
    one, t = nn.causal_conv(x[2:], w, b, silu=True, return_state=True)
    assert torch.equal(y[2:], one) and torch.equal(s[2:], t)
    del one
    dx = nn.causal_conv_grad(y, x, w, b, silu=True)["dx"]
    assert torch.equal(dx[2:], nn.causal_conv_grad(y[2:], x[2:], w, b, silu=True)["dx"])


def test_scan_past_31_bits(g):
    """[5][40000][11264]: 2.25e9 elements.  The last sequence's end, from a state, by itself: within bf16 rounding of
    the state's own fp32 differences."""
    L, d = 40000, 11264
    x, dt = randn(g, 5, L, d, dtype=BF16), torch.full((1,), 0.5, dtype=BF16, device=DEV).expand(5, L, d)
    dt = dt.contiguous()
    B, C = randn(g, 5, L, 1, 4, dtype=BF16), randn(g, 5, L, 1, 4, dtype=BF16)
    A = -torch.exp(randn(g, d, 4))
    y = nn.selective_scan(x, dt, A, B, C, softplus=True)
    cut = L - 64  # decays of exp(-0.97 * 1000 * |A|) leave nothing of the tokens before a start this far back
    far = L - 20000
    tail = nn.selective_scan(x[4:, far:], dt[4:, far:], A, B[4:, far:], C[4:, far:], softplus=True)
    a, b = y[4, cut:].float(), tail[0, cut - far:].float()
    slow = A.abs().amin(1) * 0.97 * (cut - far) > 60
    assert slow.float().mean() > 0.9
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -14)[:, slow].all()


def test_step_past_31_bits(g):
    """A pool of 2.2e9 state values: its last place."""
    pool, d, n = 34000, 4096, 16
    state = torch.zeros(pool, d, n, device=DEV)
    x, dt = randn(g, 2, d, dtype=BF16), randn(g, 2, d, dtype=BF16)
    B, C = randn(g, 2, 1, n, dtype=BF16), randn(g, 2, 1, n, dtype=BF16)
    A = -torch.exp(randn(g, d, n))
    last = torch.tensor([pool - 1, 7], dtype=torch.int32, device=DEV)
    y = nn.selective_scan_step(x, dt, A, B, C, state, softplus=True, slots=last)
    small = torch.zeros(2, d, n, device=DEV)
    assert torch.equal(y, nn.selective_scan_step(x, dt, A, B, C, small, softplus=True))
    assert torch.equal(state[pool - 1], small[0]) and torch.equal(state[7], small[1])
    conv = torch.zeros(180000, 3, d, dtype=BF16, device=DEV)
    last = torch.tensor([179999, 7], dtype=torch.int32, device=DEV)
    w = randn(g, d, 4, dtype=BF16)
    y = nn.causal_conv_step(x, conv, w, slots=last)
    assert y.isfinite().all() and torch.equal(conv[179999, 2], x[0]) and torch.equal(conv[7, 2], x[1])


def test_product_past_31_bits(g):
    """65600 x 32832 results; its last rows and columns by themselves (other tiles: within a rounding)."""
    a, b = randn(g, 65600, 128, dtype=BF16), randn(g, 32832, 128, dtype=BF16)
    qa, sa = nn.fp8_quantize(a)
    qb, sb = nn.fp8_quantize(b)
    out = nn.fp8_matmul(qa, sa, qb, sb)
    one = nn.fp8_matmul(qa[-200:].contiguous(), sa[-200:].contiguous(), qb[-200:].contiguous(), sb[-200:].contiguous())
    assert ((out[-200:, -200:].float() - one.float()).abs() <= 2.0 ** -7 * one.float().abs() + 1e-3).all()


def sequences(g, d, lens, typ):
    start = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    return randn(g, sum(lens), d, dtype=typ), start


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_infinities_stay_in_their_sequence(g, bad):
    """One sequence of a packed batch, and one channel of it, is spoilt: the others keep their bits."""
    d, lens = 70, [37, 130, 3, 40]
    x, start = sequences(g, d, lens, BF16)
    w, b, dy = randn(g, d, 4, dtype=BF16), randn(g, d, dtype=BF16), randn(g, sum(lens), d, dtype=BF16)
    dt, B, C = randn(g, sum(lens), d, dtype=BF16), randn(g, sum(lens), 1, 16, dtype=BF16), randn(g, sum(lens), 1, 16, dtype=BF16)
    A, z = -torch.exp(randn(g, d, 16)), randn(g, sum(lens), d, dtype=BF16)

    def run(x, dy):
        y, s = nn.causal_conv(x, w, b, silu=True, seq_start=start, return_state=True)
        c = nn.causal_conv_grad(dy, x, w, b, silu=True, seq_start=start)
        v, t = nn.selective_scan(x, dt, A, B, C, z=z, softplus=True, seq_start=start, return_state=True)
        r = nn.selective_scan_grad(dy, x, dt, A, B, C, z=z, softplus=True, seq_start=start)
        return (y, c["dx"], v, r["du"], r["ddt"], r["dz"], r["dB"].flatten(1), r["dC"].flatten(1)), (s, t)

    ref, ref_states = run(x, dy)
    x2, dy2 = x.clone(), dy.clone()
    x2[166, 5] = dy2[40, 69] = bad  # the second sequence: its last token, and one near its first
    got, states = run(x2, dy2)
    other = torch.ones(sum(lens), dtype=torch.bool, device=DEV)
    other[37:167] = False
    for u, v in zip(ref, got):
        assert torch.equal(u[other], v[other])
    for u, v in zip(ref_states, states):
        assert torch.equal(u[[0, 2, 3]], v[[0, 2, 3]])
    clean = [c for c in range(d) if c not in (5, 69)]
    for u, v in zip(ref[:6], got[:6]):  # channels have nothing to do with one another but in dB and dC
        assert torch.equal(u[:, clean], v[:, clean])


def bits(a, b):
    """The same bits; states that grow past the largest number give NaN on both sides."""
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_expanded_inputs(g):
    """Inputs that repeat one row (stride 0) give what their copies give, bit for bit."""
    d, n = 40, 16
    row = lambda *s: randn(g, *s, dtype=BF16)
    x, dt, z, dy = (row(1, 1, d).expand(2, 53, d) for _ in range(4))
    B, C = (row(1, 1, 1, n).expand(2, 53, 2, n) for _ in range(2))
    A, w = -torch.exp(randn(g, d, n)), randn(g, d, 3, dtype=BF16)
    full = lambda *ts: [t.contiguous() for t in ts]
    assert bits(nn.causal_conv(x, w), nn.causal_conv(x.contiguous(), w))
    a, b = nn.causal_conv_grad(dy, x, w), nn.causal_conv_grad(*full(dy, x), w)
    assert bits(a["dx"], b["dx"]) and bits(a["dw"], b["dw"])
    xc, dtc, Bc, Cc, zc, dyc = full(x, dt, B, C, z, dy)
    assert bits(nn.selective_scan(x, dt, A, B, C, z=z), nn.selective_scan(xc, dtc, A, Bc, Cc, z=zc))
    a, b = nn.selective_scan_grad(dy, x, dt, A, B, C, z=z), nn.selective_scan_grad(dyc, xc, dtc, A, Bc, Cc, z=zc)
    assert all(bits(a[k], b[k]) for k in a if a[k] is not None)


def test_starts_out_of_range_are_clamped(g):
    """Starts past the tokens or below zero lead nowhere: what lies in the sequences that remain is right."""
    d = 24
    x, _ = sequences(g, d, [50], BF16)
    w = randn(g, d, 4, dtype=BF16)
    dt, B, C, A = randn(g, 50, d, dtype=BF16), randn(g, 50, 1, 8, dtype=BF16), randn(g, 50, 1, 8, dtype=BF16), -torch.exp(randn(g, d, 8))
    good = torch.tensor([0, 20, 50, 50], dtype=torch.int32, device=DEV)
    odd = torch.tensor([-9, 20, 50, 2 ** 30], dtype=torch.int32, device=DEV)
    assert torch.equal(nn.causal_conv(x, w, seq_start=odd), nn.causal_conv(x, w, seq_start=good))
    assert torch.equal(nn.selective_scan(x, dt, A, B, C, softplus=True, seq_start=odd),
                       nn.selective_scan(x, dt, A, B, C, softplus=True, seq_start=good))
