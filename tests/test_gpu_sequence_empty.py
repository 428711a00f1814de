"""Batches without a token: the outputs are empty, states pass through, and gradients of weights are zero."""
import pytest
import torch

import convolution_nhwc_implicit_amd as nn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def batch(packed, seqs, *inner, dtype):
    lead = (0,) if packed else (seqs, 0)
    start = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV) if packed else None
    return torch.empty(lead + inner, dtype=dtype, device=DEV), start


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("packed,seqs,d,typ", [(False, 1, 40, BF16), (False, 3, 300, F32), (True, 4, 2, F16)])
def test_conv(packed, seqs, d, typ, state):
    x, start = batch(packed, seqs, d, dtype=typ)
    w, b = torch.randn(d, 4, device=DEV).to(typ), torch.randn(d, device=DEV).to(typ)
    s0 = torch.randn(seqs, 3, d, device=DEV).to(typ) if state else None
    ds = torch.randn(seqs, 3, d, device=DEV).to(typ)
    y, s1 = nn.causal_conv(x, w, b, silu=True, initial_state=s0, seq_start=start, return_state=True)
    assert y.shape == x.shape and torch.equal(s1, s0 if state else torch.zeros_like(ds))
    assert nn.causal_conv(x, w, b, silu=True, initial_state=s0, seq_start=start).shape == x.shape
    g = nn.causal_conv_grad(x, x, w, b, silu=True, initial_state=s0, seq_start=start, dfinal_state=ds)
    assert g["dx"].shape == x.shape
    assert torch.equal(g["dw"], torch.zeros_like(w)) and torch.equal(g["db"], torch.zeros_like(b))
    assert torch.equal(g["dinitial_state"], ds) if state else g["dinitial_state"] is None


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("packed,seqs,d,n,typ", [(False, 1, 40, 16, BF16), (False, 3, 70, 33, F32), (True, 4, 2, 3, F16)])
def test_scan(packed, seqs, d, n, typ, state):
    x, start = batch(packed, seqs, d, dtype=typ)
    B, _ = batch(packed, seqs, 1, n, dtype=typ)
    A, D, bias = -torch.rand(d, n, device=DEV), torch.randn(d, device=DEV), torch.randn(d, device=DEV)
    s0 = torch.randn(seqs, d, n, device=DEV) if state else None
    ds = torch.randn(seqs, d, n, device=DEV)
    kw = dict(D=D, z=x, dt_bias=bias, softplus=True, initial_state=s0, seq_start=start)
    y, s1 = nn.selective_scan(x, x, A, B, B, return_state=True, **kw)
    assert y.shape == x.shape and torch.equal(s1, s0 if state else torch.zeros_like(ds))
    assert nn.selective_scan(x, x, A, B, B, **kw).shape == x.shape
    g = nn.selective_scan_grad(x, x, x, A, B, B, dfinal_state=ds, **kw)
    for k, t in (("du", x), ("ddt", x), ("dz", x), ("dB", B), ("dC", B)):
        assert g[k].shape == t.shape
    for k, t in (("dA", A), ("dD", D), ("ddt_bias", bias)):
        assert torch.equal(g[k], torch.zeros_like(t))
    assert torch.equal(g["dinitial_state"], ds) if state else g["dinitial_state"] is None


def test_steps():
    w, pool = torch.randn(8, 4, device=DEV), torch.randn(2, 3, 8, device=DEV)
    before, none = pool.clone(), torch.empty(0, dtype=torch.int32, device=DEV)
    assert nn.causal_conv_step(torch.empty(0, 8, device=DEV), pool, w, slots=none).shape == (0, 8)
    assert torch.equal(pool, before)
    state, x, B = torch.randn(2, 8, 4, device=DEV), torch.empty(0, 8, device=DEV), torch.empty(0, 1, 4, device=DEV)
    before = state.clone()
    assert nn.selective_scan_step(x, x, -torch.rand(8, 4, device=DEV), B, B, state, slots=none).shape == (0, 8)
    assert torch.equal(state, before)
