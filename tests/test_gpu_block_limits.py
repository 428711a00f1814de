"""Recurrence, norm and 4-bit products past 2^31 elements: offsets that pass 32 bits."""
import pytest
import torch

import convolution_nhwc_implicit_amd as nn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def close(a, b, tol):
    """Two chunkings' results differ by fp32 roundings and the step of a bf16 result that they may move."""
    return bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + tol).all())


@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_rows_far_apart(packed):
    t, d, row = 40000, 24, 65536
    wide = torch.empty(t, row, dtype=BF16, device=DEV)  # 2.6e9 elements
    parts = [wide[:, k * 1000:k * 1000 + d] for k in range(5)]
    for p in parts:
        p.normal_()
    x, r, i, z, dy = parts
    A = torch.full((d,), -0.02, device=DEV)
    start = torch.tensor([0, 100, 39000, t], dtype=torch.int32, device=DEV) if packed else None
    y, f = nn.gated_recurrence(x, r, i, A, z=z, seq_start=start, return_state=True)
    small = [v.contiguous() for v in parts]
    y2, f2 = nn.gated_recurrence(*small[:3], A, z=small[3], seq_start=start, return_state=True)
    assert torch.equal(y, y2) and torch.equal(f, f2)
    g, g2 = (nn.gated_recurrence_grad(v[4], *v[:3], A, z=v[3], seq_start=start) for v in (parts, small))
    assert all(torch.equal(g[k], g2[k]) for k in ("dx", "dr", "di", "dz", "dA"))


def test_recurrence_many_elements():
    t, d = 280000, 8192  # 2.3e9 elements
    x = torch.empty(t, d, dtype=BF16, device=DEV).normal_()
    gate = torch.zeros(1, d, dtype=BF16, device=DEV).expand(t, d)
    A = torch.full((d,), -1.0, device=DEV)
    y = nn.gated_recurrence(x, gate, gate, A)
    # a decay of exp(-1/2) a token: 60 tokens before the last ones are all that matters
    want = nn.gated_recurrence(x[-100:].contiguous(), gate[-100:], gate[-100:], A)
    assert close(y[-20:], want[-20:], 1e-5)
    g = nn.gated_recurrence_grad(x, x, gate, gate, A)
    want = nn.gated_recurrence_grad(x[-100:].contiguous(), x[-100:].contiguous(), gate[-100:], gate[-100:], A)
    assert all(close(g[k][-20:], want[k][-20:], 1e-4) for k in ("dx", "dr", "di"))


def test_norm_many_elements():
    t, d = 530000, 4096  # 2.2e9 elements
    x = torch.empty(t, d, dtype=BF16, device=DEV).normal_()
    y, total = nn.layer_norm(x, residual=x)
    want = nn.layer_norm(x[-50:].contiguous(), residual=x[-50:].contiguous())
    assert torch.equal(y[-50:], want[0]) and torch.equal(total[-50:], want[1])
    del total
    g = nn.layer_norm_grad(y, x, torch.ones(d, device=DEV))
    want = nn.layer_norm_grad(y[-50:].contiguous(), x[-50:].contiguous())
    assert torch.equal(g["dx"][-50:], want["dx"]) and bool(g["dw"].isfinite().all())


def test_norm_long_rows():
    d = (1 << 24) - 1
    x = torch.empty(3, d, device=DEV).normal_()
    y = nn.layer_norm(x)
    # the mean and the deviation of so many values in 64 bits; fp32 sums of 16384 values a lane round by 2^-24 each
    want = (x.double() - x.double().mean(1, keepdim=True)) / (x.double().var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    assert float((y.double() - want).abs().max()) <= 2e-3
    g = nn.layer_norm_grad(x, x, torch.ones(d, device=DEV))
    assert bool(g["dx"].isfinite().all()) and bool(g["dw"].isfinite().all())


def test_fp4_many_weights():
    n, k = 70000, 65536  # 2.3e9 bytes of weights
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV)
    scale = torch.full((n, k // 32), 120, dtype=torch.uint8, device=DEV)
    for m in (2, 20):
        x = torch.randn(m, k, device=DEV).to(BF16)
        out = nn.fp4_matmul(x, q, scale)
        want = nn.fp4_matmul(x, q[-128:].contiguous(), scale[-128:].contiguous())
        # k may be split in other places: 2^-24 of the sums' terms (some hundreds), and a bf16 step
        assert close(out[:, -128:], want, 1e-2)


def test_fp4_many_results():
    m, n, k = 40000, 60000, 64  # 2.4e9 results
    x = torch.randn(m, k, device=DEV).to(BF16)
    q, scale = nn.fp4_quantize(torch.randn(n, k, device=DEV))
    out = nn.fp4_matmul(x, q, scale)
    assert torch.equal(out[-16:], nn.fp4_matmul(x[-16:].contiguous(), q, scale))
    assert torch.equal(out[:16], nn.fp4_matmul(x[:16].contiguous(), q, scale))


def test_fp4_quantize_many_values():
    m, k = 35000, 65536  # 2.3e9 values
    x = torch.empty(m, k, dtype=BF16, device=DEV).normal_()
    q, scale = nn.fp4_quantize(x)
    q2, scale2 = nn.fp4_quantize(x[-64:].contiguous())
    assert torch.equal(q[-64:], q2) and torch.equal(scale[-64:], scale2)
