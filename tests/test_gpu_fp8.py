"""Block-scaled fp8 products against plain 64-bit forms: quantisation value for value, products over types, ragged
sizes, row and block scales, scales that are no powers of two, and operands with rubbish past their rows' ends."""
import pytest
import torch

import convolution_nhwc_implicit_amd as nn

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def e4m3(v):
    """v (64 bits, |v| <= 448) to the nearest e4m3 value, ties to even."""
    unit = torch.exp2((torch.frexp(v)[1].double() - 1).clamp_min(-6) - 3)
    return torch.round(v / unit) * unit


def scales_of(x, rows):
    """The least power of two s >= 2^-126 with 448 s >= every finite |value| of a block of `rows` x 128."""
    m, k = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -k % 128, 0, -m % rows))
    v = torch.where(torch.isfinite(v), v.abs(), 0).view(-(-m // rows), rows, -(-k // 128), 128).amax((1, 3))
    s = torch.full_like(v, 2.0 ** -126)
    e = torch.ceil(torch.log2((v / 448).clamp_min(2.0 ** -126)))
    s = torch.maximum(s, torch.exp2(e))
    s = torch.where(448 * s < v, 2 * s, s)  # the logarithm may have rounded
    return torch.where((s / 2 >= 2.0 ** -126) & (448 * (s / 2) >= v), s / 2, s)


def spread(s, rows, m, k):
    return s.double().repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :k]


QUANT = [(1, 1), (3, 127), (5, 128), (130, 300), (129, 1025), (257, 16)]


@pytest.mark.parametrize("typ", [F16, BF16, F32])
@pytest.mark.parametrize("form", ["rows", "transpose", "blocks"])
@pytest.mark.parametrize("m,k", QUANT)
def test_quantize(m, k, form, typ):
    g = gen(m * 1000 + k)
    x = (torch.randn(m, k, generator=g) * torch.exp(2 * torch.randn(m, 1, generator=g))).to(typ)
    x[0, : k // 2] = 0
    x.view(-1)[-1] = 448.0  # the border: scale 1 where nothing is larger
    wide = torch.full((m, k + 3), float("nan"), dtype=typ, device=DEV)
    wide[:, :k] = x.to(DEV)
    q, s = nn.fp8_quantize(wide[:, :k], transpose=form == "transpose", blocks=form == "blocks")
    v = x.t() if form == "transpose" else x
    rows = 128 if form == "blocks" else 1
    want_s = scales_of(v, rows)
    assert torch.equal(s.double().cpu(), want_s)
    want = e4m3(v.double() / spread(want_s, rows, *v.shape))
    assert torch.equal(q.cpu().double(), want)
    assert q.stride(0) % 16 == 0 or q.shape[0] == 1
    if q.stride(0) > q.shape[1]:  # padding is zero
        whole = q.as_strided((q.shape[0], q.stride(0)), (q.stride(0), 1))
        assert not whole[:, q.shape[1]:].view(torch.uint8).any()


@pytest.mark.parametrize("form", ["rows", "transpose", "blocks"])
def test_quantize_borders(form):
    """Values at the format's borders, infinities and NaN: they stay in their places and out of the scale."""
    x = torch.randn(128, 256, generator=gen(5))
    x[3, 7], x[40, 9], x[41, 200] = float("inf"), float("nan"), -float("inf")
    x[:, 130] = 0
    x[64] = 2.0 ** -133  # below the least scale's steps
    x[65] = 3e38
    q, s = nn.fp8_quantize(x.to(DEV), transpose=form == "transpose", blocks=form == "blocks")
    v = x.t() if form == "transpose" else x
    rows = 128 if form == "blocks" else 1
    want_s = scales_of(v, rows)
    assert torch.equal(s.double().cpu(), want_s)
    got, fin = q.cpu().double(), torch.isfinite(v)
    want = e4m3(torch.where(fin, v.double(), 0) / spread(want_s, rows, *v.shape))
    assert torch.equal(got[fin], want[fin]) and got[~fin].isnan().all()


def operand(g, rows, k, block_rows, pow2, pad, rubbish):
    """Random e4m3 values with scales on the CPU, and the same on the GPU with `rubbish` past each row."""
    q = (torch.randn(rows, k, generator=g) * 40).clamp(-448, 448).to(E4M3)
    kb = -(-k // 128)
    s = torch.exp2(torch.randint(-8, 3, (-(-rows // block_rows), kb), generator=g).float())
    if not pow2:
        s = s * (1 + torch.rand(s.shape, generator=g))
    pitch = -(-k // 16) * 16 + pad
    buf = torch.full((rows, pitch), rubbish, dtype=torch.uint8, device=DEV)
    buf[:, :k] = q.view(torch.uint8).to(DEV)
    return q.double() * spread(s, block_rows, rows, k), buf.view(E4M3)[:, :k], s.to(DEV)


# m, n, k: single rows, odd and ragged sizes, k below, at and past one block, n and m past tiles
MATMUL = [(1, 1, 1), (1, 200, 4096), (3, 129, 127), (8, 640, 300), (16, 512, 1024), (17, 130, 128), (33, 1000, 515),
          (64, 384, 2048), (65, 257, 640), (130, 260, 129), (300, 515, 1111), (513, 1030, 264), (1030, 700, 96)]


@pytest.mark.parametrize("m,n,k", MATMUL)
@pytest.mark.parametrize("typ,block_rows,pow2", [(BF16, 128, True), (F32, 1, True), (F16, 128, False), (F32, 128, False),
                                                 (F32, 1, False)])
def test_matmul(m, n, k, typ, block_rows, pow2):
    g = gen(m * 7 + n * 3 + k)
    av, a, sa = operand(g, m, k, 1, pow2, 0, 0x7f)   # NaN past the rows' ends
    bv, b, sb = operand(g, n, k, block_rows, pow2, 16, 0x7f)
    scale = 2.0 ** -6 if typ == F16 else 1.0  # keeps fp16 results in range
    sa = sa * scale
    av = av * scale
    got = nn.fp8_matmul(a, sa, b, sb, out_dtype=typ)
    want = av @ bv.t()
    mag = av.abs() @ bv.abs().t()
    # fp32 sums: of 128 exact products inside the matrix unit (at most 128 roundings or cuts of 2^-23), of the
    # blocks, and with scales that are no powers of two three roundings more a block
    kb = -(-k // 128)
    tol = (torch.finfo(typ).eps / 2 * want.abs() if typ != F32 else 0) + U * (256 + 4 * kb) * mag
    if typ != F32:
        # 16-bit results come from the fp8 unit, which cuts each of 8 neighbouring products at 2^-13 of the power of
        # two of the largest: 7 such cuts for every 8 terms, none larger than 2^-13 of the largest term
        group = [torch.nn.functional.pad(v.abs(), (0, -k % 8)).unflatten(1, (-1, 8)).amax(-1) for v in (av, bv)]
        tol = tol + 7 * 2.0 ** -13 * (group[0] @ group[1].t())
    if typ == F16:
        tol = tol + 2.0 ** -25
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), f"worst {float((err / mag.clamp_min(1e-300)).max() / U):.1f} units of the terms"


def test_matmul_special_scales():
    """Scales beyond the powers of two that the matrix unit takes: zero, subnormal, negative, and one of them alone
    among powers of two; infinities and NaN in operands and scales reach the rows and columns that hold them only."""
    g = gen(77)
    m, n, k = 150, 140, 400
    av, a, sa = operand(g, m, k, 1, True, 0, 0)
    bv, b, sb = operand(g, n, k, 1, True, 0, 0)
    ref = av @ bv.t()

    def check(sa2, sb2, rows=None):
        got = nn.fp8_matmul(a, sa2, b, sb2, out_dtype=F32).double().cpu()
        x = a.double().cpu() * spread(sa2.cpu(), 1, m, k)
        y = b.double().cpu() * spread(sb2.cpu(), 1, n, k)
        want, mag = x @ y.t(), x.abs() @ y.abs().t()
        assert ((got - want).abs() <= U * 300 * mag + 2.0 ** -140).all()

    for v in (0.0, 2.0 ** -130, -2.0, 3.0):
        sa2, sb2 = sa.clone(), sb.clone()
        sa2[17, 1] = v
        check(sa2, sb)
        sb2[130, 2] = v
        check(sa, sb2)
    sa2 = sa.clone()
    sa2[5, 0], sa2[140, 3] = float("inf"), float("nan")
    got = nn.fp8_matmul(a, sa2, b, sb, out_dtype=F32).double().cpu()
    assert not torch.isfinite(got[5]).any() and got[140].isnan().all()
    rest = [r for r in range(m) if r not in (5, 140)]
    assert ((got - ref)[rest].abs() <= U * 300 * (av.abs() @ bv.abs().t())[rest]).all()


def test_matmul_empty():
    for m, n, k in ((0, 5, 16), (5, 0, 16), (4, 3, 0)):
        a = torch.zeros(m, k, dtype=E4M3, device=DEV)
        b = torch.zeros(n, k, dtype=E4M3, device=DEV)
        kb = -(-k // 128)
        got = nn.fp8_matmul(a, torch.ones(m, kb, device=DEV), b, torch.ones(n, kb, device=DEV), out_dtype=F32)
        assert got.shape == (m, n) and not got.any()


def test_linear_and_its_gradients():
    """A projection from 16-bit activations, and both its gradients: against the products of
    the values that the quantised operands stand for."""
    g = gen(9)
    m, n, k = 70, 200, 333
    x, w, dy = torch.randn(m, k, generator=g), torch.randn(n, k, generator=g), torch.randn(m, n, generator=g) * 1e-3
    x, w, dy = (v.to(BF16).to(DEV) for v in (x, w, dy))

    def held(q, s, rows=1):
        return q.double().cpu() * spread(s.cpu(), rows, *q.shape)

    qx, sx = nn.fp8_quantize(x)
    qw, sw = nn.fp8_quantize(w, blocks=True)
    qd, sd = nn.fp8_quantize(dy)
    qwt, swt = nn.fp8_quantize(w.t().contiguous(), blocks=True)
    assert torch.equal(swt, sw.t()) and torch.equal(held(qwt, swt, 128), held(qw, sw, 128).t())
    qdt, sdt = nn.fp8_quantize(dy, transpose=True)
    qxt, sxt = nn.fp8_quantize(x, transpose=True)
    for got, p, q in ((nn.fp8_matmul(qx, sx, qw, sw, out_dtype=F32), held(qx, sx), held(qw, sw, 128)),
                      (nn.fp8_matmul(qd, sd, qwt, swt, out_dtype=F32), held(qd, sd), held(qwt, swt, 128)),
                      (nn.fp8_matmul(qdt, sdt, qxt, sxt, out_dtype=F32), held(qdt, sdt), held(qxt, sxt))):
        assert ((got.double().cpu() - p @ q.t()).abs() <= U * 300 * (p.abs() @ q.abs().t())).all()


def test_streams_repeats_and_graph():
    g = gen(10)
    x, w = torch.randn(200, 600, generator=g).to(BF16).to(DEV), torch.randn(260, 600, generator=g).to(BF16).to(DEV)
    few = x[:5]

    def run():
        qw, sw = nn.fp8_quantize(w, blocks=True)
        out = [nn.fp8_matmul(*nn.fp8_quantize(v), qw, sw) for v in (x, few)]
        out.append(nn.fp8_matmul(*nn.fp8_quantize(w, transpose=True), *nn.fp8_quantize(w, transpose=True), out_dtype=F32))
        return out

    ref = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(u, v) for u, v in zip(ref, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for rep in range(4):
        for t in out:
            t.fill_(float("nan"))
        eager = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) and torch.equal(u, e) for u, v, e in zip(ref, out, eager)), f"replay {rep}"
