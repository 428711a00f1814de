"""Every path of the fp8 products against the 64-bit product: tiles of both sizes over many blocks (even and odd counts
of them, k that ends inside 16 bytes), rows left to the narrow kernel, k split, float32 results, and scales that take a
tile to its second path.  Each size first asks the host's plan whether it reaches the path that it stands for."""
import pytest
import torch

import convolution_nhwc_implicit_amd as nn
import sequence_plans as plans

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24

# m, n, k, type of the result, rows of b to a scale; the plan: tile, splits, odd count of blocks, rows of a and of b left
PATHS = [
    (1557, 5031, 512, BF16, 128, 256, 1, False, False, False),
    (2705, 3109, 643, BF16, 128, 256, 1, False, False, False),
    (1726, 4680, 528, F16, 1, 256, 1, True, False, False),
    (3250, 2448, 514, BF16, 1, 256, 1, True, False, False),
    (3529, 4629, 757, BF16, 128, 256, 1, False, False, True),
    (3894, 4270, 526, F16, 1, 256, 1, True, True, False),
    (3867, 4415, 642, BF16, 128, 256, 1, False, True, True),
    (836, 4773, 7917, BF16, 128, 256, 3, True, False, False),
    (4679, 835, 7639, F16, 1, 256, 3, False, False, False),
    (577, 2519, 512, BF16, 128, 128, 1, False, False, False),
    (327, 3505, 643, F16, 1, 128, 1, False, False, False),
    (204, 5014, 529, BF16, 128, 128, 1, True, False, False),
    (1284, 2976, 1159, BF16, 1, 128, 1, False, False, True),
    (4105, 921, 1034, F16, 128, 128, 1, True, True, False),
    (3901, 2186, 1691, BF16, 128, 128, 1, False, True, True),
    (69, 70, 5151, F16, 1, 128, 11, False, False, False),
    (1053, 130, 7284, BF16, 128, 128, 12, True, False, False),
    (132, 4808, 688, F32, 128, 128, 1, False, False, False),
    (133, 4460, 529, F32, 1, 128, 1, True, False, False),
    (1672, 2308, 651, F32, 128, 128, 1, False, False, True),
    (4647, 779, 645, F32, 1, 128, 1, False, True, False),
    (3335, 2453, 947, F32, 1, 128, 1, False, True, True),
    (71, 68, 2067, F32, 128, 128, 5, False, False, False),
    (129, 2314, 3098, F32, 1, 128, 5, True, False, False),
    (300, 40, 1111, BF16, 1, 0, 1, True, False, True),
    (90, 700, 300, F16, 128, 0, 1, True, True, False),
]


def spread(s, rows, m, k):
    return s.double().repeat_interleave(rows, 0)[:m].repeat_interleave(128, 1)[:, :k]


def operand(g, rows, k, pad):
    """e4m3 values in rows with NaN past their ends."""
    q = (torch.randn(rows, k, generator=g, device=DEV) * 40).clamp(-448, 448).to(E4M3)
    buf = torch.full((rows, -(-k // 16) * 16 + pad), 0x7f, dtype=torch.uint8, device=DEV)
    buf[:, :k] = q.view(torch.uint8)
    return q.double(), buf.view(E4M3)[:, :k]


def scales(g, rows, kb, low):
    return torch.exp2(torch.randint(low, low + 11, (rows, kb), generator=g, device=DEV).float())


@pytest.mark.parametrize("m,n,k,typ,rows,tile,splits,odd,left_m,left_n", PATHS)
def test_path(m, n, k, typ, rows, tile, splits, odd, left_m, left_n):
    got_tile, got_splits, per, nm, nn_ = plans.product(m, n, k, typ)
    assert (got_tile, got_splits, per % 2 == 1, nm, nn_) == (tile, splits, odd, left_m, left_n)
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    kb = -(-k // 128)
    (aq, a), (bq, b) = operand(g, m, k, 0), operand(g, n, k, 16)
    sa, sb = scales(g, m, kb, -18 if typ == F16 else -8), scales(g, -(-n // rows), kb, -8)
    sums = {}
    for which in ("powers", "one", "any"):
        if which == "one":  # one row's scale in one block: only its tiles leave the first path
            sa, sb = sa.clone(), sb.clone()
            sa[m // 3, kb // 2] *= 1.25
            sb[-1, kb - 1] *= -1.5
        if which == "any":
            sa, sb = (s * (1 + torch.rand(s.shape, generator=g, device=DEV)) for s in (sa, sb))
        got = sums[which] = nn.fp8_matmul(a, sa, b, sb, out_dtype=typ)
        av, bv = aq * spread(sa, 1, m, k), bq * spread(sb, rows, n, k)
        want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
        # fp32 sums of 128 exact products (at most 128 roundings or cuts of 2^-23), of the blocks and the splits, and
        # three roundings a block more where scales are no powers of two
        tol = U * (256 + 4 * kb + splits) * mag
        if typ != F32:
            # the fp8 unit cuts each of 8 neighbouring products at 2^-13 of the largest: 7 such cuts in 8 terms
            top = [torch.nn.functional.pad(v.abs(), (0, -k % 8)).unflatten(1, (-1, 8)).amax(-1) for v in (av, bv)]
            tol = tol + torch.finfo(typ).eps / 2 * want.abs() + 7 * 2.0 ** -13 * (top[0] @ top[1].t())
        if typ == F16:
            tol = tol + 2.0 ** -25
        err = (got.double() - want).abs()
        assert (err <= tol).all(), f"{which}: {int((~(err <= tol)).sum())} off, worst {float((err / mag).max() / U):.1f} units of the terms"
        assert torch.equal(got, nn.fp8_matmul(a, sa, b, sb, out_dtype=typ))


@pytest.mark.parametrize("m,n,k,typ", [(1726, 4680, 528, BF16), (327, 3505, 643, BF16), (133, 4460, 529, F32), (1053, 130, 7284, BF16)])
def test_nan_stays_in_its_row(m, n, k, typ):
    """A NaN in one row of each operand, and an infinite scale in another of a: the other results keep their bits."""
    g = torch.Generator(device=DEV).manual_seed(5)
    kb = -(-k // 128)
    (_, a), (_, b) = operand(g, m, k, 0), operand(g, n, k, 0)
    sa, sb = scales(g, m, kb, -8), scales(g, n, kb, -8)
    want = nn.fp8_matmul(a, sa, b, sb, out_dtype=typ)
    a.view(torch.uint8)[m - 1, k - 1] = 0x7f
    b.view(torch.uint8)[0, 130] = 0xff
    got = nn.fp8_matmul(a, sa, b, sb, out_dtype=typ)
    assert got[m - 1].isnan().all() and got[:, 0].isnan().all() and torch.equal(got[:m - 1, 1:], want[:m - 1, 1:])
    sa[1, kb - 1] = float("inf")
    got = nn.fp8_matmul(a, sa, b, sb, out_dtype=typ)
    assert not got[1].isfinite().any() and got[m - 1].isnan().all() and got[:, 0].isnan().all()
    rest = torch.ones(m, dtype=torch.bool, device=DEV)
    rest[[1, m - 1]] = False
    # tiles with the infinite scale take the second path: its sums may round otherwise
    near = got[rest][:, 1:].double() - want[rest][:, 1:].double()
    assert near.isfinite().all()


def test_zero_blocks():
    """Rows and blocks of zeros, which the quantisation gives its least scale: zeros out, the rest as without them."""
    for m, n, k, typ in ((1726, 4680, 528, BF16), (327, 3505, 643, BF16), (132, 4808, 688, F32)):
        g = torch.Generator(device=DEV).manual_seed(6)
        x, w = torch.randn(m, k, generator=g, device=DEV), torch.randn(n, k, generator=g, device=DEV)
        x[m // 2:m // 2 + 3], x[:, 128:256], w[:, 256:384] = 0, 0, 0
        (qa, sa), (qb, sb) = nn.fp8_quantize(x), nn.fp8_quantize(w)
        got = nn.fp8_matmul(qa, sa, qb, sb, out_dtype=typ)
        av, bv = qa.double() * spread(sa, 1, m, k), qb.double() * spread(sb, 1, n, k)
        want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
        tol = U * (256 + 4 * 6) * mag
        if typ != F32:
            top = [torch.nn.functional.pad(v.abs(), (0, -k % 8)).unflatten(1, (-1, 8)).amax(-1) for v in (av, bv)]
            tol = tol + torch.finfo(typ).eps / 2 * want.abs() + 7 * 2.0 ** -13 * (top[0] @ top[1].t())
        assert ((got.double() - want).abs() <= tol).all() and not got[m // 2:m // 2 + 3].any()
