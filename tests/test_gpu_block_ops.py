"""Gated recurrence, layer norm and 4-bit products against plain 64-bit forms: outputs, states, gradients and single
tokens, over types, odd widths, strided inputs, dense and packed sequences (empty and one-token ones among them), chunk
borders, padding slots, spoilt neighbours, other streams and captured graphs."""
import pytest
import torch

import block_ref as R
import convolution_nhwc_implicit_amd as nn

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, scale=1.0, dtype=F32):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def strided(t, extra):
    """t on the GPU as a slice of a wider tensor."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), float("nan"), dtype=t.dtype, device=DEV)
    wide[..., :t.shape[-1]] = t.to(DEV)
    return wide[..., :t.shape[-1]]


def close(got, want, err, typ, what):
    got, want = got.detach().double().cpu(), want.detach()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    tol = err + R.half_step(typ) * (want.abs() + err) + torch.finfo(typ).smallest_normal * torch.finfo(typ).eps
    bad = ~((got - want).abs() <= tol)  # NaN is bad
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() / tol).max()):.3g} of its bound"


def cut(lens, packed):
    """(leading shape, seq_start)"""
    if not packed:
        assert len(set(lens)) == 1
        return (len(lens), lens[0]), None
    return (sum(lens),), torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)


def f64(t):
    return None if t is None else t.double()


# ---------------------------------------------------------------------------------- gated recurrence
RECUR = [
    # lens, packed, d, type, gate, biases, states
    ([1], False, 1, F32, False, False, False),
    ([5, 5, 5], False, 8, BF16, True, True, True),
    ([300, 300], False, 131, F16, True, True, False),
    ([128, 128, 128], False, 70, F32, True, False, True),
    ([0, 1, 2, 3, 0, 131, 7, 0], True, 129, BF16, True, True, True),
    ([0, 1, 2, 3, 0, 131, 7, 0], True, 129, F32, True, True, False),
    ([33, 64, 31], True, 2, F16, False, True, True),
    ([1] * 70 + [0] * 9 + [2] * 40, True, 65, BF16, True, True, True),
    ([0] * 600 + [1, 0] * 300 + [5], True, 3, F32, True, False, True),
    ([1000], False, 67, BF16, True, True, True),
    ([1500], False, 64, F32, False, False, True),
    ([700, 900], True, 64, F16, True, True, True),
    ([0, 0], True, 5, F32, True, True, True),
    ([4, 0, 3], True, 1, BF16, True, True, True),
    (list(range(64)), True, 258, BF16, True, True, True),
    (list(range(65)), True, 100, F32, True, False, True),
    ([3, 7000, 2, 1500, 1], True, 7, F32, True, True, True),
    ([1, 0, 2, 1] * 1024, True, 40, BF16, True, True, True),
    ([0, 1, 1] * 1370, True, 5, F32, True, True, True),
    ([2500], False, 300, F16, True, True, True),
    ([16] * 300, False, 300, BF16, True, True, True),
    ([5] * 300, False, 40, F32, True, True, True),
    ([64] * 70, False, 256, F16, True, True, False),
]


def recur_case(case, seed=1):
    lens, packed, d, typ, gate, biases, states = case
    g = gen(seed)
    t, n = sum(lens), len(lens)
    c = dict(x=randn(g, t, d, dtype=typ), r=randn(g, t, d, scale=2.0, dtype=typ), i=randn(g, t, d, scale=2.0, dtype=typ),
             A=2 * torch.log(0.8 + 0.1999 * torch.rand(d, generator=g)), z=randn(g, t, d, dtype=typ) if gate else None,
             rb=randn(g, d, scale=0.5) if biases else None, ib=randn(g, d, scale=0.5) if biases else None,
             init=randn(g, n, d) if states else None, dy=randn(g, t, d, dtype=typ), dfinal=randn(g, n, d) if states else None)
    lead, start = cut(lens, packed)
    dev = {k: None if v is None else strided(v.view(lead + (d,)), e) if k in ("x", "r", "i", "z", "dy") else v.to(DEV)
           for (k, v), e in zip(c.items(), (d, 3, 1, 0, 2, 0, 0, 0, 5, 0))}
    return c, dev, lead, start


def recur_call(p, start, state=False):
    return nn.gated_recurrence(p["x"], p["r"], p["i"], p["A"], z=p["z"], r_bias=p["rb"], i_bias=p["ib"],
                               initial_state=p["init"], seq_start=start, return_state=state)


def recur_grads(p, start):
    return nn.gated_recurrence_grad(p["dy"], p["x"], p["r"], p["i"], p["A"], z=p["z"], r_bias=p["rb"], i_bias=p["ib"],
                                    initial_state=p["init"], seq_start=start, dfinal_state=p["dfinal"])


def recur_ref(c, lens, grad=False):
    v = {k: f64(t) for k, t in c.items()}
    if grad:
        for k in ("x", "r", "i", "A", "z", "rb", "ib", "init"):
            if v[k] is not None:
                v[k].requires_grad_()
    return v, R.recurrence(v["x"], v["r"], v["i"], v["A"], v["z"], v["rb"], v["ib"], lens, v["init"])


@pytest.mark.parametrize("case", RECUR, ids=str)
def test_recurrence(case):
    lens, packed, d, typ, _, _, states = case
    c, p, lead, start = recur_case(case)
    y, final = recur_call(p, start, state=True)
    _, (wy, wf, ey, ef) = recur_ref(c, lens)
    assert y.dtype == typ and y.shape == lead + (d,) and final.dtype == F32
    close(y.flatten(0, -2), wy, ey, typ, "y")
    close(final, wf, ef, F32, "final state")
    assert torch.equal(recur_call(p, start), y)


@pytest.mark.parametrize("case", RECUR, ids=str)
def test_recurrence_grad(case):
    lens, packed, d, typ, gate, biases, states = case
    c, p, lead, start = recur_case(case)
    got = recur_grads(p, start)
    v, (wy, wf, _, _) = recur_ref(c, lens, grad=True)
    out = (wy * v["dy"]).sum() + (0 if v["dfinal"] is None else (wf * v["dfinal"]).sum())
    names = dict(x="dx", r="dr", i="di", A="dA", z="dz", rb="dr_bias", ib="di_bias", init="dinitial_state")
    have = [k for k in names if v[k] is not None]
    want = torch.autograd.grad(out, [v[k] for k in have], allow_unused=True)
    with torch.no_grad():
        bound = R.recurrence_grad_bounds(v["dy"], *(v[k] for k in ("x", "r", "i", "A", "z", "rb", "ib")), lens, v["init"], v["dfinal"])
    for k, w in zip(have, want):
        w = torch.zeros_like(v[k]) if w is None else w
        n = names[k]
        typ_ = typ if n in ("dx", "dr", "di", "dz") else F32
        assert got[n].dtype == typ_
        close(got[n].reshape(w.shape), w, bound[n], typ_, n)
    assert all(got[names[k]] is None for k in names if v[k] is None)


def test_recurrence_gradient_against_differences():
    case = ([40, 1, 90], True, 33, F32, True, True, True)
    c, p, lead, start = recur_case(case, seed=3)
    got = recur_grads(p, start)
    g = gen(4)
    names = dict(x="dx", r="dr", i="di", A="dA", z="dz", rb="dr_bias", ib="di_bias", init="dinitial_state")
    v = {k: f64(t) for k, t in c.items()}

    def loss(step, name, way):
        w = dict(v)
        w[name] = v[name] + step * way
        y, f, _, _ = R.recurrence(w["x"], w["r"], w["i"], w["A"], w["z"], w["rb"], w["ib"], case[0], w["init"])
        return float((y * v["dy"]).sum() + (f * v["dfinal"]).sum())

    for name, grad in names.items():
        way = randn(g, *v[name].shape).double() * (1e-3 if name == "A" else 1.0)
        h = 1e-5
        slope = (loss(h, name, way) - loss(-h, name, way)) / (2 * h)
        mine = float((got[grad].double().cpu() * way).sum())
        # central differences are off by h^2 times a third derivative (1e-10 times some tens) and 1e-16 / h of the
        # loss's terms; the gradient by fp32 roundings of its terms
        size = float((got[grad].double().cpu() * way).abs().sum())
        assert abs(slope - mine) <= 1e-4 * size + 1e-6, (name, slope, mine)


@pytest.mark.parametrize("rows,pool,d,typ,gate", [(1, 1, 1, F32, True), (4, 9, 130, BF16, True), (7, 7, 4097, F16, False),
                                                  (300, 400, 256, BF16, True), (33, 40, 6, F32, True)], ids=str)
def test_recurrence_step(rows, pool, d, typ, gate):
    g = gen(5)
    c, _, _, _ = recur_case(([1] * rows, True, d, typ, gate, True, True), seed=6)
    state = randn(g, pool, d)
    slots = torch.randperm(pool, generator=g)[:rows].to(torch.int32)
    if rows > 3:
        slots[1], slots[2] = -1, pool  # padding
    real = (slots >= 0) & (slots < pool)
    c["init"] = torch.where(real[:, None], state[slots.long().clamp(0, pool - 1)], 0)
    _, (wy, wf, ey, ef) = recur_ref(c, [1] * rows)
    held = state.to(DEV)
    kw = {k: None if c[v] is None else c[v].to(DEV) for k, v in (("r_bias", "rb"), ("i_bias", "ib"))}
    y = nn.gated_recurrence_step(strided(c["x"], 1), strided(c["r"], d), strided(c["i"], 2), c["A"].to(DEV), held,
                                 z=strided(c["z"], 3) if gate else None, slots=slots.to(DEV), **kw)
    assert not y.cpu()[~real].any()
    close(y[real.to(DEV)], wy[real], ey[real], typ, "y")
    want, err = state.double(), torch.zeros(pool, d, dtype=torch.float64)
    want[slots[real].long()], err[slots[real].long()] = wf[real], ef[real]
    close(held, want, err, F32, "states")
    if rows <= pool and not (~real).any():
        again = state.to(DEV)
        y2 = nn.gated_recurrence_step(c["x"].to(DEV), c["r"].to(DEV), c["i"].to(DEV), c["A"].to(DEV), again[slots.long().to(DEV)].contiguous(),
                                      z=c["z"].to(DEV) if gate else None, **kw)
        assert torch.equal(y2, y)


def test_recurrence_step_goes_on_from_a_prompt():
    case = ([50], False, 200, BF16, True, True, False)
    c, p, _, _ = recur_case(case)
    whole = recur_call(p, None)
    head = {k: v[:, :47] if k in ("x", "r", "i", "z") else v for k, v in p.items()}
    y, state = recur_call(head, None, state=True)
    assert torch.equal(y, whole[:, :47])
    for t in range(47, 50):
        y = nn.gated_recurrence_step(*(p[k][:, t] for k in ("x", "r", "i")), p["A"], state, z=p["z"][:, t], r_bias=p["rb"], i_bias=p["ib"])
        # the same operations, in a run's order or one by one: a rounding or two of the state, then one of the result
        assert ((y - whole[:, t]).abs() <= 2.0 ** -7 * whole[:, t].abs()).all()


@pytest.mark.parametrize("typ", [F16, BF16, F32], ids=str)
def test_recurrence_extreme_gates(typ):
    """Gates that are shut, open and infinite, and rates from none to infinite."""
    inf = float("inf")
    r = torch.tensor([-inf, -100.0, 0.0, 100.0, inf])
    A = torch.tensor([0.0, -1e-30, -1e-6, -1.0, -100.0, -3e38, -inf])
    t, d = 5 * 5, len(A)
    c = dict(x=randn(gen(7), t, d, dtype=typ), r=r.repeat(5)[:, None].expand(t, d).to(typ),
             i=r.repeat_interleave(5)[:, None].expand(t, d).to(typ), A=A)
    got, state = nn.gated_recurrence(*(c[k].to(DEV) for k in ("x", "r", "i", "A")), return_state=True)
    h = torch.zeros(d, dtype=torch.float64)
    ref = torch.clamp(A, min=-2e38).double()
    for k in range(t):
        g = torch.sigmoid(c["r"][k].double())
        g[g < 2.0 ** -126] = 0  # sigmoid(-100) = 3.7e-44 is below fp32's normal numbers: 0, also times a rate of 2e38
        L = ref * g
        h = torch.exp(L) * h + torch.sqrt(-torch.expm1(2 * L)) * torch.sigmoid(c["i"][k].double()) * c["x"][k].double()
        # 1e-6 of what came in: 16 roundings of each term
        err = 1e-5 * h.abs() + 1e-6
        close(got[k], h, err, typ, f"token {k}")
    g = nn.gated_recurrence_grad(torch.ones_like(got), *(c[k].to(DEV) for k in ("x", "r", "i", "A")))
    assert all(bool(g[k].isfinite().all()) for k in ("dx", "dr", "di"))
    assert float(g["dA"][0]) == 0.0


@pytest.mark.parametrize("spoil", ["x", "r", "init", "dy"])
def test_recurrence_spoilt_sequences_stay_alone(spoil):
    lens = [3, 130, 40, 9, 300]
    case = (lens, True, 66, F32, True, True, True)
    c, p, _, start = recur_case(case)
    y, f = recur_call(p, start, state=True)
    g = recur_grads(p, start)
    p2 = {k: None if v is None else v.clone() for k, v in p.items()}
    a, b = 133, 173  # the third sequence
    for bad in (float("nan"), float("inf")):
        if spoil == "init":
            p2["init"][2] = bad
        else:
            p2[spoil][a:b] = bad
        y2, f2 = recur_call(p2, start, state=True)
        g2 = recur_grads(p2, start)
        rest = torch.cat([torch.arange(a), torch.arange(b, sum(lens))]).to(DEV)
        assert torch.equal(y2[rest], y[rest]) and torch.equal(f2[[0, 1, 3, 4]], f[[0, 1, 3, 4]])
        for k in ("dx", "dr", "di", "dz"):
            assert torch.equal(g2[k][rest], g[k][rest]), k
        assert torch.equal(g2["dinitial_state"][[0, 1, 3, 4]], g["dinitial_state"][[0, 1, 3, 4]])


def test_recurrence_rows_behind_the_last_sequence():
    """A padded packed batch: rows that no sequence covers are not looked at."""
    lens, pad = [70, 0, 200, 33], 90
    case = (lens, True, 40, BF16, True, True, True)
    c, p, _, start = recur_case(case)
    y, f = recur_call(p, start, state=True)
    g = recur_grads(p, start)
    t = sum(lens)
    wide = {k: torch.cat([v, torch.full((pad, 40), float("nan"), dtype=BF16, device=DEV)]) if k in ("x", "r", "i", "z", "dy") else v
            for k, v in p.items()}
    y2, f2 = recur_call(wide, start, state=True)
    g2 = recur_grads(wide, start)
    same = {**{k: g[k] for k in ("dA", "dr_bias", "di_bias", "dinitial_state")}, **{k: g[k] for k in ("dx", "dr", "di", "dz")}}
    close(y2[:t], y.double().cpu(), 0.0, BF16, "y")
    assert torch.allclose(f2, f, rtol=1e-5, atol=1e-6)
    for k, v in same.items():
        got = g2[k][:t] if k in ("dx", "dr", "di", "dz") else g2[k]
        assert bool(got.isfinite().all()) and torch.allclose(got.float(), v.float(), rtol=2.0 ** -6 if got.dtype == BF16 else 1e-3, atol=1e-3), k


def same_but_for_chunks(a, b):
    """Results of two chunkings: states differ by fp32 roundings, which move a result to its neighbour at most; cancelling
    sums keep 1e-5 of values of size 1."""
    return bool(((a.double() - b.double()).abs() <= torch.finfo(a.dtype).eps * b.double().abs() + 1e-5).all())


def test_recurrence_batch_strides():
    """Sequences of a dense batch that lie apart (walked one by one), and one row for all tokens."""
    g = gen(8)
    d = 96
    x, r, i, z = (randn(g, 3, 50, d, dtype=BF16).to(DEV) for _ in range(4))
    A = torch.full((d,), -0.3, device=DEV)
    want = nn.gated_recurrence(x[:, 7:45].contiguous(), r[:, 7:45].contiguous(), i[:, :38].contiguous(), A, z=z[:, 7:45].contiguous())
    got = nn.gated_recurrence(x[:, 7:45], r[:, 7:45], i[:, :38], A, z=z[:, 7:45])
    assert same_but_for_chunks(got, want)
    one = r[:1, :1].expand(3, 38, d)
    args = (x[:, 7:45], one, i[:, :38], A)
    assert same_but_for_chunks(nn.gated_recurrence(*args), nn.gated_recurrence(args[0].contiguous(), one.contiguous(), args[2].contiguous(), A))
    dy = z[:, 12:]
    a, b = (nn.gated_recurrence_grad(*v) for v in ((dy, *args), tuple(t.contiguous() for t in (dy, *args))))
    assert all(same_but_for_chunks(a[k], b[k]) for k in ("dx", "dr", "di"))
    # 114 terms of size 1, each with some tens of roundings
    assert float((a["dA"] - b["dA"]).abs().max()) <= 114 * 64 * R.U


def test_recurrence_long_sequences_that_lie_apart():
    """A dense batch with gaps, long enough to be cut: against its sequences one by one."""
    g = gen(9)
    d = 70
    x, r, i, z, dy = (randn(g, 2, 1500, d, dtype=F32).to(DEV)[:, 100:1400] for _ in range(5))
    A, h0, df = torch.full((d,), -0.05, device=DEV), randn(g, 2, d).to(DEV), randn(g, 2, d).to(DEV)
    y, f = nn.gated_recurrence(x, r, i, A, z=z, initial_state=h0, return_state=True)
    k = nn.gated_recurrence_grad(dy, x, r, i, A, z=z, initial_state=h0, dfinal_state=df)
    for s in range(2):
        y1, f1 = nn.gated_recurrence(x[s], r[s], i[s], A, z=z[s], initial_state=h0[s:s + 1], return_state=True)
        k1 = nn.gated_recurrence_grad(dy[s], x[s], r[s], i[s], A, z=z[s], initial_state=h0[s:s + 1], dfinal_state=df[s:s + 1])
        assert same_but_for_chunks(y[s], y1) and same_but_for_chunks(f[s], f1[0])
        assert same_but_for_chunks(k["dinitial_state"][s], k1["dinitial_state"][0])
        # gradients of gates add terms of some tens
        assert all(float((k[n][s] - k1[n]).abs().max()) <= 1e-4 for n in ("dx", "dr", "di", "dz"))


def test_recurrence_least_rates():
    """Rates whose inverses pass float32's range: below 2^-126 they count as 0."""
    A = -torch.tensor([1e-45, 1e-40, 1.1754942e-38, 1.1754944e-38, 3e-38, 1e-36])
    g = gen(15)
    c = [randn(g, 300, 6).to(DEV) for _ in range(4)]
    dA = A.to(DEV)
    y = nn.gated_recurrence(*c[:3], dA, z=c[3])
    k = nn.gated_recurrence_grad(c[0], *c[:3], dA, z=c[3])
    assert bool(y.isfinite().all()) and all(bool(k[n].isfinite().all()) for n in ("dx", "dr", "di", "dz", "dA"))
    assert not y[:, :3].any() and not any(k[n][:, :3].any() for n in ("dx", "dr", "di", "dz")) and not k["dA"][:3].any()
    h, lost = torch.zeros(3, dtype=torch.float64), torch.zeros(3, dtype=torch.float64)
    x, r, i, z = (v[:, 3:].double().cpu() for v in c)
    for t in range(300):
        L = A[3:].double() * torch.sigmoid(r[t])
        b = torch.sqrt(-torch.expm1(2 * L)) * torch.sigmoid(i[t]) * x[t]
        h = torch.exp(L) * h + b
        # log2 e L may count as 0 below 2^-126: a root of at most (2 ln 2)^0.5 2^-63; else 64 roundings of a term and
        # one of the sum so far, at most 300 of them
        lost += 2.0 ** -62 * x[t].abs() + (64 + 300) * R.U * b.abs()
        silu = z[t] * torch.sigmoid(z[t])
        assert bool(((y[t, 3:].double().cpu() - h * silu).abs() <= lost * silu.abs() + 64 * R.U * (h * silu).abs()).all())


def test_recurrence_starts_out_of_order():
    """Starts that descend or lie outside give unspecified results, and nothing else."""
    case = ([40, 50, 60, 70], True, 66, BF16, True, True, True)
    c, p, _, start = recur_case(case)
    y, k = recur_call(p, start), recur_grads(p, start)
    for bad in ([0, 90, 40, 150, 220], [220, 150, 90, 40, 0], [-7, 40, 1 << 30, 150, 220], [5, 5, 5, 5, 5], [-(1 << 31), 0, 0, 0, (1 << 31) - 1]):
        t = torch.tensor(bad, dtype=torch.int32, device=DEV)
        recur_call(p, t, state=True)
        recur_grads(p, t)
        torch.cuda.synchronize()
    assert torch.equal(recur_call(p, start), y)
    again = recur_grads(p, start)
    assert all(torch.equal(again[n], k[n]) for n in k)


# ------------------------------------------------------------------------------------------ layer norm
NORM = [
    # rows, d, type, float32 parameters, weight, bias, residual
    (1, 1, F32, True, True, True, False), (5, 3, BF16, False, True, True, True), (9, 7, F16, True, True, False, False),
    (33, 8, BF16, False, True, True, True), (130, 100, F32, True, False, True, True), (4, 128, F16, False, True, True, False),
    (70, 515, BF16, True, True, True, True), (3, 768, F32, True, True, True, True), (17, 1024, F16, False, False, False, True),
    (9, 2731, F16, False, True, True, True), (40, 4096, BF16, False, True, True, True), (6, 5000, F32, True, True, True, True),
    (3, 8191, BF16, True, True, True, True), (5, 16384, F16, False, True, True, False), (2, 16387, F32, True, True, True, True),
    (2000, 200, F16, False, True, True, True), (300, 129, BF16, True, True, True, False), (70, 12000, BF16, True, True, True, True),
    (9, 130, F32, True, True, True, True), (5, 256, BF16, False, True, True, True),
    (3, 33001, BF16, False, True, True, True), (1200, 264, BF16, True, True, True, True),
]


def norm_case(case, seed=11):
    rows, d, typ, f32, weight, bias, residual = case
    g = gen(seed)
    pt = F32 if f32 else typ
    return dict(x=(randn(g, rows, d) * torch.exp(randn(g, d, scale=0.5)) + randn(g, d, scale=0.5)).to(typ),
                w=(1 + randn(g, d, scale=0.2)).to(pt) if weight else None, b=randn(g, d, scale=0.2, dtype=pt) if bias else None,
                res=randn(g, rows, d, dtype=typ) if residual else None, dy=randn(g, rows, d, dtype=typ),
                dt=randn(g, rows, d, dtype=typ) if residual else None)


def dev(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm(case):
    rows, d, typ, f32, _, _, residual = case
    c = norm_case(case)
    got = nn.layer_norm(strided(c["x"], 5), dev(c["w"]), dev(c["b"]), eps=1e-5, residual=strided(c["res"], 1) if residual else None)
    t = c["x"].double() + (c["res"].double() if residual else 0)
    y, err = R.norm(t, f64(c["w"]), f64(c["b"]), 1e-5)
    if residual:
        close(got[1], t, R.U * t.abs(), typ, "total")
        got = got[0]
    assert got.dtype == typ
    close(got, y, err, typ, "y")


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_grad(case):
    rows, d, typ, f32, weight, bias, residual = case
    c = norm_case(case)
    got = nn.layer_norm_grad(strided(c["dy"], 2), strided(c["x"], 5), dev(c["w"]), dev(c["b"]), eps=1e-5,
                             dtotal=strided(c["dt"], 3) if residual else None)
    v = {k: f64(t) for k, t in c.items()}
    t = v["x"].requires_grad_()
    w = torch.ones(d, dtype=torch.float64) if v["w"] is None else v["w"]
    b = torch.zeros(d, dtype=torch.float64) if v["b"] is None else v["b"]
    w.requires_grad_()
    b.requires_grad_()
    y, _ = R.norm(t, w, b, 1e-5)
    dx, dw, db = torch.autograd.grad((y * v["dy"]).sum() + (0 if v["dt"] is None else (t * v["dt"]).sum()), (t, w, b))
    with torch.no_grad():
        bound = R.norm_grad_bounds(v["dy"], t.detach(), f64(c["w"]), 1e-5, v["dt"])
    close(got["dx"], dx, bound["dx"], typ, "dx")
    pt = F32 if f32 else typ
    assert (got["dw"] is None) == (not weight) and (got["db"] is None) == (not bias)
    if weight:
        assert got["dw"].dtype == pt
        close(got["dw"], dw, bound["dw"], pt, "dw")
    if bias:
        close(got["db"], db, bound["db"], pt, "db")


def test_norm_gradient_against_differences():
    c = norm_case((12, 50, F32, True, True, True, False))
    got = nn.layer_norm_grad(dev(c["dy"]), dev(c["x"]), dev(c["w"]), dev(c["b"]))
    g = gen(12)
    v = {k: f64(t) for k, t in c.items()}
    for name, grad in (("x", "dx"), ("w", "dw"), ("b", "db")):
        way = randn(g, *v[name].shape).double()

        def loss(h):
            w = dict(v)
            w[name] = v[name] + h * way
            return float((R.norm(w["x"], w["w"], w["b"], 1e-5)[0] * v["dy"]).sum())

        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        terms = got[grad].double().cpu() * way
        # h^2 times a third derivative, and fp32 roundings of the gradient's terms
        assert abs(slope - float(terms.sum())) <= 1e-4 * float(terms.abs().sum()) + 1e-6, name


def test_norm_keeps_small_deviations_around_a_large_mean():
    """Deviations of 2^-10 around 1000: squares minus the mean's square would lose them."""
    g = gen(13)
    x = (1000 + randn(g, 8, 4096).sign() * 2.0 ** -10)
    got = nn.layer_norm(x.to(DEV), eps=0.0)
    y, err = R.norm(x.double(), None, None, 0.0)
    # the mean's error, 96 U 1000 at most in the bound, is about the deviations' size; sums of 64 neighbours and 6 levels
    # of equal numbers round by U 1000 each level: 70 roundings of half a step in random directions, 8 of them in norm
    assert float((got.double().cpu() - y).abs().max()) <= 0.25


def test_norm_rows_apart():
    g = gen(14)
    x, res = (randn(g, 4, 30, 264, dtype=BF16).to(DEV) for _ in range(2))
    w = randn(g, 264, dtype=BF16).to(DEV)
    a = nn.layer_norm(x[:, 3:20], w, residual=res[1:2, :17].expand(4, 17, 264))
    b = nn.layer_norm(x[:, 3:20].contiguous(), w, residual=res[1:2, :17].expand(4, 17, 264).contiguous())
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = nn.layer_norm_grad(x[:, 3:20], res[:, 10:27], w, dtotal=x[:, :17])
    b = nn.layer_norm_grad(x[:, 3:20].contiguous(), res[:, 10:27].contiguous(), w, dtotal=x[:, :17].contiguous())
    assert all(torch.equal(a[k], b[k]) for k in ("dx", "dw"))


@pytest.mark.parametrize("typ", [F16, BF16, F32], ids=str)
def test_norm_constant_and_spoilt_rows(typ):
    x = randn(gen(15), 40, 520, dtype=typ)
    x[3] = 2.5
    b = torch.arange(520).to(typ) / 64
    want = nn.layer_norm(x.to(DEV), bias=b.to(DEV))
    assert torch.equal(want[3].cpu(), b)  # no deviation: the bias
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[7, 100] = bad
        got = nn.layer_norm(y.to(DEV), bias=b.to(DEV))
        rest = [k for k in range(40) if k != 7]
        assert torch.equal(got[rest], want[rest]) and bool(got[7].isnan().any())


def test_norm_without_rows():
    x = torch.zeros(0, 64, dtype=BF16, device=DEV)
    w = torch.ones(64, device=DEV)
    y, total = nn.layer_norm(x, w, w, residual=x)
    assert y.shape == (0, 64) and total.shape == (0, 64)
    g = nn.layer_norm_grad(x, x, w, w)
    assert not g["dw"].any() and not g["db"].any() and g["dx"].shape == (0, 64)


# -------------------------------------------------------------------------------------- 4-bit products
@pytest.mark.parametrize("m,k,typ", [(1, 1, F32), (3, 31, BF16), (5, 32, F16), (7, 33, F32), (64, 200, BF16), (9, 4104, F16)], ids=str)
def test_fp4_quantize(m, k, typ):
    x = randn(gen(21), m, k, dtype=typ)
    if m > 4:
        x[2] = 0
        x[3, :k // 2] = 6 * 2.0 ** -9
        x[4] *= 2.0 ** -12
    q, scale = nn.fp4_quantize(strided(x, 3))
    assert q.shape == (m, (k + 1) // 2) and q.dtype == torch.uint8 and scale.shape == (m, -(-k // 32))
    value, want = R.fp4_quantize(x)
    assert torch.equal(scale.cpu(), want)
    assert torch.equal(R.fp4_values(q.cpu(), scale.cpu(), k), value)
    if k % 2:
        assert not (q[:, -1] >> 4).any()


def test_fp4_quantize_borders_and_extremes():
    """Every border between neighbouring values, its neighbours, the largest and least numbers, and spoilt groups."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = torch.cat([edges, torch.nextafter(edges, torch.tensor(0.0)), torch.nextafter(edges, torch.tensor(9.0)), -edges])
    x = torch.zeros(6, 32)
    x[0, :28], x[0, 28] = near, 6.0
    x[1, :28], x[1, 28] = near * 2.0 ** -100, 6.0 * 2.0 ** -100
    x[2] = torch.finfo(F32).max
    x[2, 3] = 1.0
    x[3, :4] = torch.tensor([1.0, 2.0, 3.0, 7.0]) * 2.0 ** -149
    x[4] = torch.linspace(-1, 1, 32)
    x[5] = torch.linspace(-1, 1, 32)
    x[4, 9], x[5, 8] = float("nan"), float("-inf")
    q, scale = nn.fp4_quantize(x.to(DEV))
    q, scale = q.cpu(), scale.cpu()
    value, want = R.fp4_quantize(x[:4])
    assert torch.equal(scale[:4], want) and scale[4:].eq(255).all()
    assert torch.equal(R.fp4_values(q[:4], scale[:4], 32), value)


def fp4_weights(g, n, k):
    q, scale = nn.fp4_quantize(randn(g, n, k, scale=k ** -0.5).to(DEV))
    return q, scale, R.fp4_values(q.cpu(), scale.cpu(), k)


FP4 = [(4, 300, 30000, BF16), (16, 70, 7000, F16), (6, 8200, 8200, BF16), (20, 130, 4096, BF16), (64, 300, 2050, F16), (40, 129, 1024, F16), (17, 128, 8200, BF16), (100, 257, 700, F16), (33, 1, 600, BF16), (1, 1, 1, F32), (1, 16, 32, BF16), (1, 300, 4096, BF16), (2, 17, 33, F16), (16, 100, 1000, BF16), (17, 64, 160, F32),
       (33, 257, 4104, F16), (48, 40, 777, BF16), (64, 130, 2048, F32), (65, 31, 511, BF16), (150, 96, 95, F16), (5, 1000, 31, F32)]


@pytest.mark.parametrize("m,n,k,typ", FP4, ids=str)
def test_fp4_matmul(m, n, k, typ):
    g = gen(22)
    x = (randn(g, m, k) * torch.exp(randn(g, 1, k))).to(typ)
    q, scale, w = fp4_weights(g, n, k)
    got = nn.fp4_matmul(strided(x, 1), q, scale)
    assert got.dtype == typ and got.shape == (m, n)
    want, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    # in a row: 32 products of an instruction, the instructions of a wave (an eighth of them), three parts of x, the waves
    close(got, want, (3 * k / 256 + 64) * R.U * mag, typ, "out")


@pytest.mark.parametrize("typ", [F16, BF16, F32], ids=str)
def test_fp4_matmul_keeps_every_bit_of_x(typ):
    """One product each: values with all their bits set, large and small, come back as they are."""
    fi = torch.finfo(typ)
    one = torch.tensor(2.0, dtype=typ) - torch.tensor(fi.eps, dtype=typ)
    x = torch.zeros(16, 64, dtype=typ)
    for k in range(16):
        x[k, 3 * k] = one * 2.0 ** (k - 8) * (-1) ** k
    q, scale = nn.fp4_quantize(torch.eye(64, device=DEV))
    assert torch.equal(nn.fp4_matmul(x.to(DEV), q, scale).cpu(), x)


def test_fp4_matmul_scales():
    """Every scale byte, the least ones (2^-127 and up) and NaN among them."""
    n = 256
    q = torch.full((n, 16), 0x22, dtype=torch.uint8, device=DEV)  # ones
    scale = torch.arange(n, device=DEV).to(torch.uint8)[:, None]
    x = torch.zeros(2, 32, device=DEV)
    x[0, 5], x[1, 30] = 1.0, 2.0 ** -20
    got = nn.fp4_matmul(x, q, scale).double().cpu()
    want = torch.exp2(torch.arange(n).double() - 127)
    assert torch.equal(got[0, :255], want[:255]) and bool(got[:, 255].isnan().all())
    normal = want[:255] * 2.0 ** -20 >= 2.0 ** -126
    assert torch.equal(got[1, :255][normal], (want[:255] * 2.0 ** -20)[normal])


@pytest.mark.parametrize("m", [2, 40])
@pytest.mark.parametrize("typ", [F16, BF16], ids=str)
def test_fp4_matmul_scales_in_16_bits(typ, m):
    """Every scale byte next to every other (256 rows of two groups): fp16 weights hold only some of them."""
    g = gen(24)
    n, k = 256, 64
    q = torch.randint(0, 256, (n, 32), generator=g).to(torch.uint8)
    scale = torch.stack([torch.arange(n), torch.arange(n).roll(1)], 1).to(torch.uint8)
    x = randn(g, m, k, dtype=typ)
    x[1] *= 2.0 ** -14  # fp16's subnormal numbers among them
    got = nn.fp4_matmul(x.to(DEV), q.to(DEV), scale.to(DEV)).double().cpu()
    w = R.fp4_values(q, scale, k)
    want, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    top = torch.finfo(typ).max
    # a sum's roundings, below fp32's normal numbers half its least step each; the result's half step, or its least
    tol = 70 * R.U * mag + R.half_step(typ) * want.abs() + torch.finfo(typ).smallest_normal * torch.finfo(typ).eps + 70 * 2.0 ** -150
    ok = ((got - want).abs() <= tol) | (want.isnan() & got.isnan()) | ((want.abs() >= top * 0.99) & (got.abs() >= top * 0.99))
    # past fp32's range: between the terms of a sum, or the weights themselves (6 * 2^126 is 2^128.6)
    assert (ok | (mag >= 2.0 ** 127) | (w.abs().amax(1) >= 2.0 ** 128)).all()


@pytest.mark.parametrize("typ", [F16, BF16, F32], ids=str)
def test_fp4_matmul_spoilt_rows_and_padding(typ):
    g = gen(23)
    x = randn(g, 20, 100, dtype=typ)
    q, scale, w = fp4_weights(g, 50, 100)
    want = nn.fp4_matmul(x.to(DEV), q, scale)
    y = x.clone()
    y[4, 7], y[9, 99] = float("nan"), float("inf")
    got = nn.fp4_matmul(y.to(DEV), q, scale)
    rest = [k for k in range(20) if k not in (4, 9)]
    assert torch.equal(got[rest], want[rest]) and bool(got[4].isnan().all())
    hit = w[:, 99] != 0
    assert torch.equal(got[9].cpu()[hit], (torch.sign(w[:, 99]) * float("inf")).to(typ)[hit]) and bool(got[9].cpu()[~hit].isnan().all())
    # halves of bytes behind the last value have no influence
    big = torch.full((50, 64), 0x77, dtype=torch.uint8, device=DEV)
    big[:, :50] = q
    assert torch.equal(nn.fp4_matmul(x.to(DEV), big[:, :50], scale), want)
    # x behind its last value neither
    assert torch.equal(nn.fp4_matmul(strided(x, 40), q, scale), want)


def test_fp4_matmul_of_nothing():
    q, scale = nn.fp4_quantize(torch.zeros(5, 0, device=DEV))
    out = nn.fp4_matmul(torch.zeros(3, 0, device=DEV), q, scale)
    assert out.shape == (3, 5) and not out.any()
    q, scale = nn.fp4_quantize(torch.zeros(0, 40, device=DEV))
    assert nn.fp4_matmul(torch.zeros(3, 40, device=DEV), q, scale).shape == (3, 0)
    q, scale = nn.fp4_quantize(torch.zeros(4, 40, device=DEV))
    assert nn.fp4_matmul(torch.zeros(0, 40, device=DEV), q, scale).shape == (0, 4)


# ------------------------------------------------------------------------------- streams and captured graphs
def together(p, start, nrm, q, scale, state):
    y = recur_call(p, start)
    n, total = nn.layer_norm(y, *nrm, residual=p["x"])
    g = nn.layer_norm_grad(p["dy"], total, *nrm, dtotal=y)
    r = recur_grads({**p, "dy": g["dx"]}, start)
    out = nn.fp4_matmul(n[:5], q, scale)
    s = nn.gated_recurrence_step(p["x"][:5], p["r"][:5], p["i"][:5], p["A"], state, z=p["z"][:5])
    return [y, n, total, *(v for v in g.values() if v is not None), *(v for v in r.values() if v is not None), out, s, state]


@pytest.mark.parametrize("graph", [False, True])
def test_streams_and_graphs(graph):
    d = 256
    case = ([300, 1, 0, 90], True, d, BF16, True, True, True)
    c, p, _, start = recur_case(case)
    g = gen(31)
    nrm = (1 + randn(g, d, scale=0.1, dtype=BF16)).to(DEV), randn(g, d, dtype=BF16).to(DEV)
    q, scale, _ = fp4_weights(g, 100, d)
    begin = randn(g, 5, d).to(DEV)
    want = [v.clone() for v in together(p, start, nrm, q, scale, begin.clone())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    state = begin.clone()
    torch.cuda.synchronize()
    if not graph:
        with torch.cuda.stream(side):
            got = together(p, start, nrm, q, scale, state)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        return
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        got = together(p, start, nrm, q, scale, state)
    for _ in range(3):
        state.copy_(begin)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        together(p, start, nrm, q, scale, begin.clone())  # eager work between
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Calls that run side by side share nothing."""
    cases = [([3000], False, 64, BF16, True, True, True), ([900, 0, 1300], True, 200, BF16, True, True, True)]
    args = []
    for case in cases:
        c, p, _, start = recur_case(case)
        d = case[2]
        g = gen(33)
        nrm = (1 + randn(g, d, scale=0.1, dtype=BF16)).to(DEV), randn(g, d, dtype=BF16).to(DEV)
        flat = {k: v.reshape(-1, d) if k in ("x", "r", "i", "z", "dy") else v for k, v in p.items()}
        args.append((flat, start if start is not None else torch.tensor([0, 3000], dtype=torch.int32, device=DEV), nrm,
                     *fp4_weights(g, 300, d)[:2], randn(g, 5, d).to(DEV)))
    run = lambda a: together(*a[:-1], a[-1].clone())
    want = [run(a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = []
    for _ in range(10):
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                got.append(run(a))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[k % 2]))


def test_fp4_one_row_for_all():
    """x with one row for all, and in a matrix with a row to spare."""
    g = gen(35)
    q, scale, _ = fp4_weights(g, 70, 200)
    x = randn(g, 1, 200, dtype=F16).to(DEV)
    want = nn.fp4_matmul(x, q, scale)
    for m in (3, 40, 70):
        got = nn.fp4_matmul(x.expand(m, 200), q, scale)
        assert torch.equal(got, got[:1].expand(m, 70))
        # sums of another order: both within 200 roundings of the sum of sizes
        size = x.float().abs().max() * 200 * 6 * 2.0 ** (int(scale.max()) - 127)
        assert bool(((got[0].double() - want[0].double()).abs() <= torch.finfo(F16).eps * want[0].double().abs() + 2.0 ** -24 + 400 * R.U * float(size)).all())
