"""Causal convolution and selective scan against plain 64-bit forms: outputs, states, gradients and single tokens,
over types, widths, odd channel counts, strided inputs, dense and packed sequences (empty and one-token ones among
them), chunk borders, padding slots, other streams and captured graphs."""
import pytest
import torch

import convolution_nhwc_implicit_amd as nn
import sequence_ref as R

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


def close(got, want, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)  # NaN is bad
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((got - want).abs().max()):.3g}"


def cut(lens, packed):
    """(leading shape, seq_start)"""
    if not packed:
        assert len(set(lens)) == 1
        return (len(lens), lens[0]), None
    return (sum(lens),), torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)


# ------------------------------------------------------------------------------ causal convolution
CONV = [
    # lens, packed, d, w, type, silu, bias, state
    ([1], False, 1, 2, F32, False, False, False),
    ([5, 5, 5], False, 8, 4, BF16, True, True, True),
    ([300, 300], False, 515, 4, F16, True, True, False),
    ([0, 1, 2, 3, 0, 131, 7, 0], True, 129, 4, BF16, True, True, True),
    ([0, 1, 2, 3, 0, 131, 7, 0], True, 129, 4, F32, True, True, False),
    ([33, 64, 31], True, 2, 3, F16, False, True, True),
    ([2, 2, 2, 2], False, 2056, 2, F32, True, False, True),
    ([1000], False, 67, 3, BF16, True, True, True),
]


def conv_case(case, seed=1):
    lens, packed, d, w, typ, silu, bias, state = case
    g = gen(seed)
    t = sum(lens)
    c = dict(x=randn(g, t, d, dtype=typ), w=randn(g, d, w, scale=w ** -0.5, dtype=typ),
             bias=randn(g, d, scale=0.3, dtype=typ) if bias else None,
             init=randn(g, len(lens), w - 1, d, dtype=typ) if state else None,
             dy=randn(g, t, d, dtype=typ), dfinal=randn(g, len(lens), w - 1, d, dtype=typ))
    lead, start = cut(lens, packed)
    x = strided(c["x"].view(lead + (d,)), d + 3)
    return c, x, {k: None if c[k] is None else c[k].to(DEV) for k in ("w", "bias", "init")}, lead, start


def f64(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(case):
    lens, packed, d, w, typ, silu, _, state = case
    c, x, p, lead, start = conv_case(case)
    y, final = nn.causal_conv(x, p["w"], p["bias"], silu=silu, initial_state=p["init"], seq_start=start,
                              return_state=True)
    only = nn.causal_conv(x, p["w"], p["bias"], silu=silu, initial_state=p["init"], seq_start=start)
    want, fin, mag = R.conv(f64(c["x"]), f64(c["w"]), f64(c["bias"]), silu, lens, f64(c["init"]))
    # w + 1 sums of products; |d silu| < 1.1; the sigmoid's exp2, its argument and reciprocal: 8 roundings of silu
    tol = R.half_step(typ) * want.abs() + R.U * ((w + 2) * 1.1 * mag + 8 * (1 + mag) * want.abs()) + 1e-30
    if typ == F16:
        tol = tol + 2.0 ** -25
    close(y.view(-1, d), want, tol, "y")
    close(final, fin, 0 * fin, "final state")
    assert torch.equal(y, only)


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_grad(case):
    lens, packed, d, w, typ, silu, _, state = case
    c, x, p, lead, start = conv_case(case, 2)
    dy = strided(c["dy"].view(lead + (d,)), 5)
    dfin = c["dfinal"].to(DEV) if state else None
    got = nn.causal_conv_grad(dy, x, p["w"], p["bias"], silu=silu, initial_state=p["init"], seq_start=start,
                              dfinal_state=dfin)
    leaves = {k: f64(c[k]).requires_grad_() for k in ("x", "w", "bias", "init") if c[k] is not None}
    y, fin, mag = R.conv(leaves["x"], leaves["w"], leaves.get("bias"), silu, lens, leaves.get("init"))
    loss = (y * f64(c["dy"])).sum() + ((fin * f64(c["dfinal"])).sum() if state else 0)
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    # the same with sizes: |g| from below (silu' <= 1.1) with its own roundings, then the sums'
    pre_err = R.U * ((w + 2) * mag + 16 * (1 + mag))  # of pre, through silu' (slope <= 0.5), and of silu' itself
    g = 1.1 * f64(c["dy"]).abs()
    gerr = f64(c["dy"]).abs() * pre_err + 4 * R.U * g
    n = (sum(lens) + 64) * R.U  # a sum of all rows rounds at most so often
    a = {k: v.detach().abs() for k, v in leaves.items()}
    dfa = f64(c["dfinal"]).abs() if state else None

    def spread(gv):  # the linear parts of the gradient of sizes gv
        lv = {k: a[k].clone().requires_grad_() for k in a}
        yy, ff, _ = R.conv(lv["x"], lv["w"], lv.get("bias"), False, lens, lv.get("init"))
        ls = (yy * gv).sum() + ((ff * dfa).sum() if state else 0)
        return dict(zip(lv, torch.autograd.grad(ls, list(lv.values()))))

    m, e = spread(g), spread(gerr)
    dfin_part = spread(0 * g)
    for name, key in (("dx", "x"), ("dw", "w"), ("db", "bias"), ("dinitial_state", "init")):
        if key not in leaves:
            assert got[name] is None
            continue
        many = n if key in ("w", "bias") else 8 * R.U
        tol = R.half_step(typ) * want[key].abs() + (e[key] - dfin_part[key]) + many * m[key] + 1e-30
        if typ == F16:
            tol = tol + 2.0 ** -25
        close(got[name].view(want[key].shape), want[key], tol, name)


@pytest.mark.parametrize("rows,pool,d,w,typ", [(1, 1, 1, 2, F32), (5, 9, 130, 4, BF16), (3, 4, 2731, 3, F16),
                                               (70, 70, 64, 4, F32)])
def test_conv_step(rows, pool, d, w, typ):
    g = gen(3)
    x, wt, b = randn(g, rows, d, dtype=typ), randn(g, d, w, scale=0.5, dtype=typ), randn(g, d, dtype=typ)
    state = randn(g, pool, w - 1, d, dtype=typ)
    slots = torch.randperm(pool, generator=g)[:rows].to(torch.int32)
    if rows > 2:
        slots[1] = -1
        slots[2] = pool
    sd = state.to(DEV)
    y = nn.causal_conv_step(strided(x, 7), sd, wt.to(DEV), b.to(DEV), silu=True, slots=slots.to(DEV))
    expect = state.clone()
    for r in range(rows):
        s = int(slots[r])
        if not 0 <= s < pool:
            assert not y[r].any()
            continue
        want, fin, mag = R.conv(f64(x[r:r + 1]), f64(wt), f64(b), True, [1], f64(state[s:s + 1]))
        tol = R.half_step(typ) * want.abs() + R.U * ((w + 2) * 1.1 * mag + 8 * (1 + mag) * want.abs()) + 2.0 ** -25
        close(y[r:r + 1], want, tol, f"row {r}")
        expect[s] = fin[0].to(typ)
    assert torch.equal(sd.cpu(), expect)


def test_conv_token_by_token_is_the_prompt():
    """A prompt in one call, and the same tokens one by one from its start state: the same bits."""
    g = gen(4)
    x, w, b = randn(g, 2, 9, 40, dtype=BF16).to(DEV), randn(g, 40, 4, dtype=BF16).to(DEV), randn(g, 40, dtype=BF16).to(DEV)
    y, final = nn.causal_conv(x, w, b, silu=True, return_state=True)
    state = torch.zeros(2, 3, 40, dtype=BF16, device=DEV)
    steps = [nn.causal_conv_step(x[:, t], state, w, b, silu=True) for t in range(9)]
    assert torch.equal(torch.stack(steps, 1), y) and torch.equal(state, final)


# ---------------------------------------------------------------------------------- selective scan
SCAN = [
    # lens, packed, d, n, groups, type, softplus, D, z, dt_bias, state
    ([1], False, 1, 1, 1, F32, True, False, False, False, False),
    ([37, 37], False, 70, 16, 1, BF16, True, True, True, True, False),
    ([200], False, 36, 8, 2, F32, True, True, True, True, True),
    ([0, 1, 65, 2, 0, 130, 16, 0], True, 67, 16, 1, F16, True, True, True, True, True),
    ([19, 3, 64], True, 12, 5, 4, BF16, False, False, True, False, False),
    ([70], False, 130, 32, 2, F32, True, True, False, True, True),
    ([33, 33], False, 20, 64, 1, F16, True, True, True, True, True),
    ([21, 21], False, 20, 33, 1, F32, True, True, True, True, True),
    ([260, 130], True, 8, 3, 1, F32, True, True, True, True, True),
]


def scan_case(case, seed=11):
    lens, packed, d, n, groups, typ, soft, hasD, hasz, hasb, state = case
    g = gen(seed)
    t = sum(lens)
    c = dict(x=randn(g, t, d, dtype=typ), dt=randn(g, t, d, scale=0.5, dtype=typ),
             A=-torch.exp(randn(g, d, n, scale=0.7)), B=randn(g, t, groups, n, dtype=typ),
             C=randn(g, t, groups, n, dtype=typ), D=randn(g, d) if hasD else None,
             z=randn(g, t, d, dtype=typ) if hasz else None, dt_bias=randn(g, d) - 2 if hasb else None,
             initial=randn(g, len(lens), d, n) if state else None, dy=randn(g, t, d, dtype=typ),
             dfinal=randn(g, len(lens), d, n))
    if not soft:
        c["dt"] = c["dt"].abs()
    lead, start = cut(lens, packed)
    dev = {"x": strided(c["x"].view(lead + (d,)), 3), "dt": strided(c["dt"].view(lead + (d,)), d)}
    bc = torch.cat([c["B"].flatten(1), c["C"].flatten(1)], 1).view(lead + (2 * groups * n,)).to(DEV)
    dev["B"], dev["C"] = (v.unflatten(-1, (groups, n)) for v in bc.split(groups * n, -1))
    for k in ("A", "D", "dt_bias", "initial"):
        dev[k] = None if c[k] is None else c[k].to(DEV)
    dev["z"] = None if c["z"] is None else strided(c["z"].view(lead + (d,)), 1)
    kw = dict(D=dev["D"], z=dev["z"], dt_bias=dev["dt_bias"], softplus=soft, initial_state=dev["initial"],
              seq_start=start)
    return c, dev, kw, lead


KEYS = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan(case):
    lens, packed, d, n, groups, typ, soft = case[:7]
    c, dev, kw, lead = scan_case(case)
    y, final = nn.selective_scan(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], return_state=True, **kw)
    only = nn.selective_scan(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], **kw)
    want, fin, mag, worst = R.scan(*(f64(c[k]) for k in KEYS), soft, lens, f64(c["initial"]))
    extra = R.U * (worst + n + 24)  # a state's roundings, the sum over n, the gate
    close(y.view(-1, d), want, R.half_step(typ) * want.abs() + extra * mag + (2.0 ** -25 if typ == F16 else 1e-30), "y")
    ref_mag = R.scan(*(f64(c[k]) if k not in ("x", "B") else f64(c[k]).abs() for k in KEYS), soft, lens,
                     None if c["initial"] is None else f64(c["initial"]).abs())[1]
    close(final, fin, extra * ref_mag + 1e-30, "final state")
    assert torch.equal(y, only)


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan_grad(case):
    lens, packed, d, n, groups, typ, soft = case[:7]
    c, dev, kw, lead = scan_case(case, 12)
    dfin = c["dfinal"].to(DEV) if case[-1] else None
    got = nn.selective_scan_grad(strided(c["dy"].view(lead + (d,)), 2), dev["x"], dev["dt"], dev["A"], dev["B"],
                                 dev["C"], dfinal_state=dfin, **kw)
    leaves = {k: f64(c[k]).requires_grad_() for k in KEYS + ("initial",) if c[k] is not None}
    y, fin, _, worst = R.scan(*(leaves.get(k) for k in KEYS), soft, lens, leaves.get("initial"))
    loss = (y * f64(c["dy"])).sum() + ((fin * f64(c["dfinal"])).sum() if case[-1] else 0)
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    mag = R.scan_grad_mag(f64(c["dy"]), *(f64(c[k]) for k in KEYS), soft, lens, f64(c["initial"]),
                          f64(c["dfinal"]) if case[-1] else None)
    for name, key in (("du", "x"), ("ddt", "dt"), ("dA", "A"), ("dB", "B"), ("dC", "C"), ("dD", "D"), ("dz", "z"),
                      ("ddt_bias", "dt_bias"), ("dinitial_state", "initial")):
        if key not in leaves:
            assert got[name] is None
            continue
        t = got[name].dtype
        # states forwards, carries backwards (as many roundings again), then the sums over n, channels or rows
        adds = {"A": sum(lens), "D": sum(lens), "dt_bias": sum(lens), "B": d, "C": d}.get(key, n) + 32
        tol = (R.half_step(t) * want[key].abs() if t != F32 else 0) + R.U * (2 * worst + adds) * mag[key] + 1e-30
        if t == F16:
            tol = tol + 2.0 ** -25
        close(got[name].view(want[key].shape), want[key], tol, name)


def test_scan_grad_against_differences():
    """The gradients' sum along random directions against central differences of the kernel's own forward pass."""
    case = ([40, 25], True, 24, 16, 2, F32, True, True, True, True, True)
    c, dev, kw, lead = scan_case(case, 13)
    dy, dfin = c["dy"].to(DEV), c["dfinal"].to(DEV)
    got = nn.selective_scan_grad(dy, dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dfinal_state=dfin, **kw)
    start = kw["seq_start"]
    base = dict(x=dev["x"], dt=dev["dt"], A=dev["A"], B=dev["B"], C=dev["C"], D=dev["D"], z=dev["z"],
                dt_bias=dev["dt_bias"], initial_state=dev["initial"])

    def loss(v):
        y, f = nn.selective_scan(softplus=True, seq_start=start, return_state=True, **v)
        return (y.double() * dy.double()).sum() + (f.double() * dfin.double()).sum(), (y * dy).abs().sum() + (f * dfin).abs().sum()

    eps = 2.0 ** -8
    for k, gk in (("x", "du"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"),
                  ("dt_bias", "ddt_bias"), ("initial_state", "dinitial_state")):
        step = torch.randn(base[k].shape, generator=gen(14)).to(DEV)
        hi, size = loss({**base, k: base[k] + eps * step})
        lo, _ = loss({**base, k: base[k] - eps * step})
        want = float((hi - lo) / (2 * eps))
        have = float((got[gk].double() * step.double()).sum())
        scale = float((got[gk].double() * step.double()).abs().sum())
        # differences: the third derivative's share (eps^2 of the sum of terms), and the losses' own rounding over eps
        assert abs(want - have) <= 8 * eps ** 2 * scale + 64 * R.U * float(size) / eps, (k, want, have, scale)


@pytest.mark.parametrize("rows,pool,d,n,groups,typ", [(1, 1, 1, 1, 1, F32), (5, 7, 66, 16, 1, BF16),
                                                      (3, 3, 24, 8, 4, F16), (2, 5, 10, 50, 2, F32), (4, 4, 130, 32, 1, BF16)])
def test_scan_step(rows, pool, d, n, groups, typ):
    case = ([rows], False, d, n, groups, typ, True, True, True, True, False)
    c, dev, kw, lead = scan_case(case, 15)
    state = randn(gen(16), pool, d, n)
    slots = torch.randperm(pool, generator=gen(17))[:rows].to(torch.int32)
    if rows > 2:
        slots[0], slots[2] = pool + 3, -5
    sd = state.to(DEV)
    y = nn.selective_scan_step(dev["x"][0], dev["dt"][0], dev["A"], dev["B"][0], dev["C"][0], sd, D=dev["D"],
                               z=dev["z"][0], dt_bias=dev["dt_bias"], softplus=True, slots=slots.to(DEV))
    untouched = torch.ones(pool, dtype=torch.bool)
    for r in range(rows):
        s = int(slots[r])
        if not 0 <= s < pool:
            assert not y[r].any()
            continue
        untouched[s] = False
        one = {k: f64(c[k][r:r + 1]) if k in ("x", "dt", "B", "C", "z") else f64(c[k]) for k in KEYS}
        want, fin, mag, worst = R.scan(*(one[k] for k in KEYS), True, [1], f64(state[s:s + 1]))
        fmag = R.scan(*(one[k].abs() if k in ("x", "B") else one[k] for k in KEYS), True, [1], f64(state[s:s + 1]).abs())[1]
        extra = R.U * (worst + n + 24)
        close(y[r:r + 1], want, R.half_step(typ) * want.abs() + extra * mag + 2.0 ** -25, f"row {r}")
        close(sd[s:s + 1], fin, extra * fmag, f"state {s}")
    assert torch.equal(sd.cpu()[untouched], state[untouched])


def test_scan_in_pieces_is_the_whole():
    """A prompt in one call, and in pieces through the state: within the bound of both."""
    case = ([90], False, 40, 16, 1, F32, True, True, True, True, False)
    c, dev, kw, lead = scan_case(case, 18)
    kw.pop("initial_state")
    a = [dev[k] for k in ("x", "dt", "B", "C")]
    want, fin, mag, worst = R.scan(*(f64(c[k]) for k in KEYS), True, [90])
    ys, state = [], None
    for lo, hi in ((0, 1), (1, 33), (33, 90)):
        x, dt, B, C = (v[:, lo:hi] for v in a)
        y, state = nn.selective_scan(x, dt, dev["A"], B, C, initial_state=state, return_state=True,
                                     **{**kw, "z": dev["z"][:, lo:hi]})
        ys.append(y)
    close(torch.cat(ys, 1)[0], want, R.U * (worst + 40) * mag, "y")


# --------------------------------------------------------------------------- streams, graphs, repeats
def all_passes(seed=21):
    """Every operator once, as a function of nothing that returns its outputs."""
    conv = conv_case(([0, 1, 40, 7], True, 35, 4, BF16, True, True, True), seed)
    scan = scan_case(([0, 1, 165, 7], True, 35, 16, 1, BF16, True, True, True, True, True), seed)
    c, x, p, lead, start = conv
    cdy = c["dy"].to(DEV)
    sc, sdev, kw, _ = scan
    sdy = sc["dy"].to(DEV)
    sa = [sdev[k] for k in ("x", "dt", "A", "B", "C")]

    def run():
        out = list(nn.causal_conv(x, p["w"], p["bias"], silu=True, initial_state=p["init"], seq_start=start,
                                  return_state=True))
        g = nn.causal_conv_grad(cdy, x, p["w"], p["bias"], silu=True, initial_state=p["init"], seq_start=start)
        out += [g[k] for k in sorted(g)]
        out += list(nn.selective_scan(*sa, return_state=True, **kw))
        g = nn.selective_scan_grad(sdy, *sa, **kw)
        return out + [g[k] for k in sorted(g)]
    return run


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_repeats_and_other_stream_give_the_same_bits():
    run = all_passes()
    ref = run()
    assert same(ref, run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert same(ref, got)


def test_graph_replays():
    run = all_passes()
    ref = run()
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
        assert same(ref, eager) and same(ref, out), f"replay {rep}"
