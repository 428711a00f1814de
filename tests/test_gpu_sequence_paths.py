"""The scan's paths against the 64-bit form: forward passes that cut sequences into chunks and join them (dense and
packed, borders inside sequences, states in and out), every number of waves on long sequences, more than 16 states, and
gradients of batches that are not cut.  Each size first asks the host's plan whether it reaches the path it stands for.

A dense batch becomes one sequence for the reference: its sequences side by side as channels, each with its own groups."""
import pytest
import torch

import convolution_nhwc_implicit_amd as nn
import sequence_plans as plans
import sequence_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
KEYS = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")


def inputs(lens, packed, d, n, groups, typ, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    lead = (sum(lens),) if packed else (len(lens), lens[0])

    def randn(*shape, dtype=F32):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)

    c = dict(x=randn(*lead, d, dtype=typ), dt=(0.5 * randn(*lead, d)).to(typ), A=-torch.exp(0.7 * randn(d, n)),
             B=randn(*lead, groups, n, dtype=typ), C=randn(*lead, groups, n, dtype=typ), D=randn(d),
             z=randn(*lead, d, dtype=typ), dt_bias=randn(d) - 4)  # small steps: states reach over many chunks
    start = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32) if packed else None
    return c, dict(dy=randn(*lead, d, dtype=typ), initial=randn(len(lens), d, n), dfinal=randn(len(lens), d, n)), start


def fold(t):
    """[seqs][len][..][k] -> [len][seqs * ..][k] or, of channels, [len][seqs * d]."""
    t = t.transpose(0, 1).double()
    return t.flatten(1, 2)


def unfold(t, seqs):
    """Of a folded tensor [len][seqs * ..]: [seqs][len][..]."""
    return t.unflatten(1, (seqs, -1)).transpose(0, 1)


def reference(c, lens, packed, initial):
    """The arguments of the 64-bit form, its lengths and first states."""
    if packed:
        return {k: c[k].double() for k in KEYS}, lens, initial.double()
    s = len(lens)
    v = {k: fold(c[k]) for k in ("x", "dt", "B", "C", "z")}
    v.update({k: c[k].double().repeat((s,) + (1,) * (c[k].dim() - 1)) for k in ("A", "D", "dt_bias")})
    return v, [lens[0]], initial.double().flatten(0, 1)[None]


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)  # NaN is bad
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((got.double() - want).abs().max()):.3g}"


FORWARD = [
    # lens, packed, d, n, groups, type; whether it is cut
    ([1024], False, 64, 16, 1, BF16, True),
    ([1024], False, 64, 33, 1, F32, True),
    ([2000, 2000], False, 70, 16, 2, F32, True),
    ([1777], False, 12, 8, 3, F16, True),
    ([400], False, 70, 64, 1, BF16, True),
    ([700, 1, 333], True, 64, 16, 1, F16, True),
    ([1000, 5, 0, 800], True, 67, 16, 1, F32, True),
    ([0, 500, 1, 700, 0], True, 64, 33, 2, BF16, True),
    ([1] * 20 + [1200] + [1] * 11, True, 64, 16, 1, BF16, False),
    ([100] * 600, False, 64, 16, 1, BF16, False),   # one wave a workgroup, several runs of each
    ([150] * 300, False, 64, 16, 2, F16, False),    # two
    ([210] * 150, False, 64, 16, 1, F32, False),    # four
    ([300], False, 64, 16, 1, F32, False),          # eight
    ([90] * 600, False, 64, 32, 1, F32, False),
    ([70] * 600, False, 64, 33, 1, BF16, False),
    ([90] * 300, False, 64, 64, 1, F32, False),
]


@pytest.mark.parametrize("case", FORWARD, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1:]}")
def test_scan(case):
    lens, packed, d, n, groups, typ, cut = case
    assert plans.scan_is_cut(lens, packed, d, n, groups, typ) == cut
    c, more, start = inputs(lens, packed, d, n, groups, typ, 41)
    y, final = nn.selective_scan(*(c[k] for k in ("x", "dt", "A", "B", "C")), D=c["D"], z=c["z"], dt_bias=c["dt_bias"],
                                 softplus=True, initial_state=more["initial"], seq_start=start, return_state=True)
    v, ls, first = reference(c, lens, packed, more["initial"])
    want, fin, mag, worst = R.scan(*(v[k] for k in KEYS), True, ls, first)
    # a state's roundings, the sum over n, the gate; joins of runs and chunks round a state once more each
    extra = R.U * (worst + n + 24 + max(lens) // 4)
    fmag = R.scan(*(v[k].abs() if k in ("x", "B") else v[k] for k in KEYS), True, ls, first.abs())[1]
    if not packed:
        want, mag = unfold(want, len(lens)), unfold(mag, len(lens))
    close(y, want, R.half_step(typ) * want.abs() + extra * mag + (2.0 ** -25 if typ == F16 else 1e-30), "y")
    close(final, fin.view(final.shape), extra * fmag.view(final.shape) + 1e-30, "final state")
    # from a zero state, without the last: the same path of the kernel without what states take
    y = nn.selective_scan(*(c[k] for k in ("x", "dt", "A", "B", "C")), softplus=True, dt_bias=c["dt_bias"], seq_start=start)
    v.update(D=None, z=None)
    want, _, mag, worst = R.scan(*(v[k] for k in KEYS), True, ls, None)
    if not packed:
        want, mag = unfold(want, len(lens)), unfold(mag, len(lens))
    extra = R.U * (worst + n + 24 + max(lens) // 4)
    close(y, want, R.half_step(typ) * want.abs() + extra * mag + (2.0 ** -25 if typ == F16 else 1e-30), "y from zero")


GRAD = [
    ([64] * 512, False, 64, 16, 1, BF16, False),
    ([40] * 512, False, 70, 16, 2, F32, False),
    ([100] * 512, False, 64, 8, 1, F16, False),
    ([64] * 1024, False, 20, 16, 1, F32, False),
    ([5, 0, 3, 8], True, 70, 16, 1, BF16, False),
    ([7, 0, 11] * 100, True, 64, 16, 1, F32, False),
    ([1] * 20 + [1200] + [1] * 11, True, 64, 16, 1, F32, True),
    ([500], False, 40, 33, 1, F32, True),
    ([300, 300], False, 70, 64, 1, BF16, True),
    ([700, 1, 0, 333], True, 64, 32, 2, F16, True),
]


@pytest.mark.parametrize("case", GRAD, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1:]}")
def test_scan_grad(case):
    lens, packed, d, n, groups, typ, cut = case
    assert plans.scan_grad_is_cut(lens, packed, d, n, groups, typ) == cut
    c, more, start = inputs(lens, packed, d, n, groups, typ, 42)
    got = nn.selective_scan_grad(more["dy"], *(c[k] for k in ("x", "dt", "A", "B", "C")), D=c["D"], z=c["z"],
                                 dt_bias=c["dt_bias"], softplus=True, initial_state=more["initial"], seq_start=start,
                                 dfinal_state=more["dfinal"])
    v, ls, first = reference(c, lens, packed, more["initial"])
    seqs = len(lens)
    dy = more["dy"].double() if packed else fold(more["dy"])
    dfinal = more["dfinal"].double() if packed else more["dfinal"].double().flatten(0, 1)[None]
    leaves = {**v, "initial": first}
    for t in leaves.values():
        t.requires_grad_()
    y, fin, _, worst = R.scan(*(v[k] for k in KEYS), True, ls, first)
    want = dict(zip(leaves, torch.autograd.grad((y * dy).sum() + (fin * dfinal).sum(), list(leaves.values()))))
    plain = {k: t.detach() for k, t in leaves.items()}
    mag = R.scan_grad_mag(dy, *(plain[k] for k in KEYS), True, ls, plain["initial"], dfinal)
    for name, key in (("du", "x"), ("ddt", "dt"), ("dA", "A"), ("dB", "B"), ("dC", "C"), ("dD", "D"), ("dz", "z"),
                      ("ddt_bias", "dt_bias"), ("dinitial_state", "initial")):
        w, m = want[key], mag[key]
        if not packed and key in ("A", "D", "dt_bias"):  # of every sequence's copy
            w, m = (t.unflatten(0, (seqs, -1)).sum(0) for t in (w, m))
        elif not packed and key != "initial":
            w, m = unfold(w, seqs), unfold(m, seqs)
        t = got[name].dtype
        # states forwards, carries backwards (as many roundings again, and the chunks' joins), then the sums over n,
        # channels or tokens
        adds = {"A": sum(lens), "D": sum(lens), "dt_bias": sum(lens), "B": d, "C": d}.get(key, n) + 32 + max(lens) // 4
        tol = (R.half_step(t) * w.abs() if t != F32 else 0) + R.U * (2 * worst + adds) * m + 1e-30
        if t == F16:
            tol = tol + 2.0 ** -25
        close(got[name], w.view(got[name].shape), tol.view(got[name].shape), name)
