"""Plain 64-bit forms (CPU) of a recurrent block's operators: gated recurrence, layer norm and 4-bit products, with the
bounds that their fp32 kernels are held to.

Bounds.  An output of type t is rounded once: half a step, eps(t)/2 relative.  Before that each fp32 operation rounds by
at most U = 2^-24 of its result (the exponential, reciprocal and root instructions by a step, 2 U); a count of such
roundings times U times the size of the terms bounds an error."""
import torch

U = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def sequences(lens):
    at = 0
    for n in lens:
        yield at, at + n
        at += n


# ---------------------------------------------------------------------------------- gated recurrence
def gates(x, r, i, A, rb, ib):
    g, u = torch.sigmoid(r + rb), torch.sigmoid(i + ib)
    L = A * g
    return g, u, L, torch.exp(L), torch.sqrt(-torch.expm1(2 * L))


def recurrence(x, r, i, A, z, rb, ib, lens, initial=None):
    """x, r, i, z [T][d] in 64 bits -> y, final states, and bounds of the errors of y (before its rounding) and of the
    final states.

    A sigmoid's exponent is off by |v| U and its operations by 4 steps: (8 + 4 |v|) U relative.  So is L, and a by that
    times |L| and 8 U.  1 - a^2 loses 16 U a^2 U at the border of its series, relative 32 U, and the root halves; with
    the other gate and three products (32 + 4 |r| + 4 |i|) U."""
    d = A.shape[0]
    rb, ib = (x.new_zeros(d) if v is None else v for v in (rb, ib))
    g, u, L, a, s = gates(x, r, i, A, rb, ib)
    b = s * u * x
    ad, bd, Ld = a.detach(), b.detach().abs(), L.detach().abs()
    vr, vi = (r + rb).detach().abs(), (i + ib).detach().abs()
    ea, eb = 10 + Ld * (8 + 4 * vr), 32 + 4 * vr + 4 * vi
    hs, errs, finals, final_errs = [], [], [], []
    for q, (p, e) in enumerate(sequences(lens)):
        h = x.new_zeros(d) if initial is None else initial[q]
        hm, err = h.detach().abs(), torch.zeros(d, dtype=x.dtype)
        for t in range(p, e):
            h = a[t] * h + b[t]
            err = ad[t] * err + U * (ea[t] * ad[t] * hm + eb[t] * bd[t])
            hm = ad[t] * hm + bd[t]
            hs.append(h)
            errs.append(err)
        finals.append(h)
        final_errs.append(err)
    h = torch.stack(hs) if hs else x.new_zeros(0, d)
    err = torch.stack(errs) if errs else h
    y, ey = h, err
    if z is not None:
        gate = z * torch.sigmoid(z)
        y = h * gate
        gd, zd = gate.detach().abs(), z.detach().abs()
        ey = err * gd + U * (8 + 4 * zd) * y.detach().abs()
    return y, torch.stack(finals), ey, torch.stack(final_errs)


def recurrence_grad_bounds(dy, x, r, i, A, z, rb, ib, lens, initial=None, dfinal=None):
    """Bounds of the errors of the gradients before their rounding: the formulas with every term's size, times the
    roundings that the states (and likewise their gradients) carry at most and those of a term itself."""
    d = A.shape[0]
    rb, ib = (x.new_zeros(d) if v is None else v for v in (rb, ib))
    g, u, L, a, s = gates(x, r, i, A, rb, ib)
    b = (s * u * x).abs()
    vr, vi = (r + rb).abs(), (i + ib).abs()
    ea, eb = 10 + L.abs() * (8 + 4 * vr), 32 + 4 * vr + 4 * vi
    gate = torch.ones_like(x) if z is None else (z * torch.sigmoid(z)).abs()
    G = dy.abs() * gate
    zs = torch.zeros_like(x) if z is None else z.abs()
    before, hm, km = (torch.zeros_like(x) for _ in range(3))
    eh, ek = torch.zeros_like(x), torch.zeros_like(x)  # in roundings times size
    ebefore = torch.zeros_like(x)
    d0, ed0 = x.new_zeros(len(lens), d), x.new_zeros(len(lens), d)
    for q, (p, e) in enumerate(sequences(lens)):
        h = x.new_zeros(d) if initial is None else initial[q].abs()
        err = torch.zeros(d, dtype=x.dtype)
        for t in range(p, e):
            before[t], ebefore[t] = h, err
            err = a[t] * err + ea[t] * a[t] * h + eb[t] * b[t]
            h = a[t] * h + b[t]
            hm[t], eh[t] = h, err
        k = x.new_zeros(d) if dfinal is None else dfinal[q].abs()
        err = torch.zeros(d, dtype=x.dtype)
        for t in range(e - 1, p - 1, -1):
            k = k + G[t]
            err = err + (8 + 4 * zs[t]) * G[t] + k
            km[t], ek[t] = k, err
            err = a[t] * err + ea[t] * a[t] * k
            k = a[t] * k
        d0[q], ed0[q] = k, err
    sig = torch.sigmoid(zs)
    term = 48 + 8 * vr + 8 * vi + 8 * zs + ea + eb
    root = torch.where(s > 0, L.abs() / s.clamp_min(1e-300), torch.zeros_like(s))
    inner = a * before * L.abs() + a * a * (u * x).abs() * root
    dll = km * inner
    edll = ek * inner + km * a * L.abs() * ebefore + term * dll
    out = dict(dx=(ek + term * km) * s * u, di=(ek + term * km) * b, dr=edll,
               dz=dy.abs() * (eh + term * hm) * sig * (1 + zs), dinitial_state=ed0)
    # the sums: those of the terms, and a rounding for every addition in a row (an eighth of the tokens, and 64)
    adds = x.shape[0] / 8 + 64
    sums = dict(dA=(edll.sum(0) + adds * dll.sum(0)) / A.abs().clamp_min(1e-300), dr_bias=edll.sum(0) + adds * dll.sum(0),
                di_bias=out["di"].sum(0) + adds * (km * b).sum(0))
    return {k: U * v for k, v in {**out, **sums}.items()}


# ------------------------------------------------------------------------------------------ layer norm
ADDS = 96  # roundings of a sum over a row: what a lane adds in a row, the lanes' levels, the waves


def norm(t, w, b, eps):
    """y of t [rows][d] in 64 bits, and the bound of its error: the mean is off by ADDS U mean|t|, the deviation by
    that and 2 U |t|, the reciprocal deviation by 2 ADDS U and what the mean's error does to the variance."""
    mean = t.mean(-1, keepdim=True)
    c = t - mean
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    w = torch.ones(t.shape[-1], dtype=t.dtype) if w is None else w
    y = c * rstd * w + (0 if b is None else b)
    cd, rd, wd = c.detach(), rstd.detach(), w.detach().abs()
    ec = norm_deviation_bound(t.detach())
    ey = rd * wd * ec + (rd * cd.abs() * wd) * (2 * ADDS * U + rd * ec.mean(-1, keepdim=True)) + 4 * U * y.detach().abs()
    return y, ey + (0 if b is None else 2 * U * b.detach().abs())


def norm_deviation_bound(t):
    return U * (ADDS * t.abs().mean(-1, keepdim=True) + 4 * t.abs())


def norm_grad_bounds(dy, t, w, eps, dtotal):
    mean = t.mean(-1, keepdim=True)
    c = t - mean
    rstd = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    xh = (c * rstd).abs()
    ec = rstd * norm_deviation_bound(t)
    e = 3 * ADDS * U + 2 * ec.mean(-1, keepdim=True)  # relative, of rstd and of the two means
    gw = (dy * (1 if w is None else w)).abs()
    m1, m2 = gw.mean(-1, keepdim=True), (gw * xh).mean(-1, keepdim=True)
    dx = rstd * ((gw + m1 + xh * m2) * e + ec * m2 + xh * (gw * ec).mean(-1, keepdim=True))
    adds = U * (t.shape[0] / 8 + 64)
    return dict(dx=dx + (0 if dtotal is None else 2 * U * dtotal.abs()),
                dw=(dy.abs() * (ec + xh * (e + adds))).sum(0), db=adds * dy.abs().sum(0))


# -------------------------------------------------------------------------------------- 4-bit products
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def fp4_values(q, scale, k):
    """What q [n][ceil(k/2)] and scale [n][ceil(k/32)] stand for, in 64 bits."""
    code = torch.stack([q % 16, q // 16], -1).flatten(1)[:, :k].long()
    v = E2M1[code % 8] * torch.where(code >= 8, -1.0, 1.0).double()
    e = torch.where(scale == 255, float("nan"), torch.exp2(scale.double() - 127))
    return v * e.repeat_interleave(32, 1)[:, :k]


def fp4_quantize(x):
    """Codes' values and scale bytes of x [m][k] in 64 bits."""
    m, k = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -k % 32)).view(m, -1, 32)
    top = v.abs().amax(-1)
    e = torch.where(top > 0, torch.ceil(torch.log2(top / 6)), -127.0).clamp(-127, 127)
    scaled = v / torch.exp2(e)[..., None]
    # the nearest value; of two as near the one with an even code (its place in the table)
    far = (scaled.abs()[..., None] - E2M1).abs()
    least = far.amin(-1, keepdim=True)
    near = far == least
    place = torch.arange(8).expand_as(near)
    pick = torch.where(near & (place % 2 == 0), place, 99).amin(-1)
    pick = torch.where(pick == 99, torch.where(near, place, 99).amin(-1), pick)
    value = E2M1[pick] * torch.sign(scaled) * torch.exp2(e)[..., None]
    return value.flatten(1)[:, :k], (e + 127).to(torch.uint8)
