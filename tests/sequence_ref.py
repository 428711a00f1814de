"""Plain 64-bit forms of the sequence operators (CPU), with the error bounds that their fp32 kernels are held to.

Bounds.  An output of type t is rounded once: half a step, eps(t)/2 relative.  Before that, fp32 arithmetic
rounds each product and each sum by at most 2^-24 of a term, so an error is bounded by the number of roundings
times 2^-24 times the same formula evaluated with absolute values ("mag")."""
import torch

U = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def sequences(lens):
    at = 0
    for n in lens:
        yield at, at + n
        at += n


# ------------------------------------------------------------------------------ causal convolution
def conv(x, w, bias, silu, lens, initial=None):
    """x [T][d] (sequences end to end) in 64 bits -> y, final states, and the sum of the terms' sizes."""
    d, wd = w.shape
    ys, mags, finals = [], [], []
    for s, (a, b) in enumerate(sequences(lens)):
        before = x.new_zeros(wd - 1, d) if initial is None else initial[s]
        full = torch.cat([before, x[a:b]])
        pre = x.new_zeros(b - a, d) + (0 if bias is None else bias)
        mag = pre.abs()
        for k in range(wd):
            pre = pre + w[:, k] * full[k:k + b - a]
            mag = mag + (w[:, k] * full[k:k + b - a]).abs()
        ys.append(pre * torch.sigmoid(pre) if silu else pre)
        mags.append(mag)
        finals.append(full[b - a:])
    return torch.cat(ys), torch.stack(finals), torch.cat(mags).detach()


# ---------------------------------------------------------------------------------- selective scan
def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def scan(x, dt, A, B, C, D, z, dt_bias, soft, lens, initial=None):
    """x, dt, z [T][d], B, C [T][g][n] in 64 bits -> y, final states, the size of y's terms, and how many roundings
    of a state's terms a state carries at most (decayed with the state)."""
    d, n = A.shape
    rep = d // B.shape[1]
    Bc, Cc = B.repeat_interleave(rep, 1), C.repeat_interleave(rep, 1)
    raw = dt + (0 if dt_bias is None else dt_bias)
    delta = softplus(raw) if soft else raw
    ys, finals, mags, worst = [], [], [], 0.0
    for s, (a, b) in enumerate(sequences(lens)):
        h = x.new_zeros(d, n) if initial is None else initial[s]
        hm, err = h.detach().abs(), torch.zeros_like(h.detach())
        for t in range(a, b):
            e = torch.exp(delta[t][:, None] * A)
            h = e * h + (delta[t] * x[t])[:, None] * Bc[t]
            ed = e.detach()
            hm = ed * hm + (delta[t] * x[t])[:, None].abs().detach() * Bc[t].abs().detach()
            # a step's roundings: the exponent's (its size relative), the exponential's, the step size's, products, sum
            err = ed * err + (16 + 4 * (delta[t][:, None] * A).abs().detach()) * hm
            worst = max(worst, float((err / hm.clamp_min(1e-300)).max()))
            y = (h * Cc[t]).sum(-1)
            m = (hm * Cc[t].abs()).sum(-1).detach()
            if D is not None:
                y = y + D * x[t]
                m = m + (D * x[t]).abs().detach()
            if z is not None:
                gate = z[t] * torch.sigmoid(z[t])
                y = y * gate
                m = m * gate.abs().detach()
            ys.append(y)
            mags.append(m)
        finals.append(h)
    y = torch.stack(ys) if ys else x.new_zeros(0, d)
    return y, torch.stack(finals), (torch.stack(mags) if mags else y), worst


def scan_grad_mag(dy, x, dt, A, B, C, D, z, dt_bias, soft, lens, initial=None, dfinal=None):
    """The gradients' formulas with every term's size in place of the term (no sums cancel): bounds for the terms
    that each gradient adds up."""
    names = ["x", "dt", "A", "B", "C", "D", "z", "dt_bias", "initial"]
    d, n = A.shape
    rep = d // B.shape[1]
    raw = dt + (0 if dt_bias is None else dt_bias)
    delta = softplus(raw) if soft else raw
    back = torch.sigmoid(raw) if soft else torch.ones_like(raw)
    Bc, Cc = B.abs().repeat_interleave(rep, 1), C.abs().repeat_interleave(rep, 1)
    sig = torch.ones_like(x) if z is None else torch.sigmoid(z)
    gate = torch.ones_like(x) if z is None else (z * sig).abs()
    g = dy.abs() * gate
    Dm = torch.zeros(d, dtype=x.dtype) if D is None else D.abs()
    out = {k: None for k in names}
    du, ddl, dB, dC, dz = (torch.zeros_like(v) for v in (x, x, B, C, x))
    dA, dD = torch.zeros_like(A), torch.zeros_like(Dm)
    dinit = x.new_zeros(len(lens), d, n)
    for s, (a, b) in enumerate(sequences(lens)):
        h = x.new_zeros(d, n) if initial is None else initial[s].abs()
        hs = [h]
        for t in range(a, b):
            h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * x[t]).abs()[:, None] * Bc[t]
            hs.append(h)
        k = x.new_zeros(d, n) if dfinal is None else dfinal[s].abs()
        for t in range(b - 1, a - 1, -1):
            dh = k + g[t][:, None] * Cc[t]
            h = hs[t - a + 1]
            ys = (h * Cc[t]).sum(-1) + Dm * x[t].abs()
            dz[t] = dy[t].abs() * ys * (sig[t] * (1 + (0 if z is None else z[t].abs() * (1 - sig[t]))))
            dC[t] = (g[t][:, None] * h).view(B.shape[1], rep, n).sum(1)
            dB[t] = ((delta[t] * x[t]).abs()[:, None] * dh).view(B.shape[1], rep, n).sum(1)
            inner = (dh * Bc[t]).sum(-1)
            k = dh * torch.exp(delta[t][:, None] * A)
            f = k * hs[t - a]
            du[t] = delta[t].abs() * inner + Dm * g[t]
            ddl[t] = (x[t].abs() * inner + (f * A.abs()).sum(-1)) * back[t]
            dA += f * delta[t].abs()[:, None]
            dD += g[t] * x[t].abs()
        dinit[s] = k
    out.update(x=du, dt=ddl, A=dA, B=dB, C=dC, D=dD, z=dz, dt_bias=ddl.sum(0), initial=dinit)
    return out
