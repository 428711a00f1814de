"""More sequence operators' measured cases: the gated linear recurrence for prompts, training and single tokens, the
layer norm in front of a block with its gradients, and products with 4-bit weights for single tokens.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and this package's kernels."""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
GROUP = 32  # 4-bit values that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token for few requests: latency
        dict(name="recur_step_few", op="recur_step", rows=4, pool=8, d=4096, type="bf16"),
        # one new token for a full serving batch: the states' traffic
        dict(name="recur_step_batch", op="recur_step", rows=256, pool=320, d=5120, type="bf16"),
        # one long prompt
        dict(name="recur_prompt", op="recur", lens="8192", d=4096, type="bf16", state=False),
        # the next pieces of ragged prompts, states in and out; odd channel count
        dict(name="recur_packed", op="recur", lens="700,1,129,950,64,3,500,654", d=1999, type="f16", state=True),
        # a layer's recurrence in a training step: forward and all gradients
        dict(name="recur_train", op="recur_grad", lens="4096,4096,4096,4096", d=4096, type="bf16"),
        # the same in full precision, on sequences of odd length
        dict(name="recur_train_f32", op="recur_grad", lens="517,517,517", d=768, type="f32"),
        # the norm in front of a block for the new tokens of 32 requests, with the residual sum: latency
        dict(name="norm_step", op="norm", rows=32, d=4096, type="bf16", wtype="bf16"),
        # the same for packed prompts; odd width
        dict(name="norm_prompt", op="norm", rows=4057, d=2731, type="f16", wtype="f16"),
        # a layer's norm in a training step: forward and all gradients, parameters kept in full precision
        dict(name="norm_train", op="norm_grad", rows=16384, d=4096, type="bf16", wtype="f32"),
        # the same in full precision, for a narrow model
        dict(name="norm_train_f32", op="norm_grad", rows=1551, d=768, type="f32", wtype="f32"),
        # a projection of one new token: the weights' traffic
        dict(name="fp4_step", op="fp4", m=1, n=8192, k=4096, type="bf16"),
        # a projection of the new tokens of 48 requests; no size is a whole tile
        dict(name="fp4_batch", op="fp4", m=48, n=8200, k=4104, type="f16"),
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cut(rng, total, most):
    """`total` tokens cut at random places into at most `most` sequences (none of them empty)."""
    parts = rng.randint(1, min(most, total))
    cuts = sorted(rng.sample(range(1, total), parts - 1)) if parts > 1 else []
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["recur_step", "recur", "recur_grad", "norm", "norm_grad", "fp4"])
    kind = rng.choice(["f16", "bf16", "f32"])
    if op == "recur_step":
        rows = _log(rng, 1, 512)
        return dict(op=op, rows=rows, pool=rows + rng.randint(0, rows), d=_log(rng, 64, 8192), type=kind)
    if op.startswith("recur"):
        d = _log(rng, 64, 6000)
        lens = _cut(rng, _log(rng, 1, min(16384, (1 << (25 if kind == "f32" else 26)) // d)), 12)
        c = dict(op=op, lens=lens, d=d, type=kind)
        return dict(c, state=rng.random() < 0.5) if op == "recur" else c
    if op.startswith("norm"):
        d = _log(rng, 64, 16384)
        rows = _log(rng, 1, min(16384, (1 << (25 if kind == "f32" else 26)) // d))
        return dict(op=op, rows=rows, d=d, type=kind, wtype=rng.choice([kind, "f32"]))
    return dict(op=op, m=_log(rng, 1, 64), n=_log(rng, 200, 8192), k=_log(rng, 200, 8192), type=kind)


# ------------------------------------------------------------------------------------------------- the inputs
def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def _dense(lens):
    """Sequences of one length are a batch [B][L]; others lie end to end, with their starts."""
    return len(set(lens)) == 1


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)

    op, dt = case["op"], TYPES[case["type"]]
    s = {"op": op, "type": dt}
    if op == "fp4":
        m, n, k = case["m"], case["n"], case["k"]
        q, scale = _quantize(randn(n, k, scale=k ** -0.5))
        # rows of whole 16-byte pieces, as the package lays them out
        buf = torch.zeros((n, -(-k // GROUP) * 16), dtype=torch.uint8, device=DEV)
        buf[:, :q.shape[1]] = q
        s.update(x=randn(m, k, dtype=dt) * torch.exp(randn(1, k, scale=0.5)).to(dt),  # some features are larger
                 w=buf[:, :q.shape[1]], w_scale=scale)
        return s
    d = case["d"]
    if op.startswith("norm"):
        rows, wt = case["rows"], TYPES[case["wtype"]]
        # channels of different sizes around different means, as they grow along a residual stream
        level, size = randn(d, scale=0.3), torch.exp(randn(d, scale=0.5))
        s.update(x=(randn(rows, d) * size + level).to(dt), residual=randn(rows, d, dtype=dt),
                 weight=(1.0 + randn(d, scale=0.1)).to(wt), bias=randn(d, scale=0.1, dtype=wt))
        if op == "norm_grad":
            s.update(dy=randn(rows, d, dtype=dt), dtotal=randn(rows, d, dtype=dt))
        return s
    if "rows" in case:
        rows, pool = case["rows"], case["pool"]
        lead = (rows,)
        s.update(slots=torch.randperm(pool, generator=gen, device=DEV)[:rows].to(torch.int32))
        count = pool
    else:
        lens = _lens(case)
        lead = (len(lens), lens[0]) if _dense(lens) else (sum(lens),)
        count = len(lens)
        starts = torch.tensor([0] + lens, device=DEV).cumsum(0)
        s.update(starts=starts, seq_start=None if _dense(lens) else starts.to(torch.int32))
    gates = randn(*lead, 2 * d, dtype=dt)  # both gates are halves of one projection's output
    # at an open gate of one half, decays between 0.9 and 0.999 a token
    s.update(x=randn(*lead, d, dtype=dt), r=gates[..., :d], i=gates[..., d:], z=randn(*lead, d, dtype=dt),
             A=2.0 * torch.log(0.9 + 0.099 * torch.rand(d, generator=gen, device=DEV)),
             r_bias=randn(d, scale=0.3), i_bias=randn(d, scale=0.3))
    s["state"] = randn(count, d) if op == "recur_step" or case.get("state") else None
    if op == "recur_grad":
        s["dy"] = randn(*lead, d, dtype=dt)
    return s


# ------------------------------------------------------------------------------------------- the plain forms
def _quantize(w):
    """4-bit values of w [n][k], two to a byte (the even one in the low half), and exponents of scales for 32 values of
    a row: the least power of two that brings them all into e2m1's range."""
    n, k = w.shape
    v = F.pad(w.float(), (0, -k % GROUP)).view(n, -1, GROUP)
    part, exp = torch.frexp(v.abs().amax(-1))  # part in [0.5, 1); 6 is 0.75 * 2^3
    exp = torch.where(part == 0, torch.full_like(exp, -127), exp - 3 + (part > 0.75).int()).clamp(-127, 127)
    v = torch.ldexp(v, -exp[..., None])
    # nearest of the eight sizes; the borders between them go to the even one
    size = v.abs()
    code = sum((size > b).int() for b in (0.25, 1.25, 2.5, 5.0)) + sum((size >= b).int() for b in (0.75, 1.75, 3.5))
    code = (code + 8 * (v < 0).int()).flatten(1)[:, :k]
    code = F.pad(code, (0, k % 2)).view(n, -1, 2)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), (exp + 127).to(torch.uint8)


def _values(q, scale, k):
    """What the 4-bit values stand for, in 32 bits."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(1)[:, :k].long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    size = torch.exp2(scale.float() - 127).repeat_interleave(GROUP, 1)[:, :k]
    return table[code] * size


def _plain_fp4(s):
    x = s["x"].float()
    return (x @ _values(s["w"], s["w_scale"], x.shape[1]).t()).to(s["type"])


def _normed(t):
    mean = t.mean(-1, keepdim=True)
    rstd = torch.rsqrt(((t - mean) ** 2).mean(-1, keepdim=True) + EPS)
    return (t - mean) * rstd, rstd


def _plain_norm(s):
    t = s["x"].float() + s["residual"].float()
    y = _normed(t)[0] * s["weight"].float() + s["bias"].float()
    return y.to(s["type"]), t.to(s["type"])


def _plain_norm_grad(s):
    y, total = _plain_norm(s)
    dy = s["dy"].float()
    xh, rstd = _normed(total.float())
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True)) + s["dtotal"].float()
    wt = s["weight"].dtype
    return y, total, dx.to(s["type"]), (dy * xh).sum(0).to(wt), dy.sum(0).to(wt)


def _running(a, b):
    """h[t] = a[t] * h[t-1] + b[t] along the first axis, by doubling."""
    reach = 1
    while reach < b.shape[0]:
        b = torch.cat([b[:reach], torch.addcmul(b[reach:], a[reach:], b[:-reach])])
        a = torch.cat([a[:reach], a[reach:] * a[:-reach]])
        reach *= 2
    return b


def _gates(s):
    flat = [s[k].flatten(0, -2).float() for k in ("x", "r", "i", "z")]
    g, u = torch.sigmoid(flat[1] + s["r_bias"]), torch.sigmoid(flat[2] + s["i_bias"])
    a = torch.exp(s["A"] * g)
    return flat[0], g, u, flat[3], a, torch.sqrt(-torch.expm1(2 * s["A"] * g))


def _recur(s):
    x, g, u, z, a, size = _gates(s)
    b = size * u * x
    first = s["starts"][:-1]
    a = a.clone()
    if s["state"] is not None:
        b[first] += a[first] * s["state"]
    a[first] = 0
    return x, g, u, z, a, size, _running(a, b)


def _plain_recur(s):
    z, h = _recur(s)[3::3]
    y = (h * z * torch.sigmoid(z)).to(s["type"]).view(s["x"].shape)
    return y if s["state"] is None else (y, h[s["starts"][1:] - 1])


def _plain_recur_grad(s):
    x, g, u, z, a, size, h = _recur(s)
    dt, lead = s["type"], s["x"].shape
    dy, sig = s["dy"].flatten(0, -2).float(), torch.sigmoid(z)
    # the states' gradients run backwards; a at a sequence's first token is already 0
    k = _running(torch.cat([torch.zeros_like(a[:1]), a[1:].flip(0)]), (dy * z * sig).flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    full = torch.exp(s["A"] * g)
    dl = k * (a * before - full * full / size * u * x)
    dr = dl * s["A"] * g * (1 - g)
    di = k * size * x * u * (1 - u)
    return {"y": (h * z * sig).to(dt).view(lead), "dx": (k * size * u).to(dt).view(lead), "dr": dr.to(dt).view(lead),
            "di": di.to(dt).view(lead), "dA": (dl * g).sum(0),
            "dz": (dy * h * sig * (1 + z * (1 - sig))).to(dt).view(lead), "dr_bias": dr.sum(0), "di_bias": di.sum(0)}


def _plain_recur_step(s):
    slots = s["slots"].long()
    x, g, u, z, a, size = _gates(s)
    h = a * s["state"][slots] + size * u * x
    s["state"][slots] = h
    return (h * z * torch.sigmoid(z)).to(s["type"]), s["state"]


# ------------------------------------------------------------------------------------------ the package's calls
def _own_recur(s):
    import convolution_nhwc_implicit_amd as nn
    return nn.gated_recurrence(s["x"], s["r"], s["i"], s["A"], z=s["z"], r_bias=s["r_bias"], i_bias=s["i_bias"],
                               initial_state=s["state"], seq_start=s["seq_start"], return_state=s["state"] is not None)


def _own_recur_grad(s):
    import convolution_nhwc_implicit_amd as nn
    kw = dict(z=s["z"], r_bias=s["r_bias"], i_bias=s["i_bias"], seq_start=s["seq_start"])
    y = nn.gated_recurrence(s["x"], s["r"], s["i"], s["A"], **kw)
    g = nn.gated_recurrence_grad(s["dy"], s["x"], s["r"], s["i"], s["A"], **kw)
    return {"y": y, **{k: g[k] for k in ("dx", "dr", "di", "dA", "dz", "dr_bias", "di_bias")}}


def _own_recur_step(s):
    import convolution_nhwc_implicit_amd as nn
    return nn.gated_recurrence_step(s["x"], s["r"], s["i"], s["A"], s["state"], z=s["z"], r_bias=s["r_bias"],
                                    i_bias=s["i_bias"], slots=s["slots"]), s["state"]


def _own_norm(s):
    import convolution_nhwc_implicit_amd as nn
    return nn.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, residual=s["residual"])


def _own_norm_grad(s):
    import convolution_nhwc_implicit_amd as nn
    y, total = nn.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, residual=s["residual"])
    g = nn.layer_norm_grad(s["dy"], total, s["weight"], s["bias"], eps=EPS, dtotal=s["dtotal"])
    return y, total, g["dx"], g["dw"], g["db"]


def _own_fp4(s):
    import convolution_nhwc_implicit_amd as nn
    return nn.fp4_matmul(s["x"], s["w"], s["w_scale"])


PLAIN = {"recur": _plain_recur, "recur_grad": _plain_recur_grad, "recur_step": _plain_recur_step, "norm": _plain_norm,
         "norm_grad": _plain_norm_grad, "fp4": _plain_fp4}
OWN = {"recur": _own_recur, "recur_grad": _own_recur_grad, "recur_step": _own_recur_step, "norm": _own_norm,
       "norm_grad": _own_norm_grad, "fp4": _own_fp4}


def run(state):
    if own:
        return OWN[state["op"]](state)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------------- the work
def work(case):
    op, e = case["op"], 4 if case["type"] == "f32" else 2
    if op == "fp4":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": e * m * (k + n) + n * (-(-k // 2) + -(-k // GROUP)), "flops": 2 * m * n * k}
    d = case["d"]
    if op.startswith("norm"):
        grad, we = op == "norm_grad", 4 if case["wtype"] == "f32" else 2
        # x, residual, y, total; dy, dtotal, dx; and the parameters with their gradients
        return {"bytes": e * (7 if grad else 4) * case["rows"] * d + we * d * (4 if grad else 2),
                "flops": case["rows"] * d * (22 if grad else 8)}
    t = case["rows"] if "rows" in case else sum(_lens(case))
    seqs = case["rows"] if "rows" in case else len(_lens(case))
    states = 2 if op == "recur_step" or case.get("state") else 0
    grad = op == "recur_grad"
    # x, r, i, z, y; dy, dx, dr, di, dz; and the three parameters with their gradients
    return {"bytes": e * (10 if grad else 5) * t * d + 4 * d * (3 * (2 if grad else 1) + states * seqs),
            "flops": t * d * (60 if grad else 20)}


# --------------------------------------------------------------------------------- the definition in 64 bits
def _exact_fp4(s):
    x, q = s["x"].double(), s["w"].int()
    pairs = torch.stack([torch.bitwise_and(q, 15), torch.div(q, 16, rounding_mode="floor")], 2)
    code = pairs.reshape(q.shape[0], -1)[:, :x.shape[1]]
    low = code % 8
    # an exponent of two bits and one bit behind the leading one, which the exponent 0 lacks
    exp, half = torch.div(low, 2, rounding_mode="floor"), (low % 2).double()
    size = torch.where(exp == 0, 0.5 * half, torch.exp2(exp.double() - 1) * (1 + 0.5 * half))
    group = torch.arange(x.shape[1], device=DEV) // GROUP
    w = torch.where(code >= 8, -size, size) * torch.exp2(s["w_scale"].double() - 127)[:, group]
    return torch.mm(x, w.t())


def _exact_norm(s):
    x, res, w, b = (s[k].double() for k in ("x", "residual", "weight", "bias"))
    t = x + res
    var, mean = torch.var_mean(t, dim=1, correction=0, keepdim=True)
    y = w * ((t - mean) / torch.sqrt(var + EPS)) + b
    if s["op"] == "norm":
        return y, t
    dy = s["dy"].double()
    held = t.to(s["type"]).double()  # the gradients are those at the sum as it is held
    n = t.shape[1]
    var, mean = torch.var_mean(held, dim=1, correction=0, keepdim=True)
    dev = torch.sqrt(var + EPS)
    c = held - mean
    dc = dy * w / dev - c * ((dy * w * c).sum(1, keepdim=True) / (n * dev ** 3))
    return (y, t, dc - dc.sum(1, keepdim=True) / n + s["dtotal"].double(),
            torch.einsum("td,td->d", dy, c / dev), dy.sum(0))


def _pieces(s, names):
    """The tensors of each batch of sequences of one length, [b][l][...] in 64 bits."""
    if s["seq_start"] is None:
        return [[s[k].double() for k in names]]
    ends = s["starts"].tolist()
    return [[s[k][a:b].double()[None] for k in names] for a, b in zip(ends, ends[1:])]


def _joined(s, parts):
    return parts[0] if s["seq_start"] is None else torch.cat([p[0] for p in parts])


def _exact_recur(s):
    """One token after another, forwards and then backwards."""
    A, rb, ib = s["A"].double(), s["r_bias"].double(), s["i_bias"].double()
    step, grad = s["op"] == "recur_step", "dy" in s
    names = ["x", "r", "i", "z"] + (["dy"] if grad else [])
    parts = [[s[k].double()[:, None] for k in names]] if step else _pieces(s, names)
    out = {k: [] for k in ("y", "dx", "dr", "di", "dz")}
    total = {"dA": torch.zeros_like(A), "dr_bias": torch.zeros_like(A), "di_bias": torch.zeros_like(A)}
    ends = []
    for n, p in enumerate(parts):
        x, z = p[0], p[3]
        gate, take = 1 / (1 + torch.exp(-(p[1] + rb))), 1 / (1 + torch.exp(-(p[2] + ib)))
        a = torch.exp(A * gate)
        size = torch.sqrt(-torch.expm1(2 * A * gate))
        fresh = size * take * x
        h = torch.zeros_like(x[:, 0])
        if step:
            h = s["state"][s["slots"].long()].double()
        elif s["state"] is not None:
            h = (s["state"] if s["seq_start"] is None else s["state"][n:n + 1]).double()
        states = torch.empty_like(x)
        for t in range(x.shape[1]):
            h = a[:, t] * h + fresh[:, t]
            states[:, t] = h
        ends.append(h)
        sig = 1 / (1 + torch.exp(-z))
        out["y"].append(states * z * sig)
        if not grad:
            continue
        out["dz"].append(p[4] * states * (sig + z * sig * (1 - sig)))
        k = p[4] * z * sig
        for t in range(x.shape[1] - 2, -1, -1):
            k[:, t] += a[:, t + 1] * k[:, t + 1]
        out["dx"].append(k * size * take)
        di = k * size * x * take * (1 - take)
        da = -k * take * x * a / size
        da[:, 1:] += k[:, 1:] * states[:, :-1]
        dr = da * a * A * gate * (1 - gate)
        out["di"].append(di)
        out["dr"].append(dr)
        for name, v in (("dA", da * a * gate), ("dr_bias", dr), ("di_bias", di)):
            total[name] += v.sum((0, 1))
    if step:
        pool = s["state"].double()
        pool[s["slots"].long()] = ends[0]
        return out["y"][0][:, 0], pool
    y = _joined(s, out["y"])
    if not grad:
        return y if s["state"] is None else (y, torch.cat(ends))
    res = {k: _joined(s, out[k]) for k in ("dx", "dr", "di", "dz")}
    return {"y": y, **{k: res[k] if k in res else total[k]
                       for k in ("dx", "dr", "di", "dA", "dz", "dr_bias", "di_bias")}}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "fp4":
        return _exact_fp4(s)
    return _exact_norm(s) if s["op"].startswith("norm") else _exact_recur(s)
