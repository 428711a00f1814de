"""A gated state space block on the sequence operators, for prompts, single tokens and training.

    python -m convolution_nhwc_implicit_amd.gated_block

runs one on the GPU: a packed batch of prompts, the next tokens one by one, and a training step.

    x, z  = split(in_proj(u));   x = causal_conv(x, silu)
    dt, B, C = split(x_proj(x)); y = selective_scan(x, dt, A, B, C, D, z)
    out   = out_proj(y)

The projections are fp8 products with a scale for every 128 values: weights are quantised once in blocks of
128 x 128, both as they are and transposed (for the inputs' gradients), activations and gradients by rows in each
call.
"""
import torch

from . import sequence as S


class Fp8Linear:
    """y = x W^T for x [tokens][k] and W [n][k]."""

    def __init__(self, weight):
        self.n, self.k = weight.shape
        self.w = S.fp8_quantize(weight, blocks=True)
        self.wt = S.fp8_quantize(weight.t().contiguous(), blocks=True)

    def __call__(self, x):
        return S.fp8_matmul(*S.fp8_quantize(x), *self.w, out_dtype=x.dtype)

    def grad(self, dy, x):
        """(dx in dy's type, dW in float32)."""
        dx = S.fp8_matmul(*S.fp8_quantize(dy), *self.wt, out_dtype=dy.dtype)
        dw = S.fp8_matmul(*S.fp8_quantize(dy, transpose=True), *S.fp8_quantize(x, transpose=True),
                          out_dtype=torch.float32)
        return dx, dw


class GatedBlock:
    """Weights in float32: in_proj [2d][model], conv [d][w], conv_bias [d], x_proj [d + 2 groups n][d],
    dt_bias [d], A [d][n] (negative), D [d], out_proj [model][d]."""

    def __init__(self, weights, groups=1, dtype=torch.bfloat16):
        self.d, self.n = weights["A"].shape
        self.groups, self.dtype = groups, dtype
        self.in_proj, self.x_proj, self.out_proj = (Fp8Linear(weights[k]) for k in ("in_proj", "x_proj", "out_proj"))
        self.conv, self.conv_bias = weights["conv"].to(dtype), weights["conv_bias"].to(dtype)
        self.A, self.D, self.dt_bias = (weights[k].float().contiguous() for k in ("A", "D", "dt_bias"))

    @staticmethod
    def random(model, d, n, w=4, groups=1, dtype=torch.bfloat16, device="cuda", generator=None):
        def randn(*shape, scale=1.0):
            return torch.randn(shape, device=device, generator=generator) * scale

        return GatedBlock(dict(
            in_proj=randn(2 * d, model, scale=model ** -0.5), conv=randn(d, w, scale=w ** -0.5),
            conv_bias=randn(d, scale=0.1), x_proj=randn(d + 2 * groups * n, d, scale=d ** -0.5),
            dt_bias=randn(d, scale=0.5) - 3.0, A=-torch.exp(randn(d, n, scale=0.5)), D=1.0 + randn(d, scale=0.1),
            out_proj=randn(model, d, scale=d ** -0.5)), groups, dtype)

    def states(self, pool):
        """Empty states for `pool` requests: the convolution's last rows and the scan's states."""
        dev = self.A.device
        return (torch.zeros(pool, self.conv.shape[1] - 1, self.d, dtype=self.dtype, device=dev),
                torch.zeros(pool, self.d, self.n, device=dev))

    def _split(self, p):
        gn = self.groups * self.n
        dt, B, C = p.split([self.d, gn, gn], -1)
        return dt, B.unflatten(-1, (self.groups, self.n)), C.unflatten(-1, (self.groups, self.n))

    def _scan(self, z):
        return dict(D=self.D, z=z, dt_bias=self.dt_bias, softplus=True)

    def prompt(self, u, seq_start, states=None):
        """u [tokens][model] of sequences packed by seq_start, from `states` (one for each sequence) or from
        empty ones; the outputs and the states to go on from."""
        x, z = self.in_proj(u).split(self.d, -1)
        conv, scan = states if states is not None else (None, None)
        x, conv = S.causal_conv(x, self.conv, self.conv_bias, silu=True, initial_state=conv, seq_start=seq_start,
                                return_state=True)
        dt, B, C = self._split(self.x_proj(x))
        y, scan = S.selective_scan(x, dt, self.A, B, C, initial_state=scan, seq_start=seq_start, return_state=True,
                                   **self._scan(z))
        return self.out_proj(y), (conv, scan)

    def step(self, u, states, slots=None):
        """One token for each request, u [rows][model]; states are pools, updated in place."""
        x, z = self.in_proj(u).split(self.d, -1)
        x = S.causal_conv_step(x, states[0], self.conv, self.conv_bias, silu=True, slots=slots)
        dt, B, C = self._split(self.x_proj(x))
        y = S.selective_scan_step(x, dt, self.A, B, C, states[1], slots=slots, **self._scan(z))
        return self.out_proj(y)

    def train(self, u, dout, seq_start=None):
        """Outputs for u [tokens][model] and, for the output gradients dout(outputs), the gradients of u and of
        every weight: (out, dict)."""
        xz = self.in_proj(u)
        x0, z = xz.split(self.d, -1)
        conv = dict(silu=True, seq_start=seq_start)
        x = S.causal_conv(x0, self.conv, self.conv_bias, **conv)
        dt, B, C = self._split(self.x_proj(x))
        scan = dict(seq_start=seq_start, **self._scan(z))
        y = S.selective_scan(x, dt, self.A, B, C, **scan)
        out = self.out_proj(y)

        g = {}
        dy, g["out_proj"] = self.out_proj.grad(dout(out), y)
        s = S.selective_scan_grad(dy, x, dt, self.A, B, C, **scan)
        dp = torch.cat([s["ddt"], s["dB"].flatten(-2), s["dC"].flatten(-2)], -1)
        dx, g["x_proj"] = self.x_proj.grad(dp, x)
        c = S.causal_conv_grad(s["du"] + dx, x0, self.conv, self.conv_bias, **conv)
        g["u"], g["in_proj"] = self.in_proj.grad(torch.cat([c["dx"], s["dz"]], -1), u)
        g.update(conv=c["dw"], conv_bias=c["db"], A=s["dA"], D=s["dD"], dt_bias=s["ddt_bias"])
        return out, g


def main():
    gen = torch.Generator(device="cuda").manual_seed(0)
    block = GatedBlock.random(1024, 2048, 16, generator=gen)
    lens = [300, 1, 77, 640]
    start = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    u = torch.randn(sum(lens), 1024, device="cuda", generator=gen).to(torch.bfloat16)
    out, states = block.prompt(u, start)
    print("prompts of", lens, "tokens:", tuple(out.shape))
    token = out[start[1:].long() - 1]
    for _ in range(4):
        token = block.step(token, states)
    print("four tokens more for each:", tuple(token.shape), "finite:", bool(token.isfinite().all()))
    out, g = block.train(u, lambda y: y * 1e-3, start)
    print("training step:", {k: tuple(v.shape) for k, v in g.items()})


if __name__ == "__main__":
    main()
