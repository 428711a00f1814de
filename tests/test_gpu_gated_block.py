"""The gated block that runs the sequence operators together: prompts against single tokens, and a training step
against the same block in 64 bits without quantisation."""
import pytest
import torch

import sequence_ref as R
from convolution_nhwc_implicit_amd.gated_block import GatedBlock

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(groups=2):
    g = torch.Generator().manual_seed(3)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g) * scale

    model, d, n, w = 136, 200, 16, 4
    weights = dict(in_proj=randn(2 * d, model, scale=model ** -0.5), conv=randn(d, w, scale=0.5),
                   conv_bias=randn(d, scale=0.1), x_proj=randn(d + 2 * groups * n, d, scale=d ** -0.5),
                   dt_bias=randn(d, scale=0.5) - 3.0, A=-torch.exp(randn(d, n, scale=0.5)),
                   D=1 + randn(d, scale=0.1), out_proj=randn(model, d, scale=d ** -0.5))
    return weights, GatedBlock({k: v.to(DEV) for k, v in weights.items()}, groups), randn


def off(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    return float((got - want).norm() / want.norm())


def test_prompts_and_tokens_agree():
    """Prompts in one packed call against the same tokens one by one on pooled states.  The two sides sum products in
    different orders and round to bf16 at five places on the way: five half steps of 2^-8 in norm, and as much again
    where a rounding moves an fp8 value to its neighbour."""
    _, block, randn = make()
    lens = [9, 4, 6]
    start = torch.tensor([0] + lens).cumsum(0)
    u = randn(sum(lens), 136).to(torch.bfloat16).to(DEV)
    out, (conv, scan) = block.prompt(u, start.to(torch.int32).to(DEV))
    pool = block.states(5)
    places = [4, 0, 2]
    outs = [[] for _ in lens]
    for t in range(max(lens)):
        live = [i for i, n in enumerate(lens) if t < n]
        rows = torch.stack([u[start[i] + t] for i in live])
        slots = torch.tensor([places[i] for i in live], dtype=torch.int32, device=DEV)
        for i, y in zip(live, block.step(rows, pool, slots)):
            outs[i].append(y)
    got = torch.cat([torch.stack(o) for o in outs])
    assert off(got, out) <= 10 * 2.0 ** -8
    at = torch.tensor(places, device=DEV)
    assert off(pool[0][at], conv) <= 10 * 2.0 ** -8 and off(pool[1][at], scan) <= 10 * 2.0 ** -8
    # a second piece of every prompt, from the states
    more, _ = block.prompt(u, start.to(torch.int32).to(DEV), (conv, scan))
    assert more.shape == out.shape and more.isfinite().all()


def test_training_step():
    """Outputs and gradients against the block in 64 bits.  e4m3 rounds by at most 2^-4 of a value, 2^-4 / sqrt(3) in
    norm; a gradient's path crosses at most eight quantised operands."""
    weights, block, randn = make()
    lens = [30, 1, 22]
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    u, dout = randn(53, 136).to(torch.bfloat16), randn(53, 136).to(torch.bfloat16)
    out, g = block.train(u.to(DEV), lambda y: dout.to(DEV), start)
    leaves = {k: v.double().requires_grad_() for k, v in {**weights, "u": u}.items()}
    d = 200
    x0, z = (leaves["u"] @ leaves["in_proj"].t()).split(d, -1)
    x = R.conv(x0, leaves["conv"], leaves["conv_bias"], True, lens)[0]
    dt, B, C = (x @ leaves["x_proj"].t()).split([d, 32, 32], -1)
    y = R.scan(x, dt, leaves["A"], B.unflatten(-1, (2, 16)), C.unflatten(-1, (2, 16)), leaves["D"], z,
               leaves["dt_bias"], True, lens)[0]
    want = y @ leaves["out_proj"].t()
    bound = 8 * 2.0 ** -4 / 3 ** 0.5
    assert off(out, want.detach()) <= bound
    grads = dict(zip(leaves, torch.autograd.grad((want * dout.double()).sum(), list(leaves.values()))))
    assert set(g) == set(grads)
    for k in grads:
        assert off(g[k], grads[k]) <= bound, (k, off(g[k], grads[k]))
