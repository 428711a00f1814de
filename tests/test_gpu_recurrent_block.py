"""The recurrent block that runs norm, recurrence and 4-bit products together with the operators that were there: prompts
against single tokens, a training step against the block in 64 bits without quantisation, and both blocks on one stream."""
import pytest
import torch

import block_ref as B
import sequence_ref as R
from convolution_nhwc_implicit_amd import gated_block
from convolution_nhwc_implicit_amd.gated_block import Fp4Linear, Fp8Linear, GatedBlock, RecurrentBlock

pytestmark = pytest.mark.gpu
DEV = "cuda"
MODEL, D = 136, 200


def make(four_bit=False):
    g = torch.Generator().manual_seed(5)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g) * scale

    weights = dict(norm=1 + randn(MODEL, scale=0.1), norm_bias=randn(MODEL, scale=0.1),
                   in_proj=randn(2 * D, MODEL, scale=MODEL ** -0.5), conv=randn(D, 4, scale=0.5), conv_bias=randn(D, scale=0.1),
                   gate_proj=randn(2 * D, D, scale=D ** -0.5), r_bias=randn(D, scale=0.3), i_bias=randn(D, scale=0.3),
                   A=2 * torch.log(0.9 + 0.099 * torch.rand(D, generator=g)), out_proj=randn(MODEL, D, scale=D ** -0.5))
    return weights, RecurrentBlock({k: v.to(DEV) for k, v in weights.items()}, four_bit=four_bit), randn


def off(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    return float((got - want).norm() / want.norm())


def test_prompts_and_tokens_agree():
    """Prompts in one packed call against the same tokens one by one on pooled states. The two sides sum products in
    different orders and round to bf16 at six places on the way: six half steps of 2^-8 in norm, and as much again
    where a rounding moves an fp8 value to its neighbour."""
    _, block, randn = make()
    lens = [9, 4, 6]
    start = torch.tensor([0] + lens).cumsum(0)
    u, res = (randn(sum(lens), MODEL).to(torch.bfloat16).to(DEV) for _ in range(2))
    out, total, (conv, state) = block.prompt(u, start.to(torch.int32).to(DEV), residual=res)
    pool = block.states(5)
    places = [4, 0, 2]
    outs, totals = [[] for _ in lens], [[] for _ in lens]
    for t in range(max(lens)):
        live = [i for i, n in enumerate(lens) if t < n]
        rows = [int(start[i]) + t for i in live]
        slots = torch.tensor([places[i] for i in live], dtype=torch.int32, device=DEV)
        for i, y, s in zip(live, *block.step(u[rows], pool, slots, residual=res[rows])):
            outs[i].append(y)
            totals[i].append(s)
    assert off(torch.cat([torch.stack(o) for o in outs]), out) <= 12 * 2.0 ** -8
    assert torch.equal(torch.cat([torch.stack(o) for o in totals]), total)
    at = torch.tensor(places, device=DEV)
    assert off(pool[0][at], conv) <= 12 * 2.0 ** -8 and off(pool[1][at], state) <= 12 * 2.0 ** -8


def test_four_bit_tokens():
    """A token's projections in 4 bits: e2m1 rounds a value by at most a quarter of it, in norm a quarter over sqrt(3);
    three products one behind the other."""
    weights, block, randn = make(four_bit=True)
    assert isinstance(block.token["in_proj"], Fp4Linear)
    eight = make()[1]
    u = randn(7, MODEL).to(torch.bfloat16).to(DEV)
    a, b = block.step(u, block.states(7)), eight.step(u, eight.states(7))
    assert torch.equal(a[1], b[1]) and off(a[0], b[0]) <= 3 * 0.25 / 3 ** 0.5


def test_training_step():
    """Outputs and gradients against the block in 64 bits. e4m3 rounds by at most 2^-4 of a value, 2^-4 / sqrt(3) in
    norm; a gradient's path crosses at most eight quantised operands."""
    weights, block, randn = make()
    lens = [30, 1, 22]
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    u, res, dout, dtot = (randn(53, MODEL).to(torch.bfloat16) for _ in range(4))
    out, total, g = block.train(u.to(DEV), lambda y, t: (dout.to(DEV), dtot.to(DEV)), start, residual=res.to(DEV))
    leaves = {k: v.double().requires_grad_() for k, v in {**weights, "u": u}.items()}
    t = leaves["u"] + res.double()
    h, _ = B.norm(t, leaves["norm"], leaves["norm_bias"], 1e-5)
    x0, z = (h @ leaves["in_proj"].t()).split(D, -1)
    x = R.conv(x0, leaves["conv"], leaves["conv_bias"], True, lens)[0]
    r, i = (x @ leaves["gate_proj"].t()).split(D, -1)
    y = B.recurrence(x, r, i, leaves["A"], z, leaves["r_bias"], leaves["i_bias"], lens)[0]
    want = y @ leaves["out_proj"].t()
    bound = 8 * 2.0 ** -4 / 3 ** 0.5
    assert off(out, want.detach()) <= bound and off(total, t.detach()) <= 2.0 ** -8
    loss = (want * dout.double()).sum() + (t * dtot.double()).sum()
    grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    assert set(g) == set(grads)
    for k in grads:
        assert off(g[k], grads[k]) <= bound, (k, off(g[k], grads[k]))


def test_both_blocks_on_one_stream():
    gen = torch.Generator(device=DEV).manual_seed(1)
    first = GatedBlock.random(128, 192, 16, generator=gen, four_bit=True)
    second = RecurrentBlock.random(128, 192, generator=gen, four_bit=True)
    start = torch.tensor([0, 11, 12, 40], dtype=torch.int32, device=DEV)
    u = torch.randn(40, 128, device=DEV, generator=gen).to(torch.bfloat16)
    out, states = first.prompt(u, start)
    out, total, states2 = second.prompt(out, start, residual=u)
    assert out.shape == total.shape == u.shape
    token = out[-3:] + total[-3:]
    for _ in range(3):
        out = first.step(token, states)
        out, total = second.step(out, states2, residual=token)
        token = out + total
    assert token.shape == (3, 128) and token.isfinite().all()


def test_command(capsys):
    gated_block.main()
    assert capsys.readouterr().out.count("training step") == 2


@pytest.mark.parametrize("kind", ["gated", "recurrent"])
def test_tokens_take_a_projection_that_was_replaced(kind):
    """New weights on a block, as after a training step: single tokens take them too."""
    def block():
        gen = torch.Generator(device=DEV).manual_seed(9)
        return GatedBlock.random(128, 192, 16, generator=gen) if kind == "gated" else RecurrentBlock.random(128, 192, generator=gen)

    gen = torch.Generator(device=DEV).manual_seed(10)
    one = block()
    u = torch.randn(5, 128, device=DEV, generator=gen).to(torch.bfloat16)
    weight = torch.randn(128, 192, device=DEV, generator=gen) * 192 ** -0.5

    def step(b):
        y = b.step(u, b.states(5))
        return y if kind == "gated" else y[0]

    before = step(one)
    one.out_proj = Fp8Linear(-weight)
    after = step(one)
    one.out_proj = Fp8Linear(weight)
    assert torch.equal(step(one), -after) and not torch.equal(after, before)
