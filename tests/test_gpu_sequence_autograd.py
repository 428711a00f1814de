"""The sequence operators beside autograd: inputs that require a gradient are not dropped without a word, and states
that a step writes in place count as written."""
import warnings

import pytest
import torch

import convolution_nhwc_implicit_amd as nn

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def t(*shape, dtype=torch.float32):
    return torch.full(shape, 0.5, device=DEV).to(dtype)


# the operator, its arguments, and which of them may require a gradient
CALLS = {
    "causal_conv": (dict(x=t(5, 8), weight=t(8, 4), bias=t(8)), ("x", "weight", "bias")),
    "causal_conv_step": (dict(x=t(2, 8), state=t(2, 3, 8), weight=t(8, 4)), ("x", "weight")),
    "selective_scan": (dict(x=t(5, 8), dt=t(5, 8), A=-t(8, 4), B=t(5, 1, 4), C=t(5, 1, 4), D=t(8), z=t(5, 8)),
                       ("x", "dt", "A", "B", "C", "D", "z")),
    "selective_scan_step": (dict(x=t(2, 8), dt=t(2, 8), A=-t(8, 4), B=t(2, 1, 4), C=t(2, 1, 4), state=t(2, 8, 4)), ("x", "A")),
    "fp8_quantize": (dict(x=t(5, 8)), ("x",)),
    "fp8_matmul": (dict(a=t(5, 16, dtype=E4M3), a_scale=t(5, 1), b=t(7, 16, dtype=E4M3), b_scale=t(7, 1)), ("a_scale", "b_scale")),
} if torch.cuda.is_available() else {}


@pytest.mark.parametrize("name", ["causal_conv", "causal_conv_step", "selective_scan", "selective_scan_step", "fp8_quantize",
                                  "fp8_matmul"])
def test_inputs_that_require_a_gradient(name):
    args, leaves = CALLS[name]
    fn = getattr(nn, name)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        want = fn(**args)  # without such inputs: no warning
        for leaf in leaves:
            given = {**args, leaf: args[leaf].clone().requires_grad_()}
            with torch.no_grad():
                fn(**given)
            with torch.inference_mode():
                fn(**given)
            with pytest.raises(UserWarning, match=f"{name}: {leaf} requires a gradient"):
                fn(**given)
    if "state" in args:
        return
    with pytest.warns(UserWarning) as seen:
        got = fn(**given)
    assert seen[0].filename == __file__  # the caller's line
    for u, v in zip(*(r if isinstance(r, tuple) else (r,) for r in (want, got))):
        assert torch.equal(u.float(), v.float()) and not v.requires_grad


def test_gradient_calls_take_parameters():
    args, _ = CALLS["selective_scan"]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        given = {k: v.clone().requires_grad_() for k, v in args.items()}
        got = nn.selective_scan_grad(t(5, 8), **given)
        assert not any(v is not None and v.requires_grad for v in got.values())
        conv = {k: v.clone().requires_grad_() for k, v in CALLS["causal_conv"][0].items()}
        assert not nn.causal_conv_grad(t(5, 8), **conv)["dw"].requires_grad


@pytest.mark.parametrize("name", ["causal_conv_step", "selective_scan_step"])
def test_steps_count_as_writes(name):
    args, _ = CALLS[name]
    state = args["state"].clone()
    before = state._version
    view = state[:]
    getattr(nn, name)(**{**args, "state": state})
    assert state._version > before and view._version == state._version
    # what autograd saved of a state before a step is not used after it
    w = torch.ones_like(state, requires_grad=True)
    out = (w * state).sum()
    getattr(nn, name)(**{**args, "state": state})
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward()
    with torch.inference_mode():
        inner = state.clone()
        getattr(nn, name)(**{**args, "state": inner})
    getattr(nn, name)(**{**args, "state": inner})  # an inference tensor has no version
