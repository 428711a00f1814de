"""The sequence operators on torch tensors.

``causal_conv``, ``selective_scan`` and ``gated_recurrence`` with their gradients
(``*_grad``) and their single-token forms on pooled states (``*_step``),
``layer_norm`` with its gradients, the block-scaled fp8 products
(``fp8_quantize``, ``fp8_matmul``) and products with 4-bit weights
(``fp4_quantize``, ``fp4_matmul``).  The native module _sequence
checks the arguments, allocates outputs and workspaces on the current stream
and calls the C ABI in include/sequence_ops.h; the computation runs in the HIP
kernels of libconv2d_nhwc.so.  The step forms write their states in place.

Shapes.  Tensors of tokens are [B][L][...] (a dense batch of sequences of one
length), [T][...] (one sequence), or [T][...] with ``seq_start`` (int32,
[seqs + 1], on the GPU): sequences packed end to end, sequence s in rows
seq_start[s] to seq_start[s + 1] - 1.  They need unit stride over their last
axis and may be slices of a wider projection's output.  ``seq_start`` is not
read on the host: it must rise from 0 to T; rows outside every sequence stay
unspecified.

Gradients are calls of their own: results carry no autograd history.  With
gradients enabled, an input that requires one draws a UserWarning.

Wrong types raise TypeError, wrong shapes, strides and devices ValueError, and
what the kernels do not support Conv2dError, before anything is enqueued.
"""
import importlib.util
import os

import torch

from . import binding

MODULE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_sequence.so")

_module = None


def load():
    """The native module (raises if it has not been built)."""
    global _module
    if _module is None:
        binding.load()
        if not os.path.exists(MODULE_PATH):
            raise RuntimeError(f"{MODULE_PATH} is missing: build it with "
                               "`python -m convolution_nhwc_implicit_amd.build`")
        spec = importlib.util.spec_from_file_location("_sequence", MODULE_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _module = module
    return _module


# ------------------------------------------------------------ causal convolution

def causal_conv(x, weight, bias=None, silu=False, initial_state=None, seq_start=None, return_state=False):
    """y[t][c] = act(bias[c] + sum_k weight[c][k] x[t - (w-1) + k][c]) within each sequence.

    x [..][d]; weight [d][w], 2 <= w <= 4; bias [d]; act is SiLU or nothing.  Rows before a
    sequence's first come from initial_state [seqs][w-1][d] (oldest first), or are zero.  With
    return_state the result is (y, final_state), the last w-1 rows each sequence has seen."""
    return load().causal_conv(x, weight, bias, silu, initial_state, seq_start, return_state)


def causal_conv_grad(dy, x, weight, bias=None, silu=False, initial_state=None, seq_start=None, dfinal_state=None):
    """Gradients of causal_conv for the output gradient dy (and that of the returned state, if given):
    a dict of dx, dw, db (None without bias) and dinitial_state (None without initial_state), in x's type,
    each rounded once from fp32 sums."""
    return load().causal_conv_grad(dy, x, weight, bias, silu, initial_state, seq_start, dfinal_state)


def causal_conv_step(x, state, weight, bias=None, silu=False, slots=None):
    """causal_conv for one token per request: x [rows][d], state [pool][w-1][d] (updated in place),
    slots [rows] int32 the requests' places in the pool (default: row r has place r).  Rows with a
    slot outside the pool give zeros and touch nothing; no place may appear twice."""
    return load().causal_conv_step(x, state, weight, bias, silu, slots)


# ---------------------------------------------------------------- selective scan

def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False, initial_state=None,
                   seq_start=None, return_state=False):
    """h = exp(delta A) h + delta x B;  y = (sum over n of h C + D x) silu(z), token after token, with
    delta = softplus(dt + dt_bias) (or the sum itself).

    x, dt, z [..][d] and B, C [..][groups][n] in one type, A [d][n], D [d], dt_bias [d] and the states
    [seqs][d][n] in float32; channel c belongs to group c // (d / groups); n <= 64, fastest up to 16.
    Rates of A past 2e38 in size (infinite ones) count as 2e38.  With return_state the result is
    (y, final_state)."""
    return load().selective_scan(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seq_start, return_state)


def selective_scan_grad(dy, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False, initial_state=None,
                        seq_start=None, dfinal_state=None):
    """Gradients of selective_scan for the output gradient dy (and that of the returned state, if given):
    a dict of du (of x), ddt, dB, dC, dz in x's type and dA, dD, ddt_bias, dinitial_state in float32;
    None where the input is None.  The forward pass is computed again, not kept."""
    return load().selective_scan_grad(dy, x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seq_start,
                                      dfinal_state)


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus=False, slots=None):
    """selective_scan for one token per request: x, dt, z [rows][d], B, C [rows][groups][n], state
    [pool][d][n] float32 (updated in place), slots as for causal_conv_step."""
    return load().selective_scan_step(x, dt, A, B, C, D, z, dt_bias, state, softplus, slots)


# -------------------------------------------------------------- gated recurrence

def gated_recurrence(x, r, i, A, z=None, r_bias=None, i_bias=None, initial_state=None, seq_start=None,
                     return_state=False):
    """a = exp(A sigmoid(r + r_bias));  h = a h + sqrt(1 - a^2) sigmoid(i + i_bias) x;  y = h silu(z) (without z: h),
    token after token and channel by channel.

    x, r, i, z [..][d] in one type; A (log decays, at most 0), r_bias, i_bias [d] and the states [seqs][d] in float32.
    Positive A gives NaN; rates below -2e38 count as -2e38, those nearer to 0 than 2^-126 as 0. With return_state the result is (y, final_state)."""
    return load().gated_recurrence(x, r, i, A, z, r_bias, i_bias, initial_state, seq_start, return_state)


def gated_recurrence_grad(dy, x, r, i, A, z=None, r_bias=None, i_bias=None, initial_state=None, seq_start=None,
                          dfinal_state=None):
    """Gradients of gated_recurrence for the output gradient dy (and that of the returned state, if given): a dict of
    dx, dr, di, dz in x's type and dA, dr_bias, di_bias, dinitial_state in float32; None where the input is None.
    The forward pass is computed again, not kept. dA is 0 where A is 0 (the square root has no derivative there)."""
    return load().gated_recurrence_grad(dy, x, r, i, A, z, r_bias, i_bias, initial_state, seq_start, dfinal_state)


def gated_recurrence_step(x, r, i, A, state, z=None, r_bias=None, i_bias=None, slots=None):
    """gated_recurrence for one token per request: x, r, i, z [rows][d], state [pool][d] float32 (updated in place),
    slots as for causal_conv_step."""
    return load().gated_recurrence_step(x, r, i, A, z, r_bias, i_bias, state, slots)


# -------------------------------------------------------------------- layer norm

def layer_norm(x, weight=None, bias=None, eps=1e-5, residual=None):
    """y = (t - mean) / sqrt(var + eps) * weight + bias over the last axis, of t = x, or of t = x + residual: then the
    result is (y, total) with total = t in x's type. y comes from the unrounded sum, statistics are float32.

    x, residual [tokens][d] or [sequences][tokens][d]; weight and bias [d] in x's type or both in float32."""
    return load().layer_norm(x, weight, bias, eps, residual)


def layer_norm_grad(dy, x, weight=None, bias=None, eps=1e-5, dtotal=None):
    """Gradients of layer_norm at t = x (its total, where there was a residual) for the output gradient dy: a dict of
    dx in x's type (also the residual's gradient; dtotal, the gradient that reaches total on other ways, is added to
    it) and dw, db in the parameters' type (None where the parameter is None)."""
    return load().layer_norm_grad(dy, x, weight, bias, eps, dtotal)


# ------------------------------------------------------------ block-scaled fp8 products

def fp8_quantize(x, transpose=False, blocks=False):
    """x [m][k] to e4m3 with a scale for every 128 values of a row: (q [m][k], scale [m][ceil(k/128)]).

    transpose: of x's transpose, q [k][m] and scale [k][ceil(m/128)].  blocks: a scale for every 128 x 128
    values (weights), scale [ceil(m/128)][ceil(k/128)].  Scales are the least powers of two (at least 2^-126)
    that bring a block's finite values into e4m3's range (2^-126 for a block of zeros, which costs fp8_matmul
    time); infinities and NaN become NaN.  q's rows are padded with zeros to a multiple of 128 bytes; q is a
    view of them."""
    return load().fp8_quantize(x, transpose, blocks)


def fp8_matmul(a, a_scale, b, b_scale, out_dtype=torch.bfloat16):
    """a times b's transpose: out [m][n] in out_dtype (float16, bfloat16 or float32) of e4m3 operands a [m][k]
    and b [n][k] with float32 scales of 128 values along k: a_scale [m][ceil(k/128)], and b_scale
    [n][ceil(k/128)] or [ceil(n/128)][ceil(k/128)].  Scales may be any values; powers of two from 2^-62 to 2^62
    cost no time, others more than double it.  Sums are float32, rounded once; for a 16-bit result the fp8 matrix unit
    cuts each group of 8 neighbouring products at 2^-13 of its largest, below the result's own rounding (a float32
    result has no such cut, and may be rounded afterwards)."""
    return load().fp8_matmul(a, a_scale, b, b_scale, out_dtype)


# ---------------------------------------------------------------- 4-bit products

def fp4_quantize(x):
    """x [m][k] to e2m1 values with a power-of-two scale for every 32 values of a row: (q [m][ceil(k/2)], scale
    [m][ceil(k/32)]), both uint8. Byte j of a row of q holds values 2j (low half) and 2j + 1; a scale byte e stands for
    2^(e - 127). Scales are the least that bring a group's values into e2m1's range; a group with an infinity or a NaN
    becomes NaN (e = 255). q's rows are padded with zeros to whole groups; q is a view of them."""
    return load().fp4_quantize(x)


def fp4_matmul(x, w, w_scale):
    """x times w's transpose: out [m][n] in x's type, of x [m][k] in float16, bfloat16 or float32 and 4-bit w (as
    fp4_quantize makes it: [n][ceil(k/2)], w_scale [n][ceil(k/32)]). Products are exact, sums float32, rounded once.
    Made for few rows of x (new tokens), where the weights' bytes are what there is to do; for many rows fp8_matmul is
    faster."""
    return load().fp4_matmul(x, w, w_scale)
