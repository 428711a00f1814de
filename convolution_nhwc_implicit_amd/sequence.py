"""The sequence operators: ctypes binding of the C ABI in include/sequence_ops.h.

``causal_conv`` and ``selective_scan`` with their gradients (``*_grad``) and
their single-token forms on pooled states (``*_step``), and the block-scaled
fp8 products (``fp8_quantize``, ``fp8_matmul``).  As in the convolution's
binding, Python checks the arguments and allocates outputs and workspaces on
the current stream; the computation runs in the HIP kernels.  The step forms
write their states in place.

Shapes.  Tensors of tokens are [B][L][...] (a dense batch of sequences of one
length), [T][...] (one sequence), or [T][...] with ``seq_start`` (int32,
[seqs + 1], on the GPU): sequences packed end to end, sequence s in rows
seq_start[s] to seq_start[s + 1] - 1.  They need unit stride over their last
axis and may be slices of a wider projection's output.  ``seq_start`` is not
read on the host: it must rise from 0 to T; rows outside every sequence stay
unspecified.
"""
import ctypes

import torch

from . import binding
from .binding import CONV2D_DTYPE_BF16, CONV2D_DTYPE_F16, Conv2dError

CONV2D_DTYPE_F32 = 3
_CODE = {torch.float16: CONV2D_DTYPE_F16, torch.bfloat16: CONV2D_DTYPE_BF16, torch.float32: CONV2D_DTYPE_F32}

_i, _ll, _vp, _sz = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_size_t


class SeqBatch(ctypes.Structure):
    _fields_ = [("seq_start", _vp), ("seqs", _i), ("len", _i), ("tokens", _ll)]


class SeqStride(ctypes.Structure):
    _fields_ = [("row", _ll), ("seq", _ll)]


class CausalConvProblem(ctypes.Structure):
    _fields_ = [("batch", SeqBatch), ("d", _i), ("w", _i), ("silu", _i), ("x", SeqStride), ("dy", SeqStride)]


class CausalConvStepProblem(ctypes.Structure):
    _fields_ = [(f, _i) for f in ("rows", "pool", "d", "w", "silu")] + [("x_row", _ll)]


class SelectiveScanProblem(ctypes.Structure):
    _fields_ = ([("batch", SeqBatch)] + [(f, _i) for f in ("d", "n", "groups", "softplus")] +
                [(f, SeqStride) for f in ("x", "dt", "B", "C", "z", "dy")] + [("b_group", _ll), ("c_group", _ll)])


class SelectiveScanGrads(ctypes.Structure):
    _fields_ = [(f, _vp) for f in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinitial")]


class SelectiveScanStepProblem(ctypes.Structure):
    _fields_ = ([(f, _i) for f in ("rows", "pool", "d", "n", "groups", "softplus")] +
                [(f, _ll) for f in ("x_row", "dt_row", "b_row", "c_row", "z_row", "b_group", "c_group")])


class Fp8MatmulProblem(ctypes.Structure):
    _fields_ = [(f, _i) for f in ("m", "n", "k", "b_blocks")] + [("a_pitch", _ll), ("b_pitch", _ll)]


FP8_ROWS, FP8_TRANSPOSE, FP8_BLOCKS = 0, 1, 2
FP8_BLOCK = 128  # values along the summed axis that share a scale

_P = ctypes.POINTER
_SIGNATURES = {
    "causal_conv": [_P(CausalConvProblem), _i] + [_vp] * 7,
    "causal_conv_grad_workspace_size": [_P(CausalConvProblem), _i, _P(_sz)],
    "causal_conv_grad": [_P(CausalConvProblem), _i] + [_vp] * 11 + [_sz, _vp],
    "causal_conv_step": [_P(CausalConvStepProblem), _i] + [_vp] * 7,
    "selective_scan_workspace_size": [_P(SelectiveScanProblem), _i, _P(_sz)],
    "selective_scan": [_P(SelectiveScanProblem), _i] + [_vp] * 12 + [_sz, _vp],
    "selective_scan_grad_workspace_size": [_P(SelectiveScanProblem), _i, _P(_sz)],
    "selective_scan_grad": [_P(SelectiveScanProblem), _i] + [_vp] * 11 + [_P(SelectiveScanGrads), _vp, _sz, _vp],
    "selective_scan_step": [_P(SelectiveScanStepProblem), _i] + [_vp] * 12,
    "fp8_quantize": [_i, _i, _i, _i, _vp, _ll, _vp, _ll, _vp, _vp],
    "fp8_matmul_workspace_size": [_P(Fp8MatmulProblem), _i, _P(_sz)],
    "fp8_matmul": [_P(Fp8MatmulProblem), _i] + [_vp] * 6 + [_sz, _vp],
}
_lib = None


def load():
    """The library, with the sequence operators' signatures set."""
    global _lib
    if _lib is None:
        lib = binding.load()
        for name, args in _SIGNATURES.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, ctypes.c_int
        _lib = lib
    return _lib


# ------------------------------------------------------------------ arguments

def _tensor(t, name, dtype, shape, device=None):
    """A GPU tensor of this type and shape with unit stride over its last axis."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride over its last axis")


def _dense(t, name, dtype, shape, device):
    if t is None:
        return None
    _tensor(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _float(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {t.dtype}")
    return code


def _ptr(t):
    return None if t is None else t.data_ptr()


def _int32(t, name, count, device):
    if t is None:
        return None
    _tensor(t, name, torch.int32, None, device)
    if t.dim() != 1 or (count is not None and t.shape[0] != count):
        raise ValueError(f"{name} must be a vector" + ("" if count is None else f" of {count}"))
    return t.data_ptr()


def _batch(lead, seq_start, device):
    """The sequences of tensors [*lead][...]; (seq_batch, number of sequences)."""
    if seq_start is not None:
        if len(lead) != 1:
            raise ValueError("with seq_start, tokens lie along one axis")
        p = _int32(seq_start, "seq_start", None, device)
        if seq_start.shape[0] < 2:
            raise ValueError("seq_start must have an entry for every sequence and one more")
        return SeqBatch(p, seq_start.shape[0] - 1, 0, lead[0]), seq_start.shape[0] - 1
    if len(lead) == 1:
        return SeqBatch(None, 1, lead[0], lead[0]), 1
    if len(lead) != 2:
        raise ValueError("tokens must lie along one axis, or along two as [sequences][tokens]")
    if lead[0] < 1:
        raise ValueError("there must be at least one sequence")
    return SeqBatch(None, lead[0], lead[1], lead[0] * lead[1]), lead[0]


def _strides(t, lead):
    """Strides over tokens and sequences; an axis of one element has any stride."""
    row = t.stride(len(lead) - 1) if lead[-1] > 1 else 0
    return SeqStride(row, t.stride(0) if len(lead) == 2 and lead[0] > 1 else 0)


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else 0


class _On:
    """The tensors' device made current, where it is not."""

    def __init__(self, device):
        self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _raise(status, where):
    if status:
        raise Conv2dError(status, where)


def _workspace(fn, prob, code, device):
    n = _sz()
    _raise(getattr(load(), fn)(prob, code, n), fn)
    return (torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None), n.value


# ------------------------------------------------------------ causal convolution

def _conv_problem(x, weight, bias, silu, initial_state, seq_start):
    code = _float(x, "x")
    if x.dim() < 2:
        raise ValueError("x must be [tokens][d] or [sequences][tokens][d]")
    lead, d, dev = x.shape[:-1], x.shape[-1], x.device
    _tensor(x, "x", x.dtype, None)
    if weight.dim() != 2:
        raise ValueError("weight must be [d][w]")
    w = weight.shape[1]
    _dense(weight, "weight", x.dtype, (d, w), dev)
    _dense(bias, "bias", x.dtype, (d,), dev)
    batch, seqs = _batch(lead, seq_start, dev)
    _dense(initial_state, "initial_state", x.dtype, (seqs, w - 1, d), dev)
    return CausalConvProblem(batch, d, w, int(bool(silu)), _strides(x, lead)), code, (seqs, w - 1, d)


def causal_conv(x, weight, bias=None, silu=False, initial_state=None, seq_start=None, return_state=False):
    """y[t][c] = act(bias[c] + sum_k weight[c][k] x[t - (w-1) + k][c]) within each sequence.

    x [..][d]; weight [d][w], 2 <= w <= 4; bias [d]; act is SiLU or nothing.  Rows before a
    sequence's first come from initial_state [seqs][w-1][d] (oldest first), or are zero.  With
    return_state the result is (y, final_state), the last w-1 rows each sequence has seen."""
    prob, code, sshape = _conv_problem(x, weight, bias, silu, initial_state, seq_start)
    with _On(x.device) as stream:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        state = torch.empty(sshape, dtype=x.dtype, device=x.device) if return_state else None
        _raise(load().causal_conv(prob, code, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state),
                                  y.data_ptr(), _ptr(state), stream), "causal_conv")
    return (y, state) if return_state else y


def causal_conv_grad(dy, x, weight, bias=None, silu=False, initial_state=None, seq_start=None, dfinal_state=None):
    """Gradients of causal_conv for the output gradient dy (and that of the returned state, if given):
    a dict of dx, dw, db (None without bias) and dinitial_state (None without initial_state), in x's type,
    each rounded once from fp32 sums."""
    prob, code, sshape = _conv_problem(x, weight, bias, silu, initial_state, seq_start)
    dev = x.device
    _tensor(dy, "dy", x.dtype, x.shape, dev)
    _dense(dfinal_state, "dfinal_state", x.dtype, sshape, dev)
    prob.dy = _strides(dy, x.shape[:-1])
    with _On(dev) as stream:
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
        dw = torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        dinit = None if initial_state is None else torch.empty_like(initial_state)
        ws, need = _workspace("causal_conv_grad_workspace_size", prob, code, dev)
        _raise(load().causal_conv_grad(prob, code, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), _ptr(bias),
                                       _ptr(initial_state), _ptr(dfinal_state), dx.data_ptr(), dw.data_ptr(),
                                       _ptr(db), _ptr(dinit), _ptr(ws), need, stream), "causal_conv_grad")
    return {"dx": dx, "dw": dw, "db": db, "dinitial_state": dinit}


def causal_conv_step(x, state, weight, bias=None, silu=False, slots=None):
    """causal_conv for one token per request: x [rows][d], state [pool][w-1][d] (updated in place),
    slots [rows] int32 the requests' places in the pool (default: row r has place r).  Rows with a
    slot outside the pool give zeros and touch nothing; no place may appear twice."""
    code = _float(x, "x")
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be [rows][d], weight [d][w] and state [pool][w-1][d]")
    (rows, d), w, pool, dev = x.shape, weight.shape[1], state.shape[0], x.device
    _tensor(x, "x", x.dtype, None)
    _dense(weight, "weight", x.dtype, (d, w), dev)
    _dense(bias, "bias", x.dtype, (d,), dev)
    _dense(state, "state", x.dtype, (pool, w - 1, d), dev)
    if slots is None and rows > pool:
        raise ValueError("without slots, state must have a place for every row")
    sp = _int32(slots, "slots", rows, dev)
    prob = CausalConvStepProblem(rows, pool, d, w, int(bool(silu)), _row_stride(x))
    with _On(dev) as stream:
        y = torch.empty((rows, d), dtype=x.dtype, device=dev)
        _raise(load().causal_conv_step(prob, code, x.data_ptr(), state.data_ptr(), weight.data_ptr(), _ptr(bias),
                                       sp, y.data_ptr(), stream), "causal_conv_step")
    return y


# ---------------------------------------------------------------- selective scan

def _scan_sizes(x, dt, A, B, C, D, z, dt_bias):
    code = _float(x, "x")
    if x.dim() < 2 or A.dim() != 2 or B.dim() < 3:
        raise ValueError("x must be [tokens][d] or [sequences][tokens][d], A [d][n] and B [tokens][groups][n] likewise")
    lead, d, dev, typ = x.shape[:-1], x.shape[-1], x.device, x.dtype
    n, groups = A.shape[1], B.shape[-2]
    _tensor(x, "x", typ, None)
    _tensor(dt, "dt", typ, x.shape, dev)
    for t, name in ((B, "B"), (C, "C")):
        _tensor(t, name, typ, lead + (groups, n), dev)
    if z is not None:
        _tensor(z, "z", typ, x.shape, dev)
    _dense(A, "A", torch.float32, (d, n), dev)
    _dense(D, "D", torch.float32, (d,), dev)
    _dense(dt_bias, "dt_bias", torch.float32, (d,), dev)
    if groups < 1 or d % groups:
        raise ValueError(f"the {groups} groups of B must divide the {d} channels")
    return code, lead, d, n, groups


def _group_stride(t, groups):
    return t.stride(-2) if groups > 1 else 0


def _scan_problem(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seq_start):
    code, lead, d, n, groups = _scan_sizes(x, dt, A, B, C, D, z, dt_bias)
    batch, seqs = _batch(lead, seq_start, x.device)
    _dense(initial_state, "initial_state", torch.float32, (seqs, d, n), x.device)
    prob = SelectiveScanProblem(batch, d, n, groups, int(bool(softplus)), _strides(x, lead), _strides(dt, lead),
                                _strides(B, lead), _strides(C, lead),
                                SeqStride() if z is None else _strides(z, lead), SeqStride(),
                                _group_stride(B, groups), _group_stride(C, groups))
    return prob, code, (seqs, d, n)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False, initial_state=None,
                   seq_start=None, return_state=False):
    """h = exp(delta A) h + delta x B;  y = (sum over n of h C + D x) silu(z), token after token, with
    delta = softplus(dt + dt_bias) (or the sum itself).

    x, dt, z [..][d] and B, C [..][groups][n] in one type, A [d][n], D [d], dt_bias [d] and the states
    [seqs][d][n] in float32; channel c belongs to group c // (d / groups); n <= 64.  With return_state
    the result is (y, final_state)."""
    prob, code, sshape = _scan_problem(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seq_start)
    dev = x.device
    with _On(dev) as stream:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
        state = torch.empty(sshape, dtype=torch.float32, device=dev) if return_state else None
        ws, need = _workspace("selective_scan_workspace_size", prob, code, dev)
        _raise(load().selective_scan(prob, code, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
                                     C.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(initial_state),
                                     y.data_ptr(), _ptr(state), _ptr(ws), need, stream), "selective_scan")
    return (y, state) if return_state else y


def selective_scan_grad(dy, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False, initial_state=None,
                        seq_start=None, dfinal_state=None):
    """Gradients of selective_scan for the output gradient dy (and that of the returned state, if given):
    a dict of du (of x), ddt, dB, dC, dz in x's type and dA, dD, ddt_bias, dinitial_state in float32;
    None where the input is None.  The forward pass is computed again, not kept."""
    prob, code, sshape = _scan_problem(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seq_start)
    dev, typ = x.device, x.dtype
    _tensor(dy, "dy", typ, x.shape, dev)
    _dense(dfinal_state, "dfinal_state", torch.float32, sshape, dev)
    prob.dy = _strides(dy, x.shape[:-1])
    with _On(dev) as stream:
        def like(t):
            return None if t is None else torch.empty(t.shape, dtype=t.dtype, device=dev)

        g = {"du": like(x), "ddt": like(dt), "dA": like(A), "dB": like(B), "dC": like(C), "dD": like(D),
             "dz": like(z), "ddt_bias": like(dt_bias), "dinitial_state": like(initial_state)}
        ws, need = _workspace("selective_scan_grad_workspace_size", prob, code, dev)
        out = SelectiveScanGrads(*[_ptr(g[k]) for k in g])
        _raise(load().selective_scan_grad(prob, code, dy.data_ptr(), x.data_ptr(), dt.data_ptr(), A.data_ptr(),
                                          B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias),
                                          _ptr(initial_state), _ptr(dfinal_state), out, _ptr(ws), need, stream),
               "selective_scan_grad")
    return g


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus=False, slots=None):
    """selective_scan for one token per request: x, dt, z [rows][d], B, C [rows][groups][n], state
    [pool][d][n] float32 (updated in place), slots as for causal_conv_step."""
    code, lead, d, n, groups = _scan_sizes(x, dt, A, B, C, D, z, dt_bias)
    if len(lead) != 1 or state.dim() != 3:
        raise ValueError("x must be [rows][d] and state [pool][d][n]")
    rows, pool, dev = lead[0], state.shape[0], x.device
    sp_state = _dense(state, "state", torch.float32, (pool, d, n), dev)
    if slots is None and rows > pool:
        raise ValueError("without slots, state must have a place for every row")
    sp = _int32(slots, "slots", rows, dev)
    prob = SelectiveScanStepProblem(rows, pool, d, n, groups, int(bool(softplus)), _row_stride(x), _row_stride(dt),
                                    _row_stride(B), _row_stride(C), 0 if z is None else _row_stride(z),
                                    _group_stride(B, groups), _group_stride(C, groups))
    with _On(dev) as stream:
        y = torch.empty((rows, d), dtype=x.dtype, device=dev)
        _raise(load().selective_scan_step(prob, code, x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
                                          C.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias), sp_state, sp,
                                          y.data_ptr(), stream), "selective_scan_step")
    return y


# ------------------------------------------------------------ block-scaled fp8 products

def _blocks(v):
    return -(-v // FP8_BLOCK)


def fp8_quantize(x, transpose=False, blocks=False):
    """x [m][k] to e4m3 with a scale for every 128 values of a row: (q [m][k], scale [m][ceil(k/128)]).

    transpose: of x's transpose, q [k][m] and scale [k][ceil(m/128)].  blocks: a scale for every 128 x 128
    values (weights), scale [ceil(m/128)][ceil(k/128)].  Scales are the least powers of two (at least 2^-126)
    that bring a block's finite values into e4m3's range; infinities and NaN become NaN.  q's rows are padded
    with zeros to a multiple of 16 bytes; q is a view of them."""
    code = _float(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [m][k]")
    if transpose and blocks:
        raise ValueError("blocks of 128 x 128 are quantised as they lie")
    _tensor(x, "x", x.dtype, None)
    (m, k), dev = x.shape, x.device
    rows, cols = (k, m) if transpose else (m, k)
    pitch = -(-cols // 16) * 16
    form = FP8_TRANSPOSE if transpose else FP8_BLOCKS if blocks else FP8_ROWS
    with _On(dev) as stream:
        q = torch.empty((rows, pitch), dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty((_blocks(rows) if blocks else rows, _blocks(cols)), dtype=torch.float32, device=dev)
        _raise(load().fp8_quantize(form, code, m, k, x.data_ptr(), _row_stride(x), q.data_ptr(), pitch,
                                   scale.data_ptr(), stream), "fp8_quantize")
    return (q if pitch == cols else q[:, :cols]), scale


def _fp8_operand(q, scale, name, rows):
    _tensor(q, name, torch.float8_e4m3fn, None)
    if q.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    kb = _blocks(q.shape[1])
    blocks = rows == "blocks" and q.shape[0] != 1 and scale.shape[0] != q.shape[0]
    _dense(scale, f"{name}_scale", torch.float32, (_blocks(q.shape[0]) if blocks else q.shape[0], kb), q.device)
    pitch = q.stride(0) if q.shape[0] > 1 and q.shape[1] > 0 else -(-q.shape[1] // 16) * 16
    if pitch % 16 or pitch < q.shape[1]:
        raise ValueError(f"{name}'s rows must start on 16-byte steps (fp8_quantize lays them out so)")
    return pitch, blocks


def fp8_matmul(a, a_scale, b, b_scale, out_dtype=torch.bfloat16):
    """a times b's transpose: out [m][n] in out_dtype (float16, bfloat16 or float32) of e4m3 operands a [m][k]
    and b [n][k] with float32 scales of 128 values along k: a_scale [m][ceil(k/128)], and b_scale
    [n][ceil(k/128)] or [ceil(n/128)][ceil(k/128)].  Scales may be any values; powers of two cost no time.
    Sums are float32, rounded once."""
    a_pitch, _ = _fp8_operand(a, a_scale, "a", "rows")
    b_pitch, blocks = _fp8_operand(b, b_scale, "b", "blocks")
    (m, k), n, dev = a.shape, b.shape[0], a.device
    if b.shape[1] != k or b.device != dev:
        raise ValueError(f"b must be [n][{k}] on {dev}, got {tuple(b.shape)} on {b.device}")
    code = _CODE.get(out_dtype)
    if code is None:
        raise TypeError(f"out_dtype must be float16, bfloat16 or float32, got {out_dtype}")
    prob = Fp8MatmulProblem(m, n, k, int(blocks), a_pitch, b_pitch)
    with _On(dev) as stream:
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
        ws, need = _workspace("fp8_matmul_workspace_size", prob, code, dev)
        _raise(load().fp8_matmul(prob, code, a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr(),
                                 out.data_ptr(), _ptr(ws), need, stream), "fp8_matmul")
    return out
