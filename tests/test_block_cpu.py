"""Refusals of the gated recurrence, the layer norm and the 4-bit products, without a GPU: through Python (types, shapes,
strides, devices) and through the C ABI (status codes; every check runs before anything could be enqueued)."""
import ctypes as ct

import pytest
import torch

import block_ref as R
import convolution_nhwc_implicit_amd as nn
from test_sequence_cpu import (AT, BF16, BF16C, F16C, F32C, I8C, INVALID, LIB, OK, SMALL, UNSUPPORTED, Batch, P, Stride,
                               size, start)

U8 = torch.uint8


# ------------------------------------------------------------------------------------ through Python
def recur_args(**kw):
    a = dict(x=torch.zeros(2, 5, 8, dtype=BF16), r=torch.zeros(2, 5, 8, dtype=BF16), i=torch.zeros(2, 5, 8, dtype=BF16),
             A=torch.zeros(8), z=torch.zeros(2, 5, 8, dtype=BF16), r_bias=torch.zeros(8), i_bias=torch.zeros(8),
             initial_state=torch.zeros(2, 8))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err,text", [
    ({}, ValueError, "on the GPU"),
    (dict(x=5), TypeError, "x must be a torch.Tensor"),
    (dict(x=torch.zeros(2, 5, 8, dtype=torch.int32)), TypeError, "float16"),
    (dict(x=torch.zeros(8, dtype=BF16)), ValueError, "tokens"),
    (dict(r=torch.zeros(2, 5, 9, dtype=BF16)), ValueError, "r must have shape"),
    (dict(i=torch.zeros(2, 5, 8)), TypeError, "i must be torch.bfloat16"),
    (dict(i=torch.zeros(2, 8, 5, dtype=BF16).transpose(1, 2)), ValueError, "i must have unit stride"),
    (dict(z=torch.zeros(2, 4, 8, dtype=BF16)), ValueError, "z must have shape"),
    (dict(A=torch.zeros(8, dtype=BF16)), TypeError, "A must be torch.float32"),
    (dict(A=torch.zeros(8, 1)), ValueError, "A must have shape"),
    (dict(r_bias=torch.zeros(16)[::2]), ValueError, "r_bias must"),
    (dict(i_bias=torch.zeros(1)), ValueError, "i_bias must have shape"),
    (dict(initial_state=torch.zeros(3, 8)), ValueError, "initial_state must have shape"),
    (dict(initial_state=torch.zeros(2, 8, dtype=BF16)), TypeError, "initial_state must be torch.float32"),
    (dict(seq_start=start(0, 5)), ValueError, "one axis"),
    (dict(x=torch.zeros(0, 5, 8, dtype=BF16), r=torch.zeros(0, 5, 8, dtype=BF16), i=torch.zeros(0, 5, 8, dtype=BF16),
          z=None), ValueError, "at least one sequence"),
])
def test_recurrence_refusals(kw, err, text):
    with pytest.raises(err, match=text):
        nn.gated_recurrence(**recur_args(**kw))
    with pytest.raises(err, match=text):
        a = recur_args(**kw)
        nn.gated_recurrence_grad(a["x"].clone() if isinstance(a["x"], torch.Tensor) else torch.zeros(1), **a)


def test_recurrence_grad_and_step_refusals():
    with pytest.raises(ValueError, match="dy must have shape"):
        nn.gated_recurrence_grad(torch.zeros(2, 4, 8, dtype=BF16), **recur_args())
    with pytest.raises(TypeError, match="dy must be torch.bfloat16"):
        nn.gated_recurrence_grad(torch.zeros(2, 5, 8), **recur_args())
    with pytest.raises(ValueError, match="dfinal_state must have shape"):
        nn.gated_recurrence_grad(torch.zeros(2, 5, 8, dtype=BF16), dfinal_state=torch.zeros(2, 9), **recur_args())
    s = {k: (v[0] if v.dim() > 2 else v) for k, v in recur_args().items() if k != "initial_state"}
    for kw, err, text in ((dict(state=torch.zeros(4, 8)), ValueError, "place for every row"),
                          (dict(state=torch.zeros(5, 9)), ValueError, "state must have shape"),
                          (dict(state=torch.zeros(5, 8, dtype=BF16)), TypeError, "state must be torch.float32"),
                          (dict(state=torch.zeros(5, 16)[:, ::2]), ValueError, "state must"),
                          (dict(state=torch.zeros(5, 8), slots=start(0, 1)), ValueError, "slots must have shape"),
                          (dict(state=torch.zeros(5, 8), slots=torch.arange(5)), TypeError, "slots must be torch.int32"),
                          (dict(state=torch.zeros(5, 1, 8)), ValueError, r"state \[pool\]\[d\]"),
                          (dict(state=torch.zeros(5, 8)), ValueError, "on the GPU")):
        with pytest.raises(err, match=text):
            nn.gated_recurrence_step(**{**s, **kw})


def norm_args(**kw):
    a = dict(x=torch.zeros(2, 5, 8, dtype=BF16), weight=torch.zeros(8), bias=torch.zeros(8))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err,text", [
    ({}, ValueError, "on the GPU"),
    (dict(x=torch.zeros(8, dtype=BF16)), ValueError, "tokens"),
    (dict(x=torch.zeros(1, 2, 5, 8, dtype=BF16)), ValueError, "tokens"),
    (dict(x=torch.zeros(5, 0, dtype=BF16), weight=None, bias=None), ValueError, "at least one element"),
    (dict(x=torch.zeros(2, 5, 8, dtype=torch.int32)), TypeError, "float16"),
    (dict(x=torch.zeros(2, 8, 5, dtype=BF16).transpose(1, 2)), ValueError, "unit stride"),
    (dict(weight=torch.zeros(7)), ValueError, "weight must have shape"),
    (dict(weight=torch.zeros(8, dtype=torch.float16), bias=None), TypeError, "weight must be torch.bfloat16"),
    (dict(bias=torch.zeros(8, dtype=BF16)), TypeError, "bias must be torch.float32"),
    (dict(weight=torch.zeros(16)[::2]), ValueError, "weight must"),
    (dict(eps=-1e-6), ValueError, "eps"), (dict(eps=float("nan")), ValueError, "eps"), (dict(eps=float("inf")), ValueError, "eps"),
    (dict(eps=1e39), ValueError, "eps"), (dict(eps="x"), TypeError, "real number"),
])
def test_norm_refusals(kw, err, text):
    with pytest.raises(err, match=text):
        nn.layer_norm(**norm_args(**kw))
    with pytest.raises(err, match=text):
        nn.layer_norm_grad(norm_args(**kw)["x"].clone(), **norm_args(**kw))


def test_norm_companions():
    with pytest.raises(ValueError, match="residual must have shape"):
        nn.layer_norm(**norm_args(), residual=torch.zeros(2, 4, 8, dtype=BF16))
    with pytest.raises(TypeError, match="residual must be torch.bfloat16"):
        nn.layer_norm(**norm_args(), residual=torch.zeros(2, 5, 8))
    with pytest.raises(ValueError, match="dy must have shape"):
        nn.layer_norm_grad(torch.zeros(2, 5, 9, dtype=BF16), **norm_args())
    with pytest.raises(ValueError, match="dtotal must have shape"):
        nn.layer_norm_grad(torch.zeros(2, 5, 8, dtype=BF16), **norm_args(), dtotal=torch.zeros(5, 8, dtype=BF16))


def test_fp4_refusals():
    x = torch.zeros(3, 100, dtype=BF16)
    for v, err, text in ((x, ValueError, "on the GPU"), (x[0], ValueError, r"\[m\]\[k\]"), (x.t(), ValueError, "unit stride"),
                         (x.int(), TypeError, "float16"), (3, TypeError, "torch.Tensor")):
        with pytest.raises(err, match=text):
            nn.fp4_quantize(v)
    wide = torch.zeros(7, 64, dtype=U8)
    w, s = wide[:, :50], torch.zeros(7, 4, dtype=U8)
    for kw, err, text in ((dict(), ValueError, "on the GPU"), (dict(x=x[0]), ValueError, r"x must be \[m\]\[k\]"),
                          (dict(x=x.int()), TypeError, "float16"), (dict(w=w[:, :49]), ValueError, "w must have shape"),
                          (dict(w=w.float()), TypeError, "w must be"), (dict(w_scale=s[:, :3]), ValueError, "w_scale must have shape"),
                          (dict(w_scale=s.float()), TypeError, "w_scale must be"),
                          (dict(w_scale=torch.zeros(7, 8, dtype=U8)[:, ::2]), ValueError, "w_scale must"),
                          (dict(w=w.contiguous()), ValueError, "16-byte steps"),
                          (dict(w=torch.zeros(400, dtype=U8).as_strided((7, 50), (48, 1))), ValueError, "whole groups"),
                          # the last row's last group would end behind the memory
                          (dict(w=torch.zeros(6 * 64 + 50, dtype=U8).as_strided((7, 50), (64, 1))), ValueError, "whole groups")):
        v = {**dict(x=x, w=w, w_scale=s), **kw}
        with pytest.raises(err, match=text):
            nn.fp4_matmul(**v)


# ------------------------------------------------------------------------------------ through the C ABI
class Recur(ct.Structure):
    _fields_ = [("batch", Batch), ("d", ct.c_int)] + [(f, Stride) for f in ("x", "r", "i", "z", "dy")]


class RecurGrads(ct.Structure):
    _fields_ = [(f, ct.c_void_p) for f in ("dx", "dr", "di", "dA", "dz", "dr_bias", "di_bias", "dinitial")]


class RecurStep(ct.Structure):
    _fields_ = [(f, ct.c_int) for f in ("rows", "pool", "d")] + [(f, ct.c_longlong) for f in ("x_row", "r_row", "i_row", "z_row")]


class Norm(ct.Structure):
    _fields_ = [("seqs", ct.c_int), ("len", ct.c_int), ("d", ct.c_int), ("eps", ct.c_float)] + [
        (f, Stride) for f in ("x", "residual", "dy", "dtotal")]


class Fp4(ct.Structure):
    _fields_ = [(f, ct.c_int) for f in ("m", "n", "k")] + [("x_row", ct.c_longlong), ("w_pitch", ct.c_longlong)]


def put(p, kw):
    for k, v in kw.items():
        setattr(p.batch if hasattr(p, "batch") and hasattr(p.batch, k) else p, k, v)
    return p


def recur(**kw):
    s = Stride(8, 40)
    return put(Recur(Batch(None, 2, 5, 10), 8, s, s, s, s, s), kw)


@pytest.mark.parametrize("kw,dtype,want", [
    ({}, BF16C, OK), ({}, F32C, OK), ({}, I8C, UNSUPPORTED), ({}, 9, UNSUPPORTED), (dict(d=0), F16C, INVALID),
    (dict(seqs=0), F16C, INVALID), (dict(tokens=11), F16C, INVALID), (dict(len=-1), F16C, INVALID),
    (dict(r=Stride(-1, 0)), F16C, INVALID), (dict(i=Stride(8, -1)), F16C, INVALID), (dict(z=Stride(1 << 24, 0)), F16C, UNSUPPORTED),
    (dict(seqs=1 << 16, len=1 << 16, tokens=1 << 32), F16C, UNSUPPORTED), (dict(d=1 << 24), F16C, UNSUPPORTED),
    (dict(d=(1 << 24) - 1), F16C, OK),
    (dict(x=Stride(0, 0), r=Stride(0, 0)), F16C, OK), (dict(seqs=1, len=(1 << 31) - 1, tokens=(1 << 31) - 1), F16C, OK),
])
def test_recurrence_abi(kw, dtype, want):
    for fn in ("gated_recurrence_workspace_size", "gated_recurrence_grad_workspace_size"):
        status, n = size(fn, recur(**kw), dtype)
        assert status == want and (n == 12345) == (want != OK)


def test_recurrence_abi_pointers():
    p = recur(seqs=1, len=1 << 14, tokens=1 << 14)
    need = size("gated_recurrence_workspace_size", p, BF16C)[1]
    assert need > 0  # one long sequence is cut into chunks
    f, s = LIB.gated_recurrence, ct.c_size_t
    args = [ct.byref(p), BF16C, AT, AT, AT, AT, AT, None, None, None, AT, None]
    assert f(*args, AT, s(need - 1), None) == SMALL
    assert f(*args, None, s(0), None) == INVALID
    assert f(*args, P(8 + (1 << 20)), s(need), None) == UNSUPPORTED
    for k, bad, want in ((2, None, INVALID), (3, None, INVALID), (4, None, INVALID), (5, None, INVALID), (10, None, INVALID),
                         (0, None, INVALID), (3, P(1 + (1 << 20)), UNSUPPORTED), (5, P(2 + (1 << 20)), UNSUPPORTED),
                         (7, P(2 + (1 << 20)), UNSUPPORTED), (11, P(2 + (1 << 20)), UNSUPPORTED)):
        a = list(args)
        a[k] = bad
        assert f(*a, AT, s(need), None) == want
    need = size("gated_recurrence_grad_workspace_size", p, BF16C)[1]
    g = RecurGrads(*([1 << 20] * 8))
    args = [ct.byref(p), BF16C, AT, AT, AT, AT, AT, AT, None, None, None, None, ct.byref(g)]
    f = LIB.gated_recurrence_grad
    assert f(*args, AT, s(need - 1), None) == SMALL and f(*args, None, s(need), None) == INVALID
    for name in ("dx", "dr", "di", "dA", "dz"):
        bad = RecurGrads(*([1 << 20] * 8))
        setattr(bad, name, None)
        assert f(*args[:-1], ct.byref(bad), AT, s(need), None) == INVALID


def test_recurrence_step_abi():
    f = LIB.gated_recurrence_step

    def call(p, dtype=F16C, **kw):
        a = dict(x=AT, r=AT, i=AT, A=AT, z=None, rb=None, ib=None, state=AT, slots=None, y=AT)
        a.update(kw)
        return f(ct.byref(p), dtype, *a.values(), None)

    assert call(RecurStep(0, 0, 8, 8, 8, 8, 8)) == OK
    for p in (RecurStep(-1, 4, 8, 8, 8, 8, 8), RecurStep(4, -1, 8, 8, 8, 8, 8), RecurStep(4, 4, 0, 8, 8, 8, 8), RecurStep(4, 4, 8, 8, -8, 8, 8)):
        assert call(p) == INVALID
    p = RecurStep(4, 4, 8, 8, 8, 8, 8)
    assert call(p, I8C) == UNSUPPORTED
    for name in ("x", "r", "i", "A", "state", "y"):
        assert call(p, **{name: None}) == INVALID
    for name in ("A", "state", "slots", "rb"):
        assert call(p, **{name: P(2 + (1 << 20))}) == UNSUPPORTED


@pytest.mark.parametrize("kw,dtype,want", [
    ({}, BF16C, OK), ({}, I8C, UNSUPPORTED), (dict(d=0), F32C, INVALID), (dict(seqs=-1), F32C, INVALID), (dict(len=-1), F32C, INVALID),
    (dict(eps=-1.0), F32C, INVALID), (dict(eps=float("nan")), F32C, INVALID), (dict(eps=float("inf")), F32C, INVALID),
    (dict(x=Stride(-1, 0)), F32C, INVALID), (dict(dtotal=Stride(0, -1)), F32C, INVALID), (dict(d=1 << 24), F32C, UNSUPPORTED),
    (dict(seqs=1 << 16, len=1 << 16), F32C, UNSUPPORTED), (dict(seqs=1, len=1 << 27), F32C, OK), (dict(seqs=1, len=1 << 29), F32C, UNSUPPORTED),  # 16 lanes a row, 2^32 threads
    (dict(seqs=1, len=(1 << 22), d=9000), F32C, UNSUPPORTED), (dict(seqs=0), F32C, OK),
])
def test_norm_abi(kw, dtype, want):
    s = Stride(8, 40)
    status, n = size("layer_norm_grad_workspace_size", put(Norm(2, 5, 8, 1e-5, s, s, s, s), kw), dtype)
    assert status == want and (n == 12345) == (want != OK)


def test_norm_abi_pointers():
    s = Stride(8, 40)
    p = Norm(2, 5, 8, 1e-5, s, s, s, s)
    f = LIB.layer_norm
    args = [ct.byref(p), BF16C, F32C, AT, AT, AT, AT, AT, AT]
    for k, bad, want in ((0, None, INVALID), (2, F16C, UNSUPPORTED), (3, None, INVALID), (7, None, INVALID),
                         (3, P(1 + (1 << 20)), UNSUPPORTED), (5, P(2 + (1 << 20)), UNSUPPORTED)):
        a = list(args)
        a[k] = bad
        assert f(*a, None) == want
    need = size("layer_norm_grad_workspace_size", p, BF16C)[1]
    f = LIB.layer_norm_grad
    args = [ct.byref(p), BF16C, BF16C, AT, AT, AT, AT, AT, AT, AT]
    assert f(*args, AT, ct.c_size_t(need - 1), None) == SMALL
    assert f(*args, None, ct.c_size_t(need), None) == INVALID
    assert f(*args, P(8 + (1 << 20)), ct.c_size_t(need), None) == UNSUPPORTED
    for k in (3, 4, 7):
        a = list(args)
        a[k] = None
        assert f(*a, AT, ct.c_size_t(need), None) == INVALID


def test_fp4_abi():
    ll = ct.c_longlong
    q = LIB.fp4_quantize
    for dtype, m, k, pitch, want in ((BF16C, -1, 4, 16, INVALID), (BF16C, 4, 4, 24, UNSUPPORTED), (BF16C, 4, 40, 16, INVALID),
                                     (I8C, 4, 4, 16, UNSUPPORTED), (BF16C, 0, 4, 16, OK), (BF16C, (1 << 31) - 1, 64, 32, UNSUPPORTED)):
        assert q(dtype, m, k, AT, ll(4), AT, ll(pitch), AT, None) == want
    assert q(BF16C, 4, 4, None, ll(4), AT, ll(16), AT, None) == INVALID
    assert q(BF16C, 4, 4, AT, ll(4), P(8 + (1 << 20)), ll(16), AT, None) == UNSUPPORTED
    f = LIB.fp4_matmul

    def call(p, dtype=BF16C, **kw):
        a = dict(x=AT, w=AT, s=AT, out=AT, work=AT, size=ct.c_size_t(1 << 40))
        a.update(kw)
        return f(ct.byref(p) if p else None, dtype, *a.values(), None)

    assert call(Fp4(0, 4, 4, 4, 16)) == OK and call(Fp4(4, 0, 4, 4, 16)) == OK and call(None) == INVALID
    for p, want in ((Fp4(-1, 4, 4, 4, 16), INVALID), (Fp4(4, 4, 40, 40, 16), INVALID), (Fp4(4, 4, 4, -4, 16), INVALID),
                    (Fp4(4, 4, 4, 4, 24), UNSUPPORTED), (Fp4(1 << 23, 4, 4, 4, 16), UNSUPPORTED), (Fp4(4, (1 << 31) - 1, 4, 4, 16), UNSUPPORTED)):
        assert call(p) == want
    p = Fp4(4, 4, 4, 4, 16)
    assert call(p, I8C) == UNSUPPORTED and call(p, w=P(8 + (1 << 20))) == UNSUPPORTED
    for name in ("x", "w", "s", "out"):
        assert call(p, **{name: None}) == INVALID
    p = Fp4(48, 1024, 8192, 8192, 4096)
    status, need = size("fp4_matmul_workspace_size", p, BF16C)
    assert status == OK and need > 0  # few columns: workgroups split k
    assert call(p, size=ct.c_size_t(need - 1)) == SMALL and call(p, work=None) == INVALID and call(p, work=P(8 + (1 << 20))) == UNSUPPORTED


# ----------------------------------------------------------------------- the plain forms that kernels are held to
def test_reference_quantisation():
    x = torch.tensor([[6.0, -6.0, 0.25, 0.26, 0.75, 2.5, -2.5, 5.0, 5.1, 0.0] + [0.0] * 22, [0.0] * 32, [7.0] + [1.0] * 31])
    value, scale = R.fp4_quantize(x)
    assert scale.flatten().tolist() == [127, 0, 128]
    assert value[0, :10].tolist() == [6, -6, 0, 0.5, 1, 2, -2, 4, 6, 0] and not value[1].any()
    assert value[2, :2].tolist() == [8.0, 1.0]  # 3.5 goes to 4, the even one; 0.5 is there


def test_reference_recurrence_differs_with_a_planted_mistake():
    """The bounds notice a forgotten bias and a decay taken from the wrong token."""
    g = torch.Generator().manual_seed(1)
    x, r, i, z = (torch.randn(30, 4, generator=g).double() for _ in range(4))
    A, b = torch.full((4,), -0.2).double(), torch.full((4,), 0.1).double()
    y, _, err, _ = R.recurrence(x, r, i, A, z, b, b, [30])
    for wrong in (R.recurrence(x, r, i, A, z, None, b, [30])[0], R.recurrence(x, r.roll(1, 0), i, A, z, b, b, [30])[0]):
        assert ((wrong - y).abs() > err + R.half_step(BF16) * y.abs()).any()
