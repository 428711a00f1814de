"""Refusals of the sequence operators, without a GPU: through Python (types, shapes, strides, devices) and through the
C ABI (status codes; every check runs before anything could be enqueued)."""
import ctypes as ct

import pytest
import torch

import convolution_nhwc_implicit_amd as nn
from convolution_nhwc_implicit_amd import binding as B

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
OK, INVALID, UNSUPPORTED, SMALL = (B.CONV2D_OK, B.CONV2D_ERR_INVALID_ARGUMENT, B.CONV2D_ERR_UNSUPPORTED,
                                   B.CONV2D_ERR_WORKSPACE_TOO_SMALL)
F16C, BF16C, I8C, F32C = B.CONV2D_DTYPE_F16, B.CONV2D_DTYPE_BF16, B.CONV2D_DTYPE_I8, 3


# ------------------------------------------------------------------------------------ through Python
def conv_args(**kw):
    a = dict(x=torch.zeros(2, 5, 8, dtype=BF16), weight=torch.zeros(8, 4, dtype=BF16), bias=torch.zeros(8, dtype=BF16),
             initial_state=torch.zeros(2, 3, 8, dtype=BF16))
    a.update(kw)
    return a


def scan_args(**kw):
    a = dict(x=torch.zeros(2, 5, 8, dtype=BF16), dt=torch.zeros(2, 5, 8, dtype=BF16), A=torch.zeros(8, 16),
             B=torch.zeros(2, 5, 2, 16, dtype=BF16), C=torch.zeros(2, 5, 2, 16, dtype=BF16), D=torch.zeros(8),
             z=torch.zeros(2, 5, 8, dtype=BF16), dt_bias=torch.zeros(8), initial_state=torch.zeros(2, 8, 16))
    a.update(kw)
    return a


def start(*v):
    return torch.tensor(v, dtype=torch.int32)


@pytest.mark.parametrize("kw,err,text", [
    ({}, ValueError, "on the GPU"),
    (dict(x=5), TypeError, "x must be a torch.Tensor"),
    (dict(x=torch.zeros(2, 5, 8, dtype=torch.int32)), TypeError, "float16"),
    (dict(x=torch.zeros(8, dtype=BF16)), ValueError, "tokens"),
    (dict(x=torch.zeros(2, 8, 5, dtype=BF16).transpose(1, 2)), ValueError, "unit stride"),
    (dict(weight=torch.zeros(8, 4)), TypeError, "weight must be torch.bfloat16"),
    (dict(weight=torch.zeros(7, 4, dtype=BF16)), ValueError, "weight must have shape"),
    (dict(weight=torch.zeros(4, 8, dtype=BF16).t()), ValueError, "weight must"),
    (dict(weight=torch.zeros(8, dtype=BF16)), ValueError, "weight must be"),
    (dict(bias=torch.zeros(9, dtype=BF16)), ValueError, "bias must have shape"),
    (dict(initial_state=torch.zeros(2, 4, 8, dtype=BF16)), ValueError, "initial_state must have shape"),
    (dict(initial_state=torch.zeros(3, 3, 8, dtype=BF16)), ValueError, "initial_state must have shape"),
    (dict(seq_start=start(0, 5)), ValueError, "one axis"),
    (dict(x=torch.zeros(5, 8, dtype=BF16), seq_start=start(0)), ValueError, "seq_start"),
    (dict(x=torch.zeros(5, 8, dtype=BF16), seq_start=torch.tensor([0, 5])), TypeError, "seq_start must be torch.int32"),
    (dict(x=torch.zeros(0, 5, 8, dtype=BF16)), ValueError, "at least one sequence"),
    (dict(x=torch.zeros(1, 2, 5, 8, dtype=BF16)), ValueError, "one axis"),
])
def test_conv_refusals(kw, err, text):
    with pytest.raises(err, match=text):
        nn.causal_conv(**conv_args(**kw))
    with pytest.raises(err, match=text):
        a = conv_args(**kw)
        dy = a["x"].clone() if isinstance(a["x"], torch.Tensor) else torch.zeros(1)
        nn.causal_conv_grad(dy, **a)


def test_grad_refusals():
    with pytest.raises(ValueError, match="dy must have shape"):
        nn.causal_conv_grad(torch.zeros(2, 4, 8, dtype=BF16), **conv_args())
    with pytest.raises(ValueError, match="dfinal_state must have shape"):
        nn.causal_conv_grad(torch.zeros(2, 5, 8, dtype=BF16), dfinal_state=torch.zeros(2, 8, 3, dtype=BF16), **conv_args())
    with pytest.raises(TypeError, match="dy must be torch.bfloat16"):
        nn.selective_scan_grad(torch.zeros(2, 5, 8), **scan_args())
    with pytest.raises(ValueError, match="dfinal_state must have shape"):
        nn.selective_scan_grad(torch.zeros(2, 5, 8, dtype=BF16), dfinal_state=torch.zeros(2, 16, 8), **scan_args())


@pytest.mark.parametrize("kw,err,text", [
    ({}, ValueError, "on the GPU"),
    (dict(dt=torch.zeros(2, 5, 9, dtype=BF16)), ValueError, "dt must have shape"),
    (dict(dt=torch.zeros(2, 5, 8)), TypeError, "dt must be torch.bfloat16"),
    (dict(A=torch.zeros(8, 16, dtype=BF16)), TypeError, "A must be torch.float32"),
    (dict(A=torch.zeros(8, 15)), ValueError, "B must have shape"),
    (dict(B=torch.zeros(2, 5, 3, 16, dtype=BF16), C=torch.zeros(2, 5, 3, 16, dtype=BF16)), ValueError, "groups"),
    (dict(B=torch.zeros(2, 5, 16, dtype=BF16)), ValueError, "x must be"),
    (dict(C=torch.zeros(2, 5, 1, 16, dtype=BF16)), ValueError, "C must have shape"),
    (dict(C=torch.zeros(2, 5, 16, 2, dtype=BF16).transpose(2, 3)), ValueError, "C must have unit stride"),
    (dict(D=torch.zeros(8, dtype=BF16)), TypeError, "D must be torch.float32"),
    (dict(z=torch.zeros(2, 4, 8, dtype=BF16)), ValueError, "z must have shape"),
    (dict(dt_bias=torch.zeros(1)), ValueError, "dt_bias must have shape"),
    (dict(initial_state=torch.zeros(2, 16, 8).transpose(1, 2)), ValueError, "initial_state must"),
    (dict(initial_state=torch.zeros(2, 8, 16, dtype=BF16)), TypeError, "initial_state must be torch.float32"),
])
def test_scan_refusals(kw, err, text):
    with pytest.raises(err, match=text):
        nn.selective_scan(**scan_args(**kw))
    with pytest.raises(err, match=text):
        nn.selective_scan_grad(torch.zeros(2, 5, 8, dtype=BF16), **scan_args(**kw))


def test_step_refusals():
    x, w = torch.zeros(3, 8, dtype=BF16), torch.zeros(8, 4, dtype=BF16)
    state = torch.zeros(4, 3, 8, dtype=BF16)
    for kw, err, text in ((dict(state=state[:2]), ValueError, "place for every row"),
                          (dict(state=state[:, :2].contiguous()), ValueError, "state must have shape"),
                          (dict(slots=start(0, 1)), ValueError, "slots must have shape"),
                          (dict(slots=torch.tensor([0, 1, 2])), TypeError, "slots must be torch.int32"),
                          (dict(), ValueError, "on the GPU")):
        with pytest.raises(err, match=text):
            nn.causal_conv_step(x, **{**dict(state=state, weight=w), **kw})
    s = {k: (v[0] if v.dim() > 2 else v) for k, v in scan_args().items() if k not in ("initial_state",)}
    for kw, err, text in ((dict(state=torch.zeros(4, 8, 16)), ValueError, "place for every row"),
                          (dict(state=torch.zeros(5, 16, 8)), ValueError, "state must have shape"),
                          (dict(state=torch.zeros(5, 8, 16, dtype=BF16)), TypeError, "state must be torch.float32"),
                          (dict(state=torch.zeros(5, 8, 16)), ValueError, "on the GPU")):
        with pytest.raises(err, match=text):
            nn.selective_scan_step(**{**s, **kw})


def test_fp8_refusals():
    x = torch.zeros(3, 200, dtype=BF16)
    for args, kw, err, text in (((x,), {}, ValueError, "on the GPU"),
                                ((x[0],), {}, ValueError, r"\[m\]\[k\]"),
                                ((x.t(),), {}, ValueError, "unit stride"),
                                ((x,), dict(transpose=True, blocks=True), ValueError, "as they lie"),
                                ((x.int(),), {}, TypeError, "float16")):
        with pytest.raises(err, match=text):
            nn.fp8_quantize(*args, **kw)
    a, sa = torch.zeros(4, 256, dtype=E4M3), torch.zeros(4, 2)
    b, sb = torch.zeros(200, 256, dtype=E4M3), torch.zeros(2, 2)
    for bad, err, text in ((dict(), ValueError, "on the GPU"),
                           (dict(a=a.view(torch.uint8)), TypeError, "a must be torch.float8_e4m3fn"),
                           (dict(a_scale=torch.zeros(4, 3)), ValueError, "a_scale must have shape"),
                           (dict(b_scale=torch.zeros(3, 2)), ValueError, "b_scale must have shape"),
                           (dict(b_scale=sb.half()), TypeError, "b_scale must be torch.float32"),
                           (dict(b=b[:, :250], ), ValueError, r"b must be \[n\]\[256\]"),
                           (dict(a=torch.zeros(4, 250, dtype=E4M3)), ValueError, "16-byte"),
                           (dict(out_dtype=torch.int32), TypeError, "out_dtype"),
                           (dict(out_dtype="bf16"), TypeError, "torch.dtype")):
        v = {**dict(a=a, a_scale=sa, b=b, b_scale=sb, out_dtype=BF16), **bad}
        with pytest.raises(err, match=text):
            nn.fp8_matmul(v["a"], v["a_scale"], v["b"], v["b_scale"], out_dtype=v["out_dtype"])


# ------------------------------------------------------------------------------------ through the C ABI
class Batch(ct.Structure):
    _fields_ = [("seq_start", ct.c_void_p), ("seqs", ct.c_int), ("len", ct.c_int), ("tokens", ct.c_longlong)]


class Stride(ct.Structure):
    _fields_ = [("row", ct.c_longlong), ("seq", ct.c_longlong)]


class Conv(ct.Structure):
    _fields_ = [("batch", Batch), ("d", ct.c_int), ("w", ct.c_int), ("silu", ct.c_int), ("x", Stride), ("dy", Stride)]


class Scan(ct.Structure):
    _fields_ = ([("batch", Batch)] + [(f, ct.c_int) for f in ("d", "n", "groups", "softplus")] +
                [(f, Stride) for f in ("x", "dt", "B", "C", "z", "dy")] +
                [("b_group", ct.c_longlong), ("c_group", ct.c_longlong)])


class Matmul(ct.Structure):
    _fields_ = [(f, ct.c_int) for f in ("m", "n", "k", "b_blocks")] + [("a_pitch", ct.c_longlong), ("b_pitch", ct.c_longlong)]


LIB = B.load()
P = ct.c_void_p
AT = P(1 << 20)  # an aligned address that no check may follow


def size(fn, prob, dtype):
    n = ct.c_size_t(12345)
    return getattr(LIB, fn)(ct.byref(prob), dtype, ct.byref(n)), n.value


def conv(**kw):
    p = Conv(Batch(None, 2, 5, 10), 8, 4, 1, Stride(8, 40), Stride(8, 40))
    for k, v in kw.items():
        setattr(p.batch if hasattr(p.batch, k) else p, k, v)
    return p


@pytest.mark.parametrize("kw,dtype,want", [
    ({}, BF16C, OK), ({}, F32C, OK), ({}, I8C, UNSUPPORTED), ({}, 9, UNSUPPORTED), (dict(w=1), F16C, UNSUPPORTED),
    (dict(w=5), F16C, UNSUPPORTED), (dict(w=0), F16C, INVALID), (dict(d=0), F16C, INVALID), (dict(silu=2), F16C, INVALID),
    (dict(seqs=0), F16C, INVALID), (dict(tokens=11), F16C, INVALID), (dict(len=-1), F16C, INVALID),
    (dict(x=Stride(-1, 0)), F16C, INVALID), (dict(dy=Stride(8, -1)), F16C, INVALID),
    (dict(seqs=1 << 16, len=1 << 16, tokens=1 << 32), F16C, UNSUPPORTED),
])
def test_conv_abi(kw, dtype, want):
    status, n = size("causal_conv_grad_workspace_size", conv(**kw), dtype)
    assert status == want and (n == 12345) == (want != OK)


def test_conv_abi_pointers():
    p, need = conv(), size("causal_conv_grad_workspace_size", conv(), F16C)[1]
    f = LIB.causal_conv
    assert f(ct.byref(p), F16C, AT, None, None, None, AT, None, None) == INVALID
    assert f(ct.byref(p), F16C, None, AT, None, None, AT, None, None) == INVALID
    assert f(ct.byref(p), F32C, P((1 << 20) + 2), AT, None, None, AT, None, None) == UNSUPPORTED
    assert f(None, F32C, AT, AT, None, None, AT, None, None) == INVALID
    g = LIB.causal_conv_grad
    args = [ct.byref(p), F16C, AT, AT, AT, None, None, None, AT, AT, None, None]
    assert g(*args, AT, ct.c_size_t(need - 1), None) == SMALL
    assert g(*args, None, ct.c_size_t(0), None) == INVALID
    assert g(*args, P((1 << 20) + 8), ct.c_size_t(need), None) == UNSUPPORTED


def scan(**kw):
    s = Stride(64, 320)
    p = Scan(Batch(None, 2, 5, 10), 8, 16, 2, 1, s, s, s, s, s, s, 16, 16)
    for k, v in kw.items():
        setattr(p.batch if hasattr(p.batch, k) else p, k, v)
    return p


@pytest.mark.parametrize("kw,dtype,want", [
    ({}, BF16C, OK), ({}, F32C, OK), ({}, I8C, UNSUPPORTED), (dict(n=64), F16C, OK), (dict(n=65), F16C, UNSUPPORTED),
    (dict(n=0), F16C, INVALID), (dict(groups=3), F16C, INVALID), (dict(groups=0), F16C, INVALID),
    (dict(softplus=-1), F16C, INVALID), (dict(tokens=9), F16C, INVALID), (dict(x=Stride(1 << 24, 0)), F16C, UNSUPPORTED),
    (dict(B=Stride(-4, 0)), F16C, INVALID), (dict(b_group=-1), F16C, INVALID), (dict(d=1 << 24), F16C, UNSUPPORTED),
    (dict(dt=Stride(0, 0), C=Stride(0, 0)), F16C, OK),
])
def test_scan_abi(kw, dtype, want):
    for fn in ("selective_scan_workspace_size", "selective_scan_grad_workspace_size"):
        status, n = size(fn, scan(**kw), dtype)
        assert status == want and (n == 12345) == (want != OK)


def test_scan_abi_pointers():
    p = scan(seqs=1, len=1 << 14, tokens=1 << 14)
    need = size("selective_scan_workspace_size", p, BF16C)[1]
    assert need > 0  # one long sequence is cut into chunks
    args = [ct.byref(p), BF16C, AT, AT, AT, AT, AT, None, None, None, None, AT, None]
    assert LIB.selective_scan(*args, AT, ct.c_size_t(need - 1), None) == SMALL
    assert LIB.selective_scan(*args, None, ct.c_size_t(0), None) == INVALID
    assert LIB.selective_scan(*args, P(8 + (1 << 20)), ct.c_size_t(need), None) == UNSUPPORTED
    for i in (2, 3, 4, 5, 6, 11):
        bad = list(args)
        bad[i] = None
        assert LIB.selective_scan(*bad, AT, ct.c_size_t(need), None) == INVALID
    bad = list(args)
    bad[4] = P(2 + (1 << 20))
    assert LIB.selective_scan(*bad, AT, ct.c_size_t(need), None) == UNSUPPORTED


@pytest.mark.parametrize("kw,dtype,want", [
    ({}, BF16C, OK), (dict(m=0), F32C, OK), (dict(k=0), F32C, OK), ({}, I8C, UNSUPPORTED), (dict(m=-1), F32C, INVALID),
    (dict(b_blocks=2), F32C, INVALID), (dict(a_pitch=128), F32C, INVALID), (dict(b_pitch=258), F32C, UNSUPPORTED),
    (dict(a_pitch=1 << 23), F32C, UNSUPPORTED),
])
def test_matmul_abi(kw, dtype, want):
    p = Matmul(40, 50, 250, 0, 256, 256)
    for k, v in kw.items():
        setattr(p, k, v)
    status, n = size("fp8_matmul_workspace_size", p, dtype)
    assert status == want and (n == 12345) == (want != OK)


def test_fp8_abi_pointers():
    p = Matmul(40, 50, 250, 0, 256, 256)
    need = size("fp8_matmul_workspace_size", p, BF16C)[1]
    f = LIB.fp8_matmul
    for i in range(2, 7):
        args = [ct.byref(p), BF16C, AT, AT, AT, AT, AT]
        args[i] = None
        assert f(*args, AT, ct.c_size_t(need), None) == INVALID
    assert f(ct.byref(p), BF16C, P((1 << 20) + 8), AT, AT, AT, AT, AT, ct.c_size_t(need), None) == UNSUPPORTED
    q = LIB.fp8_quantize
    ll = ct.c_longlong
    for form, m, k, pitch, want in ((3, 4, 4, 16, INVALID), (0, -1, 4, 16, INVALID), (0, 4, 4, 24, UNSUPPORTED),
                                    (0, 4, 40, 32, INVALID), (0, 4, 4, 256, INVALID), (1, 40, 4, 32, INVALID)):
        assert q(form, BF16C, m, k, AT, ll(4), AT, ll(pitch), AT, None) == want
    assert q(0, I8C, 4, 4, AT, ll(4), AT, ll(16), AT, None) == UNSUPPORTED
    assert q(0, BF16C, 4, 4, AT, ll(4), P((1 << 20) + 8), ll(16), AT, None) == UNSUPPORTED
    assert q(0, BF16C, 4, 4, None, ll(4), AT, ll(16), AT, None) == INVALID


def test_status_of_unsupported_is_named():
    with pytest.raises(B.Conv2dError) as e:
        raise B.Conv2dError(UNSUPPORTED, "selective_scan")
    assert e.value.status == UNSUPPORTED and "selective_scan" in str(e.value)
