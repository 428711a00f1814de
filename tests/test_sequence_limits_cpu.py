"""Sizes whose launches the device could not take (a launch's threads along an axis are counted in 32 bits), through
the C ABI and without a GPU: refused by a check, before anything is enqueued, as unsupported."""
import ctypes as ct

import pytest

from test_sequence_cpu import (AT, BF16C, F32C, LIB, OK, UNSUPPORTED, Batch, Matmul, Scan, Stride, conv, scan, size)

LL, P = ct.c_longlong, ct.c_void_p
BIG = 2 ** 31 - 1
WS = ct.c_size_t(1 << 62)  # enough for any workspace


class ConvStep(ct.Structure):
    _fields_ = [(f, ct.c_int) for f in ("rows", "pool", "d", "w", "silu")] + [("x_row", LL)]


class ScanStep(ct.Structure):
    _fields_ = ([(f, ct.c_int) for f in ("rows", "pool", "d", "n", "groups", "softplus")] +
                [(f, LL) for f in ("x_row", "dt_row", "b_row", "c_row", "z_row", "b_group", "c_group")])


def dense(seqs, length, d, n=16, groups=1):
    s = Stride(d, d * length)
    return Scan(Batch(None, seqs, length, seqs * length), d, n, groups, 1, s, s, s, s, s, s, n, n)


def packed(tokens, seqs, d, n=16, groups=1):
    s = Stride(d, 0)
    return Scan(Batch(AT, seqs, 0, tokens), d, n, groups, 1, s, s, s, s, s, s, n, n)


# a workgroup of 64 threads or more for every chunk of 16 channels
@pytest.mark.parametrize("p,want", [
    (dense(262144, 8, 4096), UNSUPPORTED), (dense(262144, 8, 4080), OK), (packed(262144 * 8, 262144, 4096), UNSUPPORTED),
    (dense(1 << 24, 1, 64), UNSUPPORTED), (dense(1 << 24, 1, 32), OK), (dense(1, BIG, 1, 1), OK),
])
def test_scan(p, want):
    assert size("selective_scan_workspace_size", p, BF16C)[0] == want
    if want != OK:
        args = [ct.byref(p), BF16C, AT, AT, AT, AT, AT, None, None, None, None, AT, None]
        assert LIB.selective_scan(*args, AT, WS, None) == want


# the sums of dB and dC have a thread to a value; sequences a workgroup of 256 each
@pytest.mark.parametrize("p,want", [
    (dense(1024, 65536, 64, 16, 4), UNSUPPORTED), (dense(1024, 65536, 64, 16, 2), OK),
    (dense(1, BIG, 1, 2), UNSUPPORTED), (dense(1, BIG, 1, 1), OK), (dense(1 << 24, 1, 1, 1), UNSUPPORTED),
    (dense((1 << 24) - 1, 1, 1, 1), OK),
])
def test_scan_grad(p, want):
    assert size("selective_scan_grad_workspace_size", p, BF16C)[0] == want
    if want != OK:
        g = (P * 9)(*[AT.value] * 9)
        args = [ct.byref(p), BF16C, AT, AT, AT, AT, AT, AT, None, None, None, None, None, ct.byref(g)]
        assert LIB.selective_scan_grad(*args, AT, WS, None) == want


def test_conv():
    p = conv(seqs=1, len=BIG, tokens=BIG, d=512)
    assert LIB.causal_conv(ct.byref(p), BF16C, AT, AT, None, None, AT, None, None) == UNSUPPORTED


def test_steps():
    p = ConvStep(1 << 26, 1, 512, 4, 1, 512)
    assert LIB.causal_conv_step(ct.byref(p), BF16C, AT, AT, AT, None, AT, AT, None) == UNSUPPORTED
    for rows, n in ((1 << 26, 16), (1 << 25, 17)):
        p = ScanStep(rows, 1, 64, n, 1, 1, 64, 64, n, n, 64, n, n)
        assert LIB.selective_scan_step(ct.byref(p), BF16C, *[AT] * 5, None, None, None, AT, AT, AT, None) == UNSUPPORTED


@pytest.mark.parametrize("form,m,k", [(0, 1 << 21, 1 << 14), (0, BIG, 128), (1, BIG, 128), (1, 128, 1 << 23),
                                      (2, 128, BIG), (2, 1 << 23, 128)])
def test_quantize(form, m, k):
    pitch = -(-(m if form == 1 else k) // 128) * 128
    assert LIB.fp8_quantize(form, BF16C, m, k, AT, LL(k), AT, LL(pitch), AT, None) == UNSUPPORTED


@pytest.mark.parametrize("m,n,k,dtype,want", [
    (1 << 28, 16, 512, BF16C, UNSUPPORTED), (16, 1 << 28, 512, F32C, UNSUPPORTED), (16, 1 << 27, 512, BF16C, OK),
    (1 << 28, 16, 128, BF16C, OK), (BIG, 100, 128, BF16C, UNSUPPORTED), (100, BIG, 128, BF16C, UNSUPPORTED),
    (BIG, BIG, 128, BF16C, UNSUPPORTED), (1 << 24, 1 << 14, 128, BF16C, OK), (0, BIG, 128, BF16C, OK),
])
def test_matmul(m, n, k, dtype, want):
    p = Matmul(m, n, k, 0, k, k)
    assert size("fp8_matmul_workspace_size", p, dtype)[0] == want
    if want != OK:
        assert LIB.fp8_matmul(ct.byref(p), dtype, AT, AT, AT, AT, AT, AT, WS, None) == want


def test_limits_leave_what_fits():
    for fn in ("selective_scan_workspace_size", "selective_scan_grad_workspace_size"):
        assert size(fn, scan(), BF16C)[0] == OK
