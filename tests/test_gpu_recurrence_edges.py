"""Calls of the gated recurrence at the edges of what its documentation allows, through the C ABI and through Python."""
import ctypes as ct

import pytest
import torch

from test_block_cpu import Recur, RecurGrads
from test_sequence_cpu import BF16C, LIB, OK, Batch, Stride, size

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def at(t):
    return None if t is None else t.data_ptr()


def abi_grads(p, dy, x, r, i, A, z=None, dz=None):
    """gated_recurrence_grad through the C ABI on bf16 tensors [..][d]: dx, dr, di, dA."""
    status, need = size("gated_recurrence_grad_workspace_size", p, BF16C)
    assert status == OK
    out = [torch.full_like(x, 7.0) for _ in range(3)] + [torch.full_like(A, 7.0)]
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    g = RecurGrads(at(out[0]), at(out[1]), at(out[2]), at(out[3]), at(dz), None, None, None)
    args = [ct.c_void_p(at(t)) for t in (dy, x, r, i, A, z)]
    stream = ct.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert LIB.gated_recurrence_grad(ct.byref(p), BF16C, *args, None, None, None, None, ct.byref(g), ct.c_void_p(at(ws)),
                                     ct.c_size_t(need), stream) == OK
    torch.cuda.synchronize()
    return out


# short, several segments, cut into chunks, many sequences walked whole, packed
GATELESS = [(1, 5, 40, None), (3, 300, 72, None), (1, 3000, 64, None), (40, 60, 1024, None), (4, 0, 66, [0, 1, 90, 90, 1000])]


@pytest.mark.parametrize("seqs,n,d,lens", GATELESS, ids=str)
def test_gradients_without_z_take_any_strides_of_it(seqs, n, d, lens):
    """z NULL: its strides do not matter."""
    g = torch.Generator(device=DEV).manual_seed(1)
    tokens = lens[-1] if lens else seqs * n
    x, r, i, dy = (torch.randn(tokens, d, device=DEV, generator=g).to(BF16) for _ in range(4))
    A = -torch.rand(d, device=DEV, generator=g)
    start = torch.tensor(lens, dtype=torch.int32, device=DEV) if lens else None
    s = Stride(d, n * d)
    out = []
    for z in (Stride(0, 0), s, Stride(8 * d, 8 * n * d)):
        p = Recur(Batch(at(start), seqs, n, tokens), d, s, s, s, z, s)
        out.append(abi_grads(p, dy, x, r, i, A))
    for got in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, out[0]))
    assert all(bool(v.isfinite().all()) for v in out[0]) and bool(out[0][0].any())


def test_gradients_without_z_leave_dz_alone():
    """z NULL and a dz given all the same: nothing is written there."""
    g = torch.Generator(device=DEV).manual_seed(2)
    x, r, i, dy = (torch.randn(70, 40, device=DEV, generator=g).to(BF16) for _ in range(4))
    A, s = -torch.rand(40, device=DEV, generator=g), Stride(40, 2800)
    p = Recur(Batch(None, 1, 70, 70), 40, s, s, s, s, s)
    dz = torch.full_like(x, 3.0)
    got = abi_grads(p, dy, x, r, i, A, dz=dz)
    assert bool((dz == 3.0).all())
    assert all(torch.equal(a, b) for a, b in zip(got, abi_grads(p, dy, x, r, i, A)))
