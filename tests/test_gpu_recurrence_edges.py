"""Calls of the gated recurrence at the edges of what its documentation allows, through the C ABI and through Python."""
import ctypes as ct

import pytest
import torch

import block_ref as R
import convolution_nhwc_implicit_amd as nn
from test_block_cpu import Recur, RecurGrads
from test_gpu_block_ops import close, recur_call, recur_case, recur_grads, recur_ref, same_but_for_chunks
from test_sequence_cpu import BF16C, LIB, OK, Batch, Stride, size

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF = float("inf")


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


# ------------------------------------------------------------------------- dense batches of one-token sequences
NAMES = dict(x="dx", r="dr", i="di", A="dA", z="dz", rb="dr_bias", ib="di_bias", init="dinitial_state")


@pytest.mark.parametrize("seqs,d,typ,states", [(2, 3, F32, True), (5, 70, BF16, True), (300, 131, F16, True), (1024, 256, BF16, False),
                                               (700, 520, F32, True)], ids=str)
def test_one_token_sequences(seqs, d, typ, states):
    lens = [1] * seqs
    c, p, lead, _ = recur_case((lens, False, d, typ, True, True, states))  # each tensor with a stride of its own
    y, final = recur_call(p, None, state=True)
    v, (wy, wf, ey, ef) = recur_ref(c, lens, grad=True)
    close(y[:, 0], wy, ey.detach(), typ, "y")
    close(final, wf, ef.detach(), F32, "final state")
    got = recur_grads(p, None)
    out = (wy * v["dy"]).sum() + (0 if v["dfinal"] is None else (wf * v["dfinal"]).sum())
    have = [k for k in NAMES if v[k] is not None]
    want = torch.autograd.grad(out, [v[k] for k in have])
    with torch.no_grad():
        bound = R.recurrence_grad_bounds(v["dy"], *(v[k] for k in ("x", "r", "i", "A", "z", "rb", "ib")), lens, v["init"], v["dfinal"])
    for k, w in zip(have, want):
        n = NAMES[k]
        close(got[n].reshape(w.shape), w, bound[n], typ if n in ("dx", "dr", "di", "dz") else F32, n)


def test_one_token_sequences_of_a_projection_and_of_one_row():
    """Both gates as halves of one product's output, and one row of x for all sequences; against the same rows packed."""
    g = torch.Generator(device=DEV).manual_seed(4)
    seqs, d = 900, 264
    gates, z, dy = (torch.randn(seqs, 1, k * d, device=DEV, generator=g).to(BF16) for k in (2, 1, 1))
    r, i = gates.split(d, -1)
    A, h0 = -torch.rand(d, device=DEV, generator=g), torch.randn(seqs, d, device=DEV, generator=g)
    one = torch.randn(1, 1, d, device=DEV, generator=g).to(BF16).expand(seqs, 1, d)
    start = torch.arange(seqs + 1, dtype=torch.int32, device=DEV)
    for x in (z.flip(0), one):
        kw = dict(z=z, initial_state=h0)
        flat = dict(z=z[:, 0], initial_state=h0, seq_start=start)
        y, f = nn.gated_recurrence(x, r, i, A, return_state=True, **kw)
        wy, wf = nn.gated_recurrence(x[:, 0], r[:, 0], i[:, 0], A, return_state=True, **flat)
        assert same_but_for_chunks(y[:, 0], wy) and same_but_for_chunks(f, wf)
        k = nn.gated_recurrence_grad(dy, x, r, i, A, **kw)
        w = nn.gated_recurrence_grad(dy[:, 0], x[:, 0], r[:, 0], i[:, 0], A, **flat)
        assert all(same_but_for_chunks(k[n].reshape(w[n].shape), w[n]) for n in ("dx", "dr", "di", "dz", "dinitial_state"))
        # 900 terms of size 1, each with some tens of roundings
        assert float((k["dA"] - w["dA"]).abs().max()) <= 900 * 64 * R.U


def test_one_token_sequences_far_apart():
    """The last tokens of long sequences, whose distance no row stride may have."""
    g = torch.Generator(device=DEV).manual_seed(5)
    wide = torch.randn(5, (1 << 25) // 64, 64, device=DEV, generator=g).to(BF16)
    x, r, i = (wide[:, -k:][:, :1] for k in (1, 2, 3))
    A = -torch.rand(64, device=DEV, generator=g)
    y = nn.gated_recurrence(x, r, i, A)
    assert same_but_for_chunks(y, nn.gated_recurrence(x.contiguous(), r.contiguous(), i.contiguous(), A))
    k = nn.gated_recurrence_grad(x, x, r, i, A)
    w = nn.gated_recurrence_grad(x.contiguous(), x.contiguous(), r.contiguous(), i.contiguous(), A)
    assert all(same_but_for_chunks(k[n], w[n]) for n in ("dx", "dr", "di"))


# --------------------------------------------------------------------------------------- single tokens without slots
@pytest.mark.parametrize("rows,pool,d,typ,gate", [(1, 3, 1, F32, True), (4, 9, 130, BF16, True), (7, 7, 4097, F16, False),
                                                  (300, 400, 256, BF16, True), (33, 40, 6, F32, True)], ids=str)
def test_step_without_slots(rows, pool, d, typ, gate):
    """Row r takes and leaves state r, every other state stays as it is."""
    c, _, _, _ = recur_case(([1] * rows, True, d, typ, gate, True, True), seed=6)
    state = torch.randn(pool, d, generator=torch.Generator().manual_seed(7))
    c["init"] = state[:rows]
    _, (wy, wf, ey, ef) = recur_ref(c, [1] * rows)
    held = state.to(DEV)
    t = {k: None if v is None else v.to(DEV) for k, v in c.items()}
    y = nn.gated_recurrence_step(t["x"], t["r"], t["i"], t["A"], held, z=t["z"], r_bias=t["rb"], i_bias=t["ib"])
    close(y, wy, ey, typ, "y")
    close(held[:rows], wf, ef, F32, "states")
    assert torch.equal(held[rows:].cpu(), state[rows:])
    again = state.to(DEV)
    slots = torch.arange(rows, dtype=torch.int32, device=DEV)
    same = nn.gated_recurrence_step(t["x"], t["r"], t["i"], t["A"], again, z=t["z"], r_bias=t["rb"], i_bias=t["ib"], slots=slots)
    assert torch.equal(same, y) and torch.equal(again, held)


@pytest.mark.parametrize("typ", [F16, BF16, F32], ids=str)
def test_growing_states_are_nan(typ):
    """A above 0: NaN where the gate is open at all, in results and gradients; other channels as ever."""
    g = torch.Generator(device=DEV).manual_seed(8)
    x, r, i, dy = (torch.randn(2, 200, 6, device=DEV, generator=g).to(typ) for _ in range(4))
    A = torch.tensor([-0.5, 1e-30, 0.01, 3.0, INF, -0.5], device=DEV)
    y, f = nn.gated_recurrence(x, r, i, A, return_state=True)
    k = nn.gated_recurrence_grad(dy, x, r, i, A)
    assert bool(y[..., 1:5].isnan().all()) and bool(f[:, 1:5].isnan().all())
    assert all(bool(k[n][..., 1:5].isnan().all()) for n in ("dx", "dr", "di", "dA"))
    assert all(bool(k[n][..., [0, 5]].isfinite().all()) for n in ("dx", "dr", "di", "dA")) and bool(y[..., [0, 5]].isfinite().all())
