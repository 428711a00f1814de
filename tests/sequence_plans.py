"""Which path the host's plans take for a size (no GPU): for tests that mean to reach one."""
import ctypes as ct

from convolution_nhwc_implicit_amd import binding as B
from test_sequence_cpu import Batch, Scan, Stride, size

AT = 1 << 20  # an address that plans do not follow
CODE = {"torch.float16": B.CONV2D_DTYPE_F16, "torch.bfloat16": B.CONV2D_DTYPE_BF16, "torch.float32": 3}


class Fp8Plan(ct.Structure):
    _fields_ = [(f, ct.c_int) for f in ("shape", "splits", "per")] + [(f, ct.c_bool) for f in ("narrow_m", "narrow_n", "all")]


def product(m, n, k, typ):
    """(tile of 256 or 128, or 0 for the narrow kernel alone; workgroups along k; the blocks of each; whether rows of
    a, and of b, past whole tiles are left to the narrow kernel)."""
    fn = B.load()._ZN3cnv15fp8_matmul_planEiiii  # cnv::fp8_matmul_plan(int, int, int, int)
    fn.restype = Fp8Plan
    p = fn(m, n, k, CODE[str(typ)])
    narrow = p.all or m <= 64 or n <= 64
    return 0 if narrow else (256, 128)[p.shape], p.splits, p.per, p.narrow_m, p.narrow_n


def _scan(lens, packed, d, n, groups, grad, typ):
    s = Stride(d, 0 if packed else d * lens[0])
    p = Scan(Batch(AT if packed else None, len(lens), 0 if packed else lens[0], sum(lens)), d, n, groups, 1, s, s, s, s, s, s, n, n)
    status, need = size("selective_scan_grad_workspace_size" if grad else "selective_scan_workspace_size", p, CODE[str(typ)])
    assert status == 0
    return need


def scan_is_cut(lens, packed, d, n, groups, typ):
    """Whether the forward pass cuts sequences into chunks: only then it has a workspace."""
    return _scan(lens, packed, d, n, groups, False, typ) > 0


def scan_grad_is_cut(lens, packed, d, n, groups, typ):
    """The same for the gradient: its workspace then holds more than the kept states and the partial sums."""
    def up(v):
        return -(-v // 256) * 256

    tokens, ts = sum(lens), 16 if n <= 8 else 8 if n <= 16 else 4
    whole = max(16, -(-(tokens if packed else lens[0]) // 16) * 16)
    slots = len(lens) + (tokens // whole if packed else 0)
    blocks = -(-(d // groups) // 64) * groups
    uncut = up((tokens // ts + slots + 1) * d * n * 4) + up(slots * d * n * 4) + 2 * up(slots * d * 4) + 2 * up(blocks * tokens * n * 4)
    return _scan(lens, packed, d, n, groups, True, typ) != uncut
