"""Operands of the 8-bit products on their way through the workspace: which rows are copied there.

Inputs are small whole numbers with scales that are powers of two, so that no addition rounds
and outputs are equal bit for bit to float64's.  The workspace starts as NaN bytes.
"""
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, DT, cuda, guarded, lib, shifted  # noqa: F401
from test_scaled_mm import cut, make, reference

gpu = pytest.mark.gpu
UNWRITTEN = 0x7F  # a NaN of e4m3


def product(a, sa, b, sb, offsets, out):
    """One call through the C entry; (y, workspace as [rows of b and then of a, bytes of a row])."""
    (M, K), N, E = a.shape, b.shape[-2], b.shape[0]
    code, td = DT[out]
    y, check = guarded((M, N), td)
    n = qb.qk_scaled_mm_workspace_size(M, N, K, E)
    ws, check_ws = guarded((n,), torch.uint8)
    ws.fill_(UNWRITTEN)
    qb.qk_scaled_mm_fwd(a, sa, b, sb, offsets, y, ws, n, M, N, K, E, 1 if sb.shape[-2] == N else 128, code)
    torch.cuda.synchronize()
    check("y")
    check_ws("workspace")
    return y, ws.view(E * N + M, -1)


# Rows by expert, rows before the first and behind the last expert's, N and K: one token's choices, one expert of many,
# experts of many rows between empty ones, none at all.
FEW = [([0] * 20 + [1] + [0] * 30 + [1, 1] + [0] * 11, 0, 0, 130, 77), ([0] * 7 + [5], 2, 3, 257, 1023),
       ([0, 40, 0, 0, 3], 1, 0, 64, 255), ([600, 0, 0, 300, 0], 4, 9, 1300, 333), ([0, 0, 0], 0, 6, 128, 100),
       ([0] * 1023 + [2], 0, 0, 129, 33)]


@gpu
@pytest.mark.parametrize("counts,before,behind,N,K", FEW)
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_what_no_row_needs_is_not_copied(cuda, counts, before, behind, N, K, out):
    offsets, end = cut(counts, before)
    M, E = end + behind, len(counts)
    a, sa, b, sb = make(M, N, K, M + N, experts=E, whole=True)
    y, ws = product(a, sa, b, sb, offsets.to(DEV), out)
    for e in (i for i in range(E) if counts[i]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        ref = reference(a[lo:hi], sa[lo:hi], b[e], sb[e])[0]
        assert torch.equal(y[lo:hi], ref.to(y.dtype)), f"expert {e}"
        assert torch.equal(ws[e * N:(e + 1) * N, :K], b[e].view(torch.uint8)), f"weights of expert {e}"
    assert (torch.cat([y[:before], y[end:]]).view(torch.uint8) == 0xA5).all(), "rows of no expert were written"
    none = torch.tensor([c == 0 for c in counts]).repeat_interleave(N).to(DEV)
    assert (ws[:E * N][none] == UNWRITTEN).all(), "weights of an expert without rows were copied"
    rows = ws[E * N:]
    assert torch.equal(rows[before:end, :K], a[before:end].view(torch.uint8))
    assert (rows[:before] == UNWRITTEN).all() and (rows[end:] == UNWRITTEN).all(), "rows of no expert were copied"


@gpu
def test_offsets_that_fall_copy_what_their_running_maximum_names(cuda):
    N, K = 136, 99
    wild = torch.tensor([-5, 10, 4, 20, 1 << 30, 7], dtype=torch.int32)
    a, sa, b, sb = make(50, N, K, 5, experts=5, whole=True)
    y, ws = product(a, sa, b, sb, wild.to(DEV), "f32")
    for e, (lo, hi) in enumerate([(0, 10), (10, 10), (10, 20), (20, 50), (50, 50)]):
        assert torch.equal(y[lo:hi].double(), reference(a[lo:hi], sa[lo:hi], b[e], sb[e])[0])
        assert lo < hi or (ws[e * N:(e + 1) * N] == UNWRITTEN).all()
