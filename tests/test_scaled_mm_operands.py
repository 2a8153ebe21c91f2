"""Operands of the 8-bit products on their way through the workspace: which rows are copied there,
and operands that start off 16 bytes.

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


OFF = [(1, 0), (0, 4), (8, 15)]  # bytes that a and b start behind 16


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 128, 16), (5, 200, 144), (70, 513, 1040), (300, 640, 256), (1030, 1100, 320),
                                   (16, 4096, 4096), (520, 2080, 640)])
def test_operands_off_16_bytes(cuda, M, N, K):
    for b_rows in (128, 1):
        a, sa, b, sb = make(M, N, K, M + N + K, b_rows=b_rows, whole=True)
        want = {t: reference(a, sa, b, sb)[0].to(t) for t in (torch.float32, torch.bfloat16)}
        for off_a, off_b in OFF:
            a1, b1 = shifted(a, off_a), shifted(b, off_b)
            for out, td in (DT["f32"], DT["bf16"]):
                assert torch.equal(qb.scaled_mm_fwd(a1, sa, b1, sb, out_dtype=td), want[td]), f"{off_a} {off_b} {td}"
                need = (M * K if off_a else 0) + (N * K if off_b else 0)
                y, check = guarded((M, N), td)
                ws, check_ws = guarded((need,), torch.uint8)
                ws.fill_(UNWRITTEN)
                call = lambda w, n: qb.qk_scaled_mm_fwd(a1, sa, b1, sb, None, y, w, n, M, N, K, 1, b_rows, out)  # noqa: E731
                call(ws, need)
                torch.cuda.synchronize()
                check("y")
                check_ws("workspace")
                assert torch.equal(y, want[td])
                for w, n in ((None, 0), (ws, need - 1)):
                    with pytest.raises(qb.QkError) as error:
                        call(w, n)
                    assert error.value.status == qb.QK_ERR_MISALIGNED


@gpu
@pytest.mark.parametrize("counts,before,behind", [([0, 5, 0, 40, 1], 2, 3), ([700, 0, 257], 0, 1)])
def test_operands_off_16_bytes_by_expert(cuda, counts, before, behind):
    N, K, E = 520, 272, len(counts)
    offsets, end = cut(counts, before)
    M = end + behind
    a, sa, b, sb = make(M, N, K, M, experts=E, whole=True)
    for off_a, off_b in OFF:
        y = torch.full((M, N), 7.0, device=DEV)
        qb.scaled_mm_fwd(shifted(a, off_a), sa, shifted(b, off_b), sb, offsets.to(DEV), out=y)
        for e in range(E):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            assert torch.equal(y[lo:hi].double(), reference(a[lo:hi], sa[lo:hi], b[e], sb[e])[0])
        assert (y[:before] == 7).all() and (y[end:] == 7).all()


@gpu
def test_operands_off_16_bytes_captured_and_on_another_stream(cuda):
    a, sa, b, sb = make(40, 300, 512, 3, whole=True)
    a, b = shifted(a, 3), shifted(b, 9)
    want = reference(a, sa, b, sb)[0].bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = qb.scaled_mm_fwd(a, sa, b, sb, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = qb.scaled_mm_fwd(a, sa, b, sb)
    for _ in range(2):
        held.fill_(3)
        graph.replay()
        assert torch.equal(held, want)


A = 1 << 32  # never read: refused on the host


def test_refusals_of_operands_off_16_bytes(lib):
    def call(a=A + 8, b=A + (2 << 24), ws=A + (5 << 24), n=4 * 128, M=4, y=A + (4 << 24)):
        return lib.qk_scaled_mm_fwd(a, A + (1 << 24), b, A + (3 << 24), None, y, ws, n, M, 256, 128, 1, 128, qb.QK_BF16, None)

    mis, bad = qb.QK_ERR_MISALIGNED, qb.QK_ERR_INVALID_ARG
    assert call(ws=None, n=0) == mis and call(n=4 * 128 - 1) == mis and call(ws=A + (5 << 24) + 16) == mis
    assert call(b=A + (2 << 24) + 4) == mis  # room for a, not for both
    assert call(ws=A) == bad and call(ws=A + (1 << 24)) == bad and call(ws=A + (4 << 24)) == bad
    assert call(M=0, ws=None, n=0) == qb.QK_OK
    assert qb.qk_scaled_mm_workspace_size(4, 256, 128, 1) == 0
