"""How far values and scales that are not finite reach in the 8-bit products: a value of a or b and a scale of a its row or
column, a scale of b the columns of its block, by expert that expert's rows.  Everything else is equal bit for bit to what
it is without them (whole numbers, see test_scaled_mm.py)."""
import pytest
import torch

from test_add_rmsnorm import DEV, cuda, lib  # noqa: F401
from test_scaled_mm import make, run

gpu = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


# narrow tiles, tiles whose k is shared, wide ones, pairs
@gpu
@pytest.mark.parametrize("M,N,K", [(5, 700, 384), (3, 300, 4096), (100, 515, 640), (300, 1800, 2048), (1500, 1600, 272)])
@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("scale", [NAN, INF])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_scales_that_are_not_finite(cuda, M, N, K, b_rows, scale, out):
    a, sa, b, sb = make(M, N, K, M + N, b_rows=b_rows, whole=True)
    want = run(a, sa, b, sb, out)
    sa[M // 2, 1] = scale
    sb[2, 0] = scale  # column 2, or columns 256 to 383
    y = run(a, sa, b, sb, out)
    hit = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    hit[M // 2] = True
    hit[:, slice(256, 384) if b_rows == 128 else slice(2, 3)] = True
    assert not y[hit].isfinite().any()  # a block's sum times infinity, or 0 times it
    assert torch.equal(y[~hit], want[~hit])


@gpu
@pytest.mark.parametrize("counts", [[3, 5, 2, 40], [130, 70, 0, 9], [300, 257, 31, 500]])
@pytest.mark.parametrize("N", [260, 2080])
def test_an_expert_that_is_not_finite_stays_by_itself(cuda, counts, N):
    K, E = 640, len(counts)
    offsets = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).int().to(DEV)
    at = offsets.tolist()
    M = at[-1] + 7
    for b_rows in (128, 1):
        a, sa, b, sb = make(M, N, K, M + N, experts=E, b_rows=b_rows, whole=True)
        want = run(a, sa, b, sb, "bf16", offsets)
        for e in range(E):
            a1, sa1, b1, sb1 = (t.clone() for t in (a, sa, b, sb))
            a1.view(torch.uint8)[at[e]:at[e + 1]] = 0x7F
            a1.view(torch.uint8)[at[-1]:] = 0xFF  # rows behind the last, of which tiles read some
            sa1[at[-1]:] = INF
            b1.view(torch.uint8)[e] = 0x7F
            sb1[e] = NAN
            y = run(a1, sa1, b1, sb1, "bf16", offsets)
            assert y[at[e]:at[e + 1]].isnan().all()
            assert torch.equal(y[:at[e]], want[:at[e]]) and torch.equal(y[at[e + 1]:at[-1]], want[at[e + 1]:at[-1]])
            assert (y[at[-1]:].contiguous().view(torch.uint8) == 0xA5).all()
