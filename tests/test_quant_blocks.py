"""Blocks of 128 x 128 in 8 bits: one scale and the same values in both directions, also where some are not finite, and
experts' weights in one matrix.  Everything is equal bit for bit: both directions round the same quotient by the same scale."""
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, cuda, lib  # noqa: F401
from test_quant import check, make
from test_scaled_mm import near, reference

gpu = pytest.mark.gpu


def equal(a, b):
    """Equal values, NaN equal to NaN."""
    torch.testing.assert_close(a, b, rtol=0, atol=0, equal_nan=True)


@gpu
@pytest.mark.parametrize("M,N", [(1, 1), (128, 128), (129, 127), (256, 384), (300, 1000), (513, 200)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("finite", [True, False])
def test_both_directions_share_scales_and_values(cuda, M, N, dtype, finite):
    x = make(M, N, dtype, M + N)
    bad = torch.zeros(-(-M // 128), -(-N // 128), dtype=torch.bool, device=DEV)
    if not finite:  # the first block and the last: others stay finite where there are more
        x[0, 0], x[-1, -1] = float("nan"), -float("inf")
        bad[0, 0] = bad[-1, -1] = True
    for qdtype in (torch.float8_e4m3fn, torch.int8):
        q, scale, qt, scale_t = qb.quant_fwd(x, block_rows=128, qdtype=qdtype, want_t=True)
        assert torch.equal(scale.isnan(), bad)
        equal(scale.T, scale_t)
        there = ~bad.repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :N]
        bits, bits_t = q.view(torch.uint8), qt.view(torch.uint8).T
        assert torch.equal(bits[there], bits_t[there])
        if finite:
            check(q, scale, x, 128, "int8" if qdtype is torch.int8 else "e4m3", f"{M}x{N}")


@gpu
def test_weights_of_experts_in_one_matrix(cuda):
    """Blocks of a matrix [experts * N, K] are the experts' own where N is a multiple of 128.  For other N a block reaches
    into the next expert's rows, whether or not the number of scales gives it away, and each expert takes a call."""
    E, K = 3, 200
    for N, own in ((256, True), (200, False), (120, False)):
        w = make(E * N, K, "bf16", N)
        q, scale, _, _ = qb.quant_fwd(w, block_rows=128)
        each = [qb.quant_fwd(w[e * N:(e + 1) * N], block_rows=128) for e in range(E)]
        qe, se = torch.stack([t[0] for t in each]), torch.stack([t[1] for t in each])
        if own:
            assert torch.equal(q.view(torch.uint8), qe.view(torch.uint8).view(E * N, K))
            assert torch.equal(scale, se.view_as(scale))
        a, sa, _, _ = qb.quant_fwd(make(9, K, "bf16", 1))
        offsets = torch.tensor([0, 3, 3, 9], dtype=torch.int32, device=DEV)
        y = qb.scaled_mm_fwd(a, sa, qe, se, offsets, out_dtype=torch.float32)
        for e, (lo, hi) in enumerate([(0, 3), (3, 3), (3, 9)]):
            if lo < hi:
                near(y[lo:hi], *reference(a[lo:hi], sa[lo:hi], qe[e], se[e]), K, f"expert {e}")
