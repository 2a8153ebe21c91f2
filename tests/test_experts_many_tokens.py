"""Gradients of the experts' weighted sum for numbers of tokens and row lengths on both sides of where a warp or a CTA takes a
token.  Tolerances as in test_experts.py: dweights 1e-5 of the sum of the products' magnitudes, drows one product rounded."""
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, DT, cuda, guarded, lib, shifted  # noqa: F401
from test_experts import choices

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("T", [2400, 2431, 2432, 2440, 9001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1, 2, 3, 9])
def test_combine_backward_of_many_tokens(cuda, T, dtype, k):
    code, td = DT[dtype]
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    P, e = T * k, 16 // td.itemsize
    g = torch.Generator(device=DEV).manual_seed(T + k)
    slot = choices(T, k, 7, P, T)
    weights = torch.randn(T, k, generator=g, device=DEV)
    t, j = torch.nonzero(slot >= 0, as_tuple=True)
    at = slot[t, j].long()
    for N in (64 * e - 1, 64 * e, 64 * e + 1, 96 * e - 2, 128 * e - 1, 128 * e, 128 * e + 1):
        off = N % 2
        rows, dy = (shifted(torch.randn(n, N, generator=g, device=DEV).to(td), off) for n in (P, T))
        drows, c1 = guarded((P, N), td, off)
        dweights, c2 = guarded((T, k), torch.float32)
        left = drows.clone()
        qb.qk_expert_combine_bwd(dy, rows, slot, weights, drows, dweights, T, k, P, N, code)
        torch.cuda.synchronize()
        c1("drows")
        c2("dweights")
        ref = weights.double()[t, j, None] * dy.double()[t]
        assert ((drows[at].double() - ref).abs() <= (half + 2.0 ** -24) * ref.abs()).all(), f"drows {N}"
        named = torch.zeros(P, dtype=torch.bool, device=DEV)
        named[at] = True
        assert torch.equal(drows[~named].view(torch.uint8), left[~named].view(torch.uint8)), f"other rows {N}"
        products = dy.double()[t] * rows.double()[at]
        want, size = torch.zeros(2, T, k, dtype=torch.float64, device=DEV)
        want[t, j], size[t, j] = products.sum(1), products.abs().sum(1)
        assert ((dweights.double() - want).abs() <= 1e-5 * size).all(), f"dweights {N}"
        again = qb.expert_combine_bwd(dy.contiguous(), rows.clone(), slot, weights)[1]
        if off == 0:
            assert torch.equal(again, dweights)
