"""The way back through experts, as a training step calls it: the weighted sum's gradients, the gradients for the rows by
both products (the weights turned, each expert's by a call of the quantiser), and the gather's gradient.

Each step against float64 of the operands that it was given; tolerances from test_scaled_mm.py and test_experts.py: a
product (2^-16 + (G + 2) 2^-24) of the sum of its terms' magnitudes for G blocks and 2^-8 of the value for its bfloat16
output, a sum of k rows (k + 1) 2^-24 of the sum of the terms' magnitudes and 2^-8 of the value."""
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, cuda, lib  # noqa: F401
from test_scaled_mm import near, reference

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("T,H,F,E,k", [(1, 128, 128, 4, 2), (96, 512, 384, 6, 2), (70, 200, 144, 5, 3), (1500, 512, 768, 4, 2),
                                       (33, 77, 130, 9, 4)])
def test_gradients_through_experts(cuda, T, H, F, E, k):
    g = torch.Generator(device=DEV).manual_seed(T + H)
    new = lambda *s, f=1.0: (torch.randn(*s, generator=g, device=DEV) * f).bfloat16()  # noqa: E731
    up = [qb.quant_fwd(new(F, H, f=H ** -0.5), block_rows=128, want_t=True) for _ in range(E)]
    down = [qb.quant_fwd(new(H, F, f=F ** -0.5), block_rows=128, want_t=True) for _ in range(E)]
    stack = lambda ws, i: torch.stack([w[i] for w in ws])  # noqa: E731
    ids = torch.stack([torch.randperm(E, generator=g, device=DEV)[:k] for _ in range(T)])
    ids[torch.rand(T, k, generator=g, device=DEV) < 0.1] = -1  # dropped: rows of no expert at the end
    weights = torch.rand(T, k, generator=g, device=DEV)
    x, dy = new(T, H), new(T, H)
    P = T * k
    nothing = lambda n: torch.full((P, n), float("nan"), dtype=torch.bfloat16, device=DEV)  # noqa: E731

    offsets, slot = qb.expert_sort(ids, E)
    end = int(offsets[-1])
    rows = qb.expert_gather_fwd(x, slot, out=nothing(H))
    a, sa, _, _ = qb.quant_fwd(rows)
    u = qb.scaled_mm_fwd(a, sa, stack(up, 0), stack(up, 1), offsets, out=nothing(F))
    m, sm, _, _ = qb.quant_fwd(u)
    d = qb.scaled_mm_fwd(m, sm, stack(down, 0), stack(down, 1), offsets, out=nothing(H))

    dd, dweights = qb.expert_combine_bwd(dy, d, slot, weights, out=nothing(H))
    gq, gs, _, _ = qb.quant_fwd(dd)
    du = qb.scaled_mm_fwd(gq, gs, stack(down, 2), stack(down, 3), offsets, out=nothing(F))
    hq, hs, _, _ = qb.quant_fwd(du)
    dx_rows = qb.scaled_mm_fwd(hq, hs, stack(up, 2), stack(up, 3), offsets, out=nothing(H))
    dx = qb.expert_combine_fwd(dx_rows, slot)

    for name, t in (("rows", rows), ("u", u), ("d", d), ("dd", dd), ("du", du), ("dx_rows", dx_rows)):
        assert t[:end].isfinite().all() and t[end:].isnan().all(), f"{name}: rows behind the last expert's"
    assert dweights.isfinite().all() and dx.isfinite().all()
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        near(du[lo:hi], *reference(gq[lo:hi], gs[lo:hi], down[e][2], down[e][3]), H, f"du of expert {e}")
        near(dx_rows[lo:hi], *reference(hq[lo:hi], hs[lo:hi], up[e][2], up[e][3]), F, f"dx of expert {e}")
        # the turned weights stand for the weights of the forward product
        for q, s, qt, st in (up[e], down[e]):
            assert torch.equal(s.T, st) and torch.equal(q.view(torch.uint8).T, qt.view(torch.uint8))
    t, j = torch.nonzero(slot >= 0, as_tuple=True)
    at = slot[t, j].long()
    ref = torch.zeros(T, H, dtype=torch.float64, device=DEV).index_add_(0, t, dx_rows[at].double())
    size = torch.zeros_like(ref).index_add_(0, t, dx_rows[at].double().abs())
    assert ((dx.double() - ref).abs() <= (k + 1) * 2.0 ** -24 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()).all()
