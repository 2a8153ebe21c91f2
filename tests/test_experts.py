"""Tokens sorted by expert and back.

The sort and the copies are exact.  Sums, against float64, tolerances fixed
before the first run: y is k fused multiply-adds in float32, (k + 1) 2^-24 of
the sum of |weight row|; dweights a float32 sum of N products, each rounding
at most 2^-24 of the sum of their magnitudes: at most 64 of them follow each
other in a thread or a join at the sizes here, and 1e-5 is allowed; bfloat16
outputs half a step more, 2^-8.  drows is one product, rounded: 2^-24, or 2^-8.
Outputs start as a byte pattern, and a guard behind each must come back as it was.
"""
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, DT, cuda, guarded, lib, shifted  # noqa: F401

gpu = pytest.mark.gpu


def sort_reference(ids, E):
    flat = ids.reshape(-1).cpu().long()
    kept = torch.nonzero((flat >= 0) & (flat < E))[:, 0]
    order = kept[torch.argsort(flat[kept], stable=True)]
    offsets = torch.zeros(E + 1, dtype=torch.int64)
    offsets[1:] = torch.bincount(flat[kept], minlength=E).cumsum(0)
    slot = torch.full_like(flat, -1)
    slot[order] = torch.arange(len(order))
    return offsets.int(), slot.int().view(ids.shape)


def run_sort(ids, E):
    T, k = ids.shape
    offsets, c1 = guarded((E + 1,), torch.int32)
    slot, c2 = guarded((T, k), torch.int32)
    n = qb.qk_expert_sort_workspace_size(T, k, E)
    ws, c3 = guarded((n,), torch.uint8)
    qb.qk_expert_sort(ids, ids.element_size(), offsets, slot, ws if n else None, n, T, k, E)
    torch.cuda.synchronize()
    for c, what in ((c1, "offsets"), (c2, "slot"), (c3, "workspace")):
        c(what)
    return offsets, slot


@gpu
@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 8), (7, 3, 5), (33, 2, 64), (128, 4, 32), (500, 8, 1024),
                                   (1024, 4, 16), (1025, 4, 3), (4097, 1, 255), (5000, 6, 64), (20000, 8, 1000),
                                   (100003, 2, 7), (90000, 8, 128)])
def test_sort(cuda, T, k, E):
    g = torch.Generator().manual_seed(T + E)
    for kind in ("even", "dropped", "one", "none"):
        ids = torch.randint(0, E, (T, k), generator=g)
        if kind == "dropped":
            ids[torch.rand(T, k, generator=g) < 0.2] = -1
            ids[torch.rand(T, k, generator=g) < 0.05] = E
        elif kind == "one":
            ids.fill_(E - 1)
        elif kind == "none":
            ids.fill_(-7)
        want = sort_reference(ids, E)
        for dtype in (torch.int32, torch.int64):
            wide = ids.to(dtype)
            if dtype == torch.int64 and kind == "none" and T:
                wide[0, 0] = (1 << 32)  # its low half would be expert 0
            got = run_sort(wide.to(DEV), E)
            assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1]), f"{kind} {dtype}"


def choices(T, k, E, P, seed, dropped=0.2):
    """slot [T, k] of a sort over E experts, on the GPU, with some choices that have no row."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    ids[torch.rand(T, k, generator=g) < dropped] = -1
    return sort_reference(ids, E)[1].to(DEV)


@gpu
@pytest.mark.parametrize("N", [1, 2, 3, 8, 16, 100, 127, 128, 500, 1024, 4096, 5001])
@pytest.mark.parametrize("T,k", [(1, 1), (5, 3), (64, 2), (300, 9)])
def test_gather(cuda, T, k, N):
    P = T * k
    slot = choices(T, k, 5, P, T + N)
    for dtype, e in ((torch.uint8, 1), (torch.bfloat16, 2), (torch.float32, 4)):
        for off in (0, 1):
            x0 = torch.randint(0, 200, (T, N), dtype=torch.uint8, device=DEV)
            x = shifted(x0.to(dtype), off)
            groups = -(-N // 128)
            scale = torch.rand(T, groups, device=DEV)
            rows, c1 = guarded((P, N), dtype, off)
            row_scale, c2 = guarded((P, groups), torch.float32)
            want, want_scale = rows.clone(), row_scale.clone()
            t, j = torch.nonzero(slot >= 0, as_tuple=True)
            want[slot[t, j].long()] = x[t]
            want_scale[slot[t, j].long()] = scale[t]
            qb.qk_expert_gather_fwd(x, scale, slot, rows, row_scale, T, k, P, N * e, groups)
            torch.cuda.synchronize()
            c1("rows")
            c2("row_scale")
            assert torch.equal(rows.view(torch.uint8), want.view(torch.uint8))
            assert torch.equal(row_scale.view(torch.uint8), want_scale.view(torch.uint8))


@gpu
@pytest.mark.parametrize("N", [1, 2, 7, 8, 64, 127, 256, 1000, 1023, 2048, 4096, 5001, 16384])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k", [(1, 1), (6, 2), (37, 8), (50, 11)])
def test_combine_and_its_gradients(cuda, T, k, dtype, N):
    code, td = DT[dtype]
    P = T * k
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    g = torch.Generator(device=DEV).manual_seed(T * N)
    slot = choices(T, k, 6, P, T + N)
    slot[0] = -1                    # a token without any
    if T > 2:
        slot[2, 0] = P + 5          # beyond the rows: none
    rows0 = torch.randn(P, N, generator=g, device=DEV).to(td)
    dy0 = torch.randn(T, N, generator=g, device=DEV).to(td)
    weights = torch.randn(T, k, generator=g, device=DEV)
    there = (slot >= 0) & (slot < P)
    t, j = torch.nonzero(there, as_tuple=True)
    at = slot[t, j].long()
    for off in (0, 1):
        rows, dy = shifted(rows0, off), shifted(dy0, off)
        r64, d64, w64 = rows.double(), dy.double(), weights.double()
        for w, ww in ((weights, w64), (None, torch.ones_like(w64))):
            ref = torch.zeros(T, N, dtype=torch.float64, device=DEV).index_add_(0, t, ww[t, j, None] * r64[at])
            size = torch.zeros_like(ref).index_add_(0, t, (ww[t, j, None] * r64[at]).abs())
            y, c = guarded((T, N), td, off)
            qb.qk_expert_combine_fwd(rows, slot, w, y, T, k, P, N, code)
            torch.cuda.synchronize()
            c("y")
            tol = (k + 1) * 2.0 ** -24 * size * (1 + half) + half * ref.abs()
            assert ((y.double() - ref).abs() <= tol).all(), f"y {T}x{k} {N} {dtype} offset {off}"
        drows, c1 = guarded((P, N), td, off)
        dweights, c2 = guarded((T, k), torch.float32)
        left = drows.clone()
        qb.qk_expert_combine_bwd(dy, rows, slot, weights, drows, dweights, T, k, P, N, code)
        torch.cuda.synchronize()
        c1("drows")
        c2("dweights")
        ref = w64[t, j, None] * d64[t]
        assert ((drows[at].double() - ref).abs() <= (half + 2.0 ** -24) * ref.abs()).all()
        named = torch.zeros(P, dtype=torch.bool, device=DEV)
        named[at] = True
        assert torch.equal(drows[~named].view(torch.uint8), left[~named].view(torch.uint8))
        want, size = torch.zeros_like(w64), torch.zeros_like(w64)
        want[t, j] = (d64[t] * r64[at]).sum(1)
        size[t, j] = (d64[t] * r64[at]).abs().sum(1)
        assert ((dweights.double() - want).abs() <= 1e-5 * size).all()
        inplace = rows.clone()
        none = qb.expert_combine_bwd(dy.contiguous(), inplace, slot, weights, out=inplace, want_dweights=False)
        assert none[1] is None and torch.equal(inplace[at], drows[at])


@gpu
def test_gradients_against_differences(cuda):
    T, k, N, P = 9, 3, 40, 27
    slot = choices(T, k, 4, P, 3)
    g = torch.Generator(device=DEV).manual_seed(8)
    rows, dy, w = (torch.randn(*s, generator=g, device=DEV) for s in ((P, N), (T, N), (T, k)))
    loss = lambda r, v: (qb.expert_combine_fwd(r, slot, v).double() * dy.double()).sum().item()  # noqa: E731
    drows, dw = qb.expert_combine_bwd(dy, rows, slot, w, out=torch.zeros(P, N, device=DEV))
    # linear in each: a central difference with a step of 1 is exact but for the float32 sums of the two
    # losses, below 2^-20 of the sum of their terms
    terms = (qb.expert_combine_fwd(rows.abs(), slot, w.abs()) * dy.abs()).sum().item() + 100
    for p, n in ((0, 0), (5, 17), (11, 39), (26, 3)):
        up, down = rows.clone(), rows.clone()
        up[p, n] += 1
        down[p, n] -= 1
        assert abs((loss(up, w) - loss(down, w)) / 2 - drows[p, n].item()) <= 2.0 ** -20 * terms
    for t in range(T):
        up, down = w.clone(), w.clone()
        up[t, 1] += 1
        down[t, 1] -= 1
        assert abs((loss(rows, up) - loss(rows, down)) / 2 - dw[t, 1].item()) <= 2.0 ** -20 * terms
    # the gather's gradient: <rows(x), d> = <x, combine(d)>
    x = torch.randn(T, N, generator=g, device=DEV)
    d = torch.randn(P, N, generator=g, device=DEV)
    moved = qb.expert_gather_fwd(x, slot, out=torch.zeros(P, N, device=DEV))
    back = qb.expert_combine_fwd(d, slot)
    a, b = (moved.double() * d.double()).sum(), (x.double() * back.double()).sum()
    assert abs(a - b) <= 2.0 ** -20 * (moved.double() * d.double()).abs().sum()


@gpu
def test_offsets_beyond_32_bits(cuda):
    T, k, N = 70001, 2, 16384  # 2.3e9 elements of rows
    g = torch.Generator(device=DEV).manual_seed(2)
    ids = torch.randint(0, 8, (T, k), generator=g, device=DEV)
    offsets, slot = qb.expert_sort(ids, 8)
    x = torch.randint(0, 100, (T, N), generator=g, device=DEV, dtype=torch.int16).view(torch.bfloat16)
    rows = qb.expert_gather_fwd(x, slot)
    for t in (0, 1, T // 2, T - 1):
        for j in range(k):
            assert torch.equal(rows[slot[t, j]].view(torch.int16), x[t].view(torch.int16))
    rows.fill_(2)
    y = qb.expert_combine_fwd(rows, slot)
    assert (y == 4).all()
    del y
    w = torch.full((T, k), 0.5, device=DEV)
    drows, dw = qb.expert_combine_bwd(torch.ones_like(x), rows, slot, w, out=rows)
    assert (drows == 0.5).all() and (dw == 2.0 * N).all()


@gpu
def test_layer_of_experts(cuda):
    """A decoder block's experts, as they are called one after the other: the norm in 8 bits, the sort, the rows'
    way to the experts, both products with the activation between them, the way back with weights, the next norm;
    each step against float64 of what it was given.  Then once more as a captured graph, on new tokens."""
    T, H, F, E, k = 96, 512, 384, 6, 2
    g = torch.Generator(device=DEV).manual_seed(17)
    new = lambda *s, f=1.0: (torch.randn(*s, generator=g, device=DEV) * f).bfloat16()  # noqa: E731
    gain, router = torch.ones(H, dtype=torch.bfloat16, device=DEV), new(E, H, f=H ** -0.5)
    up = [qb.quant_fwd(new(2 * F, H, f=H ** -0.5), block_rows=128) for _ in range(E)]
    down = [qb.quant_fwd(new(H, F, f=F ** -0.5), block_rows=128) for _ in range(E)]
    b1, s1, b2, s2 = (torch.stack([w[i] for w in ws]) for ws in (up, down) for i in (0, 1))
    x, r = new(T, H), new(T, H)

    def layer():
        q, sq, h, rstd = qb.rmsnorm_quant_fwd(x, gain, residual=r, group=128)
        p, ids = (qb.rmsnorm_fwd(h, gain)[0].float() @ router.float().T).softmax(1).topk(k, dim=1)
        offsets, slot = qb.expert_sort(ids, E)
        rows, row_scale = qb.expert_gather_fwd(q, slot, scale=sq)
        u = qb.scaled_mm_fwd(rows, row_scale, b1, s1, offsets)
        act = torch.nn.functional.silu(u[:, :F]) * u[:, F:]
        qa, sa, _, _ = qb.quant_fwd(act)
        d = qb.scaled_mm_fwd(qa, sa, b2, s2, offsets)
        y = qb.expert_combine_fwd(d, slot, p.contiguous())
        out = qb.add_rmsnorm_fwd(y, h, gain)
        return {"q": q, "sq": sq, "ids": ids, "p": p, "offsets": offsets, "slot": slot, "rows": rows, "u": u, "qa": qa,
                "sa": sa, "d": d, "y": y, "h": out[1], "n": out[0]}

    def check(o):
        want = sort_reference(o["ids"], E)
        assert torch.equal(o["offsets"].cpu(), want[0]) and torch.equal(o["slot"].cpu(), want[1])
        at = o["slot"].long()
        q64 = o["q"].double() * o["sq"].double().repeat_interleave(128, 1)
        assert torch.equal(o["rows"][at.view(-1)].float(), o["q"].float().repeat_interleave(k, 0))
        act64 = o["qa"].double() * o["sa"].double().repeat_interleave(128, 1)
        wide = lambda b, s: b.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)  # noqa: E731
        y64 = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        size = torch.zeros_like(y64)
        for t in range(T):
            for j in range(k):
                e, p = int(o["ids"][t, j]), int(at[t, j])
                w1, w2 = wide(b1[e], s1[e]), wide(b2[e], s2[e])
                u64, au = w1 @ q64[t], w1.abs() @ q64[t].abs()
                assert ((o["u"][p].double() - u64).abs() <= 2.0 ** -8 * u64.abs() + 2.0 ** -15 * au).all()
                d64, ad = w2 @ act64[p], w2.abs() @ act64[p].abs()
                assert ((o["d"][p].double() - d64).abs() <= 2.0 ** -8 * d64.abs() + 2.0 ** -15 * ad).all()
                y64[t] += o["p"][t, j].double() * o["d"][p].double()
                size[t] += (o["p"][t, j].double() * o["d"][p].double()).abs()
        assert ((o["y"].double() - y64).abs() <= 2.0 ** -8 * y64.abs() + 2.0 ** -20 * size).all()

    check(layer())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for _ in range(2):
        x.copy_(new(T, H))
        graph.replay()
    torch.cuda.synchronize()
    check(held)
    fresh = layer()
    assert all(torch.equal(fresh[n].float(), held[n].float()) for n in ("y", "h", "n"))


@gpu
def test_helper_refusals(cuda):
    x, slot = torch.zeros(4, 8, device=DEV), torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    rows = torch.zeros(8, 8, device=DEV)
    for call in (lambda: qb.expert_sort(slot.float(), 4), lambda: qb.expert_sort(slot, 0), lambda: qb.expert_sort(slot[0], 4),
                 lambda: qb.expert_sort(slot.T, 4), lambda: qb.expert_sort(slot.cpu(), 4),
                 lambda: qb.expert_gather_fwd(x, slot[:3]), lambda: qb.expert_gather_fwd(x, slot.long()),
                 lambda: qb.expert_gather_fwd(x.T, slot), lambda: qb.expert_gather_fwd(x, slot, out=rows.double()),
                 lambda: qb.expert_gather_fwd(x, slot, out_scale=w), lambda: qb.expert_gather_fwd(x, slot, scale=w[:3]),
                 lambda: qb.expert_combine_fwd(rows, slot, w.T), lambda: qb.expert_combine_fwd(rows, slot, w.half()),
                 lambda: qb.expert_combine_fwd(rows.half(), slot), lambda: qb.expert_combine_bwd(x, rows.bfloat16(), slot, w),
                 lambda: qb.expert_combine_bwd(x[:3], rows, slot, w)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(qb.QkError):
        qb.expert_sort(slot, 1025)
    assert qb.expert_combine_fwd(rows[:0], slot).abs().sum().item() == 0  # no rows: zeros
    assert qb.expert_gather_fwd(x[:0], slot[:0]).shape == (0, 8)


A = 1 << 32  # never read: refused on the host


def test_refusals(lib):
    bad, mis, big = qb.QK_ERR_INVALID_ARG, qb.QK_ERR_MISALIGNED, qb.QK_ERR_UNSUPPORTED
    B, C, D, F, G = (A + (i << 24) for i in range(1, 6))

    def sort(ids=A, size=4, offsets=B, slot=C, ws=None, n=0, T=8, k=2, E=4):
        return lib.qk_expert_sort(ids, size, offsets, slot, ws, n, T, k, E, None)

    assert sort(size=2) == bad and sort(ids=None) == bad and sort(offsets=None) == bad and sort(slot=None) == bad
    assert sort(T=-1) == bad and sort(k=0) == bad and sort(E=0) == bad and sort(E=1025) == big and sort(T=2 ** 30) == big
    assert sort(ids=A + 4, size=8) == mis and sort(slot=C + 1) == mis
    assert sort(T=100000) == bad and sort(T=100000, ws=D + 4, n=1 << 20) == mis and sort(slot=A) == bad

    def gather(x=A, scale=None, slot=B, rows=C, row_scale=None, T=8, k=2, P=16, nb=64, groups=0):
        return lib.qk_expert_gather_fwd(x, scale, slot, rows, row_scale, T, k, P, nb, groups, None)

    assert gather(x=None) == bad and gather(slot=None) == bad and gather(rows=None) == bad and gather(nb=0) == bad
    assert gather(scale=D) == bad and gather(groups=1) == bad and gather(P=-1) == bad and gather(rows=A) == bad
    assert gather(slot=B + 2) == mis and gather(P=2 ** 31) == big
    assert gather(T=0, x=None) == qb.QK_OK and gather(P=0, rows=None) == qb.QK_OK

    def fwd(rows=A, slot=B, w=None, y=C, T=8, k=2, P=16, N=64, dtype=0):
        return lib.qk_expert_combine_fwd(rows, slot, w, y, T, k, P, N, dtype, None)

    assert fwd(rows=None) == bad and fwd(slot=None) == bad and fwd(y=None) == bad and fwd(N=0) == bad and fwd(dtype=2) == bad
    assert fwd(y=A) == bad and fwd(y=C + 2) == mis and fwd(w=D + 1) == mis and fwd(T=0, rows=None, y=None) == qb.QK_OK

    def bwd(dy=A, rows=B, slot=C, w=D, drows=F, dw=G, T=8, k=2, P=16, N=64, dtype=1):
        return lib.qk_expert_combine_bwd(dy, rows, slot, w, drows, dw, T, k, P, N, dtype, None)

    for name in ("dy", "rows", "slot", "w", "drows"):
        assert bwd(**{name: None}) == bad
    assert bwd(drows=A) == bad and bwd(drows=B + 16) == bad and bwd(dw=B) == bad and bwd(drows=B, dw=B) == bad
    assert bwd(dw=G + 2) == mis and bwd(dy=A + 1) == mis and bwd(T=0, dy=None) == qb.QK_OK
