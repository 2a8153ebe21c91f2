"""Cross-entropy of a linear layer's logits, forward and backward.

Against the definitions in float64 on the same inputs.  Tolerances, from the
arithmetic and fixed before the first run; with A[i,v] = sum_k |h[i,k] w[v,k]|:
  * a logit is a float32 sum of K products: |error| <= 1e-5 A (REL_F32 of the
    magnitude of its terms).  e_i, the largest over a row, bounds the error
    that the logits give lse_i; to it comes 1e-5 |lse| (parity's rule).
  * loss = lse - logit_t + z lse^2: twice that, plus 2 |z lse| of it, plus 1e-5
    of each term.
  * p = exp(logit - lse) is off by 2 e_i + 1e-5 (relative); g has terms of
    magnitude G = |dloss| (p |1 + 2 z lse| + onehot).
  * float32: |dh - ref| <= 2 (1e-5 + 2 e_i) (G |w|), dw likewise with the
    largest e_i: the products' own rounding, and g's.
  * bfloat16: g is rounded to bfloat16 (half a step: 2^-8 of it), so 2^-8 comes
    to the factor, and the output's own rounding, 2^-8 of the value.
  * A probability below 2^-126, the smallest normal float32, is formed as 0, and
    so may a product of it be: each of a sum's terms is then off by at most
    2^-126 times the factors beside it, |dloss| and |w| (or |h|), or by 2^-126
    itself.  n terms: n 2^-126 max(1, |dloss|) max(1, |w|).
Outputs start as a byte pattern, and a guard behind each must come back as it was.
"""
import ctypes

import numpy as np
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from memory_bound_row_rmsnorm_gb300 import synthetic as syn
from parity import to_f64
from test_add_rmsnorm import DEV, DT, cuda, guarded, lib, shifted  # noqa: F401

gpu = pytest.mark.gpu
IGNORE = -100


def make(M, V, K, dtype, seed, ignored=0.1):
    h = syn.normal_rows(M, K, dtype, seed, DEV)
    w = syn.normal_rows(V, K, dtype, seed + 1, DEV, sigma=2.0 / K ** 0.5)
    g = torch.Generator().manual_seed(seed + 2)
    t = torch.randint(0, V, (M,), generator=g)
    t[torch.rand(M, generator=g) < ignored] = IGNORE
    dloss = syn.uniform_weight(M, "f32", seed + 3, DEV, lo=0.25, hi=2.0)
    return {"h": h, "w": w, "t": t.to(DEV), "dloss": dloss}


def reference(c, z=0.0, ignore=IGNORE):
    """Everything in float64, on the GPU."""
    h, w, t = c["h"].double(), c["w"].double(), c["t"]
    M, V = h.shape[0], w.shape[0]
    logits = h @ w.T
    lse = torch.logsumexp(logits, 1)
    ok = (t >= 0) & (t < V)
    skip = t == ignore if ignore is not None else torch.zeros_like(ok)
    at = logits[torch.arange(M, device=DEV), torch.where(ok, t, 0)]
    nan = torch.tensor(float("nan"), dtype=torch.float64, device=DEV)
    loss = torch.where(skip, 0.0, torch.where(ok, lse - at + z * lse ** 2, nan))
    e = 1e-5 * (h.abs() @ w.abs().T).amax(1)
    out = {"lse": lse, "loss": loss, "mean": loss[~skip].mean(), "tol_lse": e + 1e-5 * lse.abs()}
    out["tol_loss"] = (2 + 2 * (z * lse).abs()) * out["tol_lse"] + 1e-5 * (lse.abs() + at.abs() + abs(z) * lse ** 2)
    f = 1 + 2 * z * lse
    p = torch.exp(logits - lse[:, None]) * f[:, None]
    one = torch.zeros_like(p)
    one[torch.arange(M, device=DEV), torch.where(ok, t, 0)] = 1.0
    d = torch.where(skip, 0.0, torch.where(ok, c["dloss"].double(), nan))
    G = d[:, None] * (p - one)
    G[skip] = 0
    size = d.abs()[:, None] * (p.abs() + one)
    size[skip] = 0
    bf = c["h"].dtype == torch.bfloat16
    rel = 2 * (1e-5 + 2 * e) + (2 ** -8 if bf else 0.0)
    out["dh"], out["dw"] = G @ w, G.T @ h
    tiny = lambda n, x: n * 2.0 ** -126 * max(1.0, c["dloss"].abs().max().item()) * max(1.0, x.abs().max().item())  # noqa: E731
    out["tol_dh"] = rel[:, None] * (size @ w.abs()) + (2 ** -8 * out["dh"].abs() if bf else 0.0) + tiny(V, w)
    out["tol_dw"] = rel.max() * (size.T @ h.abs()) + (2 ** -8 * out["dw"].abs() if bf else 0.0) + tiny(M, h)
    return out


def near(got, ref, tol, what):
    got = got.double()
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN in other places"
    ok = ~ref.isnan()
    bad = ok & ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst "
                           f"{((got - ref).abs() / tol)[bad].max().item():.3g} of the tolerance")


def run(c, z=0.0, ignore=IGNORE, off=0, dh=True, dw=True):
    """Both passes through the C entry points, guarded; a dict of the outputs."""
    dtype = c["h"].dtype
    code = qb.QK_BF16 if dtype == torch.bfloat16 else qb.QK_F32
    M, K = c["h"].shape
    V = c["w"].shape[0]
    h, w = shifted(c["h"], off), shifted(c["w"], off)
    out, checks = {}, []

    def new(name, shape, dt, o=0):
        out[name], check = guarded(shape, dt, o)
        checks.append((name, check))
        return out[name]

    for name in ("loss", "lse"):
        new(name, (M,), torch.float32)
    new("mean", (1,), torch.float32)
    n = qb.qk_linear_xent_fwd_workspace_size(M, V, K, code)
    qb.qk_linear_xent_fwd(h, w, c["t"], out["loss"], out["lse"], out["mean"], new("workspace", (n,), torch.uint8),
                          n, M, V, K, code, ignore, z)
    if dh:
        new("dh", (M, K), dtype, off)
    if dw:
        new("dw", (V, K), dtype, off)
    n = qb.qk_linear_xent_bwd_workspace_size(M, V, K, code)
    qb.qk_linear_xent_bwd(h, w, c["t"], out["lse"], c["dloss"], out.get("dh"), out.get("dw"),
                          new("workspace 2", (n,), torch.uint8), n, M, V, K, code, ignore, z)
    torch.cuda.synchronize()
    for name, check in checks:
        check(name)
    return out


def check(c, out, z=0.0, ignore=IGNORE, what=""):
    ref = reference(c, z, ignore)
    near(out["lse"], ref["lse"], ref["tol_lse"], f"lse {what}")
    near(out["loss"], ref["loss"], ref["tol_loss"], f"loss {what}")
    counted = c["t"] != ignore if ignore is not None else torch.ones_like(c["t"], dtype=torch.bool)
    if counted.any():
        near(out["mean"][0], ref["mean"], ref["tol_loss"][counted].mean() + 1e-5 * ref["loss"][counted].abs().mean(),
             f"mean {what}")
    else:
        assert out["mean"].isnan().all()
    for k in ("dh", "dw"):
        if k in out:
            near(out[k], ref[k], ref["tol_" + k], f"{k} {what}")


SIZES = [(1, 1, 1), (1, 2, 8), (2, 5, 3), (1, 300, 64), (7, 255, 16), (16, 256, 64), (17, 257, 65), (64, 1000, 100),
         (100, 63, 72), (128, 512, 128), (129, 511, 513), (255, 64, 200), (256, 256, 256), (257, 700, 192),
         (300, 1031, 96), (513, 130, 24), (33, 5003, 40), (3, 20011, 136)]


@gpu
@pytest.mark.parametrize("M,V,K", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_both_passes(cuda, dtype, M, V, K):
    c = make(M, V, K, dtype, M + V + K)
    for off, z in ((0, 0.0), (1, 1e-2)):
        check(c, run(c, z, off=off), z, what=f"{M}x{V}x{K} {dtype} offset {off}")


@gpu
@pytest.mark.parametrize("dtype,M,V,K", [("bf16", 1000, 2048, 1024), ("bf16", 4100, 40000, 64), ("f32", 2050, 20000, 40),
                                         ("bf16", 40, 33000, 512), ("f32", 24, 9000, 520), ("bf16", 2048, 300, 2056),
                                         ("bf16", 70000, 600, 32), ("bf16", 9000, 33000, 16), ("f32", 24, 50000, 520),
                                         ("bf16", 16, 20000, 2049), ("f32", 65, 30000, 513), ("bf16", 64, 19457, 1032),
                                         ("bf16", 20000, 8000, 64), ("bf16", 20000, 7901, 67), ("f32", 20000, 3001, 64),
                                         ("f32", 16, 3000, 4000), ("f32", 32, 2000, 2001)])
def test_larger(cuda, dtype, M, V, K):
    """Several pieces of the vocabulary, long sums, many tokens on few columns and the reverse."""
    c = make(M, V, K, dtype, 77)
    check(c, run(c, 1e-4), 1e-4, what=f"{M}x{V}x{K} {dtype}")


@gpu
@pytest.mark.parametrize("dtype,M,V,K", [("f32", 40, 90000, 513), ("f32", 700, 50000, 1040), ("bf16", 16, 70000, 2049),
                                         ("bf16", 200, 140000, 1025)])
def test_weights_copied_in_pieces(cuda, dtype, M, V, K):
    """More weights than the workspace holds at a time as bf16 planes or aligned
    rows, of vectors and of single elements."""
    c = make(M, V, K, dtype, 78)
    planes = 3 if dtype == "f32" else 1
    assert planes * V * ((K + 7) // 8 * 8) * 2 > 2 ** 28
    for off in (0, 1):
        check(c, run(c, 1e-4, off=off), 1e-4, what=f"{M}x{V}x{K} {dtype} offset {off}")


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_vocabulary_of_millions(cuda, dtype):
    """Few float32 tokens whose gradient of the logits is more than one piece."""
    c = make(20, 2200000, 8, dtype, 79)
    check(c, run(c), what=f"20x2200000x8 {dtype}")


@gpu
def test_weights_beyond_32_bit_offsets(cuda):
    """A vocabulary of 2.2e9 weights: the last rows, the targets' rows and dh
    against float64 over pieces of it."""
    M, V, K = 5, 530000, 4096
    w = torch.empty(V, K, dtype=torch.bfloat16, device=DEV)
    for v in range(0, V, 53000):
        w[v:v + 53000] = syn.normal_rows(53000, K, "bf16", 100 + v, DEV, sigma=2.0 / K ** 0.5)
    c = {"h": syn.normal_rows(M, K, "bf16", 1, DEV), "w": w, "t": torch.tensor([V - 1, 0, 524288, 524287, IGNORE], device=DEV),
         "dloss": torch.linspace(0.5, 1.5, M, device=DEV)}
    out = run(c)
    logits = torch.cat([c["h"].double() @ w[v:v + 53000].double().T for v in range(0, V, 53000)], 1)
    e = 1e-5 * torch.stack([(c["h"].double().abs() @ w[v:v + 53000].double().abs().T).amax(1)
                            for v in range(0, V, 53000)]).amax(0)
    lse = torch.logsumexp(logits, 1)
    near(out["lse"], lse, e + 1e-5 * lse.abs(), "lse")
    d = torch.where(c["t"] == IGNORE, 0.0, c["dloss"].double())
    one = torch.zeros_like(logits)
    one[torch.arange(4), c["t"][:4]] = 1.0
    p = torch.exp(logits - lse[:, None])
    g, size = d[:, None] * (p - one), d[:, None] * (p + one)
    rel = 2 * (1e-5 + 2 * e) + 2 ** -8  # as reference() has it
    ref = sum(g[:, v:v + 53000] @ w[v:v + 53000].double() for v in range(0, V, 53000))
    mag = sum(size[:, v:v + 53000] @ w[v:v + 53000].double().abs() for v in range(0, V, 53000))
    near(out["dh"], ref, rel[:, None] * mag + 2 ** -8 * ref.abs(), "dh")
    rows = torch.tensor([0, 1, 524286, 524287, 524288, V - 2, V - 1], device=DEV)
    ref = g[:, rows].T @ c["h"].double()
    near(out["dw"][rows], ref, rel.max() * (size[:, rows].T @ c["h"].double().abs()) + 2 ** -8 * ref.abs(), "dw")
    assert torch.isfinite(out["dw"].view(-1)[::4097]).all()


@gpu
@pytest.mark.parametrize("M,V,K", [(3, 21, 2 ** 18 + 4), (3, 21, 2 ** 18 + 5), (1, 2, 2 ** 19), (20, 9, 60001)])
def test_rows_of_many_chunks(cuda, M, V, K):
    """Few float32 tokens whose h is walked in tens of pieces of shared memory."""
    c = make(M, V, K, "f32", 80, ignored=0)
    check(c, run(c), what=f"{M}x{V}x{K} f32")


# --- float32 by three bf16 planes: what each pair of planes gives ---
# An output's error in norm, relative to the output, is below 1e-6:
#   * what the six plane pairs leave out, and float32's rounding of g, lse, loss
#     and the outputs: below 3e-7 (the first test below forms just that; the most
#     is the target's logit as lse - loss: two roundings of numbers from 8 to 16,
#     2^-20 / sqrt(12) each, to logits of size 2 are 2e-7, for 40 rows 3e-7);
#   * the tensor core cuts an addition's tail off, 2^-25.5 of the sum each.  Of a
#     chain's 48 additions 28 are made at the sum's full size (20 of the first 24
#     hold the small pairs, 2^-8 of it or less): 28 2^-25.5 = 5.9e-7.
# A pair that is missing in one of the three products shows as 1.2e-6 or more.
PLANE_PAIRS = [(0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)]
BOUND = 1e-6


def by_planes(a, b, pairs):
    """a b^T in float64 over the given pairs of bf16 planes."""
    def planes(x):
        out, rest = [], x.double()
        for _ in range(3):
            out.append(rest.float().bfloat16().double())
            rest = rest - out[-1]
        return out
    pa, pb = planes(a), planes(b)
    return sum(pa[i] @ pb[j].T for i, j in pairs)


def exact_step(c):
    """The targets' logits, lse, dh and dw in float64 (no row ignored, z = 0)."""
    h, w, t, d = c["h"].double(), c["w"].double(), c["t"], c["dloss"].double()
    logits = h @ w.T
    lse = torch.logsumexp(logits, 1)
    at = logits.gather(1, t[:, None])[:, 0]
    g = torch.exp(logits - lse[:, None])
    g[torch.arange(len(t), device=t.device), t] -= 1
    g *= d[:, None]
    return at, lse, g @ w, g.T @ h


def norm_errors(loss, lse, dh, dw, want):
    got = (lse.double() - loss.double(), lse.double(), dh.double(), dw.double())
    return {k: ((a - b).norm() / b.norm()).item() for k, a, b in zip(("target logits", "lse", "dh", "dw"), got, want)}


@pytest.mark.parametrize("M,V,K", [(48, 70, 64), (40, 300, 96), (130, 515, 513), (40, 5003, 72)])
def test_the_bound_sees_each_plane_pair(M, V, K):
    gen = torch.Generator().manual_seed(M + V)
    c = {"h": syn.normal_rows(M, K, "f32", 1, "cpu"), "w": syn.normal_rows(V, K, "f32", 2, "cpu", sigma=2 / K ** 0.5),
         "t": torch.randint(0, V, (M,), generator=gen), "dloss": syn.uniform_weight(M, "f32", 3, "cpu", lo=0.25, hi=2.0)}
    want = exact_step(c)

    def errors(logits=PLANE_PAIRS, dh=PLANE_PAIRS, dw=PLANE_PAIRS):
        x = by_planes(c["h"], c["w"], logits)
        lse = torch.logsumexp(x, 1)
        scale = c["dloss"].max()
        g = torch.exp(x - lse[:, None])
        g[torch.arange(M), c["t"]] -= 1
        g = (g * (c["dloss"] / scale).double()[:, None]).float()
        loss = (lse - x.gather(1, c["t"][:, None])[:, 0]).float()
        return norm_errors(loss, lse.float(), (by_planes(g, c["w"].T, dh) * scale).float(),
                           (by_planes(g.T, c["h"].T, dw) * scale).float(), want)

    assert max(errors().values()) < 3e-7
    for pair in PLANE_PAIRS:
        less = [p for p in PLANE_PAIRS if p != pair]
        assert errors(logits=less)["target logits"] > 1.2 * BOUND, pair
        assert errors(dh=less)["dh"] > 1.2 * BOUND, pair
        assert errors(dw=less)["dw"] > 1.2 * BOUND, pair


@gpu
@pytest.mark.parametrize("M,V,K,off", [(48, 70, 64, 0), (64, 64, 64, 1), (40, 300, 96, 0), (130, 515, 513, 0),
                                       (257, 700, 192, 0), (40, 5003, 72, 1), (2050, 3000, 65, 0), (300, 1031, 2056, 0),
                                       (40, 90000, 513, 0), (3000, 40000, 130, 0)])
def test_float32_products_use_all_planes(cuda, M, V, K, off):
    """More than 32 tokens: narrow and full column tiles, aligned and unaligned
    rows, one chain and many, one piece of the vocabulary and several."""
    c = make(M, V, K, "f32", 90 + M, ignored=0)
    out = run(c, off=off)
    errors = norm_errors(out["loss"], out["lse"], out["dh"], out["dw"], exact_step(c))
    assert max(errors.values()) < BOUND, errors


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_targets(cuda, dtype):
    """Out of range, the extremes, the first and last column, the same column
    for all, every row ignored; no ignore index at all."""
    M, V, K = 40, 515, 48
    c = make(M, V, K, dtype, 5, ignored=0)
    c["t"][:8] = torch.tensor([0, V - 1, V, -1, -(2 ** 63), 2 ** 63 - 1, IGNORE, 255])
    check(c, run(c, 1e-3, off=0), 1e-3, what="edges")
    bad = {2, 3, 4, 5}
    out = run(c, dw=False)
    for i in range(8):
        assert bool(out["dh"][i].isnan().all()) == (i in bad) and bool(out["loss"][i].isnan()) == (i in bad)
    assert (out["dh"][6] == 0).all() and out["loss"][6] == 0
    c["t"][2:7] = 3
    check(c, run(c, ignore=None), ignore=None, what="no ignore index")
    check(c, run(c, ignore=3), ignore=3, what="a column as the ignored one")
    c["t"][:] = 300
    check(c, run(c), what="one column")
    c["t"][:] = IGNORE
    out = run(c)
    assert (out["loss"] == 0).all() and out["mean"].isnan().all()
    assert (out["dh"] == 0).all() and (out["dw"] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_the_loss(cuda, dtype):
    """dloss: none (1 for every row), zeros, one constant, tiny and mixed sizes."""
    M, V, K = 70, 600, 80
    c = make(M, V, K, dtype, 9)
    lse = qb.linear_xent_fwd(c["h"], c["w"], c["t"])[1]
    for name, d in (("ones", torch.ones(M)), ("zeros", torch.zeros(M)), ("constant", torch.full((M,), 1 / 37)),
                    ("tiny", torch.full((M,), 2.0 ** -60)), ("signs", torch.linspace(-3, 2, M)),
                    ("mixed", 10.0 ** torch.linspace(-6, 1, M))):
        c["dloss"] = d.to(DEV)
        ref = reference(c)
        dh, dw = qb.linear_xent_bwd(c["h"], c["w"], c["t"], lse, dloss=None if name == "ones" else c["dloss"],
                                    ignore_index=IGNORE)
        near(dh, ref["dh"], ref["tol_dh"], f"dh {name}")
        near(dw, ref["dw"], ref["tol_dw"], f"dw {name}")


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits(cuda, dtype):
    """Logits of hundreds: probabilities of one and of nothing."""
    c = make(50, 700, 64, dtype, 3)
    c["h"] *= 64
    check(c, run(c), what="large")
    c["w"][5:9] = 0
    c["h"][4] = 0  # every logit zero: lse = log V
    out = run(c)
    check(c, out, what="zeros")
    assert abs(out["lse"][4].item() - np.log(700)) < 1e-4


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_that_are_not_finite(cuda, dtype):
    """A NaN in a row of h reaches that row's losses and gradient only, and all of dw."""
    c = make(60, 520, 72, dtype, 4, ignored=0)
    want = run(c)
    c["h"][7, 3] = float("nan")
    c["h"][9, 3] = float("inf")
    out = run(c)
    bad = torch.zeros(60, dtype=torch.bool)
    bad[[7, 9]] = True
    for k in ("loss", "lse"):
        assert not torch.isfinite(out[k][bad]).any() and torch.equal(out[k][~bad], want[k][~bad])
    assert out["dh"][7].isnan().all() and torch.equal(out["dh"][~bad], want["dh"][~bad])
    assert out["dw"][:, 3].isnan().all() and out["mean"].isnan().all()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_of_the_gradients(cuda, dtype):
    c = make(130, 900, 104, dtype, 6)
    both = run(c)
    assert torch.equal(run(c, dw=False)["dh"], both["dh"])
    assert torch.equal(run(c, dh=False)["dw"], both["dw"])


# Tokens of the float32 kernels for few tokens (4, 8, 16 and 32 in registers),
# with rows of vectors and of elements; bf16 beside them.
FEW = [(1, 64), (4, 65), (7, 136), (8, 30), (11, 64), (16, 65), (20, 136), (32, 65)]


@gpu
@pytest.mark.parametrize("M,K", FEW)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_of_the_gradients_of_few_tokens(cuda, dtype, M, K):
    c = make(M, 700, K, dtype, 6)
    for off in (0, 1):
        both = run(c, 1e-3, off=off)
        assert torch.equal(run(c, 1e-3, off=off, dw=False)["dh"], both["dh"])
        assert torch.equal(run(c, 1e-3, off=off, dh=False)["dw"], both["dw"])
        neither = run(c, 1e-3, off=off, dh=False, dw=False)
        assert torch.equal(neither["loss"], both["loss"])


@gpu
@pytest.mark.parametrize("K", [48, 49])
@pytest.mark.parametrize("M", [3, 8, 16, 17, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_targets_of_few_tokens(cuda, dtype, M, K):
    """Out of range at either end, ignored, the first and the last column; all ignored; a single column."""
    V = 515
    c = make(M, V, K, dtype, 5, ignored=0)
    for edges in ([0, V - 1, V], [-1, IGNORE, 255], [-(2 ** 63), 2 ** 63 - 1, 1]):
        c["t"][:3] = torch.tensor(edges)
        out = run(c, 1e-3)
        check(c, out, 1e-3, what=f"{edges}")
        for i, t in enumerate(edges):
            bad = t != IGNORE and not 0 <= t < V
            assert bool(out["dh"][i].isnan().all()) == bad and bool(out["loss"][i].isnan()) == bad
    check(c, run(c, ignore=None), ignore=None, what="no ignore index")
    c["t"][:] = 3
    check(c, run(c), what="one column")
    check(c, run(c, ignore=3), ignore=3, what="every row ignored by a column")
    c["t"][:] = IGNORE
    out = run(c)
    assert (out["loss"] == 0).all() and out["mean"].isnan().all()
    assert (out["dh"] == 0).all() and (out["dw"] == 0).all()
    c = make(M, 1, K, dtype, 5, ignored=0)
    check(c, run(c), what="a vocabulary of one")


@gpu
@pytest.mark.parametrize("M,K", [(3, 72), (8, 73), (16, 72), (30, 73)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_values_that_are_not_finite(cuda, dtype, M, K):
    """A NaN or infinity in a row of h or of w, and NaN in an ignored row's dloss and lse."""
    V = 520
    c = make(M, V, K, dtype, 4, ignored=0)
    want = run(c)
    keep = {k: v.clone() for k, v in c.items()}
    c["h"][1, 3] = float("nan")
    c["h"][2, K - 1] = float("inf")
    out = run(c)
    bad = torch.zeros(M, dtype=torch.bool)
    bad[1:3] = True
    for k in ("loss", "lse"):
        assert not torch.isfinite(out[k][bad]).any() and torch.equal(out[k][~bad], want[k][~bad])
    assert out["dh"][1].isnan().all() and torch.equal(out["dh"][~bad], want["dh"][~bad])
    assert out["dw"].isnan().all() and out["mean"].isnan().all()
    c["h"].copy_(keep["h"])
    c["w"][V - 1, 0] = float("nan")  # every token's logit of that row
    out = run(c)
    assert out["lse"].isnan().all() and out["loss"].isnan().all() and out["dh"].isnan().all()
    c["w"].copy_(keep["w"])
    c["t"][0] = IGNORE
    want = run(c)
    c["dloss"][0] = float("nan")
    lse = want["lse"].clone()
    lse[0] = float("nan")
    dh, dw = qb.linear_xent_bwd(c["h"], c["w"], c["t"], lse, c["dloss"], ignore_index=IGNORE)
    assert torch.equal(dh, want["dh"]) and torch.equal(dw, want["dw"]) and (dh[0] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_same_bits_every_time(cuda, dtype):
    c = make(700, 3000, 264, dtype, 8)
    first = run(c, 1e-4)
    for _ in range(3):
        again = run(c, 1e-4)
        for k in ("loss", "lse", "mean", "dh", "dw"):
            assert torch.equal(first[k], again[k]), k


@gpu
def test_gradients_against_differences(cuda):
    """The float32 kernels' gradients against central differences of the 64-bit
    loss, along random directions (the differences' own error is below 1e-6)."""
    M, V, K, z = 9, 310, 40, 1e-2
    c = make(M, V, K, "f32", 11)

    def f(h, w):
        logits = h @ w.T
        lse = torch.logsumexp(logits, 1)
        skip = c["t"] == IGNORE
        loss = lse - logits[torch.arange(M, device=DEV), torch.where(skip, 0, c["t"])] + z * lse ** 2
        return (torch.where(skip, 0.0, loss) * c["dloss"].double()).sum()

    lse = qb.linear_xent_fwd(c["h"], c["w"], c["t"], ignore_index=IGNORE, z_loss=z)[1]
    dh, dw = qb.linear_xent_bwd(c["h"], c["w"], c["t"], lse, c["dloss"], ignore_index=IGNORE, z_loss=z)
    h, w = c["h"].double(), c["w"].double()
    gen = torch.Generator(device=DEV).manual_seed(0)
    for _ in range(4):
        u, v = (torch.randn(t.shape, generator=gen, device=DEV, dtype=torch.float64) for t in (h, w))
        e = 1e-5
        slope = (f(h + e * u, w + e * v) - f(h - e * u, w - e * v)) / (2 * e)
        got = (dh.double() * u).sum() + (dw.double() * v).sum()
        size = (dh.double() * u).abs().sum() + (dw.double() * v).abs().sum()
        assert (got - slope).abs() <= 2e-5 * size


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_end_of_a_model(cuda, dtype):
    """The last norm and the loss, forward and backward, as a training step
    calls them, against float64 autograd over the same operators (h rounded
    where the path keeps it, y and dy in the working type)."""
    M, N, V = 150, 192, 1100
    _, td = DT[dtype]
    x, r = syn.normal_rows(M, N, dtype, 1, DEV), syn.normal_rows(M, N, dtype, 2, DEV, sigma=3.0)
    g = syn.uniform_weight(N, dtype, 3, DEV)
    c = make(M, V, N, dtype, 4)
    dh_up = syn.normal_rows(M, N, dtype, 5, DEV)
    y, h, rstd = qb.add_rmsnorm_fwd(x, r, g)
    loss, lse, mean = qb.linear_xent_fwd(y, c["w"], c["t"], ignore_index=IGNORE, want_mean=True)
    dloss = torch.full((M,), 1.0 / int((c["t"] != IGNORE).sum()), device=DEV)
    dy, dw = qb.linear_xent_bwd(y, c["w"], c["t"], lse, dloss, ignore_index=IGNORE)
    dx, dg = qb.add_rmsnorm_bwd(h, g, rstd, dy, dh_up)

    h64, g64, w64 = (t.double().requires_grad_() for t in (h, g, c["w"]))
    y64 = h64 * (h64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * g64
    want = torch.nn.functional.cross_entropy(y64 @ w64.T, c["t"], ignore_index=IGNORE)
    gh, gg, gw = torch.autograd.grad(want, (h64, g64, w64))
    # Each stage is off by its half step (2^-8 relative for bf16, float32's
    # otherwise) of the largest values it works on; three stages follow each other.
    step = 3 * 2 ** -8 if dtype == "bf16" else 3e-5
    assert abs(mean.item() - want.item()) <= step * max(1.0, want.item())
    for got, ref in ((dx.double() - dh_up.double(), gh), (dg.double(), gg), (dw.double(), gw)):
        slack = 2 ** -8 * dh_up.double().abs().max() if got.shape == gh.shape and dtype == "bf16" else 0.0
        off = (got - ref).norm() / ref.norm()
        if got.shape == dx.shape:  # dx is rounded at the size of dh, not of its own part
            assert ((got - ref).abs() <= slack + 4 * step * ref.abs().max() + 1e-6).all()
        else:
            assert off <= step


@gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_gradient_that_leaves_the_end_of_a_model(cuda, dtype, residual):
    """dx of the same path in norm, the norm's part alone and beside a residual
    gradient of its size.  Three stages each round what they pass on (dy, g and
    the output: half steps of 2^-8 for bf16, independent), so the whole is off by
    3 half steps in norm at most, float32 by its sums' 3e-5 as above."""
    M, N, V = 150, 192, 1100
    x, r = syn.normal_rows(M, N, dtype, 1, DEV), syn.normal_rows(M, N, dtype, 2, DEV, sigma=3.0)
    g = syn.uniform_weight(N, dtype, 3, DEV)
    c = make(M, V, N, dtype, 4)
    y, h, rstd = qb.add_rmsnorm_fwd(x, r, g)
    lse = qb.linear_xent_fwd(y, c["w"], c["t"], ignore_index=IGNORE)[1]
    dy, dw = qb.linear_xent_bwd(y, c["w"], c["t"], lse, c["dloss"], ignore_index=IGNORE)
    h64, g64, w64 = (t.double().requires_grad_() for t in (h, g, c["w"]))
    y64 = h64 * (h64.square().mean(1, keepdim=True) + 1e-6).rsqrt() * g64
    each = torch.nn.functional.cross_entropy(y64 @ w64.T, c["t"], ignore_index=IGNORE, reduction="none")
    gh, gg, gw = torch.autograd.grad(each, (h64, g64, w64), c["dloss"].double())
    up = None
    if residual:
        up = syn.normal_rows(M, N, dtype, 5, DEV, sigma=gh.std().item())
    dx, dg = qb.add_rmsnorm_bwd(h, g, rstd, dy, up)
    step = 3 * 2 ** -8 if dtype == "bf16" else 3e-5
    want = gh if up is None else gh + up.double()
    assert (want - (0 if up is None else up.double())).norm() > 0.5 * want.norm()  # the norm's part weighs
    for got, ref in ((dx, want), (dg, gg), (dw, gw)):
        assert (got.double() - ref).norm() <= step * ref.norm()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_another_stream_and_a_captured_graph(cuda, dtype):
    c = make(200, 1500, 128, dtype, 21)
    c2 = make(200, 1500, 128, dtype, 22)

    def step(stream=None):
        loss, lse, mean = qb.linear_xent_fwd(c["h"], c["w"], c["t"], ignore_index=IGNORE, want_mean=True, stream=stream)
        dh, dw = qb.linear_xent_bwd(c["h"], c["w"], c["t"], lse, c["dloss"], ignore_index=IGNORE, stream=stream)
        return [loss, lse, mean, dh, dw]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):  # two graphs, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    keep = {k: v.clone() for k, v in c.items()}
    for values in (c2, keep):
        for k in c:
            c[k].copy_(values[k])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        eager = step()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, eager))
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want))


@gpu
def test_two_calls_at_once(cuda):
    """Two streams, each with its own workspace, forward and backward overlapping."""
    cases = [make(600, 4000, 256, "bf16", s) for s in (31, 32)]
    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s in zip(cases, streams):
            _, lse = qb.linear_xent_fwd(c["h"], c["w"], c["t"], ignore_index=IGNORE, stream=s)
            got.append((lse, *qb.linear_xent_bwd(c["h"], c["w"], c["t"], lse, c["dloss"], ignore_index=IGNORE, stream=s)))
    torch.cuda.synchronize()
    for i, (lse, dh, dw) in enumerate(got):
        ref = want[i % 2]
        assert torch.equal(lse, ref["lse"]) and torch.equal(dh, ref["dh"]) and torch.equal(dw, ref["dw"])


@gpu
def test_zero_rows_and_leading_dimensions(cuda):
    w = syn.normal_rows(300, 64, "bf16", 1, DEV)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    loss, lse, mean = qb.linear_xent_fwd(e, w, t, want_mean=True)
    assert loss.shape == (0,) and mean.isnan()
    dh, dw = qb.linear_xent_bwd(e, w, t, lse)
    assert dh.shape == (0, 64) and (dw == 0).all()
    h = syn.normal_rows(24, 64, "bf16", 2, DEV).view(2, 12, 64)
    t = torch.arange(24, device=DEV).view(2, 12)
    loss, lse = qb.linear_xent_fwd(h, w, t)
    flat, _ = qb.linear_xent_fwd(h.view(24, 64), w, t.view(24))
    assert loss.shape == (2, 12) and torch.equal(loss.view(24), flat)
    dh, dw = qb.linear_xent_bwd(h, w, t, lse)
    assert dh.shape == h.shape and dw.shape == w.shape


# --- refusals: fake, never-dereferenced addresses; nothing touches a device ---
A, G = 1 << 32, 1 << 34


def test_forward_refusals(lib):
    f, B, F = lib.qk_linear_xent_fwd, qb.QK_BF16, qb.QK_F32
    p = [A + i * G for i in range(7)]  # h, w, targets, loss, lse, mean, workspace
    n = ctypes.c_size_t(0)
    assert lib.qk_linear_xent_fwd_workspace_size(4, 100, 64, B, ctypes.byref(n)) == qb.QK_OK and n.value > 0
    call = lambda p, size=n.value, M=4, V=100, K=64, dt=B, o=None: f(*p, size, M, V, K, dt, o, None)  # noqa: E731
    for kw in (dict(M=-1), dict(V=0), dict(K=0), dict(dt=5), dict(size=n.value - 1)):
        assert call(p, **kw) == qb.QK_ERR_INVALID_ARG, kw
    for kw in (dict(M=2 ** 31), dict(V=2 ** 31), dict(K=2 ** 31)):
        assert call(p, **kw) == qb.QK_ERR_UNSUPPORTED, kw
    assert call(p, M=2 ** 30, K=2 ** 30) == qb.QK_ERR_UNSUPPORTED  # more bytes than an int64 counts
    for z in (float("nan"), float("inf")):
        assert call(p, o=ctypes.byref(qb.qk_xent_options(0, z, 0))) == qb.QK_ERR_INVALID_ARG
    for i in (0, 1, 2, 3, 6):
        assert call(p[:i] + [None] + p[i + 1:]) == qb.QK_ERR_INVALID_ARG
    for i in range(7):
        assert call(p[:i] + [p[i] + 1] + p[i + 1:]) == qb.QK_ERR_MISALIGNED
    assert call(p[:6] + [p[6] + 128]) == qb.QK_ERR_MISALIGNED
    for i in (3, 4, 5, 6):
        for j in range(7):
            if j != i:
                bad = list(p)
                bad[i] = p[j]
                assert call(bad) == qb.QK_ERR_INVALID_ARG, (i, j)
    size = lib.qk_linear_xent_fwd_workspace_size
    assert size(4, 100, 64, B, None) == qb.QK_ERR_INVALID_ARG
    assert size(4, 100, 64, 9, ctypes.byref(n)) == qb.QK_ERR_INVALID_ARG
    assert size(0, 100, 64, F, ctypes.byref(n)) == qb.QK_OK and n.value == 0


def test_backward_refusals(lib):
    f, B = lib.qk_linear_xent_bwd, qb.QK_BF16
    p = [A + i * G for i in range(8)]  # h, w, targets, lse, dloss, dh, dw, workspace
    n = ctypes.c_size_t(0)
    assert lib.qk_linear_xent_bwd_workspace_size(4, 100, 64, B, ctypes.byref(n)) == qb.QK_OK and n.value > 0
    call = lambda p, size=n.value, M=4, V=100, K=64, dt=B, o=None: f(*p, size, M, V, K, dt, o, None)  # noqa: E731
    for kw in (dict(M=-1), dict(V=0), dict(K=0), dict(dt=5), dict(size=n.value - 1)):
        assert call(p, **kw) == qb.QK_ERR_INVALID_ARG, kw
    for i in (0, 1, 2, 3, 7):
        assert call(p[:i] + [None] + p[i + 1:]) == qb.QK_ERR_INVALID_ARG
    for i in range(8):
        assert call(p[:i] + [p[i] + 1] + p[i + 1:]) == qb.QK_ERR_MISALIGNED
    for i in (5, 6, 7):
        for j in range(8):
            if j != i:
                bad = list(p)
                bad[i] = p[j]
                assert call(bad) == qb.QK_ERR_INVALID_ARG, (i, j)


def test_workspace_does_not_grow_with_the_logits(lib):
    """The largest shapes need far less than their logits: 2 GiB in bfloat16 for 8192 x 131072."""
    n = ctypes.c_size_t(0)
    for f in (lib.qk_linear_xent_fwd_workspace_size, lib.qk_linear_xent_bwd_workspace_size):
        assert f(8192, 131072, 4096, qb.QK_BF16, ctypes.byref(n)) == qb.QK_OK
        assert n.value < 1 << 30
        assert f(65536, 262144, 4096, qb.QK_BF16, ctypes.byref(n)) == qb.QK_OK
        assert n.value < 4 << 30


def test_helpers_refuse_what_is_not_on_a_gpu():
    h, w, t = torch.zeros(2, 8), torch.zeros(5, 8), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        qb.linear_xent_fwd(h, w, t)
    with pytest.raises(ValueError):
        qb.linear_xent_bwd(h, w, t, torch.zeros(2))


@gpu
def test_helper_refusals(cuda):
    h, w = torch.zeros(4, 64, device=DEV), torch.zeros(100, 64, device=DEV)
    t, lse = torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, device=DEV)
    bad = [lambda: qb.linear_xent_fwd(h, w[:, :32], t), lambda: qb.linear_xent_fwd(h, w.bfloat16(), t),
           lambda: qb.linear_xent_fwd(h, w.view(-1), t), lambda: qb.linear_xent_fwd(h, w, t.int()),
           lambda: qb.linear_xent_fwd(h, w, t[:3]), lambda: qb.linear_xent_fwd(h, w, t.cpu()),
           lambda: qb.linear_xent_fwd(h[:, ::2], w[:, ::2], t), lambda: qb.linear_xent_bwd(h, w, t, lse[:2]),
           lambda: qb.linear_xent_bwd(h, w, t, lse.double()), lambda: qb.linear_xent_bwd(h, w, t, lse, dloss=lse[:2])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        qb.linear_xent_fwd(h.half(), w.half(), t)
