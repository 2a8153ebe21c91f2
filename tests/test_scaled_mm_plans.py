"""Every kernel of the 8-bit products, by its plan.

Which kernel a call takes is an estimate's decision from its sizes.  So sizes are drawn (with a fixed
seed) until the plan names each kernel, in each form that it is called in, several times; those calls
are compared, and a kernel that no drawn size reaches fails its test.  Inputs are small whole numbers
with scales that are powers of two: sums stay below 2^24 units, so that no addition rounds and outputs
are equal bit for bit to float64's.
"""
import random

import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, DT, cuda, guarded, lib, shifted  # noqa: F401
from test_scaled_mm import make, reference, run

gpu = pytest.mark.gpu
EACH = 3        # calls of a form
DRAWS = 30000

# (by expert, rows of a tile, CTAs that share it, output) of the tiles of a few rows ...
TILES = [(e, rows, ctas, out) for e in (False, True) for rows in (16, 32, 64, 128) for ctas in (1, 2, 4, 8)
         for out in ("f32", "bf16")]
# ... and (by expert, 256, 2, output, rows of b of a scale, rows of y on 16 bytes) of the pairs.
PAIRS = [(e, 256, 2, out, b_rows, on16) for e in (False, True) for out in ("f32", "bf16") for b_rows in (128, 1)
         for on16 in (True, False)]


def spread(rng, lo, hi, unit=1):
    n = round(lo * (hi / lo) ** rng.random())
    return max(1, n // unit * unit)


def drawn():
    """{form: calls of it}; a call is (rows of each expert or of all, rows in front and behind, N, K, rows of b of a
    scale, output, elements that y starts off 16 bytes)."""
    rng, found = random.Random(20), {}
    for _ in range(DRAWS):
        if rng.random() < 0.5:
            counts, before, behind, by_expert = [spread(rng, 1, 2500)], 0, 0, False
        else:
            most = spread(rng, 1, 900)
            counts = [rng.choice([0, 1, most, rng.randint(0, most)]) for _ in range(spread(rng, 1, 40))]
            before, behind, by_expert = rng.choice([0, 0, 3]), rng.choice([0, 0, 5]), True
        unit = rng.choice([1, 8, 32])
        N, K = spread(rng, 1, 5000, unit), spread(rng, 1, rng.choice([5000, 5000, 60000]), rng.choice([1, 16]))
        M, E = before + sum(counts) + behind, len(counts)
        if M == 0 or M * N * K > 1.5e10 or E * N * K > 4e8 or M * N > 2e7:
            continue
        out, b_rows, off = rng.choice(["f32", "bf16"]), rng.choice([128, 1]), rng.choice([0, 0, 1])
        code, td = DT[out]
        es = td.itemsize
        offsets, y = 4096 if by_expert else None, 4096 + off * es  # not read
        p = qb.qk_scaled_mm_get_plan(offsets, y, M, N, K, E, b_rows, code)
        form = (by_expert, p["rows"], p["ctas"], out)
        if p["rows"] == 256:
            form += (b_rows, off == 0 and N * es % 16 == 0)
        calls = found.setdefault(form, [])
        if len(calls) < EACH:
            calls.append((counts, before, behind, N, K, b_rows, out, off))
    return found


@pytest.fixture(scope="module")
def calls(cuda):
    return drawn()


def check(call, form):
    counts, before, behind, N, K, b_rows, out, off = call
    by_expert = form[0]
    end = before + sum(counts)
    a, sa, b, sb = make(end + behind, N, K, N + K, experts=len(counts) if by_expert else None, b_rows=b_rows, whole=True)
    if not by_expert:
        y, (ref, _) = run(a, sa, b, sb, out, off=off), reference(a, sa, b, sb)
        assert torch.equal(y, ref.to(y.dtype)), f"{form} {call}: {int((y != ref.to(y.dtype)).sum())} differ"
        return
    offsets = torch.tensor([before] + counts, dtype=torch.int32).cumsum(0).int()
    y = run(a, sa, b, sb, out, offsets.to(DEV), off=off)
    for e in range(len(counts)):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo < hi:
            ref = reference(a[lo:hi], sa[lo:hi], b[e], sb[e])[0].to(y.dtype)
            assert torch.equal(y[lo:hi], ref), f"{form} {call} expert {e}: {int((y[lo:hi] != ref).sum())} differ"
    left = torch.cat([y[:before], y[end:]]).contiguous().view(torch.uint8)
    assert (left == 0xA5).all(), f"{form} {call}: rows of no expert were written"


@gpu
@pytest.mark.parametrize("form", TILES + PAIRS, ids=str)
def test_each_kernel(calls, form):
    assert form in calls, "no drawn size reaches this kernel"
    for call in calls[form]:
        check(call, form)


@gpu
def test_no_other_plan(calls):
    assert set(calls) <= set(TILES + PAIRS)


@gpu
def test_plans_of_known_sizes(cuda):
    """What the sizes alone decide: many rows go to pairs, a few to narrow tiles, and no grid exceeds the GPU."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plan = lambda M, N, K: qb.qk_scaled_mm_get_plan(None, None, M, N, K, 1, 128, qb.QK_BF16)  # noqa: E731
    assert plan(16384, 8192, 4096)["rows"] == 256 and plan(1, 4096, 4096)["rows"] == 16
    assert set(plan(0, 4096, 4096).values()) == {0}
    for M in (1, 17, 100, 300, 1000, 5000):
        p = plan(M, 4096, 4096)
        assert 0 < p["grid"] <= sms and p["grid"] % p["ctas"] == 0


def test_refusals_of_a_plan(lib):
    import ctypes
    p = qb.qk_scaled_mm_plan()
    get = lambda offsets=None, M=4, N=256, K=128, E=1, rows=128, dtype=qb.QK_BF16, at=ctypes.byref(p): (  # noqa: E731
        lib.qk_scaled_mm_get_plan(offsets, None, M, N, K, E, rows, dtype, at))
    bad = qb.QK_ERR_INVALID_ARG
    assert get(M=-1) == bad and get(N=0) == bad and get(K=0) == bad and get(E=0) == bad and get(E=2) == bad
    assert get(rows=64) == bad and get(dtype=3) == bad and get(at=None) == bad
    assert get(offsets=4096, E=1025) == qb.QK_ERR_UNSUPPORTED and get(M=2 ** 31) == qb.QK_ERR_UNSUPPORTED
    assert get(M=0) == qb.QK_OK
