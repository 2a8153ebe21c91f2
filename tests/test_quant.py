"""A matrix in 8 bits with a scale for each 128 elements, straight and turned.

Against the definition in float64 on the same inputs.  Tolerances, from the
arithmetic and fixed before the first run:
  * scale: one division and, for bfloat16, one multiplication in float32: 3 2^-24
    relative at most, 2^-22 allowed.
  * q is rounded from the quotient x qmax / max |x| as a rounded float32: equal to
    what float64's quotient gives when rounded the same way.
  * q stands for x to half a step: 2^-4 of the value for e4m3 (or half of the
    subnormal step 2^-9), half a unit for int8.
"""
import numpy as np
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, DT, QT, cuda, guarded, lib, shifted  # noqa: F401

gpu = pytest.mark.gpu
SMALLEST = 2.0 ** -100


def reference(x, rows, qmax):
    """(x / scale in float64, scale in float64, one scale for each element) of x [M, N]."""
    d = x.double()
    M, N = d.shape
    pad = torch.nn.functional.pad(d.abs(), (0, -N % 128, 0, -M % rows))
    top = pad.view(-(-M // rows), rows, -1, 128).amax((1, 3)).clamp_min(SMALLEST)
    each = top.repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :N]
    return d * qmax / each, top / qmax, each / qmax


def rounded(v, qname):
    v = v.float()
    return v.round().double() if qname == "int8" else v.to(torch.float8_e4m3fn).double()


def check(q, scale, x, rows, qname, what):
    v, s, _ = reference(x, rows, QT[qname][2])
    assert ((scale.double() - s).abs() <= 2.0 ** -22 * s).all(), f"{what}: scale"
    got = q.double()
    assert torch.equal(got, rounded(v, qname)), f"{what}: {int((got != rounded(v, qname)).sum())} values differ"


def make(M, N, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g) * torch.exp(torch.randn(M, 1, generator=g)) * scale
    return x.to(DT[dtype][1]).to(DEV)


SIZES = [(1, 1), (1, 128), (2, 7), (3, 130), (8, 64), (16, 4096), (17, 255), (127, 129), (128, 128), (129, 127), (130, 8),
         (200, 1000), (256, 512), (257, 1023), (300, 24), (1000, 65)]


@gpu
@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_against_the_definition(cuda, dtype, M, N):
    code = DT[dtype][0]
    x0 = make(M, N, dtype, M * 1000 + N)
    for qname in ("e4m3", "int8"):
        qcode, qt_type, _ = QT[qname]
        for rows in (1, 128):
            for off in (0, 1):
                x = shifted(x0, off)
                out, checks = {}, []
                for name, shape, t in (("q", (M, N), qt_type),
                                       ("scale", (-(-M // rows), -(-N // 128)), torch.float32),
                                       ("qt", (N, M), qt_type),
                                       ("scale_t", (-(-N // rows), -(-M // 128)), torch.float32)):
                    out[name], c = guarded(shape, t, off)
                    checks.append((name, c))
                alone = []
                qb.qk_quant_fwd(x, out["q"], out["scale"], out["qt"], out["scale_t"], M, N, rows, code, qcode)
                for a, b in ((("q", "scale"), None), (None, ("qt", "scale_t"))):  # one way alone gives the same
                    t = {k: torch.empty_like(out[k]) for k in (a or b)}
                    qb.qk_quant_fwd(x, t.get("q"), t.get("scale"), t.get("qt"), t.get("scale_t"), M, N, rows, code, qcode)
                    alone.append(t)
                torch.cuda.synchronize()
                what = f"{M}x{N} {dtype} {qname} rows {rows} offset {off}"
                for name, c in checks:
                    c(f"{name} {what}")
                check(out["q"], out["scale"], x, rows, qname, "q " + what)
                check(out["qt"], out["scale_t"], x.T, rows, qname, "qt " + what)
                for t in alone:
                    for k, v in t.items():
                        assert torch.equal(v.view(torch.uint8), out[k].view(torch.uint8)), f"{k} alone {what}"


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zeros_extremes_and_values_that_are_not_finite(cuda, dtype):
    M, N = 256, 384
    td = DT[dtype][1]
    x = make(M, N, dtype, 5)
    x[0:128, 128:256] = 0                      # a block of zeros
    x[130, :128] = 2.0 ** -120                 # a group below the smallest
    x[131, :128] = torch.finfo(td).max
    x[132, 5], x[133, 200], x[134, 300] = float("nan"), float("inf"), -float("inf")
    q, scale, qt, scale_t = qb.quant_fwd(x, want_t=True)
    assert (scale[0:128, 1] > 0).all() and (q[0:128, 128:256].float() == 0).all()
    assert scale[130, 0].item() == pytest.approx(SMALLEST / 448, rel=1e-6) and (q[130, :128].float() == 0).all()
    assert (q[131, :128].float() == 448).all() and scale[131, 0].isfinite()
    bad = torch.zeros(M, 3, dtype=torch.bool, device=DEV)
    bad[132, 0] = bad[133, 1] = bad[134, 2] = True
    assert torch.equal(scale.isnan(), bad)
    bad_t = torch.zeros(N, 2, dtype=torch.bool, device=DEV)
    bad_t[5, 1] = bad_t[200, 1] = bad_t[300, 1] = True
    assert torch.equal(scale_t.isnan(), bad_t)
    stands = q.float() * scale.repeat_interleave(128, 1)
    assert torch.equal(stands.isnan().view(M, 3, 128).any(2), bad) and torch.equal(stands.isnan().view(M, 3, 128).all(2), bad)
    q, scale, qt, scale_t = qb.quant_fwd(x, block_rows=128, want_t=True)
    assert torch.equal(scale.T, scale_t) or scale.isnan().any()
    want = torch.tensor([[False] * 3, [True] * 3], device=DEV)
    assert torch.equal(scale.isnan(), want) and torch.equal(scale_t.isnan(), want.T)
    assert torch.equal(q[:128].view(torch.uint8), qt.view(torch.uint8)[:, :128].T)  # blocks: the same values turned


@gpu
def test_leading_dimensions_and_refusals(cuda):
    x = make(6, 200, "bf16", 9)
    q, scale, qt, scale_t = qb.quant_fwd(x.view(2, 3, 200))
    assert q.shape == (2, 3, 200) and scale.shape == (2, 3, 2) and qt is None and scale_t is None
    assert torch.equal(q.view(6, 200).view(torch.uint8), qb.quant_fwd(x)[0].view(torch.uint8))
    assert all(t is None or t.shape[0] == 0 for t in qb.quant_fwd(x[:0]))
    for kw in ({"block_rows": 2}, {"want_q": False}, {"qdtype": torch.float16}):
        with pytest.raises((ValueError, TypeError)):
            qb.quant_fwd(x, **kw)
    with pytest.raises(ValueError):
        qb.quant_fwd(x.view(2, 3, 200), want_t=True)
    with pytest.raises(ValueError):
        qb.quant_fwd(x.T)
    with pytest.raises(TypeError):
        qb.quant_fwd(x.half())


@gpu
def test_offsets_beyond_32_bits(cuda):
    M, N = 70001, 32768  # 2.3e9 elements
    x = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    x[-3:] = make(3, N, "bf16", 11)
    x[:, -5:] = make(M, 5, "bf16", 12)
    q, scale, qt, scale_t = qb.quant_fwd(x, want_t=True)
    check(q[-3:], scale[-3:], x[-3:], 1, "e4m3", "last rows")
    check(qt[-5:], scale_t[-5:], x[:, -5:].T.contiguous(), 1, "e4m3", "last columns")


A = 1 << 32  # never read: refused on the host


def test_refusals(lib):
    def call(x=A, q=A + (1 << 24), scale=A + (2 << 24), qt=None, scale_t=None, M=4, N=256, rows=1, dtype=qb.QK_BF16,
             qtype=qb.QK_E4M3):
        return lib.qk_quant_fwd(x, q, scale, qt, scale_t, M, N, rows, dtype, qtype, None)

    bad = qb.QK_ERR_INVALID_ARG
    assert call(M=-1) == bad and call(N=0) == bad and call(rows=64) == bad and call(dtype=5) == bad
    assert call(qtype=2) == bad and call(x=None) == bad and call(scale=None) == bad and call(q=None) == bad
    assert call(q=None, scale=None) == bad and call(qt=A + (3 << 24)) == bad
    assert call(M=2 ** 40, N=2 ** 40) == bad
    assert call(q=A + 16) == bad and call(scale=A + (1 << 24) + 64) == bad
    assert call(x=A + 1) == qb.QK_ERR_MISALIGNED and call(scale=A + (2 << 24) + 2) == qb.QK_ERR_MISALIGNED
    assert call(M=0, x=None, q=None, scale=None) == qb.QK_OK
