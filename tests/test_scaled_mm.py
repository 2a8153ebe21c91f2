"""8-bit products with a scale for each block of 128.

Against the definition in float64 on the same inputs.  Tolerances, from the
arithmetic and fixed before the first run.  With S = sum over blocks of
|a_scale b_scale| times the block's sum of |a b|:
  * products of e4m3 are exact in float32.  A block's 128 of them are added in
    float32 by the tensor cores, which cut off: at most 2^-23 of the sum of
    their magnitudes each, 2^-16 for 128.  Its two scales round 2^-24 each, and
    so does every addition of the G blocks: (2^-16 + (G + 2) 2^-24) S.
  * bfloat16 outputs: 2^-8 of the value, half a step.
  * whole numbers with scales that are powers of two: no addition rounds while the
    sums stay below 2^24 units; the outputs are equal bit for bit.
Outputs start as a byte pattern, and a guard behind each must come back as it was.
"""
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, DT, cuda, guarded, lib, shifted  # noqa: F401

gpu = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // 128)


def make(M, N, K, seed, experts=None, b_rows=128, whole=False):
    """a, a_scale, b, b_scale on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    lead = () if experts is None else (experts,)

    def values(*shape):
        if whole:
            return torch.randint(-3, 4, shape, generator=g, device=DEV).float().to(E4M3)
        return (torch.randn(*shape, generator=g, device=DEV) * 60).to(E4M3)

    def scales(*shape):
        if whole:
            return 2.0 ** torch.randint(-2, 2, shape, generator=g, device=DEV).float()
        return torch.exp(torch.randn(*shape, generator=g, device=DEV)) * 0.01

    brows = N if b_rows == 1 else blocks(N)
    return (values(M, K), scales(M, blocks(K)), values(*lead, N, K), scales(*lead, brows, blocks(K)))


def reference(a, sa, b, sb):
    """(y, S) in float64 for one set of weights."""
    K, N = a.shape[1], b.shape[0]
    wa = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    wide = sb.double().repeat_interleave(128, 1)[:, :K]
    if sb.shape[0] != N:
        wide = wide.repeat_interleave(128, 0)[:N]
    wb = b.double() * wide
    return wa @ wb.T, wa.abs() @ wb.abs().T


def near(got, ref, S, K, what):
    tol = (2.0 ** -16 + (blocks(K) + 2) * 2.0 ** -24) * S
    if got.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    d = (got.double() - ref).abs()
    assert (d <= tol).all(), f"{what}: {int((~(d <= tol)).sum())} of {d.numel()} outside, worst {(d / tol).max():.3g} of it"


def run(a, sa, b, sb, out, offsets=None, off=0):
    """One call through the C entry, guarded."""
    M, K = a.shape
    N = b.shape[-2]
    experts = 1 if offsets is None else b.shape[0]
    code, td = DT[out]
    y, check = guarded((M, N), td, off)
    n = qb.qk_scaled_mm_workspace_size(M, N, K, experts)
    ws, check_ws = guarded((n,), torch.uint8)
    if K % 16:
        a, b = shifted(a, off), shifted(b, off)
    rows = 1 if sb.shape[-2] == N else 128
    qb.qk_scaled_mm_fwd(a, shifted(sa, off), b, shifted(sb, off), offsets, y, ws if n else None, n, M, N, K, experts,
                        rows, code)
    torch.cuda.synchronize()
    check("y")
    check_ws("workspace")
    return y


SIZES = [(1, 1, 1), (1, 128, 128), (2, 5, 3), (1, 4096, 512), (3, 300, 16), (7, 129, 1040), (15, 127, 17), (16, 256, 256),
         (17, 64, 4096), (31, 1000, 100), (33, 130, 384), (64, 512, 640), (65, 96, 127), (100, 16, 2048), (127, 200, 129),
         (128, 128, 128), (129, 257, 255), (200, 1023, 272), (255, 255, 1000), (256, 256, 512), (257, 385, 513),
         (300, 700, 1152), (513, 40, 96), (700, 2000, 144), (1030, 1100, 320),
         # pairs of CTAs: odd rows, last column tiles of every width class, steps that are no whole quads
         (520, 2089, 640), (777, 2112, 1040), (1025, 1184, 129), (600, 2337, 100), (1500, 1600, 272), (1001, 2047, 1023),
         # tiles of 128 rows of a, alone and with k shared by a cluster
         (374, 1801, 4144), (218, 3612, 3950), (256, 4096, 4096), (500, 2557, 3968)]


@gpu
@pytest.mark.parametrize("M,N,K", SIZES)
def test_against_the_definition(cuda, M, N, K):
    for b_rows in (128, 1):
        for whole in (False, True):
            a, sa, b, sb = make(M, N, K, M + N + K, b_rows=b_rows, whole=whole)
            ref, S = reference(a, sa, b, sb)
            for out in ("f32", "bf16"):
                for off in (0, 1):
                    y = run(a, sa, b, sb, out, off=off)
                    what = f"{M}x{N}x{K} rows {b_rows} {out} offset {off}"
                    if whole:
                        assert torch.equal(y, ref.to(y.dtype)), f"{what}: {int((y != ref.to(y.dtype)).sum())} differ"
                    else:
                        near(y, ref, S, K, what)


def cut(counts, first=0):
    offsets = torch.tensor([first] + counts, dtype=torch.int32).cumsum(0).int()
    return offsets, int(offsets[-1])


GROUPS = [([1], 0, 0), ([0, 0, 3], 0, 0), ([5, 0, 16, 17, 1], 0, 4), ([0, 0, 0], 0, 5), ([130, 1, 0, 64, 300], 3, 0),
          ([700, 2], 0, 1), ([3] * 40, 1, 2), ([1, 0] * 100, 0, 0), ([257, 256, 255, 0, 1], 0, 0)]


def rows_by_expert(counts, before, behind, N, K):
    offsets, end = cut(counts, before)
    M, E = end + behind, len(counts)
    for b_rows in (128, 1):
        a, sa, b, sb = make(M, N, K, M + N, experts=E, b_rows=b_rows, whole=True)
        y = run(a, sa, b, sb, "f32", offsets.to(DEV))
        for e in range(E):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            ref, _ = reference(a[lo:hi], sa[lo:hi], b[e], sb[e])
            assert torch.equal(y[lo:hi].double(), ref), f"expert {e} of {counts}"
        left = torch.cat([y[:before], y[end:]]).view(torch.uint8)
        assert (left == 0xA5).all(), "rows of no expert were written"


@gpu
@pytest.mark.parametrize("counts,before,behind", GROUPS)
@pytest.mark.parametrize("N,K", [(200, 144), (384, 1280), (129, 77)])
def test_rows_by_expert(cuda, counts, before, behind, N, K):
    rows_by_expert(counts, before, behind, N, K)


MANY = [([700, 257, 0, 900, 31], 3, 2, 2080, 1280), ([300] * 6, 0, 5, 2200, 1100), ([513, 40, 800], 1, 0, 1999, 384),
        ([129, 256, 1, 700], 0, 0, 2600, 200), ([120] * 8, 2, 2, 2050, 1500), ([180, 155], 0, 1, 2391, 4128),
        ([700, 600, 65, 0, 300], 0, 0, 1500, 640)]


@gpu
@pytest.mark.parametrize("counts,before,behind,N,K", MANY)
def test_many_rows_by_expert(cuda, counts, before, behind, N, K):
    rows_by_expert(counts, before, behind, N, K)


@gpu
def test_operands_beyond_32_bits(cuda):
    K, N = 16384, 72
    a, sa, b, sb = make(1000, N, K, 71, whole=True)
    M = 270000  # 4.4e9 bytes of a
    big, scales = a.repeat(M // 1000, 1), sa.repeat(M // 1000, 1)
    y = qb.scaled_mm_fwd(big, scales, b, sb, out_dtype=torch.float32)
    ref = reference(a, sa, b, sb)[0]
    for first in (0, 130000, M - 1000):
        assert torch.equal(y[first:first + 1000].double(), ref)
    del big, scales, y
    E, N = 70, 4096  # 4.7e9 bytes of b
    a, sa, b, sb = make(9, N, K, 72, whole=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:], offsets[E] = 4, 9  # the first expert and the last
    y = qb.scaled_mm_fwd(a, sa, b.expand(E, N, K).contiguous(), sb.expand(E, *sb.shape).contiguous(), offsets.to(DEV))
    assert torch.equal(y, reference(a, sa, b, sb)[0].to(y.dtype))


@gpu
def test_many_experts_and_offsets_that_fall(cuda):
    E, N, K = 1024, 136, 256
    g = torch.Generator().manual_seed(3)
    counts = torch.randint(0, 4, (E,), generator=g).tolist()
    offsets, M = cut(counts)
    a, sa, b, sb = make(M, N, K, 4, experts=E, whole=True)
    y = run(a, sa, b, sb, "bf16", offsets.to(DEV))
    for e in range(0, E, 37):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        assert torch.equal(y[lo:hi], reference(a[lo:hi], sa[lo:hi], b[e], sb[e])[0].to(y.dtype))
    wild = torch.tensor([-5, 10, 4, 20, 1 << 30, 7], dtype=torch.int32)
    a, sa, b, sb = make(50, N, K, 5, experts=5, whole=True)
    y = run(a, sa, b, sb, "f32", wild.to(DEV))
    for e, (lo, hi) in enumerate([(0, 10), (10, 10), (10, 20), (20, 50), (50, 50)]):
        assert torch.equal(y[lo:hi].double(), reference(a[lo:hi], sa[lo:hi], b[e], sb[e])[0])


@gpu
@pytest.mark.parametrize("M", [5, 100, 600])
def test_values_that_are_not_numbers_stay_in_their_row_and_column(cuda, M):
    N, K = 700, 384
    a, sa, b, sb = make(M, N, K, 21, whole=True)
    ref, _ = reference(a, sa, b, sb)
    a.view(torch.uint8)[3, 200] = 0x7F
    b.view(torch.uint8)[150, 7] = 0xFF
    sa[1, 2] = float("nan")
    y = run(a, sa, b, sb, "f32")
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    want[3] = want[1] = want[:, 150] = True
    assert torch.equal(y.isnan(), want)
    assert torch.equal(y[~want].double(), ref[~want])
    sb[0, 0] = float("inf")
    y = run(a, sa, b, sb, "f32")
    assert not y[:, :128].isfinite().any()
    assert torch.equal(y[:, 128:].isnan(), want[:, 128:])


@gpu
def test_runs_repeat_and_graphs_replay(cuda):
    offsets, M = cut([40, 0, 90, 7])
    cases = [make(9, 512, 4096, 31) + (None,), make(300, 384, 1000, 32) + (None,), make(600, 1024, 512, 33) + (None,),
             make(M, 256, 768, 34, experts=4) + (offsets.to(DEV),)]
    first = [qb.scaled_mm_fwd(*c) for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [qb.scaled_mm_fwd(*c, stream=side) for c in cases]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [qb.scaled_mm_fwd(*c) for c in cases]
    for _ in range(2):
        for h in held:
            h.fill_(7)
        graph.replay()
    torch.cuda.synchronize()
    for f, g, h in zip(first, again, held):
        assert torch.equal(f, g) and torch.equal(f, h)


@gpu
def test_outputs_beyond_32_bits(cuda):
    M, N, K = 70001, 32768, 32
    a, sa, b, sb = make(M, N, K, 41, whole=True)
    y = qb.scaled_mm_fwd(a, sa, b, sb)
    for rows in (slice(0, 3), slice(65530, 65540), slice(M - 3, M)):
        assert torch.equal(y[rows], reference(a[rows], sa[rows], b, sb)[0].to(y.dtype))


@gpu
def test_helper_shapes_and_refusals(cuda):
    a, sa, b, sb = make(6, 200, 300, 51)
    y = qb.scaled_mm_fwd(a, sa, b, sb)
    assert y.dtype == torch.bfloat16 and y.shape == (6, 200)
    assert torch.equal(y.view(2, 3, 200), qb.scaled_mm_fwd(a.view(2, 3, 300), sa.view(2, 3, 3), b, sb))
    out = torch.empty(6, 200, device=DEV)
    assert qb.scaled_mm_fwd(a, sa, b, sb, out=out) is out
    assert torch.equal(out.bfloat16(), y)
    assert qb.scaled_mm_fwd(a[:0], sa[:0], b, sb).shape == (0, 200)
    for wrong in ((a.view(torch.int8), sa, b, sb), (a, sa[:, :2], b, sb), (a, sa, b[:, :299], sb), (a, sa, b, sb[:1]),
                  (a, sa.double(), b, sb), (a, sa, b.T, sb), (a.cpu(), sa, b, sb)):
        with pytest.raises((ValueError, TypeError)):
            qb.scaled_mm_fwd(*wrong)
    with pytest.raises(ValueError):
        qb.scaled_mm_fwd(a, sa, b, sb, offsets=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError):
        qb.scaled_mm_fwd(a, sa, b, sb, out_dtype=torch.float16)


@gpu
def test_reads_what_the_norm_and_the_quantiser_leave(cuda):
    """A linear layer behind a norm, forward and backward in 8 bits: each product against float64 of its operands."""
    M, K, N = 300, 640, 384
    g = torch.Generator(device=DEV).manual_seed(61)
    x, r = (torch.randn(M, K, generator=g, device=DEV).bfloat16() for _ in range(2))
    w = torch.randn(N, K, generator=g, device=DEV) * K ** -0.5
    dy = torch.randn(M, N, generator=g, device=DEV).bfloat16()
    gain = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    q, sq, h, rstd = qb.rmsnorm_quant_fwd(x, gain, residual=r, group=128)
    qw, sw, qwt, swt = qb.quant_fwd(w, block_rows=128, want_t=True)
    y = qb.scaled_mm_fwd(q, sq, qw, sw)
    near(y, *reference(q, sq, qw, sw), K, "y")
    gq, gs, gqt, gst = qb.quant_fwd(dy, want_t=True)
    _, _, hqt, hst = qb.quant_fwd(h, want_q=False, want_t=True)
    dx = qb.scaled_mm_fwd(gq, gs, qwt, swt)
    near(dx, *reference(gq, gs, qwt, swt), N, "dx")
    dw = qb.scaled_mm_fwd(gqt, gst, hqt, hst, out_dtype=torch.float32)
    near(dw, *reference(gqt, gst, hqt, hst), M, "dw")
    # and all of it near the unquantised products: each factor is off by 2^-4 of itself at most,
    # in a group whose smallest are off by half a step 2^-9 of a scale = max / 448
    d64 = dy.double().T @ h.double()
    off = 2 * 2.0 ** -4 * (dy.double().abs().T @ h.double().abs())
    assert ((dw.double() - d64).abs() <= 1.1 * off + 1e-3).all()


A = 1 << 32  # never read: refused on the host


def test_refusals(lib):
    def call(a=A, sa=A + (1 << 24), b=A + (2 << 24), sb=A + (3 << 24), offsets=None, y=A + (4 << 24), ws=None, n=0, M=4,
             N=256, K=128, experts=1, rows=128, dtype=qb.QK_BF16):
        return lib.qk_scaled_mm_fwd(a, sa, b, sb, offsets, y, ws, n, M, N, K, experts, rows, dtype, None)

    bad = qb.QK_ERR_INVALID_ARG
    assert call(M=-1) == bad and call(N=0) == bad and call(K=0) == bad and call(experts=0) == bad
    assert call(rows=64) == bad and call(dtype=3) == bad and call(experts=2) == bad
    for name in ("a", "sa", "b", "sb", "y"):
        assert call(**{name: None}) == bad
    assert call(K=100) == bad  # needs a workspace
    assert call(K=100, ws=A + (5 << 24), n=100) == bad
    assert call(K=100, ws=A + (5 << 24) + 16, n=1 << 20) == qb.QK_ERR_MISALIGNED
    assert call(K=100, ws=A + (4 << 24), n=1 << 20) == bad and call(K=100, ws=A, n=1 << 20) == bad
    assert call(a=A + 8) == qb.QK_ERR_MISALIGNED and call(b=A + (2 << 24) + 4) == qb.QK_ERR_MISALIGNED
    assert call(sa=A + (1 << 24) + 2) == qb.QK_ERR_MISALIGNED and call(y=A + (4 << 24) + 1) == qb.QK_ERR_MISALIGNED
    assert call(y=A) == bad and call(y=A + (3 << 24)) == bad
    assert call(offsets=A + (5 << 24), experts=1025) == qb.QK_ERR_UNSUPPORTED
    assert call(M=2 ** 31) == qb.QK_ERR_UNSUPPORTED
    assert call(M=2 ** 31 - 2000, N=2 ** 31 - 2000, K=16) == qb.QK_ERR_UNSUPPORTED  # more tiles than are counted
    assert call(M=0, a=None, y=None) == qb.QK_OK
    assert qb.qk_scaled_mm_workspace_size(5, 7, 100, 3) == (5 + 21) * 112
    assert qb.qk_scaled_mm_workspace_size(5, 7, 160, 3) == 0
