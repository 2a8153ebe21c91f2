"""RMSNorm with the residual's addition: forward, 8-bit output, backward.

Against the definitions in float64 on the same inputs.  Tolerances, fixed
before the first run:
  * h is x + residual rounded once: equal bit for bit.
  * rstd, scale: relative error 1e-5 (float32 sums); y: parity.check_rows
    (one bf16 ulp, or 1e-5 relative); dx and dw: parity.check_scaled on the
    magnitude of their terms.
  * q * scale stands for y to half a step: 2^-4 of the value for e4m3 (and half
    of the subnormal step 2^-9, in units of scale), half a unit of scale for
    int8, plus 1e-4 of the value: the float32 error of y and of y / scale (two
    parts in 1e5) may also move a value across a tie, which doubles nothing --
    either neighbour is within half a step and that error.
Outputs start as NaN (or a byte pattern), and a guard behind each one must
come back as it was.
"""
import numpy as np
import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from memory_bound_row_rmsnorm_gb300 import synthetic as syn
from parity import check_rows, check_scalars, check_scaled, to_f64

DEV = "cuda:0"
EPS = 1e-6
DT = {"f32": (qb.QK_F32, torch.float32), "bf16": (qb.QK_BF16, torch.bfloat16)}
QT = {"e4m3": (qb.QK_E4M3, torch.float8_e4m3fn, 448.0), "int8": (qb.QK_INT8, torch.int8, 127.0)}
GUARD = 64  # elements behind every output

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from memory_bound_row_rmsnorm_gb300 import build
    build.build()
    return qb.load_library()


@pytest.fixture(scope="module")
def cuda(lib):
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    torch.cuda.set_device(0)
    yield
    assert qb.qk_get_device_status() == qb.QK_OK


def guarded(shape, dtype, offset=0):
    """A contiguous tensor of that shape inside a larger buffer, `offset`
    elements after its start, and a check that nothing around it changed."""
    n = int(np.prod(shape))
    buf = torch.empty(offset + n + GUARD, dtype=dtype, device=DEV)
    raw = buf.view(torch.uint8)
    raw.fill_(0xA5)
    before = raw.clone()
    view = buf[offset:offset + n].view(shape)
    e = buf.element_size()

    def check(what):
        assert torch.equal(raw[:offset * e], before[:offset * e]), f"{what}: written before its start"
        assert torch.equal(raw[(offset + n) * e:], before[(offset + n) * e:]), f"{what}: written behind its end"
    return view, check


def shifted(t, offset):
    """t's values in a buffer that starts `offset` elements off an allocation."""
    buf = torch.empty(offset + t.numel(), dtype=t.dtype, device=DEV)
    view = buf[offset:].view(t.shape)
    view.copy_(t)
    return view


def rows(M, N, dtype, seed, sigma=1.0):
    return syn.normal_rows(M, N, dtype, seed, "cpu", sigma=sigma)


def forward64(x, r, w):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    f = to_f64(h)
    rstd = 1.0 / np.sqrt((f * f).mean(1) + EPS)
    return h, f * rstd[:, None] * to_f64(w)[None, :], rstd


NS = [1, 2, 7, 8, 31, 64, 100, 128, 255, 256, 513, 1000, 1023, 1024, 2048, 4096, 5000, 8192, 16384]
MS = [1, 3, 37]


@gpu
@pytest.mark.parametrize("N", NS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward(cuda, dtype, N):
    for M in MS:
        code, td = DT[dtype]
        x, r, w = rows(M, N, dtype, N, 1.0), rows(M, N, dtype, N + 1, 3.0), syn.uniform_weight(N, dtype, N + 2, "cpu")
        h_ref, y_ref, rstd_ref = forward64(x, r, w)
        for off in (0, 1):
            y, cy = guarded((M, N), td, off)
            h, ch = guarded((M, N), td, off)
            rstd, cr = guarded((M,), torch.float32)
            qb.qk_add_rmsnorm_fwd(shifted(x, off), shifted(r, off), shifted(w, off), y, h, rstd, M, N, EPS, code)
            torch.cuda.synchronize()
            for c, what in ((cy, "y"), (ch, "h"), (cr, "rstd")):
                c(f"{what} {M}x{N} {dtype} offset {off}")
            assert torch.equal(h.cpu(), h_ref)
            check_scalars(to_f64(rstd), rstd_ref, "rstd")
            check_rows(to_f64(y), y_ref, dtype, False, f"y {M}x{N} {dtype} offset {off}")


@gpu
@pytest.mark.parametrize("dtype,M,N", [("bf16", 3, 40000), ("f32", 2, 70001), ("bf16", 700, 4096), ("bf16", 2000, 264),
                                       ("f32", 1300, 1028), ("bf16", 5000, 72), ("bf16", 3, 131072), ("f32", 2, 32768)])
def test_forward_long_rows_and_many_rows(cuda, dtype, M, N):
    x, r, w = rows(M, N, dtype, 5), rows(M, N, dtype, 6, 3.0), syn.uniform_weight(N, dtype, 7, "cpu")
    h_ref, y_ref, rstd_ref = forward64(x, r, w)
    y, h, rstd = qb.add_rmsnorm_fwd(x.to(DEV), r.to(DEV), w.to(DEV), eps=EPS)
    assert torch.equal(h.cpu(), h_ref)
    check_scalars(to_f64(rstd), rstd_ref, "rstd")
    check_rows(to_f64(y), y_ref, dtype, False, "y")


@gpu
@pytest.mark.parametrize("N", [96, 1000, 1003, 4096, 33000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_in_place(cuda, dtype, N):
    """Every exact aliasing that the interface allows gives the same bits."""
    M = 19
    x, r, w = rows(M, N, dtype, 1), rows(M, N, dtype, 2, 3.0), syn.uniform_weight(N, dtype, 3, "cpu").to(DEV)
    y0, h0, s0 = qb.add_rmsnorm_fwd(x.to(DEV), r.to(DEV), w, eps=EPS)
    for where_y, where_h in (("x", "r"), ("r", "x"), (None, "r"), (None, "x"), ("x", None), ("r", None)):
        d = {"x": x.to(DEV), "r": r.to(DEV)}
        y, h, s = qb.add_rmsnorm_fwd(d["x"], d["r"], w, eps=EPS, out=d.get(where_y), out_h=d.get(where_h))
        assert torch.equal(y, y0) and torch.equal(h, h0) and torch.equal(s, s0), (where_y, where_h)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_is_the_norm_of_the_kept_sum(cuda, dtype):
    """h, then qk_rmsnorm_fwd on it, within a rounding of the fused call."""
    x, r = rows(50, 4096, dtype, 1).to(DEV), rows(50, 4096, dtype, 2, 3.0).to(DEV)
    w = syn.uniform_weight(4096, dtype, 3, DEV)
    y, h, rstd = qb.add_rmsnorm_fwd(x, r, w, eps=EPS)
    y2, rstd2 = qb.rmsnorm_fwd(h, w, eps=EPS)
    check_scalars(to_f64(rstd), to_f64(rstd2), "rstd")
    check_rows(to_f64(y), to_f64(y2), dtype, False, "y")


@gpu
@pytest.mark.parametrize("N", [64, 100, 4096])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_values_that_are_not_finite(cuda, dtype, N):
    """A NaN or infinity stays in its row; a row of zeros gives zeros."""
    M = 9
    x, r, w = rows(M, N, dtype, 1), rows(M, N, dtype, 2), syn.uniform_weight(N, dtype, 3, "cpu")
    x[1, N // 2] = float("nan")
    x[3, 0] = float("inf")
    x[5], r[5] = 0, 0
    with np.errstate(all="ignore"):
        h_ref, y_ref, rstd_ref = forward64(x, r, w)
    y, h, rstd = qb.add_rmsnorm_fwd(x.to(DEV), r.to(DEV), w.to(DEV), eps=EPS)
    assert torch.equal(h.cpu().isnan(), h_ref.isnan()) and rstd[3].item() == 0
    check_rows(to_f64(y), y_ref, dtype, False, "y")
    q, scale, h, rstd = qb.rmsnorm_quant_fwd(x.to(DEV), w.to(DEV), residual=r.to(DEV), eps=EPS)
    bad = torch.tensor([i in (1, 3) for i in range(M)])
    assert torch.equal(scale.cpu().isnan()[:, 0], bad)
    assert (scale.cpu()[~bad] > 0).all() and (q[5].float() == 0).all() and torch.isfinite(q[~bad].float()).all()
    group = 32
    q, scale, h, rstd = qb.rmsnorm_quant_fwd(x.to(DEV), w.to(DEV), residual=r.to(DEV), eps=EPS, group=group,
                                             qdtype=torch.int8)
    assert scale[1].isnan().all()      # the whole row is NaN with its rstd
    expect = torch.zeros(scale.shape[1], dtype=torch.bool)
    expect[0] = True                   # inf * 0 in one group, zeros in the others
    assert torch.equal(scale[3].cpu().isnan(), expect)


def check_quant(q, scale, y, group, qtype, what):
    M, N = y.shape
    qmax = QT[qtype][2]
    g = group or N
    pieces = -(-N // g)
    pad = np.zeros((M, pieces * g))
    pad[:, :N] = np.abs(y)
    want = np.maximum(pad.reshape(M, pieces, g).max(2), 2.0 ** -100) / qmax
    check_scalars(to_f64(scale), want, f"{what} scale")
    s = np.repeat(to_f64(scale).reshape(M, pieces), g, 1)[:, :N]
    v = q.float().double().cpu().numpy() if qtype == "e4m3" else to_f64(q)
    assert np.isfinite(v).all() and np.abs(v).max() <= qmax
    half = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) if qtype == "e4m3" else 0.5 * s
    err = np.abs(v * s - y)
    assert (err <= half + 1e-4 * np.abs(y)).all(), f"{what}: {(err - half).max()}"


@gpu
@pytest.mark.parametrize("N", [1, 7, 31, 64, 100, 128, 255, 1000, 1024, 1023, 4096, 8192, 16384])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("qtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quant(cuda, dtype, qtype, group, N):
    code, td = DT[dtype]
    qc, qd, _ = QT[qtype]
    groups = -(-N // group) if group else 1
    for M, residual, off in ((1, True, 0), (21, True, 1), (21, False, 0), (3, False, 1)):
        x, r, w = rows(M, N, dtype, N), rows(M, N, dtype, N + 1, 3.0), syn.uniform_weight(N, dtype, N + 2, "cpu")
        h_ref, y_ref, rstd_ref = forward64(x, r if residual else None, w)
        q, cq = guarded((M, N), torch.int8, off)
        scale, cs = guarded((M, groups), torch.float32)
        h, ch = guarded((M, N), td, off)
        rstd, cr = guarded((M,), torch.float32)
        qb.qk_rmsnorm_quant_fwd(shifted(x, off), shifted(r, off) if residual else None, shifted(w, off), q, scale,
                                h if residual else None, rstd, M, N, EPS, group, code, qc)
        torch.cuda.synchronize()
        for c, what in ((cq, "q"), (cs, "scale"), (ch, "h"), (cr, "rstd")):
            c(what)
        if residual:
            assert torch.equal(h.cpu(), h_ref)
        check_scalars(to_f64(rstd), rstd_ref, "rstd")
        check_quant(q.view(qd), scale, y_ref, group, qtype, f"{M}x{N} {dtype} {qtype} {group} offset {off}")


@gpu
@pytest.mark.parametrize("dtype,M,N,group", [("bf16", 700, 4096, 128), ("bf16", 3, 40000, 0), ("f32", 2, 20000, 64),
                                             ("bf16", 3000, 264, 32), ("f32", 1300, 1028, 0), ("bf16", 2, 70000, 128)])
def test_quant_long_rows_and_many_rows(cuda, dtype, M, N, group):
    x, r, w = rows(M, N, dtype, 5), rows(M, N, dtype, 6, 3.0), syn.uniform_weight(N, dtype, 7, "cpu")
    h_ref, y_ref, _ = forward64(x, r, w)
    q, scale, h, rstd = qb.rmsnorm_quant_fwd(x.to(DEV), w.to(DEV), residual=r.to(DEV), eps=EPS, group=group)
    assert torch.equal(h.cpu(), h_ref)
    check_quant(q, scale, y_ref, group, "e4m3", f"{M}x{N}")
    # without h, and with h over the residual: the same q
    rd = r.to(DEV)
    q2, s2, none, _ = qb.rmsnorm_quant_fwd(x.to(DEV), w.to(DEV), residual=rd, eps=EPS, group=group, want_h=False)
    q3, s3, h3, _ = qb.rmsnorm_quant_fwd(x.to(DEV), w.to(DEV), residual=rd, eps=EPS, group=group, out_h=rd)
    assert none is None and torch.equal(h3.cpu(), h_ref)
    for a, b in ((q2, s2), (q3, s3)):
        assert torch.equal(a.view(torch.int8), q.view(torch.int8)) and torch.equal(b, scale)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quant_of_a_row_that_covers_every_code(cuda, dtype):
    """Values laid out over the whole range of e4m3, from the subnormals up."""
    N = 512
    x = torch.logspace(-8, 0, N, base=4.0).to(DT[dtype][1])[None] * torch.tensor([[1.0], [-1.0]]).to(DT[dtype][1])
    w = torch.ones(N, dtype=DT[dtype][1])
    _, y_ref, _ = forward64(x, None, w)
    for qtype in QT:
        q, scale, _, _ = qb.rmsnorm_quant_fwd(x.to(DEV), w.to(DEV), eps=EPS, qdtype=QT[qtype][1])
        check_quant(q, scale, y_ref, 0, qtype, qtype)


@gpu
@pytest.mark.parametrize("N", [4096, 1000, 1023])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("qtype", ["e4m3", "int8"])
def test_quant_is_the_rounded_quotient(cuda, qtype, group, N):
    """q against the division of the float32 y that the plain norm gives (the
    same sums in the same order), rounded by torch: equal but where y itself
    differs, which the equal rstd excludes."""
    x, r, w = rows(300, N, "f32", 1).to(DEV), rows(300, N, "f32", 2, 3.0).to(DEV), syn.uniform_weight(N, "f32", 3, DEV)
    y, _, rstd = qb.add_rmsnorm_fwd(x, r, w, eps=EPS)
    _, qd, _ = QT[qtype]
    q, scale, _, rstd2 = qb.rmsnorm_quant_fwd(x, w, residual=r, eps=EPS, group=group, qdtype=qd)
    same = rstd == rstd2
    assert same.any()
    wide = torch.repeat_interleave(scale, group or N, 1)[:, :N]
    want = y / wide
    want = want.round() if qtype == "int8" else want.to(qd).float()
    assert torch.equal(q.float()[same], want[same])


def eight_bits_of_the_ratio(h, w, group, qtype):
    """q of bf16 rows by the definition alone: h w qmax / max |h w|, in which
    the row's rstd cancels.  In float64 the products are exact, the quotient is
    rounded once, and what lies on a tie is one: such a quotient has few bits.
    (One that is off a tie is so by 2^-24 of itself at least, since h w has 16
    bits, so float32's rounding on the way to e4m3 makes none.)"""
    p = to_f64(h) * to_f64(w)[None, :]
    M, N = p.shape
    g = group or N
    pieces = -(-N // g)
    pad = np.zeros((M, pieces * g))
    pad[:, :N] = np.abs(p)
    top = np.repeat(pad.reshape(M, pieces, g).max(2), g, 1)[:, :N]
    v = np.divide(p * QT[qtype][2], top, out=np.zeros_like(p), where=top > 0)
    ties = v * 2 - np.floor(v * 2) == 0 if qtype == "int8" else np.zeros_like(v, dtype=bool)
    if qtype == "e4m3":
        step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -40))), -6) - 3)
        u = np.abs(v) / step
        return torch.from_numpy(v).float().to(torch.float8_e4m3fn), int((u - np.floor(u) == 0.5).sum())
    return torch.from_numpy(np.rint(v)).to(torch.int8), int((ties & (v != np.floor(v))).sum())


@gpu
@pytest.mark.parametrize("M,N,off", [(64, 4096, 0), (200, 264, 0), (64, 1003, 0), (40, 2048, 1), (8, 8192, 0), (3, 9001, 0),
                                     (2, 32768, 0), (2, 40000, 0)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("qtype", ["e4m3", "int8"])
def test_quant_ties_go_to_even(cuda, qtype, group, M, N, off):
    """bf16 rows: every value is the rounded quotient, those on a tie the even
    one, though the order of a row's sum moves rstd by a bit."""
    code, td = DT["bf16"]
    qc, qd, _ = QT[qtype]
    gen = torch.Generator().manual_seed(N + group)
    ties = 0
    for few_bits in (False, True):  # integers up to 96 meet many ties, normal values few
        x = rows(M, N, "bf16", N, 3.0)
        w = syn.uniform_weight(N, "bf16", N + 2, "cpu")
        if few_bits:
            x = torch.randint(-96, 97, (M, N), generator=gen).to(td)
            w = torch.ones(N, dtype=td)
        for c in (1.0, 2.0 ** 20, 1.5 * 2.0 ** -9):  # rows of other sizes: another rstd, the same q
            h = x * torch.tensor(c, dtype=td) if not few_bits else (x.float() * c).to(td)
            want, n = eight_bits_of_the_ratio(h, w, group, qtype)
            ties += n
            q, cq = guarded((M, N), torch.int8, off)
            scale, cs = guarded((M, -(-N // group) if group else 1), torch.float32)
            qb.qk_rmsnorm_quant_fwd(shifted(h, off), None, shifted(w, off), q, scale, None, None, M, N, 1e-12, group, code,
                                    qc)
            torch.cuda.synchronize()
            cq("q"), cs("scale")
            assert torch.equal(q.view(qd).float().cpu(), want.float()), (few_bits, c)
    assert ties > 20


@gpu
@pytest.mark.parametrize("N,off", [(256, 0), (264, 1), (9001, 0)])
@pytest.mark.parametrize("qtype", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quant_at_the_ends_of_the_range(cuda, dtype, qtype, N, off):
    """Groups whose largest y lies about 2^-100, where the scale stops; a y
    beyond float32, and one just below its end."""
    code, td = DT[dtype]
    qc, qd, _ = QT[qtype]
    for group in (0, 32):
        groups = -(-N // group) if group else 1
        x = rows(12, N, dtype, 1) * (2.0 ** torch.arange(-116, -104, dtype=torch.float64)[:, None]).to(td)
        w = syn.uniform_weight(N, dtype, 2, "cpu")
        q, cq = guarded((12, N), torch.int8, off)
        scale, cs = guarded((12, groups), torch.float32)
        qb.qk_rmsnorm_quant_fwd(shifted(x, off), None, shifted(w, off), q, scale, None, None, 12, N, EPS, group, code, qc)
        torch.cuda.synchronize()
        cq("q"), cs("scale")
        _, y, _ = forward64(x, None, w)
        assert (np.abs(y).max(1) < 2.0 ** -100).any() and (np.abs(y).max(1) > 2.0 ** -100).any()
        check_quant(q.view(qd), scale, y, group, qtype, "tiny")
        x = torch.ones(3, N, dtype=td)
        x[0, 1] = 0.75
        x[1, 1] = 4.0
        w = torch.ones(N, dtype=td)
        w[1] = 2.0 ** 127 * 1.5  # y: below float32's end, beyond it, and by a quarter below the end again
        x[2, 1] = 1.0
        q, scale, _, rstd = qb.rmsnorm_quant_fwd(shifted(x, off), shifted(w, off), eps=EPS, group=group, qdtype=qd)
        y = to_f64(x) * to_f64(rstd)[:, None] * to_f64(w)
        over = np.abs(y).max(1) > 3.4028235e38
        assert list(over) == [False, True, False]
        assert np.array_equal(np.isnan(to_f64(scale)[:, 0]), over)
        assert torch.isfinite(scale[:, 1:]).all()
        check_quant(q[~torch.from_numpy(over)], scale[~torch.from_numpy(over)], y[~over], group, qtype, "large")


def backward64(h, w, rstd, dy, dh):
    h, w, r, dy = to_f64(h), to_f64(w), to_f64(rstd)[:, None], to_f64(dy)
    up = 0.0 if dh is None else to_f64(dh)
    N = h.shape[1]
    g = dy * w
    dx = up + r * g - h * r ** 3 * (g * h).sum(1, keepdims=True) / N
    sx = np.abs(up) + r * np.abs(g) + np.abs(h) * r ** 3 * np.abs(g * h).sum(1, keepdims=True) / N
    return dx, sx, (dy * h * r).sum(0), np.abs(dy * h * r).sum(0)


def backward_case(M, N, dtype, seed):
    h, w, dy, dh = (rows(M, N, dtype, seed, 3.0), syn.uniform_weight(N, dtype, seed + 1, "cpu"),
                    rows(M, N, dtype, seed + 2), rows(M, N, dtype, seed + 3))
    rstd = torch.from_numpy(1.0 / np.sqrt((to_f64(h) ** 2).mean(1) + EPS)).float()
    return h, w, rstd, dy, dh


@gpu
@pytest.mark.parametrize("N", NS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward(cuda, dtype, N):
    code, td = DT[dtype]
    for M in MS:
        h, w, rstd, dy, dh = backward_case(M, N, dtype, N)
        for off, up in ((0, dh), (1, dh), (0, None)):
            dx_ref, sx, dw_ref, sw = backward64(h, w, rstd, dy, up)
            dx, cx = guarded((M, N), td, off)
            dw, cw = guarded((N,), torch.float32)
            nbytes = qb.qk_add_rmsnorm_bwd_workspace_size(M, N, code)
            ws, cs = guarded((nbytes,), torch.uint8)
            qb.qk_add_rmsnorm_bwd(shifted(h, off), shifted(w, off), rstd.to(DEV), shifted(dy, off),
                                  None if up is None else shifted(up, off), dx, dw, ws, nbytes, M, N, code)
            torch.cuda.synchronize()
            for c, what in ((cx, "dx"), (cw, "dw"), (cs, "workspace")):
                c(what)
            check_scaled(to_f64(dx), dx_ref, sx, dtype, f"dx {M}x{N} {dtype} offset {off}")
            check_scaled(to_f64(dw), dw_ref, sw, "f32", f"dw {M}x{N} {dtype} offset {off}")


@gpu
@pytest.mark.parametrize("dtype,M,N", [("bf16", 3, 40000), ("f32", 2, 70001), ("bf16", 2500, 4096), ("bf16", 5000, 264),
                                       ("f32", 4095, 1023), ("bf16", 9, 32768), ("f32", 5, 16384), ("f32", 1500, 2048)])
def test_backward_long_rows_and_many_rows(cuda, dtype, M, N):
    h, w, rstd, dy, dh = backward_case(M, N, dtype, 3)
    dx_ref, sx, dw_ref, sw = backward64(h, w, rstd, dy, dh)
    args = [t.to(DEV) for t in (h, w, rstd, dy, dh)]
    dx, dw = qb.add_rmsnorm_bwd(*args)
    check_scaled(to_f64(dx), dx_ref, sx, dtype, "dx")
    check_scaled(to_f64(dw), dw_ref, sw, "f32", "dw")
    for i in (0, 3, 4):  # dx over h, dy or dh: the same bits, and the same dw every time
        again = [t.clone() for t in args]
        dx2, dw2 = qb.add_rmsnorm_bwd(*again, out=again[i])
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw), i


@gpu
@pytest.mark.parametrize("N,off", [(64, 0), (1003, 0), (4096, 0), (2048, 1), (9001, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_of_rows_of_any_size(cuda, dtype, N, off):
    """Rows around 1e-17 to 1e16 with eps = 0: rstd^3 is beyond float32 at either
    end, the gradient is not.  dh is of the size of the rest of dx, 1 / the row."""
    code, td = DT[dtype]
    size = torch.tensor([1e-17, 1e-14, 1e-13, 1e-12, 1e-7, 1.0, 1e7, 1e12, 1e14, 1e15, 1e16], dtype=torch.float64)
    M = len(size)
    h = (rows(M, N, dtype, N, 3.0).double() * size[:, None]).to(td)
    w, dy = syn.uniform_weight(N, dtype, N + 1, "cpu"), rows(M, N, dtype, N + 2)
    dh = (rows(M, N, dtype, N + 3).double() / size[:, None]).to(td)
    _, _, rstd = qb.add_rmsnorm_fwd(h.to(DEV), torch.zeros_like(h).to(DEV), w.to(DEV), eps=0.0)
    check_scalars(to_f64(rstd), 1.0 / np.sqrt((to_f64(h) ** 2).mean(1)), "rstd")
    dx_ref, sx, dw_ref, sw = backward64(h, w, rstd.cpu(), dy, dh)
    dx, cx = guarded((M, N), td, off)
    dw, cw = guarded((N,), torch.float32)
    n = qb.qk_add_rmsnorm_bwd_workspace_size(M, N, code)
    ws, cs = guarded((n,), torch.uint8)
    qb.qk_add_rmsnorm_bwd(shifted(h, off), shifted(w, off), rstd, shifted(dy, off), shifted(dh, off), dx, dw, ws, n, M, N,
                          code)
    torch.cuda.synchronize()
    cx("dx"), cw("dw"), cs("workspace")
    for i in range(M):  # each row by itself: their sizes are up to 33 decades apart
        check_scaled(to_f64(dx[i]), dx_ref[i], sx[i], dtype, f"dx of a row of {size[i]:g}")
    check_scaled(to_f64(dw), dw_ref, sw, "f32", "dw")


@gpu
def test_backward_against_differences(cuda):
    """The kernel's gradient against central differences of the 64-bit forward:
    sum(y * dy) + sum(h * dh) moved along random directions (their own error is
    below 1e-7, the kernel's is float32's)."""
    M, N = 5, 200
    x, r, w = (to_f64(rows(M, N, "f32", 1)), to_f64(rows(M, N, "f32", 2)), to_f64(syn.uniform_weight(N, "f32", 3, "cpu")))
    dy, dh = to_f64(rows(M, N, "f32", 4)), to_f64(rows(M, N, "f32", 5))

    def f(x, r, w):
        h = x + r
        return ((h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * w) * dy).sum() + (h * dh).sum()

    t = lambda a: torch.from_numpy(a).float().to(DEV)  # noqa: E731
    y, h, rstd = qb.add_rmsnorm_fwd(t(x), t(r), t(w), eps=EPS)
    dx, dw = qb.add_rmsnorm_bwd(h, t(w), rstd, t(dy), t(dh))
    rng = np.random.default_rng(0)
    for _ in range(4):
        u, v, e = rng.standard_normal((M, N)), rng.standard_normal(N), 1e-5
        slope = (f(x + e * u, r, w + e * v) - f(x - e * u, r, w - e * v)) / (2 * e)
        got = (to_f64(dx) * u).sum() + (to_f64(dw) * v).sum()
        size = np.abs(to_f64(dx) * u).sum() + np.abs(to_f64(dw) * v).sum()
        assert abs(got - slope) <= 1e-5 * size


@gpu
def test_rows_beyond_32_bit_offsets(cuda):
    """2.2e9 elements: sampled rows, the last among them, of every output."""
    M, N = 540000, 4096
    x, r = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for i in range(0, M, 54000):
        x[i:i + 54000] = syn.normal_rows(54000, N, "bf16", i, DEV)
        r[i:i + 54000] = syn.normal_rows(54000, N, "bf16", i + 1, DEV, sigma=3.0)
    w = syn.uniform_weight(N, "bf16", 3, DEV)
    at = torch.tensor([0, 1, 262143, 524287, 524288, 524289, M - 2, M - 1], device=DEV)
    h_ref, y_ref, rstd_ref = forward64(x[at].cpu(), r[at].cpu(), w.cpu())
    q, scale, none, _ = qb.rmsnorm_quant_fwd(x, w, residual=r, eps=EPS, group=128, want_h=False)
    check_quant(q[at], scale[at].cpu(), y_ref, 128, "e4m3", "quant")
    y, h, rstd = qb.add_rmsnorm_fwd(x, r, w, eps=EPS, out_h=r)
    assert torch.equal(h[at].cpu(), h_ref)
    check_scalars(to_f64(rstd[at]), rstd_ref, "rstd")
    check_rows(to_f64(y[at]), y_ref, "bf16", False, "y")
    dx, dw = qb.add_rmsnorm_bwd(h, w, rstd, x, y)
    dx_ref, sx, _, _ = backward64(h_ref, w.cpu(), rstd[at].cpu(), x[at].cpu(), y[at].cpu())
    check_scaled(to_f64(dx[at]), dx_ref, sx, "bf16", "dx")
    ref, mag = torch.zeros(N, dtype=torch.float64, device=DEV), torch.zeros(N, dtype=torch.float64, device=DEV)
    for i in range(0, M, 54000):
        term = x[i:i + 54000].double() * h[i:i + 54000].double() * rstd[i:i + 54000, None].double()
        ref += term.sum(0)
        mag += term.abs().sum(0)
    check_scaled(to_f64(dw), to_f64(ref), to_f64(mag), "f32", "dw")


@gpu
@pytest.mark.parametrize("N,off", [(64, 0), (100, 1), (1003, 0), (4096, 0), (9001, 0), (40000, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_row_of_zeros_without_eps(cuda, dtype, N, off):
    """eps = 0: rstd is infinite and the row NaN, as 1 / sqrt(0) and 0 / 0 are;
    the other rows and the dw of a gradient without that row are as always."""
    x, r = rows(5, N, dtype, 1), rows(5, N, dtype, 2)
    x[2], r[2] = 0, 0
    w = syn.uniform_weight(N, dtype, 3, "cpu")
    xs, rs, ws = (shifted(t, off) for t in (x, r, w))
    y, h, rstd = qb.add_rmsnorm_fwd(xs, rs, ws, eps=0.0)
    with np.errstate(all="ignore"):
        f = to_f64(h.cpu())
        ref_rstd = 1.0 / np.sqrt((f * f).mean(1))
        ref = f * ref_rstd[:, None] * to_f64(w)[None, :]
    assert torch.equal(h.cpu(), (x.float() + r.float()).to(x.dtype)) and rstd[2].item() == float("inf")
    keep = [0, 1, 3, 4]
    check_scalars(to_f64(rstd)[keep], ref_rstd[keep], "rstd")
    assert y[2].isnan().all()
    check_rows(to_f64(y)[keep], ref[keep], dtype, False, "y")
    for group in (0, 32):
        for qdtype in (torch.float8_e4m3fn, torch.int8):
            q, scale, _, _ = qb.rmsnorm_quant_fwd(xs, ws, residual=rs, eps=0.0, group=group, qdtype=qdtype)
            assert scale[2].isnan().all() and torch.isfinite(scale[keep]).all()
            check_quant(q[keep], scale[keep], ref[keep], group, "int8" if qdtype is torch.int8 else "e4m3", "quant")
    dy, dh = rows(5, N, dtype, 4), rows(5, N, dtype, 5)
    dx, dw = qb.add_rmsnorm_bwd(h, ws, rstd, shifted(dy, off), shifted(dh, off))
    assert dx[2].isnan().all() and dw.isnan().all()
    dx_ref, sx, _, _ = backward64(h.cpu()[keep], w, rstd.cpu()[keep], dy[keep], dh[keep])
    check_scaled(to_f64(dx)[keep], dx_ref, sx, dtype, "dx")


@gpu
def test_zero_rows(cuda):
    w = torch.ones(64, device=DEV)
    e = torch.empty(0, 64, device=DEV)
    y, h, rstd = qb.add_rmsnorm_fwd(e, e.clone(), w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = qb.add_rmsnorm_bwd(e, w, rstd, e.clone())
    assert dx.shape == (0, 64) and (dw == 0).all()
    q, scale, h, rstd = qb.rmsnorm_quant_fwd(e, w, group=32)
    assert q.shape == (0, 64) and scale.shape == (0, 2)


@gpu
def test_another_stream_and_a_captured_graph(cuda):
    M, N = 33, 4096
    x, r, w = rows(M, N, "bf16", 1).to(DEV), rows(M, N, "bf16", 2).to(DEV), syn.uniform_weight(N, "bf16", 3, DEV)
    dy, dh = rows(M, N, "bf16", 4).to(DEV), rows(M, N, "bf16", 5).to(DEV)

    def all_of_them(stream=None):
        y, h, rstd = qb.add_rmsnorm_fwd(x, r, w, stream=stream)
        q, scale, _, _ = qb.rmsnorm_quant_fwd(x, w, residual=r, group=128, stream=stream)
        dx, dw = qb.add_rmsnorm_bwd(h, w, rstd, dy, dh, stream=stream)
        return [y, h, rstd, q.view(torch.int8), scale, dx, dw]

    want = [t.clone() for t in all_of_them()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = all_of_them(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of_them()
    x2 = rows(M, N, "bf16", 9).to(DEV)
    for values in (x2, x.clone()):
        x.copy_(values)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(replayed, all_of_them()))
    assert all(torch.equal(a, b) for a, b in zip(replayed, want))


# --- refusals: fake, never-dereferenced addresses; nothing touches a device ---
A, G = 1 << 32, 1 << 28


def test_forward_refusals(lib):
    f, B, F = lib.qk_add_rmsnorm_fwd, qb.QK_BF16, qb.QK_F32
    p = [A + i * G for i in range(6)]  # x, residual, w, y, h, rstd
    for M, N, dt in ((-1, 8, B), (4, 0, B), (4, 8, 9), (2 ** 40, 2 ** 40, F)):
        assert f(*p, M, N, 1e-6, dt, None) == qb.QK_ERR_INVALID_ARG
    for eps in (-1.0, float("nan"), float("inf")):
        assert f(*p, 4, 8, eps, B, None) == qb.QK_ERR_INVALID_ARG
    for i in range(5):
        assert f(*p[:i], None, *p[i + 1:], 4, 8, 1e-6, B, None) == qb.QK_ERR_INVALID_ARG
        assert f(*p[:i], p[i] + 1, *p[i + 1:], 4, 8, 1e-6, B, None) == qb.QK_ERR_MISALIGNED
    assert f(*p[:5], p[5] + 2, 4, 8, 1e-6, B, None) == qb.QK_ERR_MISALIGNED
    for i, j, off in ((3, 0, 2), (3, 1, 2), (3, 2, 0), (3, 5, 0), (4, 0, 2), (4, 1, 2), (4, 3, 0), (4, 3, 2), (5, 0, 0),
                      (5, 2, 0), (5, 4, 0)):
        bad = list(p)
        bad[i] = p[j] + off * 2
        assert f(*bad, 4, 8, 1e-6, B, None) == qb.QK_ERR_INVALID_ARG, (i, j)
    assert f(None, None, None, None, None, None, 0, 8, 1e-6, B, None) == qb.QK_OK


def test_quant_refusals(lib):
    f, B = lib.qk_rmsnorm_quant_fwd, qb.QK_BF16
    p = [A + i * G for i in range(7)]  # x, residual, w, q, scale, h, rstd
    call = lambda p, M=4, N=256, eps=1e-6, group=0, dt=B, qt=0: f(*p, M, N, eps, group, dt, qt, None)  # noqa: E731
    for kw in (dict(M=-1), dict(N=0), dict(dt=5), dict(eps=-1.0), dict(group=-1), dict(group=16), dict(group=256),
               dict(qt=2), dict(qt=-1)):
        assert call(p, **kw) == qb.QK_ERR_INVALID_ARG, kw
    for i in (0, 2, 3, 4):
        assert call(p[:i] + [None] + p[i + 1:]) == qb.QK_ERR_INVALID_ARG
    assert call([p[0], None] + p[2:]) == qb.QK_ERR_INVALID_ARG  # h without a residual
    for i in (0, 1, 2, 4, 5, 6):
        assert call(p[:i] + [p[i] + 1] + p[i + 1:]) == qb.QK_ERR_MISALIGNED
    for i, j in ((3, 0), (3, 1), (3, 2), (3, 4), (3, 5), (3, 6), (4, 0), (4, 1), (4, 5), (4, 6), (5, 2), (6, 0), (6, 5)):
        bad = list(p)
        bad[i] = p[j]
        assert call(bad) == qb.QK_ERR_INVALID_ARG, (i, j)
    bad = list(p)
    bad[5] = p[0] + 16  # h partly over x
    assert call(bad) == qb.QK_ERR_INVALID_ARG
    assert call([None] * 7, M=0) == qb.QK_OK


def test_backward_refusals(lib):
    import ctypes
    f, B = lib.qk_add_rmsnorm_bwd, qb.QK_BF16
    p = [A + i * G for i in range(8)]  # h, w, rstd, dy, dh, dx, dw, workspace
    call = lambda p, n=1 << 20, M=4, N=8, dt=B: f(*p, n, M, N, dt, None)  # noqa: E731
    for kw in (dict(M=-1), dict(N=0), dict(dt=5)):
        assert call(p, **kw) == qb.QK_ERR_INVALID_ARG
    for i in (0, 1, 2, 3, 5, 6, 7):
        assert call(p[:i] + [None] + p[i + 1:]) == qb.QK_ERR_INVALID_ARG
    for i in range(8):
        assert call(p[:i] + [p[i] + 1] + p[i + 1:]) == qb.QK_ERR_MISALIGNED
    assert call(p[:7] + [p[7] + 8]) == qb.QK_ERR_MISALIGNED
    for i, j, off in ((5, 0, 4), (5, 3, 4), (5, 4, 4), (5, 1, 0), (5, 2, 0), (6, 0, 0), (6, 3, 0), (6, 4, 0), (6, 5, 0),
                      (7, 0, 0), (7, 3, 0), (7, 4, 0), (7, 5, 0), (7, 6, 0), (7, 1, 0), (7, 2, 0)):
        bad = list(p)
        bad[i] = p[j] + off
        assert call(bad) == qb.QK_ERR_INVALID_ARG, (i, j)
    n = ctypes.c_size_t(5)
    size = lib.qk_add_rmsnorm_bwd_workspace_size
    assert size(-1, 8, B, ctypes.byref(n)) == qb.QK_ERR_INVALID_ARG
    assert size(4, 8, B, None) == qb.QK_ERR_INVALID_ARG
    assert size(0, 8, B, ctypes.byref(n)) == qb.QK_OK and n.value == 0


def test_helpers_refuse_what_is_not_on_a_gpu():
    x, w = torch.zeros(2, 8), torch.zeros(8)
    for call in (lambda: qb.add_rmsnorm_fwd(x, x, w), lambda: qb.rmsnorm_quant_fwd(x, w),
                 lambda: qb.add_rmsnorm_bwd(x, w, torch.zeros(2), x)):
        with pytest.raises(ValueError):
            call()


@gpu
def test_helper_refusals(cuda):
    x, w = torch.zeros(4, 64, device=DEV), torch.zeros(64, device=DEV)
    rstd = torch.ones(4, device=DEV)
    bad = [lambda: qb.add_rmsnorm_fwd(x, x[:2], w), lambda: qb.add_rmsnorm_fwd(x, x.bfloat16(), w),
           lambda: qb.add_rmsnorm_fwd(x.t(), x.t(), w), lambda: qb.add_rmsnorm_fwd(x, x.clone(), w[:32]),
           lambda: qb.add_rmsnorm_fwd(x, x.cpu(), w), lambda: qb.add_rmsnorm_fwd(x, x.clone(), w, out_h=x[:, :32]),
           lambda: qb.add_rmsnorm_bwd(x, w, rstd[:3], x), lambda: qb.add_rmsnorm_bwd(x, w, rstd.double(), x),
           lambda: qb.add_rmsnorm_bwd(x, w, rstd, x, dh=x[:2]), lambda: qb.rmsnorm_quant_fwd(x, w, group=48),
           lambda: qb.rmsnorm_quant_fwd(x, w, out_h=x.clone())]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qb.rmsnorm_quant_fwd(x, w, qdtype=torch.uint8), lambda: qb.rmsnorm_quant_fwd(x.half(), w.half())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(qb.QkError):
        qb.add_rmsnorm_fwd(x, x.clone(), w, out=x, out_h=x)
