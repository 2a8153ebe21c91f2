"""Several host threads calling the library at once, each on its own CUDA
stream, with different operators and shapes (so that the per-thread plan
caches, the per-device lookups and the kernel attribute set-up all run
concurrently), then every result against the fp64 oracle."""
import threading

import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from memory_bound_row_rmsnorm_gb300 import synthetic as syn
from test_parity import DEV, DT_CODE, check_against_oracle

pytestmark = pytest.mark.gpu

CASES = [("softmax", "f32", 37, 4096), ("rmsnorm", "bf16", 64, 1003), ("xent", "bf16", 19, 50257),
         ("softmax", "bf16", 5, 65536), ("rmsnorm", "f32", 300, 256), ("xent", "f32", 41, 4096),
         ("softmax", "f32", 11, 3001), ("rmsnorm", "bf16", 3, 262144)]


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    from memory_bound_row_rmsnorm_gb300 import build
    build.build()
    qb.load_library()
    torch.cuda.set_device(0)
    yield


def _launch(op, dtype, d, out, stream):
    x = d["x"]
    M, N = x.shape
    code = DT_CODE[dtype]
    if op == "softmax":
        qb.qk_softmax_fwd(x, out["y"], M, N, code, stream)
    elif op == "rmsnorm":
        qb.qk_rmsnorm_fwd(x, d["w"], out["y"], out["rstd"], M, N, 1e-6, code, stream)
    else:
        qb.qk_xent_fwd(x, d["targets"], out["loss"], out["lse"], M, N, code, stream)


def test_threads_on_separate_streams():
    work = []
    for i, (op, dtype, M, N) in enumerate(CASES):
        inp = syn.make_inputs(op, dtype, M, N, 11000 + i, "cpu")
        d = {k: v.to(DEV) for k, v in inp.items()}
        if op == "xent":
            out = {"loss": torch.full((M,), float("nan"), device=DEV),
                   "lse": torch.full((M,), float("nan"), device=DEV)}
        else:
            out = {"y": torch.full_like(d["x"], float("nan"))}
            if op == "rmsnorm":
                out["rstd"] = torch.full((M,), float("nan"), device=DEV)
        work.append((op, dtype, inp, d, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    errors = []
    barrier = threading.Barrier(len(work))

    def worker(op, dtype, d, out, stream):
        try:
            torch.cuda.set_device(0)
            barrier.wait()
            for _ in range(20):  # the same call repeatedly: writes identical values
                _launch(op, dtype, d, out, stream)
        except Exception as e:  # reported on the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(op, dt, d, out, s)) for op, dt, _, d, out, s in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert qb.qk_get_device_status() == qb.QK_OK
    for op, dtype, inp, d, out, _ in work:
        check_against_oracle(op, dtype, inp, out, what=f"threaded {op} {dtype} {tuple(d['x'].shape)}")


def _norm_work(dtype, M, N, seed):
    """Inputs, outputs and calls of the norms with the residual's addition, through the C entry points."""
    code, td = DT_CODE[dtype], torch.bfloat16 if dtype == "bf16" else torch.float32
    x, r, dy = (syn.normal_rows(M, N, dtype, seed + i, DEV) for i in range(3))
    w = syn.uniform_weight(N, dtype, seed + 3, DEV)
    out = {"y": torch.empty_like(x), "h": torch.empty_like(x), "rstd": torch.empty(M, device=DEV),
           "q": torch.empty(M, N, dtype=torch.int8, device=DEV), "scale": torch.empty(M, -(-N // 64), device=DEV),
           "dx": torch.empty_like(x), "dw": torch.empty(N, device=DEV)}
    n = qb.qk_add_rmsnorm_bwd_workspace_size(M, N, code)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)

    def call(stream):
        size = qb.qk_add_rmsnorm_bwd_workspace_size(M, N, code)  # the plans are kept per thread
        assert size == n
        qb.qk_add_rmsnorm_fwd(x, r, w, out["y"], out["h"], out["rstd"], M, N, 1e-6, code, stream)
        qb.qk_rmsnorm_quant_fwd(x, r, w, out["q"], out["scale"], None, None, M, N, 1e-6, 64, code, qb.QK_E4M3, stream)
        qb.qk_add_rmsnorm_bwd(out["h"], w, out["rstd"], dy, r, out["dx"], out["dw"], ws, n, M, N, code, stream)
    return call, out


def _xent_work(dtype, M, V, K, seed):
    """The same of the linear cross-entropy."""
    code = DT_CODE[dtype]
    h, w = syn.normal_rows(M, K, dtype, seed, DEV), syn.normal_rows(V, K, dtype, seed + 1, DEV, sigma=2 / K ** 0.5)
    t = syn.uniform_targets(M, V, seed + 2, DEV)
    out = {"loss": torch.empty(M, device=DEV), "lse": torch.empty(M, device=DEV), "dh": torch.empty_like(h),
           "dw": torch.empty_like(w)}
    nf = qb.qk_linear_xent_fwd_workspace_size(M, V, K, code)
    nb = qb.qk_linear_xent_bwd_workspace_size(M, V, K, code)
    ws = torch.empty(max(nf, nb), dtype=torch.uint8, device=DEV)

    def call(stream):
        assert qb.qk_linear_xent_bwd_workspace_size(M, V, K, code) == nb
        qb.qk_linear_xent_fwd(h, w, t, out["loss"], out["lse"], None, ws, nf, M, V, K, code, stream=stream)
        qb.qk_linear_xent_bwd(h, w, t, out["lse"], None, out["dh"], out["dw"], ws, nb, M, V, K, code, stream=stream)
    return call, out


def _fused_work():
    """For each thread two shapes in turn, so that its kept plans change with every call."""
    return [[_norm_work("bf16", 700, 4096, 1), _norm_work("bf16", 37, 264, 11)],
            [_norm_work("f32", 300, 1023, 21), _norm_work("f32", 64, 2048, 31)],
            [_norm_work("bf16", 3, 40000, 41), _norm_work("f32", 5, 9001, 51)],
            [_xent_work("bf16", 300, 5000, 256, 61), _xent_work("bf16", 16, 4000, 512, 71)],
            [_xent_work("f32", 70, 900, 104, 81), _xent_work("f32", 9, 3000, 65, 91)],
            [_xent_work("bf16", 129, 2000, 65, 101), _norm_work("bf16", 100, 1000, 111)]]


def test_threads_on_the_fused_operators():
    """Host threads with their own streams, workspaces and outputs: the bits of each call made alone."""
    work = _fused_work()
    want = []
    for pair in work:
        for call, out in pair:
            call(None)
        torch.cuda.synchronize()
        want.append([{k: v.clone() for k, v in out.items()} for _, out in pair])
        for _, out in pair:
            for v in out.values():
                v.zero_()
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    errors = []
    barrier = threading.Barrier(len(work))

    def worker(pair, stream):
        try:
            torch.cuda.set_device(0)
            barrier.wait()
            for _ in range(15):
                for call, _ in pair:
                    call(stream)
        except Exception as e:  # reported on the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(p, s)) for p, s in zip(work, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert qb.qk_get_device_status() == qb.QK_OK
    for pair, refs in zip(work, want):
        for (_, out), ref in zip(pair, refs):
            for k in out:
                assert torch.equal(out[k], ref[k]), k


def test_one_thread_on_many_streams():
    """The same calls from one thread, their streams overlapping."""
    work = [w for pair in _fused_work() for w in pair]
    for call, out in work:
        call(None)
    torch.cuda.synchronize()
    want = [{k: v.clone() for k, v in out.items()} for _, out in work]
    for _, out in work:
        for v in out.values():
            v.zero_()
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(10):
        for (call, _), s in zip(work, streams):
            call(s)
    torch.cuda.synchronize()
    for (_, out), ref in zip(work, want):
        for k in out:
            assert torch.equal(out[k], ref[k]), k
