"""The 8-bit products, the quantiser and the experts' sort, gather and combine from several host
threads, on overlapping streams, on a stream that the caller names and in graphs that replay at one
time: every result equals the same call's alone."""
import threading

import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, cuda, lib  # noqa: F401

pytestmark = pytest.mark.gpu


def calls(seed):
    """Calls of every kernel: (a function of no arguments that returns a tuple of tensors) each."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, xf, odd = normal(700, 640).bfloat16(), normal(300, 257), normal(130, 77)
    q, s, _, _ = qb.quant_fwd(x)
    few, few_s = q[:9].contiguous(), s[:9].contiguous()
    w, ws, wt, wst = qb.quant_fwd(normal(512, 640), block_rows=128, want_t=True)
    rows_w, rows_s, _, _ = qb.quant_fwd(normal(384, 640))
    oq, os_, _, _ = qb.quant_fwd(odd)
    T, k, E = 700, 3, 12
    ids = torch.randint(-1, E, (T, k), generator=g, device=DEV)
    many = torch.randint(0, 40, (9000, 2), generator=g, device=DEV)
    offsets, slot = qb.expert_sort(ids, E)
    we, wes = (torch.stack([t] * E) for t in (w, ws))
    moved, moved_s = (torch.zeros(T * k, n, device=DEV).to(t) for n, t in ((640, q.dtype), (5, s.dtype)))
    qb.expert_gather_fwd(q, slot, scale=s, out=moved, out_scale=moved_s)
    rows, weights, dy = normal(T * k, 640).bfloat16(), normal(T, k), normal(T, 640).bfloat16()
    zeros = lambda: torch.zeros(T * k, 640, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    return [lambda: qb.quant_fwd(x, want_t=True), lambda: qb.quant_fwd(xf, block_rows=128, want_t=True),
            lambda: (qb.scaled_mm_fwd(q, s, w, ws),), lambda: (qb.scaled_mm_fwd(few, few_s, w, ws),),
            lambda: (qb.scaled_mm_fwd(q, s, rows_w, rows_s, out_dtype=torch.float32),),
            lambda: (qb.scaled_mm_fwd(oq, os_, oq, os_),),
            lambda: (qb.scaled_mm_fwd(moved, moved_s, we, wes, offsets, out=torch.zeros(T * k, 512, device=DEV)),),
            lambda: qb.expert_sort(ids, E), lambda: qb.expert_sort(many, 40),
            lambda: (qb.expert_gather_fwd(x, slot, out=zeros()),), lambda: (qb.expert_combine_fwd(rows, slot, weights),),
            lambda: qb.expert_combine_bwd(dy, rows, slot, weights, out=zeros())]


def same(got, want, what):
    for a, b in zip(got, want):
        if b is not None:
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), what


def test_threads_with_streams_of_their_own(cuda):
    work = [calls(i) for i in range(4)]
    want = [[c() for c in w] for w in work]
    torch.cuda.synchronize()
    got, errors, barrier = [None] * len(work), [], threading.Barrier(len(work))

    def worker(i):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                barrier.wait()
                for _ in range(10):
                    got[i] = [c() for c in work[i]]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported on the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i, (g, w) in enumerate(zip(got, want)):
        for j, (a, b) in enumerate(zip(g, w)):
            same(a, b, f"thread {i}, call {j}")


def test_graphs_that_replay_at_one_time(cuda):
    work = [calls(i) for i in (7, 8)]
    want = [[c() for c in w] for w in work]
    torch.cuda.synchronize()
    graphs, held = [], []
    for w in work:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append([c() for c in w])
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for g, w in zip(held, want):
        for j, (a, b) in enumerate(zip(g, w)):
            same(a, b, f"call {j}")


def test_a_stream_beside_a_busy_one(cuda):
    """Called on a named stream while the caller's is busy with memory of the same sizes."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(500, 512, generator=g, device=DEV).bfloat16()
    ids = torch.randint(0, 6, (500, 2), generator=g, device=DEV)
    w = torch.randn(384, 512, generator=g, device=DEV)
    weights = torch.rand(500, 2, generator=g, device=DEV)
    odd = torch.randn(200, 333, generator=g, device=DEV)  # a product with a workspace
    side = torch.cuda.Stream()

    def chain(s):
        q, sq, _, _ = qb.quant_fwd(x, stream=s)
        qw, sw, _, _ = qb.quant_fwd(w, block_rows=128, stream=s)
        offsets, slot = qb.expert_sort(ids, 6, stream=s)
        rows, row_s = qb.expert_gather_fwd(q, slot, scale=sq, stream=s)
        with torch.cuda.stream(s) if s is not None else torch.cuda.stream(torch.cuda.current_stream()):
            we, wes = torch.stack([qw] * 6), torch.stack([sw] * 6)
        y = qb.scaled_mm_fwd(rows, row_s, we, wes, offsets, stream=s)
        out = qb.expert_combine_fwd(y, slot, weights, stream=s)
        drows, dw = qb.expert_combine_bwd(out, y, slot, weights, stream=s)
        oq, os_, _, _ = qb.quant_fwd(odd, stream=s)
        return offsets, slot, out, drows, dw, qb.scaled_mm_fwd(oq, os_, oq, os_, stream=s)

    want = chain(None)
    torch.cuda.synchronize()
    for _ in range(3):
        busy = torch.randn(4096, 4096, device=DEV)
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            busy = busy @ busy * 1e-3
            junk = [torch.full_like(t, 3) for t in want]
            del junk
        got = chain(side)
        torch.cuda.current_stream().wait_stream(side)
        same(got, want, "on the other stream")
