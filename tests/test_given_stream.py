"""The tensor helpers on a stream that the caller names.

Torch's allocator hands freed memory out again at once, in the order of the
stream that it belongs to.  What a call on a stream writes therefore has to be
allocated as that stream's, what it returns has to be known as the caller's
too, and what it was given as that stream's.  The first test watches the
allocations with stand-ins for tensors, streams and the library, on the CPU;
the others keep the caller's stream busy with memory of the same sizes.
"""
import contextlib
import types

import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from memory_bound_row_rmsnorm_gb300 import synthetic as syn
from test_add_rmsnorm import DEV, cuda, lib  # noqa: F401

gpu = pytest.mark.gpu


class FakeStream:
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device_index = handle, device

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class FakeTensor:
    """As much of a CUDA tensor as the helpers look at."""
    device, is_cuda = "cuda:0", True

    def __init__(self, shape, dtype, stream):
        self.shape, self.dtype, self.stream, self.uses = torch.Size(shape), dtype, stream, []

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        self.uses.append(stream.cuda_stream)


CALLER, GIVEN = FakeStream(0), FakeStream(0x7f0000001000)


@pytest.fixture
def watched(monkeypatch):
    """Stand-ins; yields (new tensor, tensors allocated, stream handles of the launches)."""
    now, made, launched = [CALLER], [], []

    def empty(*shape, dtype=torch.float32, device=None):
        shape = shape[0] if len(shape) == 1 and isinstance(shape[0], (tuple, list)) else shape
        made.append(FakeTensor(shape, dtype, now[0].cuda_stream))
        return made[-1]

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s
        yield
        now[0] = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if not name.endswith("_workspace_size"):
                    launched.append(args[-1] or 0)
                return 0
            return call

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch, "cuda", types.SimpleNamespace(
        Stream=FakeStream, stream=stream, current_stream=lambda *a: now[0], default_stream=lambda *a: CALLER, is_available=lambda: True,
        is_initialized=lambda: True, ExternalStream=lambda handle, **kw: FakeStream(handle)))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: now[0].cuda_stream, raising=False)
    monkeypatch.setattr(qb, "torch", torch, raising=False)
    monkeypatch.setattr(qb, "load_library", lambda *a: Library())
    qb._workspace_bytes.cache_clear()
    yield (lambda *shape, dtype=torch.float32: FakeTensor(shape, dtype, CALLER.cuda_stream)), made, launched
    qb._workspace_bytes.cache_clear()


def helper_calls(new):
    """Every tensor helper as (name, inputs, call of a stream)."""
    x, w, b, h, v = new(6, 64), new(64), new(64), new(6, 64), new(100, 64)
    t, rstd, lse = new(6, dtype=torch.int64), new(6), new(6)
    o, o2 = new(6, 64), new(6, 64)
    return [
        ("softmax_fwd", [x], lambda s: qb.softmax_fwd(x, stream=s)),
        ("softmax_fwd out", [x, o], lambda s: qb.softmax_fwd(x, out=o, stream=s)),
        ("rmsnorm_fwd", [x, w], lambda s: qb.rmsnorm_fwd(x, w, stream=s)),
        ("layernorm_fwd", [x, w, b], lambda s: qb.layernorm_fwd(x, w, b, stream=s)),
        ("xent_fwd", [x, t], lambda s: qb.xent_fwd(x, t, stream=s)),
        ("xent_fwd mean", [x, t], lambda s: qb.xent_fwd(x, t, ignore_index=3, want_mean=True, stream=s)),
        ("softmax_bwd", [x, h], lambda s: qb.softmax_bwd(x, h, stream=s)),
        ("rmsnorm_bwd", [x, w, rstd, h], lambda s: qb.rmsnorm_bwd(x, w, rstd, h, stream=s)),
        ("xent_bwd", [x, t, lse, rstd], lambda s: qb.xent_bwd(x, t, lse, rstd, stream=s)),
        ("add_rmsnorm_fwd", [x, h, w], lambda s: qb.add_rmsnorm_fwd(x, h, w, stream=s)),
        ("add_rmsnorm_fwd out", [x, h, w, o, o2], lambda s: qb.add_rmsnorm_fwd(x, h, w, out=o, out_h=o2, stream=s)),
        ("add_rmsnorm_bwd", [x, w, rstd, h, o], lambda s: qb.add_rmsnorm_bwd(x, w, rstd, h, o, stream=s)),
        ("rmsnorm_quant_fwd", [x, w, h], lambda s: qb.rmsnorm_quant_fwd(x, w, residual=h, group=32, stream=s)),
        ("linear_xent_fwd", [x, v, t], lambda s: qb.linear_xent_fwd(x, v, t, want_mean=True, stream=s)),
        ("linear_xent_bwd", [x, v, t, lse, rstd], lambda s: qb.linear_xent_bwd(x, v, t, lse, rstd, stream=s)),
    ]


@pytest.mark.parametrize("which", range(15))
@pytest.mark.parametrize("form", ["stream", "handle"])
def test_memory_belongs_to_the_stream(watched, which, form):
    new, made, launched = watched
    name, inputs, call = helper_calls(new)[which]
    out = call(GIVEN if form == "stream" else GIVEN.cuda_stream)
    out = [o for o in (out if isinstance(out, tuple) else (out,)) if o is not None]
    assert launched == [GIVEN.cuda_stream], name
    assert all(t.stream == GIVEN.cuda_stream for t in made), f"{name}: memory of another stream"
    assert all(CALLER.cuda_stream in t.uses for t in out if t in made), f"{name}: the caller's use is not known"
    assert all(t.uses == [GIVEN.cuda_stream] for t in inputs if t not in out), f"{name}: the use of an input is not known"


@pytest.mark.parametrize("which", range(15))
def test_the_current_stream_needs_no_record(watched, which):
    new, made, launched = watched
    for given in (None, CALLER, 0):
        name, inputs, call = helper_calls(new)[which]
        del made[:], launched[:]
        call(given)
        assert launched == [CALLER.cuda_stream], name
        assert all(t.stream == CALLER.cuda_stream and not t.uses for t in made + inputs), name


@pytest.mark.parametrize("which", range(15))
def test_a_stream_of_another_device_is_refused(watched, which):
    """Torch would switch to that device, and the kernels run there on this one's memory."""
    new, made, launched = watched
    name, _, call = helper_calls(new)[which]
    with pytest.raises(ValueError, match="device"):
        call(FakeStream(0x7f0000002000, device=1))
    assert not launched and not made, name


def test_any_object_with_a_handle(watched):
    """What names its handle cuda_stream is a stream, torch's class or not."""
    new, made, launched = watched
    qb.softmax_fwd(new(6, 64), stream=types.SimpleNamespace(cuda_stream=GIVEN.cuda_stream))
    assert launched == [GIVEN.cuda_stream] and made[0].stream == GIVEN.cuda_stream


def test_tensors_off_the_gpu_are_refused_on_a_given_stream():
    x, w = torch.zeros(2, 8), torch.zeros(8)
    for call in (lambda: qb.softmax_fwd(x, stream=64), lambda: qb.add_rmsnorm_fwd(x, x, w, stream=64)):
        with pytest.raises(ValueError):
            call()


def busy(c, times):
    """Backward calls on the current stream, whose memory is free for reuse while they run."""
    for _ in range(times):
        out = qb.linear_xent_bwd(c["h"], c["w"], c["t"], c["lse"])
    return out


@gpu
@pytest.mark.parametrize("handle", [False, True])
def test_a_stream_beside_a_busy_one(cuda, handle):
    """A call on another stream, of the sizes that the busy stream has just freed."""
    cases = []
    for seed in (1, 2):
        c = {"h": syn.normal_rows(2048, 1024, "bf16", seed, DEV),
             "w": syn.normal_rows(16384, 1024, "bf16", seed + 10, DEV, sigma=2 / 32)}
        c["t"] = syn.uniform_targets(2048, 16384, seed + 20, DEV)
        c["lse"] = qb.linear_xent_fwd(c["h"], c["w"], c["t"])[1]
        cases.append(c)
    want = [[t.clone() for t in busy(c, 1)] for c in cases]
    s = torch.cuda.Stream()
    given = s.cuda_stream if handle else s
    torch.cuda.synchronize()
    for _ in range(3):
        here = busy(cases[0], 4)  # the workspaces of these calls are free again before they have run
        there = qb.linear_xent_bwd(cases[1]["h"], cases[1]["w"], cases[1]["t"], cases[1]["lse"], stream=given)
        here2 = busy(cases[0], 2)
        torch.cuda.synchronize()
        for got, ref in ((here, want[0]), (here2, want[0]), (there, want[1])):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


@gpu
def test_norms_on_a_stream_beside_a_busy_one(cuda):
    M, N = 8192, 4096
    x, r = syn.normal_rows(M, N, "bf16", 1, DEV), syn.normal_rows(M, N, "bf16", 2, DEV)
    x2 = syn.normal_rows(M, N, "bf16", 3, DEV)
    w = syn.uniform_weight(N, "bf16", 4, DEV)
    ones = torch.ones(M, device=DEV)

    def calls(x, stream=None):
        y, h, rstd = qb.add_rmsnorm_fwd(x, r, w, stream=stream)
        q, scale, _, _ = qb.rmsnorm_quant_fwd(x, w, group=128, stream=stream)
        dx, dw = qb.add_rmsnorm_bwd(h, w, rstd, y, x, stream=stream)
        y2, rstd2 = qb.rmsnorm_fwd(x, w, stream=stream)
        dx2, dw2 = qb.rmsnorm_bwd(x, w, ones, y2, stream=stream)
        return [y, h, rstd, q.view(torch.int8), scale, dx, dw, y2, rstd2, dx2, dw2, qb.softmax_fwd(x, stream=stream)]

    want = [[t.clone() for t in calls(v)] for v in (x, x2)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(3):
            here = calls(x)
        there = calls(x2, s)
        here = calls(x)
        torch.cuda.synchronize()
        for got, ref in ((here, want[0]), (there, want[1])):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


@gpu
def test_a_result_freed_while_the_caller_reads_it(cuda):
    """What came from another stream, read on the caller's and dropped at once,
    while that stream goes on with calls of the same size."""
    M, N = 8192, 8192
    x, w = syn.normal_rows(M, N, "f32", 1, DEV), torch.ones(N, device=DEV)
    zeros = torch.zeros_like(x)
    s = torch.cuda.Stream()
    want = qb.rmsnorm_fwd(x, w)[0].clone()
    torch.cuda.synchronize()
    for _ in range(5):
        y, _ = qb.rmsnorm_fwd(x, w, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        wide = zeros
        for _ in range(4):
            wide = wide + y  # the caller's reads, queued
        del y
        for _ in range(3):
            qb.rmsnorm_fwd(zeros, w, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(wide, want + want + want + want)


@gpu
def test_a_captured_fork(cuda):
    """A stream that joined a capture, given to a helper: replayed with other inputs."""
    x, w = syn.normal_rows(300, 1024, "f32", 1, DEV), torch.ones(1024, device=DEV)
    r = syn.normal_rows(300, 1024, "f32", 2, DEV)
    s = torch.cuda.Stream()
    qb.add_rmsnorm_fwd(x, r, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        s.wait_stream(main)
        y, h, rstd = qb.add_rmsnorm_fwd(x, r, w, stream=s)
        y2, _ = qb.rmsnorm_fwd(x, w)
        main.wait_stream(s)
        both = y + y2
    for seed in (3, 4):
        x.copy_(syn.normal_rows(300, 1024, "f32", seed, DEV))
        graph.replay()
        torch.cuda.synchronize()
        a, ha, _ = qb.add_rmsnorm_fwd(x, r, w)
        assert torch.equal(y, a) and torch.equal(h, ha) and torch.equal(both, a + qb.rmsnorm_fwd(x, w)[0])
