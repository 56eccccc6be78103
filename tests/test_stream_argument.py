"""A call that is given a stream: the memory it allocates belongs to that stream, so that neither what it gives back (a
workspace) is reused by the current stream before its kernels end, nor what it takes is still read there."""

import contextlib
import types

import pytest
import torch

from weight_linear_attention_gb300 import falcon as F

# ---- on the CPU: where each call allocates


class Recorder:
    """Stands in for torch's streams: knows which handle is current, and notes it at each allocation."""

    def __init__(self, monkeypatch, handle_of_current=0):
        self.current, self.seen, self.launched = handle_of_current, [], []
        real = torch.empty

        def empty(*args, **kw):
            self.seen.append(self.current)
            return real(*args, **kw)

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s.cuda_stream
            try:
                yield
            finally:
                self.current = before

        class External:
            def __init__(self, handle, device=None):
                self.cuda_stream, self.device = handle, device or torch.device("cpu")

        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", External)
        monkeypatch.setattr(torch.cuda, "Stream", External)
        F._t.cache_clear()


@pytest.fixture
def record(monkeypatch):
    from weight_linear_attention_gb300 import build

    build.build()
    F.load()
    r = Recorder(monkeypatch)

    def launch(*args, stream=None, **kw):
        r.launched.append(r.current if stream is None else stream if isinstance(stream, int) else stream.cuda_stream)
        return F.FALCON_OK

    monkeypatch.setattr(F, "falcon_fwd", launch)
    monkeypatch.setattr(F, "falcon_bwd", launch)

    def seq_call(what, choice, x, views, arrays, shape, lengths, names, stream=None):
        r.launched.append(r.current if stream is None else stream if isinstance(stream, int) else stream.cuda_stream)
        pointers = [None] * (len(views) + len(arrays) + 1)
        dims = F._PACK_DIMS(*x.shape, F.FALCON_F32, 0)
        return (lambda *a: F.FALCON_OK), pointers, dims, None, 0

    monkeypatch.setattr(F, "_seq_call", seq_call)
    yield r
    F._t.cache_clear()


def calls():
    x, s = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 64)
    b = torch.zeros(2, 3, 4)
    w = torch.zeros(3, 64)
    return {"forward": lambda st: F.forward("falcon1", x, x, x, b, b, stream=st),
            "backward": lambda st: F.backward("falcon1", x, x, x, b, b, x, stream=st),
            "glr_forward": lambda st: F.glr_forward("mix", x, x, s, stream=st),
            "glr_backward": lambda st: F.glr_backward("mix", x, x, x, x, s, stream=st),
            "groupnorm_forward": lambda st: F.groupnorm_forward(x, w, w, x, act="silu", stream=st),
            "groupnorm_backward": lambda st: F.groupnorm_backward(x, x, w, w, x, act="silu", stream=st)}


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("raw", [False, True])
def test_allocations_belong_to_the_given_stream(record, name, raw):
    handle = 0x7f00dead0000
    st = handle if raw else torch.cuda.ExternalStream(handle)
    calls()[name](st)
    assert record.seen and set(record.seen) == {handle}
    assert record.launched == [handle] and record.current == 0


@pytest.mark.parametrize("name", list(calls()))
def test_without_a_stream_the_current_one_is_taken(record, name):
    calls()[name](None)
    assert record.seen and set(record.seen) == {0} and record.launched == [0]


@pytest.mark.parametrize("name", list(calls()))
def test_a_stream_of_another_device_is_refused(record, name):
    st = torch.cuda.ExternalStream(0x7f00dead0000, device=torch.device("meta"))
    with pytest.raises(ValueError, match="stream"):
        calls()[name](st)
    assert not record.launched


def test_objects_with_a_handle_and_the_legacy_handle(record):
    calls()["glr_forward"](types.SimpleNamespace(cuda_stream=0x7f00beef0000))
    assert set(record.seen) == {0x7f00beef0000} and record.launched == [0x7f00beef0000]
    record.seen.clear()
    calls()["glr_forward"](1)  # cudaStreamLegacy: the default stream's other handle
    assert set(record.seen) == {0}


# ---- on the GPU: results with work pending on both streams

PENDING = 40_000_000  # cycles of a kernel that does nothing, some 20 ms


def _tensors():
    g = torch.Generator().manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = [r(2, 3, 700, 64).bfloat16().cuda() for _ in range(4)]
    q = [r(2, 3, 128, 64).bfloat16().cuda() for _ in range(3)]
    b = [torch.sigmoid(r(2, 3, 128)).cuda() for _ in range(2)]
    return x, q, b, r(2, 3, 64).cuda(), (1 + 0.1 * r(3, 64)).cuda()


def gpu_calls():
    x, q, b, s, w = _tensors()
    return {"forward": lambda **k: F.forward("falcon1", *q, *b, **k),
            "backward": lambda **k: F.backward("falcon1", *q, *b, q[0], **k),
            "glr_forward": lambda **k: F.glr_forward("mix", x[0], x[1], s, **k),
            "glr_backward": lambda **k: F.glr_backward("mix", x[0], x[1], x[2], x[3], s, **k),
            "groupnorm_forward": lambda **k: F.groupnorm_forward(x[0], w, w, x[1], act="silu", **k),
            "groupnorm_backward": lambda **k: F.groupnorm_backward(x[0], x[2], w, w, x[1], act="silu", **k)}


def _leaves(out):
    out = list(out.values()) if isinstance(out, dict) else list(out) if isinstance(out, tuple) else [out]
    return [t for t in out if t is not None]


def _owner(t):
    """The stream whose pool the allocator took a tensor's memory from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def _same(name, got, want):
    """Falcon's backward adds in an order that varies (its gradients are within 2e-4 of their largest value, so two of
    them within twice that); the other calls repeat their bits."""
    if name == "backward":
        return all(bool(((a - b).abs() <= 4e-4 * b.abs().max()).all()) for a, b in zip(got, want))
    return all(torch.equal(a, b) for a, b in zip(got, want))


NAMES = ["forward", "backward", "glr_forward", "glr_backward", "groupnorm_forward", "groupnorm_backward"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("raw", [False, True])
def test_given_stream_with_work_pending_on_both(name, raw):
    call = gpu_calls()[name]
    want = _leaves(call())
    assert all(bool(t.isfinite().all()) for t in want)
    sizes = [t.numel() * t.element_size() for t in want]
    sizes.append(F.falcon_gn_bwd_workspace_bytes(F.make_seq_dims(2, 3, 700, 64)))
    sizes.append(F.falcon_bwd_workspace_bytes(0, F.make_dims(2, 3, 128, 64, 64), 64))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    handle = s.cuda_stream
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        # blocks that the current stream has given back and still reads
        held = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda._sleep(PENDING)
        copies = [t.clone() for t in held]
        del held
        got = _leaves(call(stream=handle if raw else s))  # ends long before the copies begin
        torch.cuda.synchronize()
        assert all(bool((c == 3).all()) for c in copies)
        assert _same(name, got, want)
        assert all(_owner(t) == handle for t in got)
        # what the call has given back is not the current stream's to write while its kernels wait
        with torch.cuda.stream(s):
            torch.cuda._sleep(PENDING)
        got = _leaves(call(stream=handle if raw else s))
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert _same(name, got, want)
        del junk


@pytest.mark.gpu
def test_two_given_streams_without_a_workspace():
    """Two calls of the same sizes from one current stream, each on a stream of its own."""
    x, _, _, _, w = _tensors()
    pairs = [(x[0], x[2]), (x[1], x[3])]
    want = [F.groupnorm_backward(a, d, w, w, act="gelu") for a, d in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(PENDING)
    got = [F.groupnorm_backward(a, d, w, w, act="gelu", stream=s) for (a, d), s in zip(pairs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for k in ("dx", "dweight", "dbias"):
            assert torch.equal(a[k], b[k]), k


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_given_stream_and_outputs(raw):
    """With nothing to allocate the call still runs on the stream it is given, and only there."""
    x, _, _, s, w = _tensors()
    want, _ = F.glr_forward("mix", x[0], x[1], s)
    norm = F.groupnorm_forward(want, w, w, x[1], act="silu")
    out, y = torch.zeros_like(want), torch.zeros_like(norm)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    st = side.cuda_stream if raw else side
    with torch.cuda.stream(side):
        torch.cuda._sleep(PENDING)
    F.glr_forward("mix", x[0], x[1], s, out=out, want_state=False, stream=st)
    F.groupnorm_forward(out, w, w, x[1], act="silu", y=y, stream=st)
    before = [out.clone(), y.clone()]  # on the current stream, which waits for neither
    torch.cuda.current_stream().synchronize()
    assert not any(bool(t.any()) for t in before)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(y, norm)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_as_an_argument(name):
    call = gpu_calls()[name]
    want = _leaves(call())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for st in (None, side):
        with torch.cuda.stream(st):
            now = torch.cuda.current_stream()
            for arg in (now, now.cuda_stream):
                got = _leaves(call(stream=arg))
                torch.cuda.synchronize()
                assert _same(name, got, want)
                assert all(_owner(t) == now.cuda_stream for t in got)
