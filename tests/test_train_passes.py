"""The order of TrainExperts' passes, eager and in graphs, on the CPU: the library's calls are replaced by the oracle's
statements, which run at once or, while a stream is being captured, when the graph is replayed."""
import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from oracle import train as tr

T, E, k, H, I = 7, 5, 2, 16, 8
NAMES = ("dx", "dw", "dW13", "dW2")


class Stream:
    """A stream of the stand-ins: what is enqueued runs at once, or goes into `graph` while there is one."""
    graph = None

    def capture(self, enqueue):
        self.graph = g = []
        try:
            enqueue()
        finally:
            self.graph = None
        return g


@pytest.fixture
def R(monkeypatch):
    from routed_expert_layer_amd import runtime

    def put(t, v):
        t.copy_(torch.from_numpy(np.ascontiguousarray(v)))

    def group(idx, E, counts, offsets, src, pos, ws):
        c, o, p, s = tr.group(idx.numpy(), E)
        for t, v in ((counts, c), (offsets, o), (pos, p), (src[:len(s)], s)):
            put(t, v)

    def dispatch(x, pos, rows):
        for t, j in np.argwhere(pos.numpy() >= 0):
            rows[pos[t, j]] = x[t]

    def collect(rows, pos, w, out):
        put(out, tr.collect(rows.double(), pos.numpy(), None if w is None else w.numpy()))

    def collect_backward(d, rows, pos, w, drows, dw):
        a, b = tr.collect_backward(d.double(), rows.double(), pos.numpy(), w.numpy())
        put(drows, a)
        put(dw, b)

    def save(gu, h, codes, scales, n):
        n, m = int(n[0]), gu.shape[1] // 2
        for first, s in ((0, scales[:n, :1]), (m, scales[:n, 1:])):
            c, v = tr.keep(gu[:n, first:first + m].double())
            put(codes[:n, first:first + m], c)
            put(s, v)
        put(h[:n], tr.swiglu(gu[:n, :m].double().numpy(), gu[:n, m:].double().numpy()))

    def back(codes, scales, dh, dgu, h, n):
        n, m = int(n[0]), dh.shape[1]
        g, u = (tr.kept(codes[:n, a:a + m].numpy(), scales[:n, a // m:a // m + 1].numpy()) for a in (0, m))
        dg, du = tr.swiglu_backward(g, u, dh[:n].double().numpy())
        put(dgu[:n], np.concatenate([dg, du], 1))
        put(h[:n], tr.swiglu(g, u))

    def matmul(a, w, counts, offsets, c, transposed=False):
        put(c, tr.matmul(a.double(), w.double(), counts.numpy(), offsets.numpy()[:-1], transposed))

    def matmul_dw(a, dc, counts, offsets, dw):
        put(dw, tr.matmul_dw(a.double(), dc.double(), counts.numpy(), offsets.numpy()[:-1]))

    def stand_in(f, n):
        def call(*args, stream=None, **kw):
            if len(args) > n:
                args, stream = args[:n], args[n]
            if stream is not None and stream.graph is not None:
                stream.graph.append(lambda: f(*args, **kw))
            else:
                f(*args, **kw)
        return call
    for name, f, n in (("moe_group", group, 7), ("moe_dispatch", dispatch, 3), ("moe_collect", collect, 4),
                       ("moe_collect_backward", collect_backward, 6), ("moe_swiglu_save", save, 5),
                       ("moe_swiglu_backward", back, 6), ("moe_matmul_grouped", matmul, 5),
                       ("moe_matmul_grouped_dw", matmul_dw, 5)):
        monkeypatch.setattr(runtime.L, name, stand_in(f, n))
    monkeypatch.setattr(runtime.L, "moe_stream_capturing", lambda s=None: s is not None and s.graph is not None,
                        raising=False)

    class on:  # torch's context of a current stream, which the CPU has none of
        def __init__(self, s):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *a):
            pass
    monkeypatch.setattr(torch.cuda, "stream", on)
    return runtime


def case(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    idx = torch.topk(r(T, E), k, dim=1).indices.int()
    idx[torch.rand((T, k), generator=g) < 0.2] = -1
    bf = torch.bfloat16
    return dict(x=r(T, H).to(bf), idx=idx, w=torch.rand((T, k), generator=g), W13=r(E, H, 2 * I).to(bf),
                W2=r(E, I, H).to(bf), dout=r(T, H).to(bf))


def outputs(c):
    like = lambda t: torch.full(t.shape, float("nan"))  # noqa: E731
    return dict(out=like(c["x"]), dx=like(c["x"]), dw=like(c["w"]), dW13=like(c["W13"]), dW2=like(c["W2"]))


class Step:
    """A layer's passes on inputs of their own, with the gradients that they ought to give."""

    def __init__(self, R, layer, seed, stream):
        self.layer, self.c, self.s = layer, case(seed), stream
        self.o = outputs(self.c)
        alone = R.TrainExperts(H, I, E, k, T, "cpu")
        self.run(alone, None)
        self.want = {n: t.clone() for n, t in self.o.items()}
        assert all(torch.isfinite(t).all() for t in self.want.values())
        self.clear()

    def run(self, layer, s):
        self.forward(layer, s)
        self.backward(layer, s)

    def clear(self):
        for t in self.o.values():
            t.fill_(float("nan"))

    def forward(self, layer=None, s="own"):
        c = self.c
        (layer or self.layer).forward(c["x"], c["idx"], c["w"], c["W13"], c["W2"], self.o["out"],
                                      self.s if s == "own" else s)

    def backward(self, layer=None, s="own"):
        c, o = self.c, self.o
        (layer or self.layer).backward(c["dout"], c["W13"], c["W2"], o["dx"], o["dw"], o["dW13"], o["dW2"],
                                       self.s if s == "own" else s)

    def right(self, names=NAMES):
        for n in names:
            assert torch.equal(self.o[n], self.want[n]), n
        self.clear()


def replay(graph):
    for call in graph:
        call()


@pytest.fixture
def two(R):
    """Two steps of one layer and their stream."""
    s, layer = Stream(), R.TrainExperts(H, I, E, k, T, "cpu")
    return Step(R, layer, 1, s), Step(R, layer, 2, s), s


def test_eager(two):
    a, b, s = two
    for step in (a, b, a):
        step.forward()
        step.backward()
        step.right()
        with pytest.raises(RuntimeError):
            step.backward()


@pytest.mark.parametrize("same", [True, False])
def test_a_replay_between_eager_passes(two, same):
    """Replays of both passes, of a forward or of a backward pass, of other inputs or the same, between an eager forward
    and its backward."""
    a, b, s = two
    g = a if same else b
    both = s.capture(lambda: (g.forward(), g.backward()))
    first, second = s.capture(g.forward), s.capture(g.backward)
    for between in ((both,), (first,), (first, second), (first, second, second), (both, first)):
        a.forward()
        for graph in between:
            replay(graph)
        a.clear()
        a.backward()
        a.right()


def test_eager_passes_between_replays(two):
    """An eager step, of its own inputs, between the replays of a forward and of its backward; a backward replayed twice."""
    a, b, s = two
    first, second = s.capture(a.forward), s.capture(a.backward)
    for _ in range(2):
        replay(first)
        b.forward()
        b.backward()
        b.right()
        for _ in range(2):
            replay(second)
            a.right()


def test_a_capture_is_no_pass(two):
    """A forward that was only captured has kept nothing, and one that capturing took the buffers of no longer does."""
    a, b, s = two
    s.capture(a.forward)
    with pytest.raises(RuntimeError):
        a.backward()
    with pytest.raises(RuntimeError):
        b.backward()
    b.forward()
    b.backward()
    b.right()


def test_a_capture_ends_a_pending_pass(two):
    a, b, s = two
    a.forward()
    s.capture(lambda: (b.forward(), b.backward()))
    with pytest.raises(RuntimeError):
        a.backward()
    a.forward()
    s.capture(lambda: (b.forward(), b.backward()))
    a.backward()
    a.right()


def test_a_captured_backward_needs_a_captured_forward(two):
    a, b, s = two
    a.forward()
    with pytest.raises(RuntimeError):
        s.capture(a.backward)
    g = s.capture(lambda: (b.forward(), b.backward()))
    a.forward()
    with pytest.raises(RuntimeError):
        s.capture(a.backward)
    replay(g)
    b.right()
    a.clear()
    a.backward()
    a.right()


def test_capturing_refused():
    """moe_stream_capturing without a place for its answer, and of the default stream."""
    import ctypes
    from routed_expert_layer_amd import _lib as L
    on = ctypes.c_int(7)
    assert L._lib.moe_stream_capturing(None, None) == L.MOE_EINVAL and L.moe_last_error()
    assert L._lib.moe_stream_capturing(None, ctypes.byref(on)) == L.MOE_OK and on.value == 0
    assert L.moe_stream_capturing() is False


def test_buffers_are_not_filled(R):
    """Nothing is enqueued when a layer is made: a fill on the stream current then could come after a first pass on
    another stream."""
    class Calls(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.seen.add(func.overloadpacket.__name__)
            return func(*args, **(kwargs or {}))
    calls = Calls()
    calls.seen = set()
    with calls:
        R.TrainExperts(H, I, E, k, T, "cpu")
    assert calls.seen <= {"empty"}, calls.seen
