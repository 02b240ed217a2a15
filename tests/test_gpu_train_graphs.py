"""TrainExperts' eager passes among replays of its captured ones: every gradient is that of its own forward."""
import pytest
import torch

from tests.test_gpu_train_layer import R, backward, case, forward, outputs  # noqa: F401

pytestmark = pytest.mark.gpu
dev = "cuda"
T, E, k, H, I = 300, 12, 3, 256, 136
GRADS = ("dx", "dw", "dW13", "dW2")


def wanted(R, c):
    layer, o = R.TrainExperts(H, I, E, k, T, dev), outputs(c)
    forward(layer, c, o)
    backward(layer, c, o)
    torch.cuda.synchronize()
    return o


def clear(*os):
    for o in os:
        for t in o.values():
            t.fill_(float("nan"))
    torch.cuda.synchronize()


def right(o, want, names=GRADS):
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(o[n], want[n]), n


@pytest.mark.parametrize("by", ["library", "torch"])
def test_eager_passes_among_replays(R, by):  # noqa: F811
    ca, cb = (case(T, E, k, H, I, 60 + i, 0.2) for i in range(2))
    wa, wb = wanted(R, ca), wanted(R, cb)
    layer, oa, ob = R.TrainExperts(H, I, E, k, T, dev), outputs(ca), outputs(cb)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    if by == "library":
        def capture(enqueue):
            g = R.DeviceDecodeLayer.capture(lambda: enqueue(s), s)
            return lambda: R.L.moe_graph_launch(g, s)
    else:
        def capture(enqueue):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                enqueue(None)

            def launch():
                with torch.cuda.stream(s):
                    g.replay()
            return launch
    first = capture(lambda q: forward(layer, cb, ob, q))
    second = capture(lambda q: backward(layer, cb, ob, q))
    with pytest.raises(RuntimeError):
        backward(layer, ca, oa, s)  # nothing has run yet
    both = capture(lambda q: (forward(layer, cb, ob, q), backward(layer, cb, ob, q)))
    for between in ((both,), (first,), (first, second, second), (both, first)):
        forward(layer, ca, oa, s)
        for g in between:
            g()
        backward(layer, ca, oa, s)
        right(oa, wa, wa)
        if between[-1] is not first:
            right(ob, wb, wb)
        clear(oa, ob)
    first()
    forward(layer, ca, oa, s)
    backward(layer, ca, oa, s)
    for _ in range(2):
        second()
        right(ob, wb)
        clear(ob)
    right(oa, wa, wa)
    with pytest.raises(RuntimeError):
        backward(layer, ca, oa, s)


def test_capture_is_seen(R):  # noqa: F811
    """moe_stream_capturing tells a stream that is being captured, by the library or by torch, from the others."""
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []
    look = lambda *q: seen.append([R.L.moe_stream_capturing(x) for x in q])  # noqa: E731
    x = torch.zeros(4, device=dev)
    look(s, s.cuda_stream, None, 0)

    def enqueue():
        with torch.cuda.stream(s):
            x.add_(1)
        look(s, s.cuda_stream, other)
    R.DeviceDecodeLayer.capture(enqueue, s)
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
        x.add_(1)
        look(s, None, other)
    look(s, None)
    assert seen == [[False] * 4, [True, True, False], [True, True, False], [False, False]]
