"""The training operators run together as TrainExperts runs them: a forward and a backward pass against the chain in 64
bits, through a captured graph, with two layers that share scratch, and with the gate's own gradient behind it."""
import numpy as np
import pytest
import torch

from oracle import train as tr
from tests.parity import np64, npi

pytestmark = pytest.mark.gpu
dev = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def R():
    from routed_expert_layer_amd import runtime
    return runtime


def case(T, E, k, H, I, seed, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    idx = torch.topk(r(T, E) + r(E), k, dim=1).indices.int()
    idx[torch.rand((T, k), generator=g) < drop] = -1
    w = torch.rand((T, k), generator=g) + 0.1
    c = dict(x=r(T, H).to(BF), idx=idx, w=w / w.sum(1, keepdim=True), W13=(r(E, H, 2 * I) / H ** 0.5).to(BF),
             W2=(r(E, I, H) / I ** 0.5).to(BF), dout=r(T, H).to(BF))
    return {n: t.to(dev).contiguous() for n, t in c.items()}


def outputs(c, odt=torch.float32, gdt=BF):
    like = lambda t, d: torch.full(t.shape, float("nan"), dtype=d, device=dev)  # noqa: E731
    return dict(out=like(c["x"], odt), dx=like(c["x"], BF), dw=like(c["w"], torch.float32), dW13=like(c["W13"], gdt),
                dW2=like(c["W2"], gdt))


def forward(layer, c, o, stream=None):
    layer.forward(c["x"], c["idx"], c["w"], c["W13"], c["W2"], o["out"], stream)


def backward(layer, c, o, stream=None):
    layer.backward(c["dout"], c["W13"], c["W2"], o["dx"], o["dw"], o["dW13"], o["dW2"], stream)


def chain(c, codes, scales, I):
    """The layer's passes in 64 bits; the backward pass from the values that were kept."""
    E = c["W13"].shape[0]
    counts, offsets, pos, src = tr.group(npi(c["idx"]), E)
    x, w, W13, W2, d = (np64(c[n]) for n in ("x", "w", "W13", "W2", "dout"))
    n = len(src)
    xp = x[src]
    gu = tr.matmul(xp, W13, counts, offsets)
    y = tr.matmul(tr.swiglu(gu[:, :I], gu[:, I:]), W2, counts, offsets)
    out = tr.collect(y, pos, w)
    G = (I + 127) // 128
    g, u = tr.kept(codes[:n, :I], scales[:n, :G]), tr.kept(codes[:n, I:], scales[:n, G:])
    dy, dw = tr.collect_backward(d, y, pos, w)
    dh = tr.matmul(dy, W2, counts, offsets, True)
    dgu = np.concatenate(tr.swiglu_backward(g, u, dh), 1)
    return dict(out=out, dw=dw, dW2=tr.matmul_dw(tr.swiglu(g, u), dy, counts, offsets),
                dW13=tr.matmul_dw(xp, dgu, counts, offsets),
                dx=tr.collect(tr.matmul(dgu, W13, counts, offsets, True), pos)), (gu, g, u, n)


@pytest.mark.parametrize("T,E,k,H,I,drop", [(1, 8, 2, 128, 64, 0), (40, 12, 3, 256, 136, 0.3), (300, 9, 4, 512, 384, 0),
                                            (17, 64, 8, 64, 128, 0.8)])
def test_passes(R, T, E, k, H, I, drop):
    """Every result against the 64-bit chain. At most four tensors on a path are rounded to bf16, each by at most 2^-9 of
    its norm on average, which products of this kind pass on unchanged: below 4 * 2^-9 = 8e-3 of a result's norm. (Single
    entries are not held to a part of the root mean square: that is taken over the zeros of experts without rows too, and
    of one token's dW2 the largest entry is 27 times it, so its last rounding alone may be 27 * 2^-8 = 0.1 of it.) What
    8 bits keep is compared for itself: half a step of its scale."""
    c = case(T, E, k, H, I, T + H, drop)
    layer = R.TrainExperts(H, I, E, k, T + 5, dev)
    for t in (layer.x_perm, layer.y_perm, *layer.scratch.values()):
        t.fill_(float("nan"))
    o = outputs(c)
    forward(layer, c, o)
    codes, scales = layer.codes.cpu().numpy(), layer.scales.cpu().numpy()
    backward(layer, c, o)
    want, (gu, g, u, n) = chain(c, codes, scales, I)
    for name in want:
        got = np64(o[name])
        assert np.all(np.isfinite(got)), name
        assert np.linalg.norm(got - want[name]) <= 8e-3 * np.linalg.norm(want[name]), name
    step = np.repeat(scales[:n], 128, 1)
    G = (I + 127) // 128 * 128
    # half a step, and the rounding of gu to bf16 before (2^-8, beside its fp32 sums)
    for v, kept, s in ((gu[:, :I], g, step[:, :I]), (gu[:, I:], u, step[:, G:G + I])):
        assert np.all(np.abs(kept - v) <= 0.5 * s * (1 + 1e-5) + 2.0 ** -7 * np.abs(v) + 1e-4)
    with pytest.raises(RuntimeError):
        backward(layer, c, o)
    with pytest.raises(ValueError):
        layer.forward(torch.zeros((T + 6, H), dtype=BF, device=dev), c["idx"], c["w"], c["W13"], c["W2"], o["out"])


def test_gate_gradient(R):
    """dtopk_w carries on into a softmax gate: the logits' gradient against differences of the whole layer's output in
    64 bits (with the experts' outputs as they are)."""
    T, E, k, H, I = 6, 5, 2, 128, 64
    c = case(T, E, k, H, I, 3)
    g = torch.Generator().manual_seed(1)
    logits = torch.randn((T, E), generator=g).to(dev).requires_grad_()
    idx = torch.topk(logits.detach(), k, dim=1).indices
    c["idx"] = idx.int().contiguous()
    w = torch.softmax(torch.gather(logits, 1, idx), 1)
    c["w"] = w.detach().contiguous()
    layer, o = R.TrainExperts(H, I, E, k, T, dev), outputs(c)
    forward(layer, c, o)
    y = np64(layer.y_perm)
    pos = npi(layer.perm_pos)
    backward(layer, c, o)
    w.backward(o["dw"])
    l0, chosen, d = np64(logits), npi(idx), np64(c["dout"])

    def value(l):
        z = np.exp(np.take_along_axis(l, chosen, 1))
        return float((tr.collect(y, pos, z / z.sum(1, keepdims=True)) * d).sum())
    step, got, size = 1e-5, np64(logits.grad), np.abs(np64(o["dw"])).max()
    for t in range(T):
        for e in range(E):
            hi, lo = l0.copy(), l0.copy()
            hi[t, e] += step
            lo[t, e] -= step
            # the sums over H in fp32, and the difference's own error
            assert abs(got[t, e] - (value(hi) - value(lo)) / (2 * step)) <= H * 2.0 ** -23 * size * 10 + 1e-6


def test_graph(R):
    """Both passes captured and replayed with other inputs in the same buffers give the eager bits, on a stream of their
    own, with two layers that share scratch and other work between the replays."""
    T, E, k, H, I = 900, 24, 5, 256, 192
    cases = [case(T, E, k, H, I, 20 + i, 0.2) for i in range(3)]
    eager = []
    for c in cases:
        layer, o = R.TrainExperts(H, I, E, k, T, dev), outputs(c, BF, torch.float32)
        forward(layer, c, o)
        backward(layer, c, o)
        eager.append({n: t.clone() for n, t in o.items()})
    c = {n: t.clone() for n, t in cases[0].items()}
    c2 = {n: t.clone() for n, t in cases[1].items()}
    one = R.TrainExperts(H, I, E, k, T, dev)
    two = R.TrainExperts(H, I, E, k, T, dev, scratch=one.scratch)
    o, o2 = outputs(c, BF, torch.float32), outputs(c, BF, torch.float32)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step():
        forward(one, c, o, s)
        forward(two, c2, o2, s)
        backward(two, c2, o2, s)
        backward(one, c, o, s)
    graph = R.DeviceDecodeLayer.capture(step, s)
    for i, j in ((0, 1), (1, 2), (2, 0), (0, 0)):
        for n in c:
            c[n].copy_(cases[i][n])
            c2[n].copy_(cases[j][n])
        for t in (*o.values(), *o2.values()):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        R.L.moe_graph_launch(graph, s)
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(o[n], eager[i][n]) and torch.equal(o2[n], eager[j][n]), n


def test_refused_backward(R):
    """A backward pass refused at an output leaves what forward kept, or says that it is gone; never other gradients."""
    T, E, k, H, I = 40, 6, 2, 136, 72
    c = case(T, E, k, H, I, 5)
    layer = R.TrainExperts(H, I, E, k, T)
    want, got = outputs(c), outputs(c)
    with pytest.raises(RuntimeError):
        backward(layer, c, want)
    forward(layer, c, want)
    backward(layer, c, want)
    with pytest.raises(RuntimeError):
        backward(layer, c, got)
    forward(layer, c, got)
    for name in ("dw", "dW2", "dW13"):
        with pytest.raises(ValueError):
            backward(layer, c, {**got, name: got[name][:1]})
    backward(layer, c, got)
    assert all(torch.equal(want[n], got[n]) for n in want)
    forward(layer, c, got)
    with pytest.raises(ValueError):
        backward(layer, c, {**got, "dx": got["dx"][:1]})
    with pytest.raises(RuntimeError):
        backward(layer, c, got)


def test_two_streams(R):
    """Two layers at once on two streams, buffers of their own."""
    T, E, k, H, I = 700, 16, 4, 256, 128
    cs = [case(T, E, k, H, I, 40 + i) for i in range(2)]
    layers, outs = [R.TrainExperts(H, I, E, k, T, dev) for _ in cs], [outputs(c) for c in cs]
    for c, layer, o in zip(cs, layers, outs):
        forward(layer, c, o)
        backward(layer, c, o)
    want = [{n: t.clone() for n, t in o.items()} for o in outs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for f in (forward, backward):
            for c, layer, o, s in zip(cs, layers, outs, streams):
                f(layer, c, o, s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(o[n], w[n]) for n in o)
