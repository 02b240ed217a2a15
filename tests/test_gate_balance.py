"""The balance of a gate: what replaces it, what keeps it alive, and what is refused. Without a GPU the tensors are
stand-ins that have a GPU tensor's interface, and the library's calls are recorded instead of made."""
import ctypes
import gc
import weakref

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


class Tensor:
    """A GPU tensor's interface, as far as the binding asks for it."""
    dtype, is_cuda = torch.float32, True

    def __init__(self, *shape, gpu=0, at=4096):
        self.shape, self.gpu, self.at, self.device = shape, gpu, at, f"cuda:{gpu}"

    def get_device(self):
        return self.gpu

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return 4


@pytest.fixture
def calls(L, monkeypatch):
    """The gate addresses that library calls were given, by name; the calls succeed."""
    seen = []

    class Library:
        def __getattr__(self, name):
            def call(*a):
                gates = [x for x in a if type(x).__name__ == "CArgObject"]
                seen.append((name, [ctypes.cast(g, ctypes.POINTER(L.Gate)).contents._balance for g in gates]))
                return L.MOE_OK
            return call

    monkeypatch.setattr(L, "_lib", Library())
    monkeypatch.setattr(L, "_device", lambda t, name: t.get_device())
    monkeypatch.setattr(L, "_stream", lambda s: 0)
    return seen


def decoder(L, kind, E=8):
    """A decoder as the binding holds one, without the library's part."""
    d = object.__new__({"host": L.MoeDecoder, "device": L.MoeDeviceDecoder}[kind])
    d.h, d.E, d.balances, d.gpu = None, E, {}, 0
    return d, {"host": L.moe_decoder_set_gate, "device": L.moe_device_decoder_set_gate}[kind]


def test_a_replaced_balance_is_the_one_that_calls_read(L, calls):
    g = L.Gate(balance=Tensor(8, at=4096))
    assert g._balance == 4096
    g.balance = Tensor(8, at=8192)
    assert g._balance == 8192 and g.balance.at == 8192
    g.balance = None
    assert g._balance is None and g.balance is None
    g.balance = Tensor(8, at=12288)
    bad = Tensor(8, at=16384)
    bad.dtype = torch.float64
    with pytest.raises(ValueError):
        g.balance = bad
    assert g._balance == 12288 and g.balance.at == 12288


@pytest.mark.parametrize("kind", ["host", "device"])
def test_decoders_keep_every_balance_that_they_were_given(L, calls, kind):
    """Queued steps and captured graphs read the balance of the gate that they were enqueued under, whatever has been
    set since, and whatever has become of that gate."""
    d, set_gate = decoder(L, kind)
    refs = []
    g = L.Gate(balance=Tensor(8, at=4096))
    refs.append(weakref.ref(g.balance))
    set_gate(d, g)
    g.balance = Tensor(8, at=8192)  # the gate moves on, the decoder's copy does not
    gc.collect()
    assert refs[0]() is not None
    set_gate(d, g)
    refs.append(weakref.ref(g.balance))
    set_gate(d, L.Gate(balance=Tensor(8, at=12288)))
    set_gate(d, None)
    del g
    gc.collect()
    assert all(r() is not None for r in refs)
    assert [b for _, q in calls for b in q] == [4096, 8192, 12288]
    same = L.Gate(balance=Tensor(8, at=4096))
    for _ in range(3):
        set_gate(d, same)
    assert len(d.balances) == 4  # the same tensor set again takes no more
    del d
    gc.collect()
    assert all(r() is None for r in refs)


def test_prefill_layer_keeps_its_balances(L, calls):
    from routed_expert_layer_amd.runtime import PrefillLayer
    pl = object.__new__(PrefillLayer)
    pl.balances, pl.gate = {}, L.Gate(balance=Tensor(8, at=4096))
    ref = weakref.ref(pl.gate.balance)
    pl.keep_balance()
    pl.gate.balance = Tensor(8, at=8192)
    pl.keep_balance()
    pl.gate = None
    pl.keep_balance()
    gc.collect()
    assert ref() is not None and len(pl.balances) == 2


@pytest.mark.parametrize("bad", [dict(shape=(7,)), dict(shape=(9,)), dict(shape=(8, 1)), dict(shape=(8,), gpu=1)],
                         ids=lambda d: "-".join(f"{k}={v}" for k, v in d.items()))
def test_a_balance_of_another_size_or_gpu_is_refused(L, calls, bad):
    """By every entry point that takes a gate, before the library is called."""
    E, T, k, H = 8, 4, 2, 64
    g = L.Gate(balance=Tensor(*bad["shape"], gpu=bad.get("gpu", 0)))
    good = L.Gate(balance=Tensor(E))
    out = Tensor(1)
    xw = [Tensor(T, H), Tensor(H, E)]

    def scored(gate):
        L.moe_route_scored(*xw, None, gate, k, out, out, None, out, out, out, out, out)

    def prefill(gate):
        L.moe_prefill_layer_scored(*xw, None, gate, k, 128, L.MOE_W_BF16, out, 4096, L.DecoderBuffers(), out)

    entries = [scored, prefill]
    for kind in ("host", "device"):
        d, set_gate = decoder(L, kind, E)
        entries.append(lambda gate, d=d, f=set_gate: f(d, gate))
        entries.append(lambda gate, d=d, f=set_gate: f(d, gate, gate.balance.shape[0]))
    for call in entries:
        del calls[:]
        with pytest.raises(ValueError, match="balance"):
            call(g)
        assert calls == []
        call(good)
        assert len(calls) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["other", "none", "moved"])
def test_a_captured_step_keeps_its_gate(L, how):
    """Graph replays after the decoder has another gate (or none), the first one's tensor has no owner left, and memory
    of its size has been written over and over."""
    import dataclasses

    import oracle
    from routed_expert_layer_amd.runtime import DeviceDecodeLayer
    from tests.parity import np64, npi
    from tests.test_gpu_layer import make_store
    from workloads import CONFIGS, gen
    dev = "cuda"
    cfg = dataclasses.replace(CONFIGS["decode_bf16_h4096_e256"], name="keptgate", L=1, T=3, steps=20, H=256, E=16, I=128,
                              k=2, zipf_s=1.0, epoch=8, S=16)
    store = make_store(cfg)
    try:
        dl = DeviceDecodeLayer(store, cfg.S, cfg.T, cfg.k, cfg.act, dev, keep_logits=True)
        values = torch.linspace(-1, 1, cfg.E)[torch.randperm(cfg.E, generator=torch.Generator().manual_seed(1))]
        kw = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=1.5)
        s = torch.cuda.Stream()
        gate = L.Gate(balance=values.to(dev), **kw)
        dl.set_gate(gate)
        x, bias = torch.empty((cfg.T, cfg.H), dtype=torch.bfloat16, device=dev), torch.empty(cfg.E, device=dev)
        W = gen.router_weight(cfg, 0, dev)
        torch.cuda.synchronize()
        graph = dl.capture(lambda: dl.step(0, x, W, bias, s), s)
        if how == "other":
            dl.set_gate(L.Gate(balance=-values.to(dev), **kw))
            del gate
        elif how == "none":
            dl.set_gate(None)
            del gate
        else:
            gate.balance = -values.to(dev)
        gc.collect()
        for step in range(4):
            over = [torch.full((cfg.E,), 7.0 * (-1) ** i, device=dev) for i in range(64)]
            for b in over:
                b[:: 2] = 0.0
            x.copy_(gen.tokens(cfg, step, 0, dev))
            bias.copy_(gen.router_bias(cfg, 0, step, dev))
            torch.cuda.synchronize()
            dl.replay(graph, s)
            torch.cuda.synchronize()
            idx, w = oracle.gate_select(np64(dl.rb.logits), cfg.k, balance=values.numpy(), **kw)
            assert np.array_equal(npi(dl.rb.topk_idx), idx), f"replay {step}"
            assert np.all(np.abs(np64(dl.rb.topk_w) - w) <= 2.0 ** -23 * np.abs(w))
            del over
    finally:
        store.close()
