"""GPU parity of the scored gates: choices, counts and positions equal the oracle's bit for bit, weights within half an
fp32 step of the value in 64 bits."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from tests.parity import check_close, check_permutation, np64, npi
from workloads import CONFIGS, gen

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def outputs(T, E, k):
    i32 = dict(dtype=torch.int32, device=dev)
    return dict(topk_idx=torch.full((T, k), -7, **i32), topk_w=torch.full((T, k), -7.0, device=dev),
                counts=torch.full((E,), -7, **i32), offsets=torch.full((E + 1,), -7, **i32),
                perm_src=torch.full((max(T * k, 1) + 3,), -7, **i32), perm_pos=torch.full((T, k), -7, **i32))


def select(L, l, gate, k, o=None, ws=None, stream=None):
    T, E = l.shape
    o = o or outputs(T, E, k)
    if ws is None:
        ws = torch.empty(L.moe_select_workspace_size(T, E, k), dtype=torch.uint8, device=dev)
    L.moe_select(l, gate, k, o["topk_idx"], o["topk_w"], o["counts"], o["offsets"], o["perm_src"], o["perm_pos"], ws,
                 stream)
    return o


def check(o, l, k, what, **kw):
    """The outputs of a selection from logits l against the oracle's."""
    T, E = l.shape
    idx, w = oracle.gate_select(np64(l), k, **{n: np64(v) if n == "balance" and v is not None else v
                                               for n, v in kw.items()})
    got = npi(o["topk_idx"])
    assert np.array_equal(got, idx), f"{what}: {np.sum((got != idx).any(1))} of {T} tokens differ"
    # one rounding to fp32 (half a step, 2^-24, or of the smallest subnormal); the 64-bit sums differ by far less
    gw = np64(o["topk_w"])
    assert np.all(np.abs(gw - w) <= 2.0 ** -24 * (1 + 1e-6) * np.abs(w) + 2.0 ** -150), what
    check_permutation(idx, npi(o["counts"]), npi(o["offsets"]), npi(o["perm_src"]), npi(o["perm_pos"]), E)
    assert np.all(npi(o["perm_src"])[T * k:] == -7), f"{what}: wrote past the rows"


CASES = [
    # T, E, k, score, groups, kept, group_top, balance, renorm, scale
    (0, 16, 2, "softmax", 1, 1, 1, False, True, 1.0),
    (1, 1, 1, "sigmoid", 1, 1, 2, True, True, 1.0),
    (1, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5),
    (2, 64, 6, "softmax", 8, 3, 1, False, False, 16.0),
    (16, 512, 16, "sigmoid", 1, 1, 1, True, True, 1.0),
    (17, 65, 5, "softmax", 5, 2, 2, True, False, 1.0),
    (63, 128, 8, "softmax", 1, 1, 1, False, True, 1.0),
    (64, 20, 4, "sigmoid", 4, 4, 2, True, True, 1.0),
    (65, 100, 7, "sigmoid", 4, 2, 2, True, False, 0.5),
    (130, 250, 6, "softmax", 10, 3, 2, True, True, 2.5),
    (300, 256, 6, "sigmoid", 1, 1, 1, True, True, 1.0),
    (300, 1024, 16, "sigmoid", 64, 20, 2, True, True, 1.0),
    (129, 1000, 10, "softmax", 8, 8, 1, False, True, 1.0),
    (70, 16, 16, "sigmoid", 2, 2, 1, True, True, 1.0),
    (70, 32, 8, "sigmoid", 32, 8, 2, True, True, 1.0),  # groups of one expert
    (1000, 64, 6, "softmax", 8, 4, 2, False, True, 1.0),
    (5000, 160, 6, "softmax", 8, 3, 1, False, False, 16.0),
]


def ids(c):
    return f"T{c[0]}-E{c[1]}-k{c[2]}-{c[3]}-g{c[4]}.{c[5]}.{c[6]}{'-b' if c[7] else ''}"


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_select_parity(L, case):
    T, E, k, score, G, keep, top, bal, renorm, scale = case
    g = torch.Generator(device=dev).manual_seed(T * 1000 + E)
    l = torch.randn((T, E), generator=g, device=dev) * 1.5
    b = 0.2 * torch.randn(E, generator=g, device=dev) if bal else None
    kw = dict(score=score, n_group=G, topk_group=keep, group_top=top, renorm=renorm, scale=scale, balance=b)
    o = select(L, l, L.Gate(**kw), k)
    torch.cuda.synchronize()
    check(o, l, k, ids(case), **kw)


@pytest.mark.parametrize("E,G,keep", [(12, 4, 2), (256, 8, 4), (300, 1, 1), (520, 4, 3)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_ties(L, E, G, keep, score):
    """Logits and balance on a coarse grid: ties everywhere, in groups and in experts, go to the lower index."""
    g = torch.Generator(device=dev).manual_seed(E)
    l = (torch.randn((200, E), generator=g, device=dev) * 2).round() / 2
    l[:7] = 0.0
    l[3, ::2] = -0.0
    for b in (None, (torch.randn(E, generator=g, device=dev)).round() / 4, torch.zeros(E, device=dev)):
        for top in (1, 2):
            kw = dict(score=score, n_group=G, topk_group=keep, group_top=top, balance=b)
            o = select(L, l, L.Gate(**kw), 5)
            torch.cuda.synchronize()
            check(o, l, 5, f"{score} top{top}", **kw)


@pytest.mark.parametrize("T", [8, 150])
def test_select_near_ties(L, T):
    """The balance of each token's row brings every biased score within about 2^-24 of one value: the order is decided
    far below what 32-bit scores hold. (One token a call, so that each has a balance of its own.)"""
    E, k = 96, 6
    g = torch.Generator(device=dev).manual_seed(T)
    l = torch.randn((T, E), generator=g, device=dev)
    b = (0.75 - 1.0 / (1.0 + torch.exp(-l[0].double()))).float()
    l[1:] = l[0] + 1e-6 * torch.randn((T - 1, E), generator=g, device=dev)
    for G, keep, top in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
        kw = dict(score="sigmoid", n_group=G, topk_group=keep, group_top=top, balance=b)
        o = select(L, l, L.Gate(**kw), k)
        torch.cuda.synchronize()
        check(o, l, k, f"near ties g{G}", **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_extremes(L, score):
    """Masked experts (-inf and the type's lowest), rows masked throughout, infinities, NaN, and infinite balances."""
    E, k, inf, nan = 24, 4, float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    g = torch.Generator(device=dev).manual_seed(5)
    l = torch.randn((100, E), generator=g, device=dev)
    l[0, 3:] = -inf
    l[1] = -inf
    l[2] = low
    l[3, 2:] = low
    l[4] = nan
    l[5, ::2] = nan
    l[6, 5] = inf
    l[7, 5:9] = inf
    l[8] = inf
    l[9] = -low
    l[10, 4] = -low
    l[11] *= 1e4
    l[12] *= 60
    l[70, 1:] = -inf
    for bal in (None, [0.0] * E, [(-inf if e % 5 == 0 else 0.1 * e) for e in range(E)],
                [(inf if e == 7 else nan if e == 3 else -inf if e == 8 else 0.0) for e in range(E)]):
        b = None if bal is None else torch.tensor(bal, device=dev)
        for G, keep, top, renorm in ((1, 1, 1, True), (1, 1, 1, False), (6, 3, 2, True), (6, 3, 1, False)):
            kw = dict(score=score, n_group=G, topk_group=keep, group_top=top, renorm=renorm, balance=b)
            o = select(L, l, L.Gate(**kw), k)
            torch.cuda.synchronize()
            check(o, l, k, f"{score} g{G} top{top} balance {bal}", **kw)


def test_select_streams_and_graph(L):
    """On a stream of its own; captured once and replayed on new logits, a longer and a shorter call in between on
    other buffers, every replay against the oracle."""
    T, E, k = 200, 128, 6
    s = torch.cuda.Stream()
    l = torch.empty((T, E), device=dev)
    b = 0.1 * torch.randn(E, device=dev)
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5, balance=b)
    gate = L.Gate(**kw)
    o = outputs(T, E, k)
    ws = torch.empty(L.moe_select_workspace_size(T, E, k), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    L.moe_graph_begin(s)
    select(L, l, gate, k, o, ws, s)
    graph = L.moe_graph_end(s)
    for i in range(4):
        l.copy_(torch.randn((T, E), device=dev))
        torch.cuda.synchronize()
        L.moe_graph_launch(graph, s)
        other = torch.randn((300 - 90 * i, E), device=dev)
        oo = select(L, other, gate, k)
        torch.cuda.synchronize()
        check(o, l, k, f"replay {i}", **kw)
        check(oo, other, k, f"eager {i}", **kw)


def exact_gate_inputs(cfg, T, E, seed):
    """x and Wr on coarse grids whose products sum exactly in fp32 in any order, so that logits are whole-exact."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-8, 9, (T, cfg.H), generator=g).to(torch.bfloat16) / 8
    W = torch.randint(-8, 9, (cfg.H, E), generator=g).to(torch.bfloat16) / 64
    dt = torch.float32 if cfg.act == "f32" else torch.bfloat16
    return x.to(dt).to(dev), W.to(dt).to(dev)


@pytest.mark.parametrize("base,T,H,E", [("decode_bf16_h4096_e256", 1, 4096, 256), ("decode_bf16_h4096_e256", 16, 512, 512),
                                        ("tiny_f32_h256_e16", 9, 256, 48), ("decode_bf16_h4096_e256", 40, 512, 96),
                                        ("decode_bf16_h4096_e256", 300, 512, 256),
                                        ("decode_bf16_h4096_e256", 700, 1024, 128)])
def test_route_scored_parity(L, base, T, H, E):
    """Every routing path (decode, matrix cores with and without split slabs, plain) under a gate: logits exact by
    construction, choices equal the oracle's."""
    from routed_expert_layer_amd.runtime import RouteBuffers
    cfg = dataclasses.replace(CONFIGS[base], H=H)
    k = 6
    x, W = exact_gate_inputs(cfg, T, E, T)
    bias = (torch.randint(-16, 17, (E,)) / 16).to(dev)
    b = 0.1 * torch.randn(E, device=dev)
    rb = RouteBuffers(T, H, E, k, dev, keep_logits=True)
    for score in ("sigmoid", "softmax"):
        kw = dict(score=score, n_group=8, topk_group=4, group_top=2, renorm=score == "sigmoid", scale=2.5, balance=b)
        rb.perm_src.fill_(-7)
        rb.route(x, W, bias, gate=L.Gate(**kw))
        torch.cuda.synchronize()
        l64 = oracle.router_logits(x, W, bias)
        assert np.array_equal(np64(rb.logits), l64)
        o = dict(topk_idx=rb.topk_idx, topk_w=rb.topk_w, counts=rb.counts, offsets=rb.offsets, perm_src=rb.perm_src,
                 perm_pos=rb.perm_pos)
        check(o, rb.logits, k, f"route T={T} E={E} {score}", **kw)


@pytest.mark.parametrize("device", [False, True], ids=["host", "device"])
def test_decoders_under_a_gate(L, device):
    """Steps of both decoders under a gate, with evictions: choices, cache trace and outputs against the oracle; taking
    the gate off brings moe_route's choice back."""
    from routed_expert_layer_amd.runtime import DecodeLayer, DeviceDecodeLayer
    from tests.test_gpu_layer import ExpertCache64, make_store
    cfg = dataclasses.replace(CONFIGS["decode_bf16_h4096_e256"], name="gated", L=2, T=3, steps=20, H=256, E=16, I=128,
                              k=2, zipf_s=1.0, epoch=8, S=8)
    store = make_store(cfg)
    try:
        dl = (DeviceDecodeLayer(store, cfg.S, cfg.T, cfg.k, cfg.act, dev, keep_logits=True, trace_capacity=4096)
              if device else DecodeLayer(store, cfg.S, cfg.T, cfg.k, cfg.act, dev, keep_logits=True))
        b = 0.3 * torch.randn(cfg.E, device=dev)
        kw = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=1.5, balance=b)
        dl.set_gate(L.Gate(**kw))
        sim = oracle.SharedLRU(cfg.S)
        ge = [ExpertCache64(cfg, l) for l in range(cfg.L)]
        for step in range(21):
            if step == 20:
                dl.set_gate(None)
            for layer in range(cfg.L):
                x, W = gen.tokens(cfg, step, layer, dev), gen.router_weight(cfg, layer, dev)
                bias = gen.router_bias(cfg, layer, step, dev)
                out = dl.step(layer, x, W, bias) if device else dl.step(step, layer, x, W, bias)
                torch.cuda.synchronize()
                l64 = np64(dl.rb.logits)
                check_close(l64, oracle.router_logits(x, W, bias), "logits", rel_l2=1e-5, max_abs_rms=1e-4)
                idx, w = oracle.gate_select(l64, cfg.k, **dict(kw, balance=np64(b))) if step < 20 else (
                    oracle.topk_select(l64, cfg.k), oracle.topk_weights(l64, oracle.topk_select(l64, cfg.k)))
                assert np.array_equal(npi(dl.rb.topk_idx), idx)
                counts, off, pos, src = oracle.permute(idx, cfg.E)
                sim.resolve(step, layer, cfg.E, np.nonzero(counts)[0])
                y = oracle.expert_outputs(np64(x), off, src, lambda e: ge[layer](int(e)))
                check_close(np64(out), oracle.combine(y, pos, w), f"step {step} layer {layer}")
        ref = [r.hit for r in sim.trace]
        if device:
            hits, misses, _ = dl.stats()
        else:
            hits, misses = L.moe_cache_stats(dl.cache)
        assert (hits, misses) == (sum(ref), len(ref) - sum(ref))
    finally:
        store.close()


def test_prefill_layer_under_a_gate(L):
    from routed_expert_layer_amd.runtime import PrefillLayer
    from tests.test_gpu_layer import ExpertCache64
    cfg = dataclasses.replace(CONFIGS["prefill_bf16_t4096_e256"], name="gatedprefill", T=150, H=512, I=256, E=8, k=3)
    blob = L.moe_expert_bytes(L.MOE_W_BF16, cfg.H, cfg.I)
    base = torch.empty(cfg.E * blob, dtype=torch.uint8, device=dev)
    for e in range(cfg.E):
        L.moe_pack_expert(L.MOE_W_BF16, cfg.H, cfg.I, *gen.expert_weights(cfg, 0, e, dev), None, None, None,
                          base[e * blob:])
    kw = dict(score="softmax", n_group=4, topk_group=2, group_top=1, renorm=False, scale=4.0)
    pl = PrefillLayer(cfg.H, cfg.I, cfg.E, cfg.k, cfg.T, blob, dev, keep_logits=True, gate=L.Gate(**kw))
    x, W = gen.tokens(cfg, 0, 0, dev), gen.router_weight(cfg, 0, dev)
    out = pl.forward(x, W, None, base)
    torch.cuda.synchronize()
    idx, w = oracle.gate_select(np64(pl.rb.logits), cfg.k, **kw)
    assert np.array_equal(npi(pl.rb.topk_idx), idx)
    counts, off, pos, src = oracle.permute(idx, cfg.E)
    ge = ExpertCache64(cfg, 0)
    check_close(np64(out), oracle.combine(oracle.expert_outputs(np64(x), off, src, lambda e: ge(int(e))), pos, w),
                "gated prefill layer")


@pytest.mark.parametrize("T,E,k,G,keep", [(3, 1023, 5, 33, 7), (70, 1023, 16, 33, 7), (5000, 512, 8, 1, 1), (16384, 48, 2, 1, 1),
                                          (16385, 96, 6, 8, 3), (16500, 512, 4, 4, 2), (16400, 1023, 3, 33, 9)])
def test_select_long_and_wide(L, T, E, k, G, keep):
    """Past the batches that two launches group, and the shapes with most experts a lane."""
    g = torch.Generator(device=dev).manual_seed(T + E)
    l = torch.randn((T, E), generator=g, device=dev) * 1.5
    kw = dict(score="sigmoid", n_group=G, topk_group=keep, group_top=2, scale=2.0,
              balance=0.2 * torch.randn(E, generator=g, device=dev))
    o = select(L, l, L.Gate(**kw), k)
    torch.cuda.synchronize()
    check(o, l, k, f"T{T} E{E}", **kw)


def test_select_two_streams_at_once(L):
    """Calls of several sizes on two streams together, each with its own workspace and outputs."""
    E, k = 256, 8
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2)
    ls = [[torch.randn((T, E), device=dev) for T in (1, 300, 5000, 17)] for _ in range(2)]
    ws = [torch.empty(L.moe_select_workspace_size(5000, E, k), dtype=torch.uint8, device=dev) for _ in range(2)]
    outs = [[outputs(l.shape[0], E, k) for l in q] for q in ls]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(4):
        for q in range(2):
            select(L, ls[q][i], L.Gate(**kw), k, outs[q][i], ws[q], ss[q])
    torch.cuda.synchronize()
    for q in range(2):
        for l, o in zip(ls[q], outs[q]):
            check(o, l, k, f"stream {q} T{l.shape[0]}", **kw)
