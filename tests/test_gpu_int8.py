"""GPU parity of the int8 experts against their statement in 64 bits, within tolerances derived in int8_cases."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from tests import int8_cases as ic
from tests.parity import np64, npi
from workloads import CONFIGS, gen

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def pack(L, H, I, experts, slot_of, n_slots):
    """Slots of packed blobs, the unused ones and the stride's padding filled with 0xFF bytes."""
    stride = (L.moe_expert_bytes(L.MOE_W_INT8, H, I) + 511) // 512 * 512
    slots = torch.full((n_slots * stride,), 255, dtype=torch.uint8, device=dev)
    for e, w in enumerate(experts):
        if 0 <= slot_of[e] < n_slots:
            L.moe_pack_expert(L.MOE_W_INT8, H, I, w["q1"], w["q3"], w["q2"], w["s1"], w["s3"], w["s2"],
                              slots[slot_of[e] * stride:])
    return slots, stride


def tokens(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g) * (0.2 + 2 * torch.rand((T, 1), generator=g))
    return x.to(torch.bfloat16).to(dev)


def routing(T, E, k, seed, skew=0.0, never=()):
    """A routing on the GPU and its arrays on the host; experts in `never` get no token."""
    r = np.random.default_rng(seed)
    score = r.standard_normal((T, E)) + skew * r.standard_normal(E)
    score[:, list(never)] = -1e9
    idx = np.argsort(-score, axis=1, kind="stable")[:, :k]
    w = r.random((T, k)) + 0.05
    w = (w / w.sum(1, keepdims=True)).astype(np.float32)
    counts, offsets, pos, src = oracle.permute(idx, E)
    t = lambda a, d=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(d).to(dev)  # noqa: E731
    return dict(idx=idx, w=w, counts=counts, offsets=offsets, pos=pos, src=src,
                dev=dict(topk_idx=t(idx), topk_w=t(w, torch.float32), perm_src=t(src), perm_pos=t(pos),
                         counts=t(counts), offsets=t(offsets)))


def expected(x, experts, rt, slot_of, n_slots, half=False):
    """(out, tol) of the layer's expert half in 64 bits, over the experts that have a slot; half: as in reference()."""
    x64, T, H = np64(x), x.shape[0], x.shape[1]
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    for e, w in enumerate(experts):
        n = int(rt["counts"][e])
        if n == 0 or not 0 <= slot_of[e] < n_slots:
            continue
        rows = rt["src"][rt["offsets"][e]:rt["offsets"][e] + n]
        y, ty = ic.reference(x64[rows], w, half)
        wt = np.array([rt["w"][t][list(rt["idx"][t]).index(e)] for t in rows], np.float64)[:, None]
        np.add.at(out, rows, wt * y)
        # the sum of k products in fp32: k roundings of at most the sum of magnitudes
        np.add.at(tol, rows, wt * ty + rt["idx"].shape[1] * 2.0 ** -23 * wt * np.abs(y))
    return out, tol


def run(L, x, rt, slots, stride, slot_of, n_slots, H, I, dtype=torch.float32, ws=None, out=None, stream=None):
    T, k = rt["idx"].shape
    E = len(rt["counts"])
    d = rt["dev"]
    if out is None:
        out = torch.full((T, H), float("nan"), dtype=dtype, device=dev)
    if ws is None:  # NaN bytes: nothing may be read before it is written
        ws = torch.full((L.moe_experts_workspace_size(T, k, E, H, I, L.MOE_W_INT8),), 255, dtype=torch.uint8, device=dev)
    L.moe_experts(x, d["topk_idx"], d["topk_w"], d["perm_src"], d["perm_pos"], d["counts"], d["offsets"],
                  None if slot_of is None else torch.tensor(slot_of, dtype=torch.int32, device=dev), n_slots, slots,
                  stride, L.MOE_W_INT8, H, I, out, ws, stream)
    return out


CASES = [
    # T, E, k, H, I, skew
    (1, 4, 1, 64, 64, 0),
    (1, 8, 6, 512, 256, 0),
    (12, 8, 2, 256, 128, 0.5),  # the last call whose down projection forms the output
    (13, 8, 2, 256, 128, 0.5),
    (2, 3, 3, 192, 320, 0),     # K tails of the decode kernels, every expert
    (7, 16, 4, 1088, 704, 0.5),
    (16, 4, 2, 256, 128, 1.0),
    (17, 2, 1, 256, 128, 0),    # the tiled products: from 4 rows an expert on
    (40, 16, 1, 256, 128, 6.0),  # few rows an expert, but groups past one tile of 16 rows
    (6, 3, 2, 384, 128, 0),     # tiles of 128 weight rows, where H is no multiple of 256
    (700, 2, 1, 640, 384, 0),   # the same with groups of more than 256 rows
    (90, 6, 3, 128, 256, 1.0),
    (32, 2, 2, 320, 192, 0),
    (33, 8, 2, 256, 128, 0.5),
    (64, 16, 6, 512, 256, 1.5),
    (40, 4, 2, 320, 192, 0.5),  # a shape that only the decode kernels take
    (130, 5, 3, 768, 384, 0.5),
    (300, 3, 2, 256, 2176, 0),  # h rows wider than the registers of the pass between the products
    (600, 4, 2, 512, 256, 0.0),
    (900, 2, 1, 256, 128, 0.0),
    (257, 40, 8, 1024, 128, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_experts_parity(L, case, bf16):
    T, E, k, H, I, skew = case
    experts = [ic.expert(H, I, 100 * e + H, dev) for e in range(E)]
    slot_of = [(3 * e + 1) % (E + 2) if (E + 2) % 3 else E + 1 - e for e in range(E)]
    slots, stride = pack(L, H, I, experts, slot_of, E + 2)
    x, rt = tokens(T, H, T), routing(T, E, k, T + E, skew)
    out = run(L, x, rt, slots, stride, slot_of, E + 2, H, I, torch.bfloat16 if bf16 else torch.float32)
    torch.cuda.synchronize()
    ic.check(np64(out), *expected(x, experts, rt, slot_of, E + 2, half=bf16), str(case), bf16)


@pytest.mark.parametrize("T", [5, 200])
def test_experts_without_a_slot(L, T):
    """Experts whose slot is negative or past the slots are left out; tokens that chose only such experts get zeros;
    experts no token chose cost nothing."""
    E, k, H, I = 6, 2, 256, 128
    experts = [ic.expert(H, I, e, dev) for e in range(E)]
    slot_of = [2, -1, 0, 5, 1, -7]
    slots, stride = pack(L, H, I, experts, slot_of, 3)
    x, rt = tokens(T, H, 1), routing(T, E, k, 2, never=(4,))
    rt0 = dict(rt)
    out = run(L, x, rt0, slots, stride, slot_of, 3, H, I)
    torch.cuda.synchronize()
    ref, tol = expected(x, experts, rt, slot_of, 3)
    only = [t for t in range(T) if all(slot_of[e] not in (0, 1, 2) for e in rt["idx"][t])]
    assert np.all(np64(out)[only] == 0)
    ic.check(np64(out), ref, tol, "left-out experts")
    # none has a slot
    out = run(L, x, rt, slots, stride, [-1] * E, 3, H, I)
    torch.cuda.synchronize()
    assert np.all(np64(out) == 0)


@pytest.mark.parametrize("T", [6, 150])
def test_experts_special_rows(L, T):
    """A token of zeros gives zeros; halves of the largest value are rounded to even; tiny and huge tokens keep their
    relative precision; a token with an infinity or a NaN gives NaN and leaves the others as they are."""
    E, k, H, I = 3, 2, 256, 128
    experts = [ic.expert(H, I, e, dev) for e in range(E)]
    slots, stride = pack(L, H, I, experts, range(E), E)
    x = tokens(T, H, 3)
    x[0] = 0
    x[1] = torch.where(torch.arange(H, device=dev) % 2 == 0, 1.0, 0.5).to(torch.bfloat16)
    x[1, 1::4] = -0.5
    x[2] = (x[2].float() * 2.0 ** -60).to(torch.bfloat16)
    x[3] = (x[3].float() * 2.0 ** 20).to(torch.bfloat16)
    rt = routing(T, E, k, 4)
    out = run(L, x, rt, slots, stride, None, E, H, I)
    torch.cuda.synchronize()
    ref, tol = expected(x, experts, rt, range(E), E)
    assert np.all(np64(out)[0] == 0)
    keep = [t for t in range(T) if t != 3]  # |g| of token 3 is beyond what the tolerance counts
    ic.check(np64(out)[keep], ref[keep], tol[keep], "special rows")
    rel = np.linalg.norm(np64(out)[3] - ref[3]) / np.linalg.norm(ref[3])
    assert rel < 1e-3  # silu is 0 or g there: the codes' flips alone, sqrt(I) of them at most, are below this
    x[4, 7], x[T - 1, 0] = float("inf"), float("nan")
    out2 = run(L, x, rt, slots, stride, None, E, H, I)
    torch.cuda.synchronize()
    bad = [4, T - 1]
    rest = [t for t in range(T) if t not in bad]
    assert np.all(np.isnan(np64(out2)[bad]))
    assert torch.equal(out2[rest], out[rest])


def test_experts_graph_streams_and_buffers(L):
    """Captured on a stream, replayed on changing tokens and routings, eager calls of other sizes on another workspace
    in between; every replay equals the eager result bit for bit, and nothing behind the output is written."""
    E, k, H, I, T = 8, 2, 512, 256, 40
    experts = [ic.expert(H, I, e, dev) for e in range(E)]
    slots, stride = pack(L, H, I, experts, range(E), E)
    s = torch.cuda.Stream()
    x = tokens(T, H, 0)
    rt = routing(T, E, k, 0)
    size = L.moe_experts_workspace_size(T, k, E, H, I, L.MOE_W_INT8)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=dev)
    back = torch.full((T + 2, H), -7.0, device=dev)
    out = back[:T]
    torch.cuda.synchronize()
    L.moe_graph_begin(s)
    run(L, x, rt, slots, stride, None, E, H, I, ws=ws, out=out, stream=s)
    graph = L.moe_graph_end(s)
    for i in range(4):
        nx, nrt = tokens(T, H, 10 + i), routing(T, E, k, 20 + i, skew=1.0)
        x.copy_(nx)
        for n in rt["dev"]:
            rt["dev"][n].copy_(nrt["dev"][n])
        torch.cuda.synchronize()
        L.moe_graph_launch(graph, s)
        big = run(L, tokens(90, H, i), routing(90, E, k, i), slots, stride, None, E, H, I)
        eager = run(L, nx, nrt, slots, stride, None, E, H, I)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), f"replay {i}"
        assert torch.isfinite(big).all()
        assert torch.all(back[T:] == -7.0)
        ic.check(np64(out), *expected(nx, experts, nrt, range(E), E), f"replay {i}")


@pytest.mark.parametrize("rows,H,I,mode", [([1, 0, 6, 16, 17, 2, 33], 512, 256, "decode"), ([5, 1, 0, 9], 192, 320, "auto"),
                                           ([130, 0, 1, 127, 300], 512, 256, "prefill"), ([40, 2, 70], 256, 128, "auto")])
def test_ffn_list_parity(L, rows, H, I, mode):
    """moe_ffn over a host list: rows of y_perm that no item lists stay as they were."""
    E = len(rows)
    T = max(40, max(rows))
    experts = [ic.expert(H, I, e + 50, dev) for e in range(E)]
    slot_of = [(e + 1) % E for e in range(E)]
    slots, stride = pack(L, H, I, experts, slot_of, E)
    x = tokens(T, H, 9)
    r = np.random.default_rng(1)
    gap = 3  # unlisted rows between the groups
    off = np.cumsum([0] + [n + gap for n in rows])
    total = int(off[-1])
    src = r.integers(0, T, size=total).astype(np.int32)
    work = np.array([[e, slot_of[e], off[e], rows[e]] for e in range(E)], np.int32)
    y = torch.full((total, H), -7.0, device=dev)
    ws = torch.full((L.moe_ffn_workspace_size(total, H, I, L.MOE_W_INT8),), 255, dtype=torch.uint8, device=dev)
    m = dict(auto=L.MOE_FFN_AUTO, decode=L.MOE_FFN_DECODE, prefill=L.MOE_FFN_PREFILL)[mode]
    L.moe_ffn(x, torch.from_numpy(src).to(dev), work, slots, stride, L.MOE_W_INT8, H, I, y, ws, m)
    torch.cuda.synchronize()
    yg, x64 = np64(y), np64(x)
    for e in range(E):
        a, b = off[e], off[e] + rows[e]
        if rows[e]:
            ic.check(yg[a:b], *ic.reference(x64[src[a:b]], experts[e]), f"expert {e}")
        assert np.all(yg[b:b + gap] == -7.0)


def int8_config(**kw):
    return dataclasses.replace(CONFIGS["decode_bf16_h4096_e256"], **dict(dict(name="int8cfg", L=2, T=3, H=256, E=16, I=128,
                                                                             k=2, zipf_s=1.0, epoch=8, S=8), **kw))


@pytest.mark.parametrize("kind,T", [("host", 3), ("host", 20), ("device", 3), ("graph", 3)])
def test_decoders_with_int8_experts(L, kind, T):
    """Steps with evictions through each decoder under a scored gate: routing, quantisation, products and combine
    together, against the oracle on the step's own logits."""
    from routed_expert_layer_amd.runtime import DecodeLayer, DeviceDecodeLayer, ExpertStore
    cfg = int8_config(T=T, S=8 if T == 3 else 16)
    E, H, I, k = cfg.E, cfg.H, cfg.I, cfg.k
    store = ExpertStore(cfg.L, E, H, I, "int8")
    try:
        ex = [[ic.expert(H, I, 1000 * l + e, dev) for e in range(E)] for l in range(cfg.L)]
        for l in range(cfg.L):
            store.pack_layer(l, lambda e: ex[l][e], device=dev)
        dl = (DecodeLayer(store, cfg.S, T, k, "bf16", dev, keep_logits=True) if kind == "host" else
              DeviceDecodeLayer(store, cfg.S, T, k, "bf16", dev, keep_logits=True))
        kw = dict(score="sigmoid", n_group=4, topk_group=3, group_top=2, scale=1.5,
                  balance=0.2 * torch.randn(E, device=dev))
        dl.set_gate(L.Gate(**kw))
        s = torch.cuda.Stream()
        xs = [torch.empty((T, H), dtype=torch.bfloat16, device=dev) for _ in range(cfg.L)]
        bs = [torch.empty(E, device=dev) for _ in range(cfg.L)]
        Ws = [gen.router_weight(cfg, l, dev) for l in range(cfg.L)]
        outs = [torch.empty((T, H), device=dev) for _ in range(cfg.L)]
        logits = [torch.empty((T, E), device=dev) for _ in range(cfg.L)]
        idxs = [torch.empty((T, k), dtype=torch.int32, device=dev) for _ in range(cfg.L)]
        torch.cuda.synchronize()

        def step(i):
            with torch.cuda.stream(s):
                for l in range(cfg.L):
                    o = dl.step(i, l, xs[l], Ws[l], bs[l], s) if kind == "host" else dl.step(l, xs[l], Ws[l], bs[l], s)
                    for a, b in ((outs[l], o), (logits[l], dl.rb.logits), (idxs[l], dl.rb.topk_idx)):
                        a.copy_(b)

        graph = None
        if kind == "graph":
            graph = dl.capture(lambda: step(0), s)
        sim = oracle.SharedLRU(cfg.S)
        for i in range(12):
            for l in range(cfg.L):
                xs[l].copy_(gen.tokens(cfg, i, l, dev))
                bs[l].copy_(gen.router_bias(cfg, l, i, dev))
            torch.cuda.synchronize()
            if graph is not None:
                dl.replay(graph, s)
            else:
                step(i)
            torch.cuda.synchronize()
            for l in range(cfg.L):
                idx, w = oracle.gate_select(np64(logits[l]), k, **dict(kw, balance=np64(kw["balance"])))
                assert np.array_equal(npi(idxs[l]), idx)
                counts, off, pos, src = oracle.permute(idx, E)
                sim.resolve(i, l, E, np.nonzero(counts)[0])
                rt = dict(idx=idx, w=w, counts=counts, offsets=off, pos=pos, src=src)
                ref, tol = expected(xs[l], ex[l], rt, range(E), E)
                ic.check(np64(outs[l]), ref, tol + 2.0 ** -23 * np.abs(ref), f"{kind} step {i} layer {l}")
        hits = sum(r.hit for r in sim.trace)
        got = L.moe_cache_stats(dl.cache) if kind == "host" else dl.stats()[:2]
        assert tuple(got) == (hits, len(sim.trace) - hits)
        if kind == "host":  # misses cannot run on the CPU in this format
            dl.set_split(1, 1)
            with pytest.raises(L.MoEError) as ei:
                dl.step(12, 0, xs[0], Ws[0], bs[0], s)
            assert ei.value.code == L.MOE_EINVAL
            torch.cuda.synchronize()
    finally:
        store.close()


@pytest.mark.parametrize("T,H,I", [(20, 320, 192), (150, 512, 256)])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_prefill_layer_with_int8_experts(L, T, H, I, gated):
    from routed_expert_layer_amd.runtime import PrefillLayer
    cfg = int8_config(T=T, H=H, I=I, E=8, k=3)
    experts = [ic.expert(H, I, e, dev) for e in range(cfg.E)]
    slots, stride = pack(L, H, I, experts, range(cfg.E), cfg.E)
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5, balance=0.1 * torch.randn(cfg.E, device=dev))
    pl = PrefillLayer(H, I, cfg.E, cfg.k, T, stride, dev, keep_logits=True, wfmt=L.MOE_W_INT8,
                      gate=L.Gate(**kw) if gated else None)
    x, W = gen.tokens(cfg, 0, 0, dev), gen.router_weight(cfg, 0, dev)
    out = pl.forward(x, W, None, slots)
    torch.cuda.synchronize()
    l64 = np64(pl.rb.logits)
    if gated:
        idx, w = oracle.gate_select(l64, cfg.k, **dict(kw, balance=np64(kw["balance"])))
    else:
        idx = oracle.topk_select(l64, cfg.k)
        w = oracle.topk_weights(l64, idx)
    assert np.array_equal(npi(pl.rb.topk_idx), idx)
    counts, off, pos, src = oracle.permute(idx, cfg.E)
    rt = dict(idx=idx, w=w, counts=counts, offsets=off, pos=pos, src=src)
    ref, tol = expected(x, experts, rt, range(cfg.E), cfg.E)
    # moe_route's weights carry fp32 exponentials: 1e-5, as the routing tests allow
    ic.check(np64(out), ref, tol + (1e-5 * cfg.k * np.abs(ref).max() if not gated else 2.0 ** -22 * np.abs(ref).max()),
             "int8 prefill layer")


@pytest.mark.parametrize("T,E,k,H,I", [(3, 2, 2, 64, 8192), (17, 2, 1, 4160, 64), (5, 3, 2, 8256, 128), (2, 2, 1, 16384, 64),
                                       (40, 2, 1, 16384, 128), (40, 3, 2, 256, 8192), (40, 24, 12, 256, 128)])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_experts_widest_shapes(L, T, E, k, H, I, bf16):
    """The largest H and I, and choices of more experts than the combine has in flight."""
    experts = [ic.expert(H, I, e + I, dev) for e in range(E)]
    slots, stride = pack(L, H, I, experts, range(E), E)
    x, rt = tokens(T, H, T), routing(T, E, k, H)
    out = run(L, x, rt, slots, stride, None, E, H, I, torch.bfloat16 if bf16 else torch.float32)
    torch.cuda.synchronize()
    ic.check(np64(out), *expected(x, experts, rt, range(E), E, half=bf16), f"{H}x{I}", bf16)


@pytest.mark.parametrize("T", [4, 50])
def test_experts_same_expert_twice(L, T):
    """A choice that names an expert twice has a row for each, weighted by its own weight."""
    E, k, H, I = 4, 3, 256, 128
    experts = [ic.expert(H, I, e, dev) for e in range(E)]
    slots, stride = pack(L, H, I, experts, range(E), E)
    x, r = tokens(T, H, 3), np.random.default_rng(T)
    idx = r.integers(0, E, (T, k))
    idx[0] = 2
    w = r.random((T, k)).astype(np.float32)
    order = np.argsort(idx.reshape(-1), kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    counts = np.bincount(idx.reshape(-1), minlength=E)
    t = lambda a, d=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(d).to(dev)  # noqa: E731
    rt = dict(idx=idx, counts=counts,
              dev=dict(topk_idx=t(idx), topk_w=t(w, torch.float32), perm_src=t(order // k), perm_pos=t(pos.reshape(T, k)),
                       counts=t(counts), offsets=t(np.concatenate([[0], np.cumsum(counts)]))))
    out = run(L, x, rt, slots, stride, None, E, H, I)
    torch.cuda.synchronize()
    ys = [ic.reference(np64(x), e) for e in experts]
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    for j in range(k):
        yj = np.stack([ys[idx[a, j]][0][a] for a in range(T)])
        wj = w[:, j:j + 1].astype(np.float64)
        y += wj * yj
        tol += wj * np.stack([ys[idx[a, j]][1][a] for a in range(T)]) + k * 2.0 ** -23 * wj * np.abs(yj)
    ic.check(np64(out), y, tol, "twice")


def test_experts_two_streams_at_once(L):
    """Decode and prefill sizes on two streams together, each with its own workspace, equal the same calls alone."""
    E, k, H, I = 8, 2, 512, 256
    experts = [ic.expert(H, I, e, dev) for e in range(E)]
    slots, stride = pack(L, H, I, experts, range(E), E)
    calls = [[(tokens(T, H, T + q), routing(T, E, k, T + q)) for T in (1, 300, 16, 40)] for q in range(2)]
    alone = [[run(L, x, rt, slots, stride, None, E, H, I) for x, rt in q] for q in calls]
    size = L.moe_experts_workspace_size(300, k, E, H, I, L.MOE_W_INT8)
    ws = [torch.full((size,), 255, dtype=torch.uint8, device=dev) for _ in range(2)]
    outs = [[torch.full_like(o, float("nan")) for o in q] for q in alone]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(4):
        for q in range(2):
            x, rt = calls[q][i]
            run(L, x, rt, slots, stride, None, E, H, I, ws=ws[q], out=outs[q][i], stream=ss[q])
    torch.cuda.synchronize()
    for q in range(2):
        for i in range(4):
            assert torch.equal(outs[q][i], alone[q][i]), (q, i)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_ffn_list_of_many_experts(L, mode):
    """More items than one launch takes, some of them in slots shared, and tiles of 256 rows."""
    H, I, E = 256, 128, 3
    rows = [1 + (5 * i) % 9 for i in range(64)] + ([300, 520] if mode == "prefill" else [30]) + [2] * 5
    experts = [ic.expert(H, I, e, dev) for e in range(E)]
    slots, stride = pack(L, H, I, experts, range(E), E)
    total, T = sum(rows), 50
    x = tokens(T, H, 1)
    src = np.random.default_rng(2).integers(0, T, size=total).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(rows)])
    work = np.array([[i % E, i % E, off[i], n] for i, n in enumerate(rows)], np.int32)
    y = torch.full((total, H), float("nan"), device=dev)
    ws = torch.full((L.moe_ffn_workspace_size(total, H, I, L.MOE_W_INT8),), 255, dtype=torch.uint8, device=dev)
    L.moe_ffn(x, torch.from_numpy(src).to(dev), work, slots, stride, L.MOE_W_INT8, H, I, y, ws,
              L.MOE_FFN_DECODE if mode == "decode" else L.MOE_FFN_PREFILL)
    torch.cuda.synchronize()
    yg, x64 = np64(y), np64(x)
    for i, n in enumerate(rows):
        ic.check(yg[off[i]:off[i] + n], *ic.reference(x64[src[off[i]:off[i] + n]], experts[i % E]), f"item {i}")


def test_decoders_refuse_unaligned_tokens(L):
    from routed_expert_layer_amd.runtime import DecodeLayer, DeviceDecodeLayer, ExpertStore
    cfg = int8_config(L=1)
    store = ExpertStore(1, cfg.E, cfg.H, cfg.I, "int8")
    try:
        W, b = gen.router_weight(cfg, 0, dev), torch.zeros(cfg.E, device=dev)
        x = torch.zeros(cfg.T * cfg.H + 1, dtype=torch.bfloat16, device=dev)[1:].view(cfg.T, cfg.H)
        with pytest.raises(L.MoEError, match="16-byte"):
            DecodeLayer(store, cfg.S, cfg.T, cfg.k, "bf16", dev).step(0, 0, x, W, b)
        with pytest.raises(L.MoEError, match="16-byte"):
            DeviceDecodeLayer(store, cfg.S, cfg.T, cfg.k, "bf16", dev).step(0, x, W, b)
    finally:
        store.close()


def test_experts_graph_of_a_short_step(L):
    """A step whose down projection forms the output, captured and replayed on changing tokens and routings, with eager
    calls on the same workspace between the replays; an expert without a slot, and steps of which none has one."""
    E, k, H, I, T = 16, 3, 512, 256, 2
    experts = [ic.expert(H, I, e, dev) for e in range(E)]
    slot_of = list(range(E))
    slots, stride = pack(L, H, I, experts, slot_of, E)
    s = torch.cuda.Stream()
    x, rt = tokens(T, H, 0), routing(T, E, k, 0)
    size = max(L.moe_experts_workspace_size(n, k, E, H, I, L.MOE_W_INT8) for n in (T, 40))
    ws = torch.full((size,), 255, dtype=torch.uint8, device=dev)
    out = torch.empty((T, H), device=dev)
    table = torch.tensor(slot_of, dtype=torch.int32, device=dev)
    d = rt["dev"]

    def step(stream):
        L.moe_experts(x, d["topk_idx"], d["topk_w"], d["perm_src"], d["perm_pos"], d["counts"], d["offsets"], table, E,
                      slots, stride, L.MOE_W_INT8, H, I, out, ws, stream)

    torch.cuda.synchronize()
    L.moe_graph_begin(s)
    step(s)
    graph = L.moe_graph_end(s)
    for i in range(6):
        nx, nrt = tokens(T, H, 10 + i), routing(T, E, k, 20 + i)
        x.copy_(nx)
        for n in d:
            d[n].copy_(nrt["dev"][n])
        now = [-1 if i == 5 or (i % 2 and e == nrt["idx"][0][0]) else e for e in range(E)]
        table.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        L.moe_graph_launch(graph, s)
        torch.cuda.synchronize()
        replay = out.clone()
        run(L, tokens(40, H, i), routing(40, E, k, i), slots, stride, now, E, H, I, ws=ws)
        out.fill_(float("nan"))
        step(None)
        torch.cuda.synchronize()
        assert torch.equal(out, replay), f"replay {i}"
        ic.check(np64(out), *expected(nx, experts, nrt, now, E), f"replay {i}")
