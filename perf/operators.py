"""What is timed of two operators of the routed expert layer, and their plain forms.

select: from router logits to the chosen experts, their weights and the grouping of the rows by expert
        (moe_select): softmax or sigmoid scores, a balance bias that moves the choice and not the weights, groups of
        experts of which a token keeps the best few, renormalised and scaled weights.
experts: the experts' products in 8-bit integers with a scale for each token and each output channel (moe_experts):
        the tokens are quantised, each expert's group of rows goes through its SwiGLU feed-forward, the SwiGLU products
        quantised row by row in between, and a token's rows are added with its routing weights.

`own` is False: `run` computes the plain form in elementary torch operations. True: the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# -------------------------------------------------------------------------------------------------------------------
# cases
# -------------------------------------------------------------------------------------------------------------------
def _select(name, T, E, k, score, groups=1, keep=1, top=1, balance=True, renorm=True, scale=1.0):
    return dict(name=name, op="select", T=T, E=E, k=k, score=score, groups=groups, keep=keep, top=top, balance=balance,
                renorm=renorm, scale=scale)


def _experts(name, T, E, k, H, I, skew=0.0):
    return dict(name=name, op="experts", T=T, E=E, k=k, H=H, I=I, skew=skew)


def listed():
    return [
        # one token of a decode step: latency
        _select("select_one", 1, 256, 6, "sigmoid", groups=8, keep=4, top=2, scale=2.5),
        # a decode batch, plain softmax scores renormalised over the chosen
        _select("select_batch", 48, 128, 8, "softmax", balance=False),
        # a ragged chunk with an odd number of experts a group; the group's best score ranks it, weights as they are
        _select("select_odd", 777, 100, 5, "softmax", groups=4, keep=2, top=1, balance=False, renorm=False, scale=16.0),
        # a prefill chunk, balance bias without groups
        _select("select_chunk", 4096, 256, 6, "sigmoid"),
        # the longest chunk, groups and balance bias
        _select("select_long", 16384, 256, 8, "sigmoid", groups=8, keep=4, top=2, scale=2.5),
        # one decoded token: six experts' weights stream through once
        _experts("experts_one", 1, 64, 6, 4096, 2048),
        # a decode batch over small experts
        _experts("experts_small", 4, 128, 8, 2048, 768, skew=1.2),
        # a decode batch that shares experts
        _experts("experts_batch", 8, 64, 6, 4096, 2048, skew=1.0),
        # many short groups, some past one tile of tokens
        _experts("experts_mid", 64, 128, 8, 2048, 768, skew=0.5),
        # ragged groups of odd sizes
        _experts("experts_odd", 333, 20, 5, 1280, 640, skew=0.5),
        # a prefill chunk over every expert of a layer: the weights' bytes bound it
        _experts("experts_chunk", 4096, 256, 6, 4096, 2048),
        # long groups: the products bound it
        _experts("experts_long", 16384, 64, 6, 4096, 2048, skew=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(max(2, 16 // groups), 256 // groups)
        E = groups * per
        keep = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(8, keep * per))
        return dict(op="select", T=_log(rng, 1, 16384), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    groups=groups, keep=keep, top=rng.choice([1, 2]), balance=rng.random() < 0.6,
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]))
    k = rng.choice([1, 2, 4, 6, 8])
    T = _log(rng, 1, 8192)
    if T <= 96:  # a decode step
        H, I = 128 * rng.randint(4, 32), 128 * rng.randint(3, 16)
    else:
        H, I = 256 * rng.randint(2, 16), 128 * rng.randint(3, 16)
    return dict(op="experts", T=T, E=rng.randint(max(8, k), 96), k=k, H=H, I=I, skew=rng.choice([0.0, 0.4, 0.8]))


def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "select":
        # the logits (and the balance bias) in; choice, weights, counts, offsets, sources and positions out
        return {"bytes": 4 * T * E + (4 * E if case["balance"] else 0) + 16 * T * k + 8 * E + 4, "flops": 8 * T * E}
    H, I = case["H"], case["I"]
    # the experts that any token chose, estimated from their number and the rows (each is chosen with the same chance)
    used = E * (1.0 - (1.0 - k / E) ** T)
    weights = used * (3 * H * I + 4 * (2 * I + H))
    return {"bytes": int(weights + 2 * T * H + 12 * T * k + 2 * T * H), "flops": 6 * T * k * H * I}


# -------------------------------------------------------------------------------------------------------------------
# inputs
# -------------------------------------------------------------------------------------------------------------------
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + salt) & ((1 << 62) - 1))
    return g


def _codes(shape, g):
    """int8 codes of normal weights quantised with a scale per channel (the largest near 4 deviations)."""
    out = torch.empty(shape, dtype=torch.int8, device=DEV)
    for e in range(shape[0]):
        out[e] = torch.randn(shape[1:], generator=g, device=DEV).mul_(31.0).round_().clamp_(-127, 127).to(torch.int8)
    return out


def _select_inputs(case, seed):
    g = _gen(seed, 1)
    T, E = case["T"], case["E"]
    logits = torch.randn((T, E), generator=g, device=DEV)
    logits += 0.5 * torch.randn(E, generator=g, device=DEV)  # experts differ in popularity
    balance = 0.1 * torch.randn(E, generator=g, device=DEV) if case["balance"] else None
    return dict(logits=logits, balance=balance)


def _experts_inputs(case, seed):
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    g = _gen(seed, 2)
    st = dict(q1=_codes((E, H, I), g), q3=_codes((E, H, I), g), q2=_codes((E, I, H), g))
    for name, n, fan in (("s1", I, H), ("s3", I, H), ("s2", H, I)):
        st[name] = (0.5 + torch.rand((E, n), generator=g, device=DEV)) / (31.0 * math.sqrt(fan))
    st["x"] = (torch.randn((T, H), generator=g, device=DEV)
               * (0.25 + torch.rand((T, 1), generator=g, device=DEV))).to(torch.bfloat16)
    # a routing: k different experts a token, some experts more popular than others
    score = torch.randn((T, E), generator=g, device=DEV) + case["skew"] * torch.randn(E, generator=g, device=DEV)
    val, idx = torch.topk(score, k, dim=1)
    w = torch.exp(val - val[:, :1])
    st["topk_w"] = (w / w.sum(1, keepdim=True)).contiguous()
    st["topk_idx"] = idx.to(torch.int32)
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(flat, minlength=E)
    st["counts"] = counts.to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    st["offsets"] = offsets.to(torch.int32)
    st["perm_src"] = (order // k).to(torch.int32)
    st["perm_pos"] = pos.reshape(T, k).to(torch.int32)
    # {expert, first row, rows} of the experts with rows, for the plain forms
    c, o = counts.tolist(), offsets.tolist()
    st["plan"] = np.array([[e, o[e], c[e]] for e in range(E) if c[e] > 0], dtype=np.int32)
    return st


def _gate(case, st):
    from routed_expert_layer_amd import _lib as L
    return L.Gate(score=case["score"], n_group=case["groups"], topk_group=case["keep"], group_top=case["top"],
                  renorm=case["renorm"], scale=case["scale"], balance=st["balance"])


def prepare(case, seed):
    """What a serving program holds before the call: logits, gate and buffers; or tokens, a routing, the experts'
    weights (for the framework as packed blobs in their slots) and the buffers it reuses from step to step."""
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "select":
        st = _select_inputs(case, seed)
        if own:
            from routed_expert_layer_amd import _lib as L
            st["gate"] = _gate(case, st)
            i32 = dict(dtype=torch.int32, device=DEV)
            st["out"] = dict(topk_idx=torch.empty((T, k), **i32), topk_w=torch.empty((T, k), device=DEV),
                             counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                             perm_src=torch.empty(T * k, **i32), perm_pos=torch.empty((T, k), **i32))
            st["ws"] = torch.empty(L.moe_select_workspace_size(T, E, k), dtype=torch.uint8, device=DEV)
    else:
        st = _experts_inputs(case, seed)
        st["order"] = torch.from_numpy(st["plan"][:, 0].astype(np.int64)).to(DEV)
        if own:
            from routed_expert_layer_amd import _lib as L
            H, I = case["H"], case["I"]
            stride = (L.moe_expert_bytes(L.MOE_W_INT8, H, I) + 4095) // 4096 * 4096
            slots = torch.empty(E * stride, dtype=torch.uint8, device=DEV)
            for e in range(E):  # expert e in slot E - 1 - e
                L.moe_pack_expert(L.MOE_W_INT8, H, I, st["q1"][e], st["q3"][e], st["q2"][e], st["s1"][e], st["s3"][e],
                                  st["s2"][e], slots[(E - 1 - e) * stride:])
            st.update(stride=stride, slots=slots, out=torch.empty((T, H), dtype=torch.bfloat16, device=DEV),
                      slot_of=torch.arange(E - 1, -1, -1, dtype=torch.int32, device=DEV),
                      ws=torch.empty(L.moe_experts_workspace_size(T, k, E, H, I, L.MOE_W_INT8), dtype=torch.uint8,
                                     device=DEV))
    st["case"] = case
    return st


# -------------------------------------------------------------------------------------------------------------------
# one pass
# -------------------------------------------------------------------------------------------------------------------
def run(st):
    return _run_select(st) if st["case"]["op"] == "select" else _run_experts(st)


def _run_select(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    if own:
        from routed_expert_layer_amd import _lib as L
        o = st["out"]
        L.moe_select(st["logits"], st["gate"], k, o["topk_idx"], o["topk_w"], o["counts"], o["offsets"], o["perm_src"],
                     o["perm_pos"], st["ws"])
        return o
    # Scores in 64 bits: two experts' biased scores can be closer than 32 bits tell apart, and the choice is whole.
    l = st["logits"].double()
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        z = torch.exp(l - l.amax(1, keepdim=True))
        s = z / z.sum(1, keepdim=True)
    c = s if st["balance"] is None else s + st["balance"].double()
    if case["groups"] > 1:
        g = c.view(T, case["groups"], -1)
        rank = torch.sort(g, dim=2, descending=True).values[:, :, :case["top"]].sum(2)
        keep = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        kept = torch.zeros((T, case["groups"]), dtype=torch.bool, device=DEV).scatter_(1, keep, True)
        c = torch.where(kept[:, :, None], g, -math.inf).view(T, E)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(s, 1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * case["scale"]).float()
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=DEV))
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(counts, 0)])
    return dict(topk_idx=idx.int(), topk_w=w, counts=counts.int(), offsets=offsets.int(), perm_src=(order // k).int(),
                perm_pos=pos.view(T, k).int())


def _quantised(a):
    """Codes (as 32-bit floats) and scale of the rows of a (last axis), the largest magnitude at 127. The quotient is
    taken in 64 bits: halves of the largest value fall exactly between two codes."""
    amax = a.abs().amax(-1, keepdim=True)
    q = torch.round(a.double() * 127.0 / torch.where(amax > 0, amax, 1.0).double()).float()
    return q, amax / 127.0


def _run_experts(st):
    case = st["case"]
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    if own:
        from routed_expert_layer_amd import _lib as L
        L.moe_experts(st["x"], st["topk_idx"], st["topk_w"], st["perm_src"], st["perm_pos"], st["counts"],
                      st["offsets"], st["slot_of"], E, st["slots"], st["stride"], L.MOE_W_INT8, H, I, st["out"],
                      st["ws"])
        return st["out"]
    plan, ex = st["plan"], st["order"]
    n, cap = len(plan), int(plan[:, 2].max())
    # every group padded to the longest one's rows; rows past a group's end are its last row again and are not used
    first = st["offsets"][ex].long()[:, None]
    last = first + st["counts"][ex].long()[:, None] - 1
    rows = torch.minimum(first + torch.arange(cap, device=DEV)[None, :], last)
    q, s = _quantised(st["x"].float())
    src = st["perm_src"].long()[rows]
    qx, sx = q[src], s[src]
    some = n < E  # a decode step uses a few of the resident experts
    pick = (lambda t: t[ex]) if some else (lambda t: t)
    g = torch.bmm(qx, pick(st["q1"]).float()) * sx * pick(st["s1"])[:, None, :]
    u = torch.bmm(qx, pick(st["q3"]).float()) * sx * pick(st["s3"])[:, None, :]
    qh, sh = _quantised(g / (1.0 + torch.exp(-g)) * u)
    del g, u, qx
    y = torch.bmm(qh, pick(st["q2"]).float()) * sh * pick(st["s2"])[:, None, :]
    place = torch.zeros(T * k, dtype=torch.int64, device=DEV)
    place.scatter_(0, rows.reshape(-1), torch.arange(n * cap, device=DEV))  # a repeated last row: any of its copies
    yr = y.reshape(n * cap, H)[place[st["perm_pos"].long()].reshape(-1)].view(T, k, H)
    return (yr * st["topk_w"][:, :, None]).sum(1).to(torch.bfloat16)


# -------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# -------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    return _exact_select(case, seed) if case["op"] == "select" else _exact_experts(case, seed)


def _exact_select(case, seed):
    st = _select_inputs(case, seed)
    T, E, k = case["T"], case["E"], case["k"]
    l = st["logits"].cpu().numpy().astype(np.float64)
    if case["score"] == "sigmoid":
        s = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    else:
        m = np.max(l, 1, keepdims=True)
        s = np.exp(l - (m + np.log(np.exp(l - m).sum(1, keepdims=True))))
    c = s + (0.0 if st["balance"] is None else st["balance"].cpu().numpy().astype(np.float64)[None, :])
    per = E // case["groups"]
    idx = np.empty((T, k), np.int64)
    if case["groups"] > 1:
        rank = -np.sort(-c.reshape(T, case["groups"], per), axis=2)[:, :, :case["top"]].sum(2)
        best = np.argsort(-rank, axis=1, kind="stable")[:, :case["keep"]]
        dropped = np.ones((T, case["groups"]), bool)
        np.put_along_axis(dropped, best, False, 1)
        c = np.where(np.repeat(dropped, per, 1), -np.inf, c)
    for j in range(k):  # the largest left, the lowest index first
        idx[:, j] = np.argmax(c, 1)
        c[np.arange(T), idx[:, j]] = -np.inf
    w = np.take_along_axis(s, idx, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdims=True)
    w = w * case["scale"]
    counts = np.bincount(idx.reshape(-1), minlength=E)
    order = np.lexsort((np.repeat(np.arange(T), k), idx.reshape(-1)))
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    i = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32))  # noqa: E731
    return dict(topk_idx=i(idx), topk_w=torch.from_numpy(w), counts=i(counts),
                offsets=i(np.concatenate([[0], np.cumsum(counts)])), perm_src=i(order // k),
                perm_pos=i(pos.reshape(T, k)))


def _exact_experts(case, seed):
    st = _experts_inputs(case, seed)
    H = case["H"]

    def codes(a):
        m = a.abs().max(1, keepdim=True)[0]
        return torch.where(m > 0, torch.round(127 * a / m), torch.zeros_like(a)), m / 127

    out = torch.zeros((case["T"], H), dtype=torch.float64, device=DEV)
    weight = torch.zeros(case["T"] * case["k"], dtype=torch.float64, device=DEV)
    weight[st["perm_pos"].long().reshape(-1)] = st["topk_w"].double().reshape(-1)
    for e, first, rows in st["plan"].tolist():
        t = st["perm_src"][first:first + rows].long()
        qx, sx = codes(st["x"][t].double())
        g = (qx @ st["q1"][e].double()) * (sx * st["s1"][e].double())
        u = (qx @ st["q3"][e].double()) * (sx * st["s3"][e].double())
        qh, sh = codes(g * torch.sigmoid(g) * u)
        y = (qh @ st["q2"][e].double()) * (sh * st["s2"][e].double())
        out.index_add_(0, t, y * weight[first:first + rows, None])
    return out
