"""What is timed of the operators that train through the routed expert layer, and their plain forms.

sort, back, grad: tokens sorted by expert and back (moe_group and moe_dispatch; moe_collect; moe_collect_backward):
        the grouping of given choices, of which some may be dropped, the copies of the token rows, the weighted sum of
        a token's rows and that sum's gradient to the rows and the weights.
save:   SwiGLU whose inputs are kept in 8 bits with a scale for 128 columns, and its backward pass from what was kept
        (moe_swiglu_save, moe_swiglu_backward).
mm, mm_t, dw: the experts' products over their groups of rows (moe_matmul_grouped; with the weights transposed, the
        gradient of the rows; moe_matmul_grouped_dw, the gradient of the weights).

`own` is False: `run` computes the plain form in elementary torch operations. True: the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GROUP = 128  # columns that share a scale


# -------------------------------------------------------------------------------------------------------------------
# cases
# -------------------------------------------------------------------------------------------------------------------
def _rows(name, op, T, E, k, H, dtype="bfloat16", drop=0.0, weights=True):
    return dict(name=name, op=op, T=T, E=E, k=k, H=H, dtype=dtype, drop=drop, weights=weights)


def _save(name, R, I, dtype="bfloat16"):
    return dict(name=name, op="save", R=R, I=I, dtype=dtype)


def _mm(name, op, T, E, k, K, N, skew=0.0, out="bfloat16"):
    return dict(name=name, op=op, T=T, E=E, k=k, K=K, N=N, skew=skew, out=out)


def listed():
    return [
        # one token to its experts' rows: latency
        _rows("sort_one", "sort", 1, 256, 6, 4096),
        # a training chunk to rows sorted by expert
        _rows("sort_chunk", "sort", 4096, 256, 6, 4096),
        # back to tokens on a GPU that holds a part of the experts: ragged, fp32 rows
        _rows("back_odd", "back", 777, 100, 5, 1000, dtype="float32", drop=0.3),
        # the gradient of the weighted sum over a long batch
        _rows("grad_long", "grad", 16384, 64, 6, 4096),
        # a small batch of small experts: SwiGLU rows kept in 8 bits and used
        _save("save_small", 384, 768),
        # ragged rows whose length is no multiple of a scale's columns
        _save("save_odd", 1665, 645, dtype="float32"),
        # the rows of a long batch
        _save("save_long", 98304, 2048),
        # a small batch over many small experts: the weights' bytes bound it
        _mm("mm_small", "mm", 48, 128, 8, 2048, 1536, skew=0.5),
        # gate and up of a chunk
        _mm("mm_chunk", "mm", 4096, 64, 6, 4096, 4096, skew=0.3),
        # the rows' gradient through the down projection
        _mm("mm_back", "mm_t", 4096, 64, 6, 2048, 4096, skew=0.3),
        # weight gradients of a short ragged batch, some experts with few rows, kept in fp32
        _mm("dw_odd", "dw", 333, 20, 5, 1280, 648, skew=0.5, out="float32"),
        # weight gradients of a long batch: the products bound it
        _mm("dw_long", "dw", 16384, 64, 6, 4096, 4096, skew=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "back", "grad", "save", "mm", "mm_t", "dw"])
    k = rng.choice([1, 2, 4, 5, 6, 8])
    E = rng.randint(max(8, k), 256)
    if op in ("sort", "back", "grad"):
        H = rng.choice([8 * _log(rng, 8, 512), _log(rng, 64, 4096)])  # whole vectors, or any length
        return dict(op=op, T=_log(rng, 1, 12288), E=E, k=k, H=H, dtype=rng.choice(["bfloat16", "bfloat16", "float32"]),
                    drop=rng.choice([0.0, 0.0, 0.25, 0.75]), weights=op == "grad" or rng.random() < 0.7)
    if op == "save":
        I = rng.choice([64 * _log(rng, 2, 32), _log(rng, 100, 2048)])
        return dict(op=op, R=_log(rng, 1, 65536), I=I, dtype=rng.choice(["bfloat16", "bfloat16", "float32"]))
    return dict(op=op, T=_log(rng, 1, 8192), E=rng.randint(max(4, k), 64), k=k, K=8 * _log(rng, 32, 512),
                N=8 * _log(rng, 32, 512), skew=rng.choice([0.0, 0.4, 0.8]),
                out=rng.choice(["bfloat16", "bfloat16", "float32"]))


def work(case):
    op = case["op"]
    if op == "save":
        R, I, s = case["R"], case["I"], _size(case["dtype"])
        kept = 2 * I + 8 * ((I + GROUP - 1) // GROUP)
        # gate and up in, h and what is kept out; what is kept and the gradient of h in, gradients and h again out
        return {"bytes": R * (3 * I * s + kept + kept + 4 * I * s), "flops": 40 * R * I}
    T, E, k = case["T"], case["E"], case["k"]
    if op in ("sort", "back", "grad"):
        H, s = case["H"], _size(case["dtype"])
        R = T * k * (1.0 - case["drop"])
        if op == "sort":  # choices and tokens in, tables and rows out
            return {"bytes": int(4 * T * k + T * H * s + 8 * E + 4 + 4 * T * k + 4 * R + R * H * s), "flops": 0}
        tables = 4 * T * k * (2 if case["weights"] else 1)
        if op == "back":
            return {"bytes": int(tables + R * H * s + T * H * s), "flops": int(2 * R * H)}
        return {"bytes": int(tables + T * H * s + 2 * R * H * s + 4 * T * k), "flops": int(3 * R * H)}
    K, N, R = case["K"], case["N"], T * k
    # the experts that any token chose, estimated from their number and the rows (each is chosen with the same chance)
    used = E if op == "dw" else E * (1.0 - (1.0 - k / E) ** T)
    o = _size(case["out"])
    size = {"mm": R * (2 * K + o * N) + 2 * used * K * N, "mm_t": R * (o * K + 2 * N) + 2 * used * K * N,
            "dw": 2 * R * (K + N) + o * used * K * N}[op]
    return {"bytes": int(size + 8 * E), "flops": 2 * R * K * N}


def _size(dtype):
    return 2 if dtype == "bfloat16" else 4


# -------------------------------------------------------------------------------------------------------------------
# inputs
# -------------------------------------------------------------------------------------------------------------------
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + salt) & ((1 << 62) - 1))
    return g


def _choices(T, E, k, skew, drop, g):
    """k different experts a token, some more popular than others; with `drop`, the entries of experts that are held
    elsewhere are -1."""
    score = torch.randn((T, E), generator=g, device=DEV) + skew * torch.randn(E, generator=g, device=DEV)
    idx = torch.topk(score, k, dim=1).indices.to(torch.int32)
    if drop:
        idx[torch.rand((T, k), generator=g, device=DEV) < drop] = -1
    return idx


def _grouping(idx, E):
    """counts, offsets and places of given choices, for the cases that start behind the grouping."""
    T, k = idx.shape
    flat = idx.reshape(-1).long()
    kept = flat >= 0
    order = torch.argsort(torch.where(kept, flat, E), stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(flat[kept], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    return counts, offsets, torch.where(kept, pos, -1).view(T, k).int()


def _rows_inputs(case, seed):
    T, E, k, H = (case[n] for n in ("T", "E", "k", "H"))
    g = _gen(seed, 1)
    dt = getattr(torch, case["dtype"])
    st = dict(topk_idx=_choices(T, E, k, 0.4, case["drop"], g))
    spread = 0.25 + torch.rand((T, 1), generator=g, device=DEV)
    st["x"] = (torch.randn((T, H), generator=g, device=DEV) * spread).to(dt)  # the tokens, or the output's gradient
    if case["op"] != "sort":
        counts, offsets, st["perm_pos"] = _grouping(st["topk_idx"], E)
        st["R"] = int(offsets[E])
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        st["topk_w"] = (w / w.sum(1, keepdim=True)).contiguous() if case["weights"] else None
        st["rows"] = torch.randn((max(st["R"], 1), H), generator=g, device=DEV).to(dt)
    return st


def _save_inputs(case, seed):
    R, I = case["R"], case["I"]
    g = _gen(seed, 2)
    dt = getattr(torch, case["dtype"])
    gu = torch.randn((R, 2 * I), generator=g, device=DEV)
    gu *= 0.5 + torch.rand(2 * I, generator=g, device=DEV)  # columns differ in size, a few by much
    gu *= torch.where(torch.rand(2 * I, generator=g, device=DEV) < 0.01, 8.0, 1.0)
    dh = torch.randn((R, I), generator=g, device=DEV) * (0.01 + torch.rand((R, 1), generator=g, device=DEV))
    return dict(gu=gu.to(dt), dh=dh.to(dt))


def _mm_inputs(case, seed):
    T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
    g = _gen(seed, 3)
    counts, offsets, _ = _grouping(_choices(T, E, k, case["skew"], 0.0, g), E)
    st = dict(counts=counts.int(), offsets=offsets.int())
    # {expert, first row, rows} of the experts with rows, for the plain forms
    c, o = counts.tolist(), offsets.tolist()
    st["plan"] = np.array([[e, o[e], c[e]] for e in range(E) if c[e] > 0], dtype=np.int64)
    bf = torch.bfloat16
    if case["op"] != "mm_t":
        st["a"] = torch.randn((T * k, K), generator=g, device=DEV).to(bf)
    if case["op"] != "mm":
        st["dc"] = torch.randn((T * k, N), generator=g, device=DEV).to(bf)
    if case["op"] != "dw":
        st["w"] = torch.empty((E, K, N), dtype=bf, device=DEV)
        for e in range(E):
            st["w"][e] = torch.randn((K, N), generator=g, device=DEV) / math.sqrt(K if case["op"] == "mm" else N)
    return st


def _inputs(case, seed):
    return {"save": _save_inputs, "mm": _mm_inputs, "mm_t": _mm_inputs, "dw": _mm_inputs}.get(
        case["op"], _rows_inputs)(case, seed)


def prepare(case, seed):
    """What a training program holds before the call: the inputs, and the buffers that it reuses from step to step
    (rows that no choice takes stay as they are: zeros here)."""
    st = _inputs(case, seed)
    op = case["op"]
    if own and op in ("sort", "back", "grad"):
        from routed_expert_layer_amd import _lib as L
        T, E, k, H = (case[n] for n in ("T", "E", "k", "H"))
        dt = getattr(torch, case["dtype"])
        i32 = dict(dtype=torch.int32, device=DEV)
        if op == "sort":
            st["out"] = dict(counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                             perm_src=torch.zeros(T * k, **i32), perm_pos=torch.empty((T, k), **i32),
                             x_perm=torch.zeros((T * k, H), dtype=dt, device=DEV))
            st["ws"] = torch.empty(L.moe_group_workspace_size(T, k, E), dtype=torch.uint8, device=DEV)
        elif op == "back":
            st["out"] = torch.empty((T, H), dtype=dt, device=DEV)
        else:
            st["out"] = dict(drows=torch.zeros_like(st["rows"]), dw=torch.empty((T, k), device=DEV))
    elif own and op == "save":
        R, I = case["R"], case["I"]
        st["codes"] = torch.empty((R, 2 * I), dtype=torch.int8, device=DEV)
        st["scales"] = torch.empty((R, 2 * ((I + GROUP - 1) // GROUP)), device=DEV)
        st["out"] = dict(h=torch.empty_like(st["dh"]), dgu=torch.empty_like(st["gu"]), h_again=torch.empty_like(st["dh"]))
    elif own:
        shape = {"mm": (case["T"] * case["k"], case["N"]), "mm_t": (case["T"] * case["k"], case["K"]),
                 "dw": (case["E"], case["K"], case["N"])}[op]
        st["out"] = torch.empty(shape, dtype=getattr(torch, case["out"]), device=DEV)
    st["case"] = case
    return st


# -------------------------------------------------------------------------------------------------------------------
# one pass
# -------------------------------------------------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    return {"sort": _run_sort, "back": _run_back, "grad": _run_grad, "save": _run_save}.get(op, _run_mm)(st)


def _run_sort(st):
    case, x, idx = st["case"], st["x"], st["topk_idx"]
    T, E, k = case["T"], case["E"], case["k"]
    if own:
        from routed_expert_layer_amd import _lib as L
        o = st["out"]
        L.moe_group(idx, E, o["counts"], o["offsets"], o["perm_src"], o["perm_pos"], st["ws"])
        L.moe_dispatch(x, o["perm_pos"], o["x_perm"])
        return o
    flat = idx.reshape(-1).long()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, E)
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=DEV))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(counts, 0)])
    used = torch.arange(T * k, device=DEV) < offsets[E]
    src = torch.where(used, order // k, 0)
    x_perm = torch.where(used[:, None], x[src], torch.zeros((), dtype=x.dtype, device=DEV))
    return dict(counts=counts.int(), offsets=offsets.int(), perm_src=src.int(),
                perm_pos=torch.where(kept, pos, -1).view(T, k).int(), x_perm=x_perm)


def _run_back(st):
    if own:
        from routed_expert_layer_amd import _lib as L
        L.moe_collect(st["rows"], st["perm_pos"], st["topk_w"], st["out"])
        return st["out"]
    pos, rows, w = st["perm_pos"].long(), st["rows"], st["topk_w"]
    out = torch.zeros(st["x"].shape, dtype=torch.float32, device=DEV)
    for j in range(st["case"]["k"]):
        p = pos[:, j]
        v = rows[p.clamp(min=0)].float()
        if w is not None:
            v = v * w[:, j, None]
        out = out + torch.where(p[:, None] >= 0, v, 0.0)
    return out.to(rows.dtype)


def _run_grad(st):
    if own:
        from routed_expert_layer_amd import _lib as L
        o = st["out"]
        L.moe_collect_backward(st["x"], st["rows"], st["perm_pos"], st["topk_w"], o["drows"], o["dw"])
        return o
    pos, rows, w, dout = st["perm_pos"].long(), st["rows"], st["topk_w"], st["x"].float()
    drows, dw = torch.zeros_like(rows), torch.zeros_like(w)
    for j in range(st["case"]["k"]):
        p = pos[:, j]
        t = torch.nonzero(p >= 0)[:, 0] if st["case"]["drop"] else slice(None)
        p = p[t]
        d = dout[t]
        drows[p] = (d * w[t, j, None]).to(rows.dtype)
        dw[t, j] = (d * rows[p].float()).sum(1)
    return dict(drows=drows, dw=dw)


def _kept(v):
    """What 8 bits keep of v [R, I]: codes (as 32-bit floats) times the scale of their 128 columns. The quotient is
    taken in 64 bits: halves of the largest value fall exactly between two codes."""
    R, I = v.shape
    n = (I + GROUP - 1) // GROUP
    p = torch.zeros((R, n * GROUP), dtype=torch.float32, device=DEV)
    p[:, :I] = v
    p = p.view(R, n, GROUP)
    amax = p.abs().amax(2, keepdim=True)
    q = torch.round(p.double() * 127.0 / torch.where(amax > 0, amax, 1.0).double()).float()
    return (q * (amax / 127.0)).view(R, n * GROUP)[:, :I]


def _run_save(st):
    gu, dh = st["gu"], st["dh"]
    if own:
        from routed_expert_layer_amd import _lib as L
        o = st["out"]
        L.moe_swiglu_save(gu, o["h"], st["codes"], st["scales"])
        L.moe_swiglu_backward(st["codes"], st["scales"], dh, o["dgu"], o["h_again"])
        return o
    I = st["case"]["I"]
    g, u = gu[:, :I].float(), gu[:, I:].float()
    h = (g / (1.0 + torch.exp(-g)) * u).to(gu.dtype)
    g, u = _kept(g), _kept(u)
    s = 1.0 / (1.0 + torch.exp(-g))
    d = dh.float()
    dgu = torch.cat([d * u * (s * (1.0 + g * (1.0 - s))), d * (g * s)], 1).to(gu.dtype)
    return dict(h=h, dgu=dgu, h_again=(g * s * u).to(gu.dtype))


def _run_mm(st):
    case = st["case"]
    op = case["op"]
    if own:
        from routed_expert_layer_amd import _lib as L
        if op == "dw":
            L.moe_matmul_grouped_dw(st["a"], st["dc"], st["counts"], st["offsets"], st["out"])
        else:
            L.moe_matmul_grouped(st["a" if op == "mm" else "dc"], st["w"], st["counts"], st["offsets"], st["out"],
                                 transposed=op == "mm_t")
        return st["out"]
    dt = getattr(torch, case["out"])
    if op == "dw":
        out = torch.zeros((case["E"], case["K"], case["N"]), dtype=dt, device=DEV)
        for e, first, n in st["plan"].tolist():
            out[e] = (st["a"][first:first + n].float().t() @ st["dc"][first:first + n].float()).to(dt)
        return out
    rows = st["a" if op == "mm" else "dc"]
    out = torch.empty((rows.shape[0], case["N"] if op == "mm" else case["K"]), dtype=dt, device=DEV)
    for e, first, n in st["plan"].tolist():
        w = st["w"][e].float()
        out[first:first + n] = (rows[first:first + n].float() @ (w if op == "mm" else w.t())).to(dt)
    return out


# -------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# -------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "sort":
        return _exact_sort(case, st)
    if op in ("back", "grad"):
        return _exact_rows(case, st)
    return _exact_save(case, st) if op == "save" else _exact_mm(case, st)


def _exact_sort(case, st):
    T, E, k = case["T"], case["E"], case["k"]
    idx = st["topk_idx"].cpu().numpy()
    t, j = np.nonzero(idx >= 0)
    by = np.lexsort((j, t, idx[t, j]))
    pos = np.full((T, k), -1, np.int32)
    pos[t[by], j[by]] = np.arange(len(by))
    src = np.zeros(T * k, np.int32)
    src[:len(by)] = t[by]
    counts = np.array([(idx == e).sum() for e in range(E)], np.int32)
    x_perm = torch.zeros((T * k, case["H"]), dtype=st["x"].dtype, device=DEV)
    x_perm[:len(by)] = st["x"][torch.from_numpy(t[by]).to(DEV)]
    i = torch.from_numpy
    return dict(counts=i(counts), offsets=i(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)),
                perm_src=i(src), perm_pos=i(pos), x_perm=x_perm)


def _exact_rows(case, st):
    """Row by row: the token and the weight of each, then the sums over the tokens' rows."""
    T, k, H, R = case["T"], case["k"], case["H"], st["R"]
    pos = st["perm_pos"].long().reshape(-1)
    entry = torch.nonzero(pos >= 0).reshape(-1)  # entries of the choices that are kept, and their rows
    row, token = pos[entry], entry // k
    w = torch.ones(T * k, dtype=torch.float64, device=DEV) if st["topk_w"] is None else st["topk_w"].double().reshape(-1)
    step = max(1, (1 << 27) // H)
    if case["op"] == "back":
        out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        for a in range(0, len(entry), step):
            c = slice(a, a + step)
            out.index_add_(0, token[c], st["rows"][row[c]].double() * w[entry[c], None])
        return out
    drows = torch.zeros((max(R, 1), H), dtype=torch.float64, device=DEV)
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    for a in range(0, len(entry), step):
        c = slice(a, a + step)
        d = st["x"][token[c]].double()
        drows[row[c]] = d * w[entry[c], None]
        dw[entry[c]] = torch.linalg.vecdot(d, st["rows"][row[c]].double())
    return dict(drows=drows, dw=dw.view(T, k))


def _exact_save(case, st):
    R, I = case["R"], case["I"]
    out = {n: torch.empty((R, m), dtype=torch.float64, device=DEV) for n, m in (("h", I), ("dgu", 2 * I), ("h_again", I))}
    step = max(1, (1 << 25) // I)
    for a in range(0, R, step):
        c = slice(a, min(a + step, R))
        v = st["gu"][c].double()
        g, u, d = v[:, :I], v[:, I:], st["dh"][c].double()
        out["h"][c] = g * torch.sigmoid(g) * u
        k = torch.empty_like(v)
        for first in range(0, 2 * I, I):
            for b in range(first, first + I, GROUP):
                part = v[:, b:min(b + GROUP, first + I)]
                top = part.abs().max(1, keepdim=True)[0]
                k[:, b:b + part.shape[1]] = torch.where(top > 0, torch.round(127 * part / top) * top / 127, 0.0)
        g, u = k[:, :I], k[:, I:]
        s = torch.sigmoid(g)
        out["dgu"][c, :I] = d * u * (s + g * s * torch.sigmoid(-g))
        out["dgu"][c, I:] = d * g * s
        out["h_again"][c] = g * s * u
    return out


def _exact_mm(case, st):
    op = case["op"]
    shape = {"mm": (case["T"] * case["k"], case["N"]), "mm_t": (case["T"] * case["k"], case["K"]),
             "dw": (case["E"], case["K"], case["N"])}[op]
    out = torch.zeros(shape, dtype=torch.float64, device=DEV)
    for e, first, n in st["plan"].tolist():
        c = slice(first, first + n)
        if op == "dw":
            out[e] = torch.mm(st["a"][c].double().t(), st["dc"][c].double())
        elif op == "mm":
            out[c] = torch.mm(st["a"][c].double(), st["w"][e].double())
        else:
            out[c] = torch.mm(st["w"][e].double(), st["dc"][c].double().t()).t()
    return out
