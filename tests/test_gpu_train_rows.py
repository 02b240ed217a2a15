"""Tokens sorted by expert and back (moe_group, moe_dispatch, moe_collect, moe_collect_backward) against their
statement in 64 bits. Whole numbers and copies are equal; a sum of n terms in fp32 is off by at most n 2^-24 of the
terms' magnitudes, and its rounding by half a step of the type (2^-24 or 2^-8 of the value)."""
import numpy as np
import pytest
import torch

from oracle import train as tr
from tests.parity import np64, npi

pytestmark = pytest.mark.gpu
dev = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
FILL = -7


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def choices(T, E, k, seed, drop=0.0, skew=0.0, repeat=False):
    r = np.random.default_rng(seed)
    if repeat:
        idx = r.integers(0, E, (T, k))
    else:
        idx = np.argsort(-(r.standard_normal((T, E)) + skew * r.standard_normal(E)), axis=1)[:, :k].reshape(T, k)
    out = r.random((T, k)) < drop
    return np.where(out, r.choice([-1, -5, E, 2 ** 31 - 1, -2 ** 31], (T, k)), idx).astype(np.int32)


def grouped(L, idx, E):
    """moe_group on the GPU; every output filled with a mark before."""
    T, k = idx.shape
    i32 = dict(dtype=torch.int32, device=dev)
    o = dict(counts=torch.full((E,), FILL, **i32), offsets=torch.full((E + 1,), FILL, **i32),
             perm_src=torch.full((max(T * k, 1),), FILL, **i32), perm_pos=torch.full((T, k), FILL, **i32))
    ws = torch.full((L.moe_group_workspace_size(T, k, E),), 255, dtype=torch.uint8, device=dev)
    L.moe_group(torch.from_numpy(idx).to(dev), E, o["counts"], o["offsets"], o["perm_src"], o["perm_pos"],
                ws if ws.numel() else None)
    return o


def fast_group(idx, E):
    """tr.group for long batches."""
    flat = idx.reshape(-1).astype(np.int64)
    kept = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(kept, flat, E), kind="stable")
    pos = np.empty(len(flat), np.int64)
    pos[order] = np.arange(len(flat))
    counts = np.bincount(flat[kept], minlength=E)
    return (counts, np.concatenate([[0], np.cumsum(counts)]), np.where(kept, pos, -1).reshape(idx.shape),
            order[:counts.sum()] // idx.shape[1])


GROUPS = [(0, 4, 2, 0, 0), (1, 1, 1, 0, 0), (1, 256, 6, 0, 0), (1, 1024, 16, 0, 0), (3, 5, 2, 1.0, 0), (63, 7, 1, .3, 0),
          (64, 64, 8, 0, 0), (65, 1023, 3, .5, 0), (333, 20, 5, .2, 1.), (512, 1024, 8, 0, 0), (513, 255, 8, 0, 0),
          (682, 33, 6, .1, 2.), (683, 33, 6, .1, 2.), (4097, 256, 1, 0, 0), (8192, 1, 1, .5, 0), (20000, 100, 16, .25, 1.),
          (70001, 1024, 5, 0, .5)]


@pytest.mark.parametrize("T,E,k,drop,skew", GROUPS)
@pytest.mark.parametrize("repeat", [False, True])
def test_group(L, T, E, k, drop, skew, repeat):
    idx = choices(T, E, k, T + E, drop, skew, repeat)
    counts, offsets, pos, src = (tr.group if T < 700 else fast_group)(idx, E)
    o = grouped(L, idx, E)
    assert np.array_equal(npi(o["counts"]), counts) and np.array_equal(npi(o["offsets"]), offsets)
    assert np.array_equal(npi(o["perm_pos"]), pos)
    got = npi(o["perm_src"])
    assert np.array_equal(got[:len(src)], src) and np.all(got[len(src):] == FILL)


def test_group_is_the_routings(L):
    """The grouping of a routing's choices is the routing's own."""
    from routed_expert_layer_amd.runtime import RouteBuffers
    T, H, E, k = 777, 256, 96, 6
    g = torch.Generator().manual_seed(1)
    x, Wr = (torch.randn(s, generator=g).to(torch.bfloat16).to(dev) for s in ((T, H), (H, E)))
    rb = RouteBuffers(T, H, E, k, dev)
    rb.route(x, Wr, None)
    o = grouped(L, npi(rb.topk_idx).astype(np.int32), E)
    for n in o:
        assert np.array_equal(npi(o[n]), npi(getattr(rb, n))), n


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (512, 64, 8), (6000, 40, 6)])
def test_group_in_a_graph(L, T, E, k):
    """Every form of the grouping captured, and replayed with other choices in the same buffer."""
    from routed_expert_layer_amd.runtime import DeviceDecodeLayer
    cases = [choices(T, E, k, 50 + i, 0.1 * i, float(i)) for i in range(3)]
    want = [{n: t.clone() for n, t in grouped(L, c, E).items()} for c in cases]
    idx = torch.from_numpy(cases[0]).to(dev)
    o = {n: torch.empty_like(t) for n, t in want[0].items()}
    ws = torch.empty(max(L.moe_group_workspace_size(T, k, E), 4), dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = DeviceDecodeLayer.capture(
        lambda: L.moe_group(idx, E, o["counts"], o["offsets"], o["perm_src"], o["perm_pos"], ws, s), s)
    for i in (1, 0, 2, 2, 1):
        idx.copy_(torch.from_numpy(cases[i]).to(dev))
        for t in (*o.values(), ws):
            t.fill_(FILL if t.dtype == torch.int32 else 255)
        torch.cuda.synchronize()
        L.moe_graph_launch(graph, s)
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(o[n], want[i][n]), n


def test_binding_refuses(L):
    """Types, shapes, layouts and host tensors that the kernels do not take are turned away by name."""
    f = lambda *s: torch.zeros(s, device=dev)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    c8 = torch.zeros((4, 16), dtype=torch.int8, device=dev)
    calls = [lambda: L.moe_group(i(4, 2), 4, i(4), i(4), i(8), i(4, 2)), lambda: L.moe_group(f(4, 2), 4, i(4), i(5), i(8), i(4, 2)),
             lambda: L.moe_group(i(4, 2), 4, i(4), i(5), i(7), i(4, 2)), lambda: L.moe_group(i(2, 4).t(), 4, i(4), i(5), i(8), i(4, 2)),
             lambda: L.moe_group(i(4, 2), 4, i(4), i(5), i(8), i(4, 2).cpu()),
             lambda: L.moe_dispatch(f(4, 8), i(4, 2), b(8, 8)), lambda: L.moe_dispatch(f(4, 8), i(5, 2), f(8, 8)),
             lambda: L.moe_dispatch(f(8, 4).t(), i(4, 2), f(8, 8)), lambda: L.moe_dispatch(f(4, 8).half(), i(4, 2), f(8, 8).half()),
             lambda: L.moe_dispatch(f(4, 8), i(4, 2).long(), f(8, 8)), lambda: L.moe_dispatch(f(4, 8), i(4, 2), f(8, 7)),
             lambda: L.moe_collect(f(8, 8), i(4, 2), f(4, 3), f(4, 8)), lambda: L.moe_collect(f(8, 8), i(4, 2), b(4, 2), f(4, 8)),
             lambda: L.moe_collect(f(8, 8), i(4, 2), None, f(4, 9)), lambda: L.moe_collect(f(8, 16)[:, ::2], i(4, 2), None, f(4, 8)),
             lambda: L.moe_collect_backward(f(4, 8), f(8, 9), i(4, 2), None, None, f(4, 2)),
             lambda: L.moe_collect_backward(f(4, 8), f(8, 8), i(4, 2), None, b(8, 8), f(4, 2)),
             lambda: L.moe_collect_backward(f(4, 8), f(8, 8), i(4, 2), None, None, b(4, 2)),
             lambda: L.moe_swiglu_save(f(4, 16), b(4, 8), c8, f(4, 2)), lambda: L.moe_swiglu_save(f(4, 16), f(4, 8), c8, f(4, 3)),
             lambda: L.moe_swiglu_save(f(4, 16), f(4, 8), c8, f(4, 2), i(2)), lambda: L.moe_swiglu_save(f(4, 16), f(4, 8), c8.float(), f(4, 2)),
             lambda: L.moe_swiglu_backward(c8, f(4, 2), f(4, 8), f(4, 8)),
             lambda: L.moe_swiglu_backward(c8, f(4, 2), b(4, 8), b(4, 16), f(4, 8)),
             lambda: L.moe_matmul_grouped(b(4, 8), b(2, 8, 16), i(2), i(3), b(4, 8)),
             lambda: L.moe_matmul_grouped(b(4, 8), b(2, 8, 16), i(2), i(3), b(4, 16), transposed=True),
             lambda: L.moe_matmul_grouped(f(4, 8), b(2, 8, 16), i(2), i(3), b(4, 16)),
             lambda: L.moe_matmul_grouped(b(4, 8), b(2, 16, 8).transpose(1, 2), i(2), i(3), b(4, 16)),
             lambda: L.moe_matmul_grouped(b(4, 8), b(2, 8, 16), i(3), i(3), b(4, 16)),
             lambda: L.moe_matmul_grouped_dw(b(4, 8), b(5, 16), i(2), i(3), b(2, 8, 16)),
             lambda: L.moe_matmul_grouped_dw(b(4, 8), b(4, 16), i(2), i(3), b(2, 8, 16).half())]
    for n, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was taken")
    with pytest.raises(L.MoEError):
        L.moe_matmul_grouped(b(4, 12), b(2, 12, 16), i(2), i(3), b(4, 16))


def rows_case(L, T, E, k, H, dt, drop, seed, spare=3):
    """Positions, rows (NaN where no entry names them) and tokens; rows_max is `spare` above the rows in use."""
    idx = choices(T, E, k, seed, drop)
    counts, offsets, pos, src = fast_group(idx, E)
    g = torch.Generator().manual_seed(seed)
    n = int(offsets[-1])
    rows = torch.full((n + spare, H), float("nan"))
    rows[:n] = torch.randn((n, H), generator=g)
    x = torch.randn((T, H), generator=g) * (0.1 + 3 * torch.rand((T, 1), generator=g))
    w = torch.rand((T, k), generator=g) * 2 - 0.5
    w[torch.from_numpy(pos) < 0] = float("nan")  # the weight of an entry without a row is not used
    return n, pos, torch.from_numpy(pos).int().to(dev), rows.to(dt).to(dev), x.to(dt).to(dev), w.to(dev)


ROWS = [(1, 8, 1, 1), (1, 256, 6, 4096), (2, 4, 3, 7), (5, 16, 16, 130), (64, 12, 8, 64), (33, 40, 9, 1000),
        (129, 64, 6, 2056), (17, 9, 2, 517), (300, 20, 5, 24), (3, 8, 4, 20480)]


@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,H", ROWS)
def test_dispatch(L, T, E, k, H, dt, drop):
    n, pos, p, rows, x, w = rows_case(L, T, E, k, H, dt, drop, T + H)
    x[0, 0] = float("nan")
    x[-1, -1] = float("inf")
    out = torch.full((n + 3, H), float(FILL), dtype=dt, device=dev)
    L.moe_dispatch(x, p, out)
    want = torch.full((n + 3, H), float(FILL), dtype=dt)
    for t, j in np.argwhere(pos >= 0):
        want[pos[t, j]] = x[t].cpu()
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=12345.0), torch.nan_to_num(want, nan=12345.0))


@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16], ids=["to_f32", "to_bf16"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,H", ROWS)
def test_collect(L, T, E, k, H, dt, odt, drop):
    n, pos, p, rows, x, w = rows_case(L, T, E, k, H, dt, drop, T + H)
    for weights in (w, None):
        out = torch.full((T, H), float("nan"), dtype=odt, device=dev)
        L.moe_collect(rows, p, weights, out)
        want = tr.collect(rows, pos, None if weights is None else np64(w))
        size = tr.collect(rows.abs(), pos, None if weights is None else np.abs(np64(w)))
        tol = k * 2.0 ** -24 * size
        assert np.all(np.abs(np64(out) - want) <= tol + HALF[odt] * (np.abs(want) + tol))


@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16], ids=["of_f32", "of_bf16"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,H", ROWS)
def test_collect_backward(L, T, E, k, H, dt, odt, drop):
    n, pos, p, rows, x, w = rows_case(L, T, E, k, H, dt, drop, T + H)
    d = x.to(odt)
    named = pos[pos >= 0]
    for weights in (w, None):
        drows = torch.full((n + 3, H), float(FILL), dtype=dt, device=dev)
        dw = torch.full((T, k), float("nan"), device=dev)
        L.moe_collect_backward(d, rows, p, weights, drows, dw)
        wn = None if weights is None else np64(w)
        want, want_w = tr.collect_backward(d, rows, pos, wn)
        got = np64(drows)
        assert np.all(got[n:] == FILL)
        tol = (HALF[dt] + 2.0 ** -23) * np.abs(want)  # the product's rounding to fp32 and then to the type
        assert np.all(np.abs(got[named] - want[named]) <= tol[named])
        size = tr.collect_backward(d.abs(), rows.abs(), pos, wn)[1]
        assert np.all(np.abs(np64(dw) - want_w) <= H * 2.0 ** -24 * size)
        alone = torch.full_like(drows, float(FILL))  # each output alone is the same
        L.moe_collect_backward(d, None, p, weights, alone, None)
        assert torch.equal(alone, drows)
        alone = torch.full_like(dw, float("nan"))
        L.moe_collect_backward(d, rows, p, weights, None, alone)
        assert torch.equal(alone, dw)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("H", [*range(1, 20), 61, 509, 2050, 2063, 4099])
def test_ends_of_rows(L, H, dt):
    """Every length of a row's last piece, in every call: whole numbers, so that the sums have one value, and an infinity
    in one of the last eight columns, which is summed once like any other."""
    T, E, k = 11, 6, 3
    n, pos, p, rows, x, w = rows_case(L, T, E, k, H, dt, 0.2, H)
    g = torch.Generator().manual_seed(H)
    whole = lambda *s: torch.randint(-4, 5, s, generator=g).to(dt).to(dev)  # noqa: E731
    x, rows, w = whole(T, H), whole(n + 3, H), torch.randint(-2, 3, (T, k), generator=g).float().to(dev)
    out = torch.full((n + 3, H), float(FILL), dtype=dt, device=dev)
    L.moe_dispatch(x, p, out)
    want = torch.full((n + 3, H), float(FILL), dtype=dt)
    for t, j in np.argwhere(pos >= 0):
        want[pos[t, j]] = x[t].cpu()
    assert torch.equal(out.cpu(), want)
    got = torch.empty((T, H), device=dev)
    L.moe_collect(rows, p, w, got)
    assert np.array_equal(np64(got), tr.collect(rows, pos, np64(w)))
    out.fill_(FILL)
    dw = torch.full((T, k), float("nan"), device=dev)
    L.moe_collect_backward(x, rows, p, w, out, dw)
    want, want_w = tr.collect_backward(x, rows, pos, np64(w))
    assert np.array_equal(np64(out)[:n], want[:n]) and np.all(np64(out)[n:] == FILL)
    assert np.array_equal(np64(dw), np.where(pos >= 0, want_w, 0))
    for c in range(max(0, H - 9), H):
        ones, r = torch.ones_like(x), rows.clone()
        r[:, c] = float("inf")
        L.moe_collect_backward(ones, r, p, w, None, dw)
        assert np.array_equal(np64(dw), np.where(pos >= 0, np.inf, 0))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("H", [72, 131])
def test_positions_past_the_rows(L, H, dt):
    """Positions that lie outside the rows' buffer, on either side, count as dropped in every call; what lies behind the
    buffer stays as it was."""
    T, E, k = 50, 8, 3
    n, pos, p, rows, x, w = rows_case(L, T, E, k, H, dt, 0.1, 9)
    few = n // 2
    p = torch.where(p == 5, torch.tensor(-2 ** 31, dtype=torch.int32, device=dev), p)
    p = torch.where(p == 7, torch.tensor(2 ** 31 - 1, dtype=torch.int32, device=dev), p)
    pos = np.where((npi(p) < 0) | (npi(p) >= few), -1, npi(p))
    w = torch.nan_to_num(w, nan=0.5)
    out = torch.full((n, H), float(FILL), dtype=dt, device=dev)
    L.moe_dispatch(x, p, out[:few])
    want = torch.full((n, H), float(FILL), dtype=dt)
    for t, j in np.argwhere(pos >= 0):
        want[pos[t, j]] = x[t].cpu()
    assert torch.equal(out.cpu(), want)
    got = torch.empty((T, H), device=dev)
    L.moe_collect(rows[:few], p, w, got)
    size = tr.collect(rows[:few].abs(), pos, np.abs(np64(w)))
    assert np.all(np.abs(np64(got) - tr.collect(rows[:few], pos, np64(w))) <= (k + 1) * 2.0 ** -24 * size)
    out.fill_(FILL)
    dw = torch.full((T, k), float("nan"), device=dev)
    L.moe_collect_backward(x, rows[:few], p, w, out[:few], dw)
    want, want_w = tr.collect_backward(x, rows[:few], pos, np64(w))
    named = pos[pos >= 0]
    assert np.all(np.abs(np64(out)[named] - want[named]) <= (HALF[dt] + 2.0 ** -23) * np.abs(want[named]))
    rest = np.setdiff1d(np.arange(n), named)
    assert np.all(np64(out)[rest] == FILL)
    size = tr.collect_backward(x.abs(), rows[:few].abs(), pos)[1]
    assert np.all(np.abs(np64(dw) - want_w) <= H * 2.0 ** -24 * size) and np.all(np64(dw)[pos < 0] == 0)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_unaligned_rows(L, dt, off):
    """Buffers that start off 16 bytes take the narrower loads."""
    T, E, k, H = 40, 8, 3, 64
    n, pos, p, rows, x, w = rows_case(L, T, E, k, H, dt, 0.2, 5)

    def shifted(t):
        b = torch.zeros(t.numel() + off, dtype=t.dtype, device=dev)
        b[off:] = t.reshape(-1)
        return b[off:].view(t.shape)
    out, out2 = torch.empty_like(x), shifted(x)
    L.moe_collect(rows, p, w, out)
    L.moe_collect(shifted(rows), p, w, out2)
    assert torch.equal(out, out2)
    a, b = torch.zeros_like(rows), shifted(torch.zeros_like(rows))
    da, db = torch.empty((T, k), device=dev), torch.empty((T, k), device=dev)
    L.moe_collect_backward(x, rows, p, w, a, da)
    L.moe_collect_backward(shifted(x), shifted(rows), p, w, b, db)
    assert torch.equal(a, b)
    named = torch.from_numpy(pos).to(dev) >= 0
    size = tr.collect_backward(x.abs(), rows.abs(), pos)[1]
    assert np.all(np.abs(np64(da - db)) <= 2 * H * 2.0 ** -24 * size) and torch.all(db[~named] == 0)
    a, b = torch.zeros_like(rows), shifted(torch.zeros_like(rows))
    L.moe_dispatch(x, p, a)
    L.moe_dispatch(shifted(x), p, b)
    assert torch.equal(a, b)


def test_no_rows(L):
    """No tokens, and tokens of which no choice is held."""
    p = torch.full((3, 2), -1, dtype=torch.int32, device=dev)
    none = torch.empty((0, 8), device=dev)
    out, dw = torch.full((3, 8), 5.0, device=dev), torch.full((3, 2), 5.0, device=dev)
    L.moe_dispatch(out, p, none)
    L.moe_collect(none, p, None, out)
    L.moe_collect_backward(torch.ones((3, 8), device=dev), none, p, None, None, dw)
    assert not out.any() and not dw.any()
    L.moe_collect(none, p[:0], None, none)
    L.moe_collect_backward(none, none, p[:0], None, none, dw[:0])
    L.moe_dispatch(none, p[:0], out)
    assert not out.any()


def test_rows_past_32_bit_offsets(L):
    """Rows that lie more than 2^32 bytes into a buffer (only the ones that are named are touched)."""
    T, k, H = 6, 2, 4096
    n = (1 << 32) // (2 * H) + 1000
    rows = torch.empty((n, H), dtype=torch.bfloat16, device=dev)
    at = np.array([n - 1, 0, n - 2, 5, n - 700, 1, n // 2, 2, n - 900, 3, n - 4, 4]).reshape(T, k)
    pos = torch.from_numpy(at).int().to(dev)
    g = torch.Generator().manual_seed(2)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).to(dev)
    w = torch.rand((T, k), generator=g).to(dev)
    L.moe_dispatch(x, pos, rows)
    assert all(torch.equal(rows[at[t, j]], x[t]) for t in range(T) for j in range(k))
    out = torch.empty((T, H), device=dev)
    L.moe_collect(rows, pos, w, out)
    want = np64(x) * np64(w).sum(1)[:, None]
    assert np.all(np.abs(np64(out) - want) <= 3 * 2.0 ** -24 * np.abs(want) + 1e-30)
    dw = torch.empty((T, k), device=dev)
    L.moe_collect_backward(x, rows, pos, w, None, dw)
    size = (np64(x) ** 2).sum(1)[:, None]
    assert np.all(np.abs(np64(dw) - size) <= H * 2.0 ** -24 * size)
    L.moe_collect_backward(x, None, pos, w, rows, None)
    for t, j in ((0, 0), (2, 0), (3, 0)):
        want = np64(x[t]) * float(w[t, j])
        assert np.all(np.abs(np64(rows[at[t, j]]) - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want))
