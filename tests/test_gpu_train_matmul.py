"""The experts' products on row-major weights and their gradients (moe_matmul_grouped, moe_matmul_grouped_dw). With small
whole numbers every partial sum is exact in fp32, so results are equal to the 64-bit statement, or to its rounding;
with other inputs each of n additions and products is off by at most a step (2^-23) of the magnitudes' sum."""
import numpy as np
import pytest
import torch

from oracle import train as tr
from tests.parity import np64

pytestmark = pytest.mark.gpu
dev = "cuda"
BF = torch.bfloat16
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
FILL = -7.0


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def layout(counts, seed, gaps):
    """Offsets of the groups, in another order than the experts' and with rows of no group between, and all rows."""
    r = np.random.default_rng(seed)
    at, offsets = int(gaps), np.zeros(len(counts) + 1, np.int64)
    for e in (r.permutation(len(counts)) if gaps else range(len(counts))):
        offsets[e] = at
        at += counts[e] + (int(r.integers(0, 4)) if gaps else 0)
    offsets[-1] = at
    return offsets, at + 2 * int(gaps)


def tensors(counts, offsets, rows, K, N, seed, whole):
    g = torch.Generator(device=dev).manual_seed(seed)

    def fill(*shape):
        if whole:
            return torch.randint(-4, 5, shape, generator=g, device=dev).to(BF)
        return torch.randn(shape, generator=g, device=dev).to(BF)
    used = torch.zeros(rows, dtype=torch.bool, device=dev)
    for o, n in zip(offsets, counts):
        used[o:o + n] = True
    a, d, w = fill(rows, K), fill(rows, N), fill(len(counts), K, N)
    a[~used] = float("nan")  # rows of no group are not read into anything
    d[~used] = float("nan")
    i = lambda v: torch.from_numpy(np.asarray(v, np.int32)).to(dev)  # noqa: E731
    return a, d, w, used, i(counts), i(offsets)


def reference(fn, *args):
    """The 64-bit statement on the GPU, group by group."""
    a, b, counts, offsets, shape = args
    out = torch.zeros(shape, dtype=torch.float64, device=dev)
    size = torch.zeros(shape, dtype=torch.float64, device=dev)
    for e, (o, n) in enumerate(zip(offsets, counts)):
        s = slice(o, o + n)
        x = a[s].double()
        for r, f in ((out, lambda v: v), (size, torch.abs)):
            if fn == "dw":
                r[e] = f(x).t().contiguous() @ f(b[s].double())
            else:
                y = b[e].double()
                r[s] = f(x) @ f(y.t().contiguous() if fn == "t" else y)
    return out, size


def check(got, want, size, n, whole, what):
    dt = got.dtype
    if whole:
        assert torch.equal(got.double(), want.to(dt).double()), what
        return
    tol = n * 2.0 ** -23 * size
    assert torch.all((got.double() - want).abs() <= tol + HALF[dt] * (want.abs() + tol)), what


def run_all(L, counts, K, N, seed, gaps, whole, odt):
    counts = np.asarray(counts)
    offsets, rows = layout(counts, seed, gaps)
    a, d, w, used, c32, o32 = tensors(counts, offsets, rows, K, N, seed, whole)
    for fn, x, b, shape, n in (("n", a, w, (rows, N), K), ("t", d, w, (rows, K), N)):
        out = torch.full(shape, FILL, dtype=odt, device=dev)
        L.moe_matmul_grouped(x, b, c32, o32, out, transposed=fn == "t")
        want, size = reference(fn, x, b, counts, offsets, shape)
        check(out[used], want[used], size[used], n, whole, fn)
        assert torch.all(out[~used] == FILL)
    dw = torch.full((len(counts), K, N), FILL, dtype=odt, device=dev)
    L.moe_matmul_grouped_dw(a, d, c32, o32, dw)
    want, size = reference("dw", a, d, counts, offsets, (len(counts), K, N))
    check(dw, want, size, int(counts.max(initial=0)), whole, "dw")


COUNTS = [[0], [1], [3, 0, 1], [64, 63, 65], [0, 0, 17, 0], [128, 127, 129, 1], [255, 0, 256, 257, 2], [16] * 40,
          [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12], [513, 31], [1000]]
SHAPES = [(8, 8), (16, 64), (64, 16), (72, 136), (128, 256), (256, 128), (264, 520), (512, 40), (1000, 1008)]


@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_whole_numbers(L, counts, K, N):
    odt = BF if (K + len(counts)) % 16 == 0 else torch.float32
    run_all(L, counts, K, N, K + N + len(counts), True, True, odt)


@pytest.mark.parametrize("odt", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("gaps", [False, True], ids=["dense", "gaps"])
@pytest.mark.parametrize("K,N", [(64, 2048), (1280, 648), (2048, 1536)])
def test_many_experts(L, K, N, gaps, odt):
    r = np.random.default_rng(K)
    counts = np.where(r.random(48) < 0.3, 0, r.integers(1, 90, 48))
    counts[5] = 700
    run_all(L, counts, K, N, 7, gaps, True, odt)


@pytest.mark.parametrize("odt", [torch.float32, BF], ids=["f32", "bf16"])
def test_other_values(L, odt):
    run_all(L, [40, 0, 300, 1], 328, 200, 11, True, False, odt)


@pytest.mark.parametrize("E,most", [(1, 4), (1024, 4), (1023, 30)])
def test_expert_numbers(L, E, most):
    r = np.random.default_rng(E)
    run_all(L, r.integers(0, most, E), 64, 72, E, True, True, torch.float32)


@pytest.mark.parametrize("T", [5, 700])
def test_in_a_graph(L, T):
    """The three products captured, and replayed after the rows, the weights and the groups have changed."""
    from routed_expert_layer_amd.runtime import DeviceDecodeLayer
    E, K, N = 12, 264, 1032
    g = torch.Generator(device=dev).manual_seed(T)
    whole = lambda *s: torch.randint(-4, 5, s, generator=g, device=dev).to(BF)  # noqa: E731
    cases = []
    for i in range(3):
        counts = np.bincount(np.random.default_rng(i).integers(0, E - i, T), minlength=E)
        c = torch.from_numpy(counts.astype(np.int32)).to(dev)
        o = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
        cases.append(dict(a=whole(T, K), d=whole(T, N), w=whole(E, K, N), c=c, o=o))

    def run(v, out, s=None):
        L.moe_matmul_grouped(v["a"], v["w"], v["c"], v["o"], out[0], stream=s)
        L.moe_matmul_grouped(v["d"], v["w"], v["c"], v["o"], out[1], transposed=True, stream=s)
        L.moe_matmul_grouped_dw(v["a"], v["d"], v["c"], v["o"], out[2], stream=s)
    outs = lambda: [torch.full(s, FILL, dtype=BF, device=dev) for s in ((T, N), (T, K), (E, K, N))]  # noqa: E731
    want = []
    for v in cases:
        want.append(outs())
        run(v, want[-1])
    v, out = {n: t.clone() for n, t in cases[0].items()}, outs()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = DeviceDecodeLayer.capture(lambda: run(v, out, s), s)
    for i in (2, 0, 1, 1):
        for n in v:
            v[n].copy_(cases[i][n])
        for t in out:
            t.fill_(FILL)
        torch.cuda.synchronize()
        L.moe_graph_launch(graph, s)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want[i]))


# Cases that reach the tiles of 64, 128 and 256 rows with ragged edges on every side: short sums, many columns.
TILES = [([300, 257, 256, 255, 1, 0, 129, 31], 72, 6000), ([300, 257, 256, 255, 1, 0, 129, 31], 6000, 72),
         ([300, 257, 256, 255, 1, 0, 129, 31], 104, 4096), ([700, 600, 513, 511], 6000, 72),
         ([700, 600, 513, 511], 88, 6008), ([33, 0, 127, 90, 260, 5, 64, 1], 520, 2056), ([2, 0, 1, 7] * 16, 264, 2056),
         ([40] * 40, 1288, 96), ([1] * 300, 96, 264)]


@pytest.mark.parametrize("odt", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("counts,K,N", TILES, ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}x{max(v)}")
def test_tiles(L, counts, K, N, odt):
    run_all(L, counts, K, N, K + N, True, True, odt)


def test_groups_past_the_rows(L):
    """A group that reaches past the rows, or has a bad first row, is left out; its weight gradient is zeros."""
    K, N, rows = 64, 64, 100
    counts, offsets = np.array([10, 50, 5, 3, 2 ** 31 - 1]), np.array([0, 51, 95, -3, 2, 100])
    ok = [0, 2]
    g = torch.Generator(device=dev).manual_seed(0)
    a, d, w = (torch.randint(-4, 5, s, generator=g, device=dev).to(BF) for s in ((rows, K), (rows, N), (5, K, N)))
    c32, o32 = (torch.from_numpy(v.astype(np.int32)).to(dev) for v in (counts, offsets))
    for t, x in ((False, a), (True, d)):
        out = torch.full((rows, N), FILL, device=dev)
        L.moe_matmul_grouped(x, w, c32, o32, out, transposed=t)
        want = torch.full((rows, N), FILL, dtype=torch.float64, device=dev)
        for e in ok:
            s = slice(offsets[e], offsets[e] + counts[e])
            want[s] = x[s].double() @ (w[e].double().t().contiguous() if t else w[e].double())
        assert torch.equal(out.double(), want)
    dw = torch.full((5, K, N), FILL, device=dev)
    L.moe_matmul_grouped_dw(a, d, c32, o32, dw)
    for e in range(5):
        s = slice(offsets[e], offsets[e] + counts[e]) if e in ok else slice(0, 0)
        assert torch.equal(dw[e].double(), a[s].double().t().contiguous() @ d[s].double())


def test_no_rows(L):
    w = torch.ones((3, 16, 8), dtype=BF, device=dev)
    z, o = torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
    a, d = torch.empty((0, 16), dtype=BF, device=dev), torch.empty((0, 8), dtype=BF, device=dev)
    L.moe_matmul_grouped(a, w, z, o, d)
    dw = torch.full((3, 16, 8), FILL, dtype=BF, device=dev)
    L.moe_matmul_grouped_dw(a, d, z, o, dw)
    assert not dw.any()


def test_infinities_stay_in_their_rows(L):
    """What is not finite in one group's rows (or in a weight's part) does not reach other groups, though tiles and
    the last step along the sum reach past a group's end."""
    counts, K, N = [5, 37, 3], 72, 88
    offsets, rows = layout(counts, 0, False)
    a, d, w, used, c32, o32 = tensors(counts, offsets, rows, K, N, 3, True)
    a[5:42], d[5:42] = float("inf"), float("nan")
    w[1] = float("nan")
    for t, x, n in ((False, a, N), (True, d, K)):
        out = torch.full((rows, n), FILL, device=dev)
        L.moe_matmul_grouped(x, w, c32, o32, out, transposed=t)
        assert torch.isfinite(out[:5]).all() and torch.isfinite(out[42:]).all() and not torch.isfinite(out[5:42]).any()
    dw = torch.full((3, K, N), FILL, device=dev)
    L.moe_matmul_grouped_dw(a, d, c32, o32, dw)
    assert torch.isfinite(dw[0]).all() and torch.isfinite(dw[2]).all() and not torch.isfinite(dw[1]).any()


def test_past_32_bit_offsets(L):
    """Groups that start more than 2^32 bytes into the rows, and weights that lie as far."""
    K, N = 4096, 4096
    rows = (1 << 32) // (2 * K) + 600
    E = (1 << 32) // (2 * K * N) + 2
    a = torch.empty((rows, K), dtype=BF, device=dev)
    counts, offsets = np.zeros(E, np.int64), np.zeros(E + 1, np.int64)
    counts[0], offsets[0], counts[E - 1], offsets[E - 1] = 130, rows - 140, 7, 3
    c32, o32 = (torch.from_numpy(v.astype(np.int32)).to(dev) for v in (counts, offsets))
    w = torch.empty((E, K, N), dtype=BF, device=dev)
    g = torch.Generator(device=dev).manual_seed(0)
    for e in (0, E - 1):
        w[e] = torch.randint(-4, 5, (K, N), generator=g, device=dev).to(BF)
        a[offsets[e]:offsets[e] + counts[e]] = torch.randint(-4, 5, (int(counts[e]), K), generator=g, device=dev).to(BF)
    out = torch.empty((rows, N), dtype=BF, device=dev)
    for t in (False, True):
        L.moe_matmul_grouped(a, w, c32, o32, out, transposed=t)
        for e in (0, E - 1):
            s = slice(offsets[e], offsets[e] + counts[e])
            want = a[s].double() @ (w[e].double().t().contiguous() if t else w[e].double())
            assert torch.equal(out[s].double(), want.to(BF).double())
    want = [a[offsets[e]:offsets[e] + counts[e]].double().t().contiguous() @
            out[offsets[e]:offsets[e] + counts[e]].double() for e in (0, E - 1)]
    L.moe_matmul_grouped_dw(a, out, c32, o32, w)
    size = [a[offsets[e]:offsets[e] + counts[e]].double().abs().t().contiguous() @
            out[offsets[e]:offsets[e] + counts[e]].double().abs() for e in (0, E - 1)]
    for i, e in enumerate((0, E - 1)):
        check(w[e], want[i], size[i], int(counts[e]), False, e)
    assert not w[1].any() and not w[E - 2].any()
