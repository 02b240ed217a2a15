"""Where the training operators change their form: numbers of entries around the grouping's forms and blocks, long
batches of one or two rows a token, buffers off 16 bytes, and the whole layer against tolerances counted per result."""
import numpy as np
import pytest
import torch

from oracle import train as tr
from tests.parity import np64, npi
from tests.test_gpu_train_layer import R, backward, case, chain, forward, outputs  # noqa: F401
from tests.test_gpu_train_rows import FILL, HALF, L, choices, fast_group, grouped, rows_case  # noqa: F401

pytestmark = pytest.mark.gpu
dev = "cuda"
TYPES = pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])

# entries T * k: one block up to 1024, several blocks in one launch up to 32768, then two launches, of a block for 4096
# entries up to 64 blocks
ENTRIES = [(1023, 1), (512, 2), (205, 5), (1026, 1), (2047, 1), (1024, 2), (683, 3), (10922, 3), (32768, 1), (4096, 8),
           (10923, 3), (32770, 1), (9216, 4), (36865, 1), (262144, 1), (32768, 8), (87382, 3), (266241, 1)]


@pytest.mark.parametrize("E", [1, 7, 256, 1024])
@pytest.mark.parametrize("T,k", ENTRIES)
def test_group_forms(L, T, k, E):  # noqa: F811
    idx = choices(T, E, k, T + E, 0.2 if E > 1 else 0.5, 0.0, True)
    idx[-1, -1], idx[0, 0] = E - 1, 0
    counts, offsets, pos, src = fast_group(idx, E)
    o = grouped(L, idx, E)
    assert np.array_equal(npi(o["counts"]), counts) and np.array_equal(npi(o["offsets"]), offsets)
    assert np.array_equal(npi(o["perm_pos"]), pos)
    got = npi(o["perm_src"])
    assert np.array_equal(got[:len(src)], src) and np.all(got[len(src):] == FILL)


@TYPES
@pytest.mark.parametrize("T,k", [(2047, 2), (2048, 1), (2049, 1), (2049, 2), (2050, 2), (2051, 3)])
@pytest.mark.parametrize("H", [512, 720, 1001, 4099])
def test_gradients_of_one_or_two_rows(L, T, k, H, dt):  # noqa: F811
    """A wave a token from 2048 tokens on, whose lanes take several pieces each, the last one ending with the row."""
    n, pos, p, rows, x, w = rows_case(L, T, 16, k, H, dt, 0.3, T + H)
    drows = torch.full((n + 3, H), float(FILL), dtype=dt, device=dev)
    dw = torch.full((T, k), float("nan"), device=dev)
    L.moe_collect_backward(x, rows, p, w, drows, dw)
    t, j = np.nonzero(pos >= 0)
    d, r, wn, at = np64(x), np64(rows), np64(w), pos[t, j]
    want = wn[t, j][:, None] * d[t]
    got = np64(drows)
    assert np.all(got[n:] == FILL)
    assert np.all(np.abs(got[at] - want) <= (HALF[dt] + 2.0 ** -23) * np.abs(want))  # as in test_collect_backward
    want, size = np.zeros((T, k)), np.zeros((T, k))
    want[t, j], size[t, j] = (d[t] * r[at]).sum(1), np.abs(d[t] * r[at]).sum(1)
    assert np.all(np.abs(np64(dw) - want) <= H * 2.0 ** -24 * size)
    alone = torch.full_like(dw, float("nan"))
    L.moe_collect_backward(x, rows, p, w, None, alone)
    assert torch.equal(alone, dw)


@TYPES
@pytest.mark.parametrize("H", [64, 1001])
@pytest.mark.parametrize("off", [1, 2, 3, 4, 7])
def test_any_alignment_gives_the_same_bits(L, H, off, dt):  # noqa: F811
    """Loads and stores take rows at any element, by the same arithmetic."""
    T, E, k = 40, 8, 3
    n, pos, p, rows, x, w = rows_case(L, T, E, k, H, dt, 0.2, 5)

    def shifted(t):
        b = torch.zeros(t.numel() + off, dtype=t.dtype, device=dev)
        b[off:] = t.reshape(-1)
        return b[off:].view(t.shape)
    res = []
    for f in (lambda t: t, shifted):
        out, sent, drows = (f(torch.full_like(t, FILL)) for t in (x, rows, rows))
        dw = f(torch.full((T, k), float("nan"), device=dev))
        L.moe_collect(f(rows), p, f(w), out)
        L.moe_dispatch(f(x), p, sent)
        L.moe_collect_backward(f(x), f(rows), p, f(w), drows, dw)
        res.append((out, sent, drows, dw))
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("T,E,k,H,I,drop", [(40, 12, 3, 256, 136, 0.3), (300, 9, 4, 512, 384, 0)])
def test_passes_by_their_roundings(R, T, E, k, H, I, drop):  # noqa: F811
    """Every result of both passes against the 64-bit chain by the bf16 roundings on its way. One rounding of numbers with
    significands spread over [1, 2) is off by 2^-8 / sqrt(7) of their norm (an error uniform in half a step of 2^-8, rms
    2^-8 / sqrt(3), to an rms of sqrt(7 / 3)). Products with matrices like these pass relative errors on as they are;
    SwiGLU passes g's rounding and u's on, 2.3 in squares: 0.45 / 0.36, the mean squares of g silu'(g) and silu(g), and 1.
    Independent ones add in squares, n of them to sqrt(n); twice that is allowed for. out: gu 2.3, h, y (out fp32);
    dw: the same; dW2: h, dy, itself; dW13: dy, dh, dgu, itself; dx: dy, dh, dgu, the rows' gradient, itself."""
    c = case(T, E, k, H, I, T + H, drop)
    layer, o = R.TrainExperts(H, I, E, k, T, dev), outputs(c)
    forward(layer, c, o)
    codes, scales = layer.codes.cpu().numpy(), layer.scales.cpu().numpy()
    backward(layer, c, o)
    want, _ = chain(c, codes, scales, I)
    for name, n in dict(out=4.3, dw=4.3, dW2=3, dW13=4, dx=5).items():
        got = np64(o[name])
        off = np.linalg.norm(got - want[name]) / np.linalg.norm(want[name])
        assert off <= 2 * n ** 0.5 * 2.0 ** -8 / 7 ** 0.5, (name, off)


@pytest.mark.parametrize("T,k,H,dt", [(16384, 6, 1403, torch.bfloat16), (16389, 4, 1030, torch.float32),
                                      (8192, 6, 1371, torch.float32)])
def test_more_rows_than_the_caches_hold(L, T, k, H, dt):  # noqa: F811
    """Rows of odd lengths, more than 256 MiB of them: copies are equal, gradients the products rounded once."""
    g = torch.Generator(device=dev).manual_seed(H)
    idx = torch.randint(-1, 40, (T, k), generator=g, device=dev, dtype=torch.int32)
    o = grouped(L, npi(idx).astype(np.int32), 40)
    n, pos = int(o["offsets"][40]), o["perm_pos"]
    x = torch.randn((T, H), generator=g, device=dev).to(dt)
    w = torch.rand((T, k), generator=g, device=dev)
    rows = torch.full((T * k, H), float(FILL), dtype=dt, device=dev)
    assert rows.numel() * rows.element_size() > 1 << 28
    L.moe_dispatch(x, pos, rows)
    t, j = torch.nonzero(pos >= 0, as_tuple=True)
    at = pos[t, j].long()
    assert len(at) == n and torch.equal(rows[at], x[t]) and torch.all(rows[n:] == FILL)
    drows, dw = torch.full_like(rows, float(FILL)), torch.full((T, k), float("nan"), device=dev)
    L.moe_collect_backward(x, rows, pos, w, drows, dw)
    assert torch.equal(drows[at], (w[t, j, None] * x[t].float()).to(dt)) and torch.all(drows[n:] == FILL)
    want = (x[t].double() ** 2).sum(1)
    assert torch.all((dw[t, j].double() - want).abs() <= H * 2.0 ** -24 * want) and torch.all(dw[pos < 0] == 0)
