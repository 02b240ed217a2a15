"""SwiGLU kept in 8 bits (moe_swiglu_save, moe_swiglu_backward) against its statement in 64 bits: codes and scales are
equal, values within the roundings counted in the tests."""
import numpy as np
import pytest
import torch

from oracle import train as tr
from tests.parity import np64

pytestmark = pytest.mark.gpu
dev = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
FILL = -7


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def inputs(R, I, dt, seed):
    g = torch.Generator().manual_seed(seed)
    gu = torch.randn((R, 2 * I), generator=g) * 2
    gu *= torch.where(torch.rand(2 * I, generator=g) < 0.05, 10.0, 1.0)
    gu[0, :min(I, 128)] = 0.0  # a scale of 0
    dh = torch.randn((R, I), generator=g)
    return gu.to(dt).to(dev), dh.to(dt).to(dev)


def buffers(R, I, dt):
    return dict(h=torch.full((R, I), float(FILL), dtype=dt, device=dev),
                codes=torch.full((R, 2 * I), FILL, dtype=torch.int8, device=dev),
                scales=torch.full((R, 2 * ((I + 127) // 128)), float(FILL), device=dev),
                dgu=torch.full((R, 2 * I), float(FILL), dtype=dt, device=dev),
                again=torch.full((R, I), float(FILL), dtype=dt, device=dev))


def check_save(gu, o, rows, I, dt):
    g, u = np64(gu[:rows, :I]), np64(gu[:rows, I:])
    # half steps of 2^-24: the exponential's argument |g| and 1.5 |g| more in base 2, itself 2, the sum 1, the reciprocal
    # 2, the products 3. The hardware's exponential gives 0 for results below the smallest normal number of fp32: s(g) is
    # off by up to 2^-126 there and g s(g) u by up to |g u| 2^-126 (at g = -88, u = -3 by 264 * 2^-126, which a tolerance
    # of (1 + |u|) 2^-126 does not hold); the product itself may be lost below 2^-126
    want = tr.swiglu(g, u)
    tol = (2.5 * np.abs(g) + 9) * 2.0 ** -24 * np.abs(want) + 2.0 ** -126 * (1 + np.abs(u)) * (1 + np.abs(g))
    assert np.all(np.abs(np64(o["h"][:rows]) - want) <= tol + HALF[dt] * (np.abs(want) + tol))
    for part, first, sc in ((g, 0, o["scales"][:rows, :(I + 127) // 128]), (u, I, o["scales"][:rows, (I + 127) // 128:])):
        codes, scales = tr.keep(part)
        assert np.array_equal(o["codes"][:rows, first:first + I].cpu().numpy(), codes)
        assert np.array_equal(sc.cpu().numpy(), scales)
    for n in ("h", "codes", "scales"):
        assert torch.all(o[n][rows:] == FILL)


def check_backward(o, dh, rows, I, dt):
    G = (I + 127) // 128
    c, s = o["codes"][:rows].cpu().numpy(), o["scales"][:rows].cpu().numpy()
    g, u, d = tr.kept(c[:, :I], s[:, :G]), tr.kept(c[:, I:], s[:, G:]), np64(dh[:rows])
    dg, du = tr.swiglu_backward(g, u, d)
    sg, sn = tr.sigmoid(g), tr.sigmoid(-g)
    # as above, with a half step more each for g and u (a code times its scale), g's through the sigmoid |g| times
    k = (3.5 * np.abs(g) + 14) * 2.0 ** -24
    tiny = 2.0 ** -126 * (1 + np.abs(u)) * (1 + np.abs(d)) * (1 + np.abs(g))
    for got, want, size in ((o["dgu"][:, :I], dg, np.abs(d * u) * (sg + np.abs(g) * sg * sn)), (o["dgu"][:, I:], du, np.abs(du)),
                            (o["again"], g * sg * u, np.abs(g * sg * u))):
        tol = k * size + tiny
        assert np.all(np.abs(np64(got[:rows]) - want) <= tol + HALF[dt] * (np.abs(want) + tol))
        assert torch.all(got[rows:] == FILL)


SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 128), (2, 129), (17, 768), (9, 645), (64, 1000), (2, 255), (1, 8), (33, 264),
          (300, 64), (4, 4104)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("R,I", SHAPES)
def test_save_and_backward(L, R, I, dt):
    gu, dh = inputs(R, I, dt, R + I)
    for rows in sorted({R, R // 2, 0}, reverse=True):
        o = buffers(R, I, dt)
        n = None if rows == R else torch.tensor([rows], dtype=torch.int32, device=dev)
        L.moe_swiglu_save(gu, o["h"], o["codes"], o["scales"], n)
        check_save(gu, o, rows, I, dt)
        L.moe_swiglu_backward(o["codes"], o["scales"], dh, o["dgu"], o["again"], n)
        check_backward(o, dh, rows, I, dt)
        if rows == R:
            alone = torch.full_like(o["dgu"], float(FILL))
            L.moe_swiglu_backward(o["codes"], o["scales"], dh, alone)
            assert torch.equal(alone, o["dgu"])
            L.moe_swiglu_save(gu, o["h"], o["codes"], o["scales"], torch.tensor([R + 9], dtype=torch.int32, device=dev))
            check_save(gu, o, R, I, dt)  # more rows than there are: all of them


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("I", [*range(2, 21), *range(121, 142), *range(257, 264)])
def test_ends_of_rows(L, I, dt):
    """Every length of a row's last piece, also where it begins in the group before, whose scale is another."""
    R = 5
    gu, dh = inputs(R, I, dt, I)
    far = torch.tensor([1.0, 2.0 ** -9, 2.0 ** 3], device=dev).repeat_interleave(128)[:I].to(dt)
    gu *= torch.cat([far, far.flip(0)])
    o = buffers(R, I, dt)
    n = torch.tensor([R - 1], dtype=torch.int32, device=dev)
    L.moe_swiglu_save(gu, o["h"], o["codes"], o["scales"], n)
    check_save(gu, o, R - 1, I, dt)
    L.moe_swiglu_backward(o["codes"], o["scales"], dh, o["dgu"], o["again"], n)
    check_backward(o, dh, R - 1, I, dt)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("R,I,off", [(7, 256, 1), (7, 256, 2), (3, 384, 4)])
def test_unaligned(L, R, I, off, dt):
    """Buffers that start off 16 bytes give the same bits."""
    gu, dh = inputs(R, I, dt, 3)

    def shifted(t):
        b = torch.zeros(t.numel() + off, dtype=t.dtype, device=dev)
        b[off:] = t.reshape(-1)
        return b[off:].view(t.shape)
    a, b = buffers(R, I, dt), {n: shifted(t) for n, t in buffers(R, I, dt).items()}
    for o, x, d in ((a, gu, dh), (b, shifted(gu), shifted(dh))):
        L.moe_swiglu_save(x, o["h"], o["codes"], o["scales"])
        L.moe_swiglu_backward(o["codes"], o["scales"], d, o["dgu"], o["again"])
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e-37, 1e-30, 1.0, 1e30], ids=str)
def test_codes_of_ties_and_far_scales(L, dt, scale):
    """Values whose 127 v / max is a whole number and a half go to the even code, at any size."""
    g = torch.Generator().manual_seed(9)
    R, I = 64, 256
    k = torch.randint(-254, 255, (R, 2 * I), generator=g).float()  # halves of codes: 127 k / 254
    k[:, ::128] = 254.0
    gu = (k * scale).to(dt)  # 254 and less in bf16 are exact before the scale; the oracle takes what is there
    gu = gu.to(dev)
    o = buffers(R, I, dt)
    L.moe_swiglu_save(gu, o["h"], o["codes"], o["scales"])
    for first, sc in ((0, o["scales"][:, :2]), (I, o["scales"][:, 2:])):
        codes, scales = tr.keep(np64(gu[:, first:first + I]))
        assert np.array_equal(o["codes"][:, first:first + I].cpu().numpy(), codes)
        assert np.array_equal(sc.cpu().numpy(), scales)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_far_gates(L, dt):
    """Gates far out: silu ends at 0 and g, its derivative at 0 and 1, without a NaN."""
    I = 256
    gu = torch.zeros((2, 2 * I))
    gu[:, :I] = torch.linspace(-1000, 1000, I)
    gu[0, I:], gu[1, I:] = 1.0, -3.0
    gu, dh = gu.to(dt).to(dev), torch.ones((2, I), dtype=dt, device=dev)
    o = buffers(2, I, dt)
    L.moe_swiglu_save(gu, o["h"], o["codes"], o["scales"])
    check_save(gu, o, 2, I, dt)
    L.moe_swiglu_backward(o["codes"], o["scales"], dh, o["dgu"], o["again"])
    check_backward(o, dh, 2, I, dt)


@pytest.mark.parametrize("I", [256, 250])
def test_not_finite(L, I):
    """An infinity or NaN makes its 128 columns NaN in the backward pass and leaves the others alone."""
    gu, dh = inputs(4, I, torch.float32, 1)
    gu[1, 3], gu[2, 130], gu[3, I + 5] = float("inf"), float("nan"), -float("inf")
    o = buffers(4, I, torch.float32)
    L.moe_swiglu_save(gu, o["h"], o["codes"], o["scales"])
    assert torch.isnan(o["scales"]).sum() == 3
    assert torch.isnan(o["scales"][1, 0]) and torch.isnan(o["scales"][2, 1]) and torch.isnan(o["scales"][3, 2])
    assert torch.isnan(o["h"][2, 130]) and torch.isfinite(o["h"]).sum() == 4 * I - 3
    L.moe_swiglu_backward(o["codes"], o["scales"], dh, o["dgu"], o["again"])
    bad = torch.zeros((4, I), dtype=torch.bool)
    bad[1, :128] = bad[2, 128:] = bad[3, :128] = True
    for t in (o["dgu"][:, :I], o["again"]):
        assert torch.equal(~torch.isfinite(t.cpu()), bad)
    bad[3] = False  # the up values' gradient does not read them
    assert torch.equal(~torch.isfinite(o["dgu"][:, I:].cpu()), bad)
