"""SwiGLU kept in 8 bits where the gate's sigmoid is small and what it is multiplied by is not: results that the type
holds come out whole, forward and backward."""
import numpy as np
import pytest
import torch

from oracle import train as tr
from tests.parity import np64

pytestmark = pytest.mark.gpu
dev = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# Half steps of 2^-24 that a value may be off before it is rounded to its type: the exponent's argument is good to 2^-40
# of itself (nothing), the exponential 2 and its correction 1, 1 + e^g is 1, the reciprocal 2, e^g times it 1, times g 1,
# times u or dh 1, and dg's sum and its second factor 2: 10. Kept g and u are a code times a scale, a half step each, and
# g's shifts the exponential by |g| of it.
STEPS = 10


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def far(dt, seed, lo, hi):
    """Rows of gates from -hi to -lo in groups of 128, and factors that bring the results to about 1 in size."""
    R, I = 48, 256
    r = np.random.default_rng(seed)
    g = -np.linspace(lo, hi, R)[:, None] - r.random((R, I)) * 0.2
    u = np.exp2(np.clip(-g / np.log(2), 0, 120)) * r.uniform(0.5, 1.5, (R, I)) * r.choice([-1, 1], (R, I))
    u[:, ::128], g[:, ::128] = np.abs(u).max(), -hi - 0.2
    return torch.tensor(np.concatenate([g, u], 1)).to(dt).to(dev), R, I


def off(got, want, size, steps, dt):
    """Entries that are off by more than their steps and rounding; results that are no normal numbers are left out."""
    tol = steps * 2.0 ** -24 * size
    held = np.abs(want) >= 2.0 ** -125
    assert held.mean() > 0.4
    return (np.abs(np64(got) - want) > tol + HALF[dt] * (np.abs(want) + tol))[held]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(60, 68), (80, 90), (88, 104), (100, 130)])
def test_small_sigmoids(L, dt, lo, hi):
    gu, R, I = far(dt, lo, lo, hi)
    h, dgu, again = (torch.empty(s, dtype=dt, device=dev) for s in ((R, I), (R, 2 * I), (R, I)))
    codes = torch.empty((R, 2 * I), dtype=torch.int8, device=dev)
    scales = torch.empty((R, 4), device=dev)
    L.moe_swiglu_save(gu, h, codes, scales)
    g, u = np64(gu[:, :I]), np64(gu[:, I:])
    want = tr.swiglu(g, u)
    assert not off(h, want, np.abs(want), STEPS, dt).any()
    dh = gu[:, I:].contiguous()  # gradients as large as u: du is about 1, and dg with u of 1
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    one = torch.full_like(gu, 1.0)
    one[:, :I] = gu[:, :I]
    c1, s1 = torch.empty_like(codes), torch.empty_like(scales)
    L.moe_swiglu_save(one, again, c1, s1)
    L.moe_swiglu_backward(c1, s1, dh, dgu, again)
    s1 = s1.cpu().numpy()
    g, u, d = tr.kept(c1[:, :I].cpu().numpy(), s1[:, :2]), tr.kept(c1[:, I:].cpu().numpy(), s1[:, 2:]), np64(dh)
    dg, du = tr.swiglu_backward(g, u, d)
    steps = STEPS + 2 + np.abs(g)
    assert not off(dgu[:, :I], dg, np.abs(d * u * tr.sigmoid(g) * (1 + np.abs(g))), steps, dt).any()
    assert not off(dgu[:, I:], du, np.abs(du), steps, dt).any()
    L.moe_swiglu_backward(codes, scales, torch.ones_like(dh), dgu, again)
    g, u = tr.kept(c[:, :I], s[:, :2]), tr.kept(c[:, I:], s[:, 2:])
    want = tr.swiglu(g, u)
    held = np.abs(u) > 0
    assert not off(again, np.where(held, want, 0), np.abs(want), STEPS + 2 + np.abs(g), dt).any()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d,u", [(70, 70), (100, 40), (40, 100), (-100, 120), (120, -100), (-60, -60), (126, 0), (0, 126)])
def test_far_factors(L, dt, d, u):
    """dh and u of 2^d and 2^u whose product the type does not hold, where dgu's gate half is in its range: it comes out."""
    R, I = 8, 256
    r = np.random.default_rng(1)
    gu = torch.empty((R, 2 * I))
    gu[:, :I] = torch.tensor(-r.uniform(30, 60, (R, I)) if d + u > 128 else r.uniform(-5, 5, (R, I)))
    gu[:, I:] = 2.0 ** u * torch.tensor(r.choice([-1.0, 1.0], (R, I)))
    dh = 2.0 ** d * torch.tensor(r.choice([-1.0, 0.75, 1.25], (R, I)))
    gu, dh = gu.to(dt).to(dev), dh.to(dt).to(dev)
    h, dgu = torch.empty((R, I), dtype=dt, device=dev), torch.empty((R, 2 * I), dtype=dt, device=dev)
    codes, scales = torch.empty((R, 2 * I), dtype=torch.int8, device=dev), torch.empty((R, 4), device=dev)
    L.moe_swiglu_save(gu, h, codes, scales)
    L.moe_swiglu_backward(codes, scales, dh, dgu)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    g, u, dh = tr.kept(c[:, :I], s[:, :2]), tr.kept(c[:, I:], s[:, 2:]), np64(dh)
    dg, _ = tr.swiglu_backward(g, u, dh)
    # as above, with the larger of two factors chosen and halves exact; dg's second factor is near 0 at g = -1.3
    size = np.abs(dh * u * tr.sigmoid(g)) * (1 + np.abs(g) * tr.sigmoid(-g))
    assert np.abs(dg).max() < 2.0 ** 127.9
    assert not off(dgu[:, :I], dg, size, STEPS + 2 + np.abs(g), dt).any()
