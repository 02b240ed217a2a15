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
    """Entries that are off by more than their steps and rounding; results below 2^-120 of a type's range are left out."""
    tol = steps * 2.0 ** -24 * size
    held = np.abs(want) >= 2.0 ** -120
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
