"""Inputs and derived tolerances of the int8 expert tests."""
import numpy as np
import torch

import oracle
from tests.parity import np64


def expert(H, I, seed, device="cpu"):
    """Canonical int8 expert: codes over the whole range [-128, 127] at the edges, scales spread over a factor of 4."""
    g = torch.Generator().manual_seed(seed)
    d = {}
    for n, shape in (("q1", (H, I)), ("q3", (H, I)), ("q2", (I, H))):
        d[n] = (torch.randn(shape, generator=g) * 40).round().clamp(-128, 127).to(torch.int8)
        d[n][0, 0], d[n][-1, -1] = -128, 127
    for n, size, fan in (("s1", I, H), ("s3", I, H), ("s2", H, I)):
        d[n] = (0.25 + 0.75 * torch.rand(size, generator=g)) / (32 * fan ** 0.5)
    return {k: v.to(device) for k, v in d.items()}


def reference(X, w, half=False):
    """(y, tol) of an expert on rows X in 64 bits. The kernel's h carries fp32 roundings: the integer sum and its two
    scales 3 half steps (of 2^-24) for u and for g, g's share through silu at most (1 + |g|) times that; the exponential's
    argument in base 2 |g| + 1.5 more, it and the reciprocal a step each, the sum and the two products 3: below
    13 + 4.5 |g| half steps, 2^-18 relative for |g| < 11. As code units that is at most 127 * 2^-18; an h whose 127 h / max|h| lies nearer than that to a half may get either code, which moves y by one
    step of its scale times its weight. Beside that y carries 2^-18 relative of the row's scale and the final
    products' roundings, over the sum of magnitudes.
    half: the layer's prefill form keeps rows that go into a bf16 output in fp16, scaled by a power of two u with
    2^14 <= 127 * 128 I max(s2) u < 2^15: half a step is 2^-11 of y, or of the smallest subnormal 2^-25 / u of the row's
    scale, at most 2^-39 * 127 * 128 I max(s2) sh."""
    r = oracle.int8_expert(X, *(np64(w[n]) for n in ("q1", "q3", "q2", "s1", "s3", "s2")))
    amax = np.abs(r["h"]).max(1, keepdims=True)
    t = np.abs(r["h"]) * 127.0 / np.where(amax > 0, amax, 1.0)
    near = np.abs(t - np.floor(t) - 0.5) < 127 * 2.0 ** -18
    W2 = np.abs(np64(w["q2"])) * np64(w["s2"])[None, :]
    step = r["sh"][:, None]
    tol = (near * step) @ W2 * (1 + 1e-3) + 2.0 ** -17 * (np.abs(r["hq"]) * step) @ W2 + 1e-30
    if half:
        I = W2.shape[0]
        tol = tol + 2.0 ** -11 * (np.abs(r["y"]) + tol) + 2.0 ** -39 * 127 * 128 * I * float(np64(w["s2"]).max()) * step
    return r["y"], tol


def check(got, y, tol, what, out_bf16=False):
    got = np.asarray(got, np.float64)
    assert got.shape == y.shape and np.all(np.isfinite(got)), what
    if out_bf16:
        tol = tol + 2.0 ** -8 * (np.abs(y) + tol)
    bad = np.abs(got - y) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - y) / tol):.2f} of its tolerance"
