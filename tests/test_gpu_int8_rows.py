"""int8 experts: how a token's rows are kept between the down projection and their sum."""
import numpy as np
import pytest
import torch

from tests import int8_cases as ic
from tests.parity import np64
from tests.test_gpu_int8 import expected, pack, routing, run, tokens

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def grouped(idx, w, E):
    """A routing as `run` takes it, from the choices idx [T, k] and their weights."""
    T, k = idx.shape
    counts = np.bincount(idx.reshape(-1), minlength=E)
    order = np.argsort(idx.reshape(-1), kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    t = lambda v: torch.from_numpy(np.ascontiguousarray(v).astype(np.int32)).to(dev)  # noqa: E731
    return dict(idx=idx, counts=counts,
                dev=dict(topk_idx=t(idx), topk_w=torch.from_numpy(np.ascontiguousarray(w)).to(dev), perm_src=t(order // k),
                         perm_pos=t(pos.reshape(T, k)), counts=t(counts),
                         offsets=t(np.concatenate([[0], np.cumsum(counts)]))))


@pytest.mark.parametrize("T,H,I", [(3, 256, 128), (40, 512, 256), (70, 384, 128), (600, 512, 256)])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_rows_that_cancel(L, T, H, I, bf16):
    """Two experts whose rows nearly cancel (the second's codes are the first's negated, its scales 1 + 2^-10 of them):
    the sum is 2^-10 of its rows and carries the error of fp32 rows, also where it is rounded to bf16 at its end."""
    a = ic.expert(H, I, 7, dev)
    a["q2"] = a["q2"].clamp(-127, 127)
    b = dict(a, q2=-a["q2"], s2=a["s2"] * (1 + 2.0 ** -10))
    experts = [a, b]
    slots, stride = pack(L, H, I, experts, range(2), 2)
    x, rt = tokens(T, H, T), routing(T, 2, 2, T)
    rt["w"][:] = 0.5
    rt["dev"]["topk_w"].fill_(0.5)
    out = run(L, x, rt, slots, stride, None, 2, H, I, torch.bfloat16 if bf16 else torch.float32)
    torch.cuda.synchronize()
    ic.check(np64(out), *expected(x, experts, rt, range(2), 2), f"cancelling rows T={T} {H}x{I}", bf16)


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_a_token_gives_the_same_in_every_batch(L, bf16):
    """The integer sums are exact and the fp32 steps behind them the same in the streaming and the tiled kernels, so a
    token's output does not depend, to the bit, on the batch it is in."""
    E, k, H, I = 8, 2, 512, 256
    dtype = torch.bfloat16 if bf16 else torch.float32
    experts = [ic.expert(H, I, e, dev) for e in range(E)]
    slots, stride = pack(L, H, I, experts, range(E), E)
    T = 700  # tiles of 128 rows; of 256 from 384 rows an expert on
    x, rt = tokens(T, H, 5), routing(T, E, k, 6)
    whole = run(L, x, rt, slots, stride, None, E, H, I, dtype)
    for n in (1, 12, 13, 40, 300):
        out = run(L, x[:n].contiguous(), grouped(rt["idx"][:n], rt["w"][:n], E), slots, stride, None, E, H, I, dtype)
        torch.cuda.synchronize()
        assert torch.equal(out, whole[:n]), f"{n} tokens"
    long = run(L, torch.cat([x] * 4), grouped(np.concatenate([rt["idx"]] * 4), np.concatenate([rt["w"]] * 4), E), slots,
               stride, None, E, H, I, dtype)
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(long[i * T:(i + 1) * T], whole), f"copy {i}"
