"""Scored gates where 32-bit scores decide least, in every form of the kernels."""
import pytest
import torch

from tests.test_gpu_scored import check, select

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def run(L, l, k, what, **kw):
    o = select(L, l, L.Gate(**kw), k)
    torch.cuda.synchronize()
    check(o, l, k, what, **kw)


# one block with a wave and with a row of lanes a token; two launches with each; three launches
SIZES = [10, 16, 48, 64, 300, 5000, 16400]


@pytest.mark.parametrize("T", SIZES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_infinite_logits_in_groups_that_are_dropped(L, T, score):
    """With the two best ranking a group, one infinite logit (a score of 1) does not keep it: its expert is not chosen,
    and the others' choice is as without it."""
    g = torch.Generator().manual_seed(T + 1)
    for E, G, keep in ((16, 8, 4), (64, 8, 3), (100, 4, 2)):
        per, t = E // G, torch.arange(T)
        x = (torch.randn((T, E), generator=g) - 1.0).view(T, G, per)
        x[t, (t + 1) % G, 1:] = -6.0
        x[t, (t + 1) % G, 0] = float("inf")
        q = t[::3]
        x[q, (q + 3) % G, :per - 1] = -7.0
        x[q, (q + 3) % G, per - 1] = float("inf")
        x[t, (t + 2) % G] += 4.0
        q = t[::2]
        x[q, q % G] += 3.0
        l = x.view(T, E).to(dev)
        for k in (1, 3, 4, 6) if T < 16384 else (4,):
            if k <= keep * per:
                for top in (2, 1):
                    run(L, l, k, f"{score} E{E} k{k} top{top}", score=score, n_group=G, topk_group=keep, group_top=top)
