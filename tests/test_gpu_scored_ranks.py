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
def test_group_ranks_that_cancel(L, T, score):
    """Balances that pin one expert of a group and mask another: the group's two largest scores are near +B and -B, and
    their sum in 32 bits is off by up to 2^-24 B, far more than it is relative to itself."""
    g = torch.Generator(device=dev).manual_seed(T)
    for E, G, keep, k in ((16, 8, 4, 4), (64, 8, 3, 5), (256, 8, 4, 6)):
        if E * T > 2000000:  # the statement in Python takes a second for 3 million scores
            continue
        l = torch.randn((T, E), generator=g, device=dev)
        for B in (1e3, 1e5, 1e6):
            b = 0.1 * torch.randn(E, generator=g, device=dev)
            groups = b.view(G, E // G)
            groups[:, 0] += B
            groups[:, 1:] -= B
            run(L, l, k, f"{score} E{E} B{B:g}", score=score, n_group=G, topk_group=keep, group_top=2, balance=b)
        # one such group among ordinary ones, its rank near theirs
        b = 0.1 * torch.randn(E, generator=g, device=dev)
        groups = b.view(G, E // G)
        groups[2, 0] += 1e6
        groups[2, 1:] -= 1e6
        run(L, l, k, f"{score} E{E} one group", score=score, n_group=G, topk_group=keep, group_top=2, balance=b)


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


@pytest.mark.parametrize("T,E", [(64, 64), (5000, 64), (5000, 256), (16384, 64), (16400, 64), (16400, 256)])
def test_near_ties_in_long_batches(L, T, E):
    """Biased scores of every token within about 2^-24 of one value, so that 32 bits decide next to no token and several
    of a wave go through 64 bits, one after another."""
    g = torch.Generator(device=dev).manual_seed(T + E)
    l0 = torch.randn(E, generator=g, device=dev)
    b = (0.75 - 1.0 / (1.0 + torch.exp(-l0.double()))).float()
    l = l0 + 1e-6 * torch.randn((T, E), generator=g, device=dev)
    for G, keep, top in ((1, 1, 1), (8, 3, 2)) if T * E < 2000000 else ((8, 3, 2),):
        run(L, l, 6, f"near ties g{G}", score="sigmoid", n_group=G, topk_group=keep, group_top=top, balance=b)


@pytest.mark.parametrize("T", SIZES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_nan_logits_that_are_chosen(L, T, score):
    """A NaN logit counts as -inf: with a finite balance its expert has a finite biased score and can be chosen, always
    where every expert of the kept groups is."""
    g = torch.Generator().manual_seed(T + 2)
    for E, G, keep, k in ((1, 1, 1, 1), (2, 1, 1, 2), (16, 1, 1, 16), (16, 4, 2, 8), (12, 4, 3, 4), (64, 8, 2, 16)):
        l = torch.randn((T, E), generator=g)
        l[torch.rand((T, E), generator=g) < 0.3] = float("nan")
        l[0] = float("nan")
        b = torch.randn(E, generator=g)
        b[0] += 1.0
        for top in (1, 2):
            run(L, l.to(dev), k, f"{score} E{E} k{k} top{top}", score=score, n_group=G, topk_group=keep, group_top=top,
                balance=b.to(dev))


@pytest.mark.parametrize("T,E", [(1, 8), (9, 8), (16, 64), (40, 8), (100, 64)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_scored_with_nan_logits(L, T, E, score):
    """The same from x and Wr: experts whose bias is a NaN have NaN logits, and a balance that chooses them."""
    from routed_expert_layer_amd.runtime import RouteBuffers
    H, k = 256, 8
    g = torch.Generator().manual_seed(E)
    x, W = torch.randn((T, H), generator=g).to(dev), torch.randn((H, E), generator=g).to(dev)
    bias, b = torch.zeros(E), 0.1 * torch.randn(E, generator=g)
    bias[1::3] = float("nan")
    b[1::3] += 3.0
    kw = dict(score=score, balance=b.to(dev), scale=2.0)
    rb = RouteBuffers(T, H, E, k, dev, keep_logits=True)
    rb.topk_idx.zero_()
    rb.perm_src.fill_(-7)
    rb.route(x, W, bias.to(dev), gate=L.Gate(**kw))
    torch.cuda.synchronize()
    assert torch.isnan(rb.logits[:, 1::3]).all()
    o = dict(topk_idx=rb.topk_idx, topk_w=rb.topk_w, counts=rb.counts, offsets=rb.offsets, perm_src=rb.perm_src,
             perm_pos=rb.perm_pos)
    check(o, rb.logits, k, f"route T={T} E={E} {score}", **kw)
