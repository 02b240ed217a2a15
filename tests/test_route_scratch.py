"""moe_route's scratch: its size is the plain route's, and scored gates stay inside it."""
import pytest
import torch

dev = "cuda"


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


@pytest.mark.parametrize("T,H,E,size", [(0, 64, 7, 512), (17, 512, 5, 6400), (300, 4096, 250, 2115840),
                                        (4096, 512, 1, 33792), (16385, 64, 1021, 70065408), (15694, 64, 1021, 64 << 20)])
def test_size_for_odd_numbers_of_experts(L, T, H, E, size):
    """What callers of moe_route hold: 12 bytes for each expert and 64 tokens behind the partial sums, whatever E is
    modulo 4. The last one is the longest batch that moe_route_noalloc's 64 MiB take at 1021 experts."""
    assert L.moe_route_workspace_size(T, H, E, 1) == size


def guarded(n):
    """n bytes of scratch and 4 KiB behind them that nothing may write."""
    t = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=dev)
    return t, t[:n]


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (3, 2), (5, 2), (101, 3), (1021, 2)])
@pytest.mark.parametrize("T", [17, 64, 65, 2000, 4096, 4097, 16384, 16385])
def test_scored_calls_stay_inside_their_scratch(L, T, E, k):
    """moe_route_scored and moe_select with scratch of exactly the size asked for, against each other."""
    H = 64
    g = torch.Generator(device=dev).manual_seed(T + E)
    x, W = torch.randn((T, H), generator=g, device=dev), torch.randn((H, E), generator=g, device=dev)
    gate = L.Gate(score="sigmoid", balance=0.1 * torch.randn(E, generator=g, device=dev))
    i32 = dict(dtype=torch.int32, device=dev)
    outs = [dict(topk_idx=torch.empty((T, k), **i32), topk_w=torch.empty((T, k), device=dev),
                 counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                 perm_src=torch.empty(T * k, **i32), perm_pos=torch.empty((T, k), **i32)) for _ in range(2)]
    args = lambda o: [o[n] for n in ("counts", "offsets", "perm_src", "perm_pos")]  # noqa: E731
    logits = torch.empty((T, E), device=dev)
    a, ws = guarded(L.moe_route_workspace_size(T, H, E, k))
    L.moe_route_scored(x, W, None, gate, k, outs[0]["topk_idx"], outs[0]["topk_w"], logits, *args(outs[0]), ws)
    b, ws2 = guarded(L.moe_select_workspace_size(T, E, k))
    L.moe_select(logits, gate, k, outs[1]["topk_idx"], outs[1]["topk_w"], *args(outs[1]), ws2)
    torch.cuda.synchronize()
    assert torch.all(a[len(ws):] == 0xA5) and torch.all(b[len(ws2):] == 0xA5)
    for n in outs[0]:
        assert torch.equal(outs[0][n], outs[1][n]), n
    assert int(outs[0]["counts"].sum()) == T * k
