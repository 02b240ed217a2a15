"""Calls of no tokens, at every number of experts that the routing's paths divide at."""
import pytest
import torch

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


@pytest.mark.parametrize("E", [1, 256, 512, 513, 1000, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_no_tokens_write_empty_groups(L, E, dtype):
    """moe_route, moe_route_noalloc, moe_route_scored and moe_select with T = 0 write counts = offsets = 0, and the next
    call of each works."""
    H = 64
    i32 = dict(dtype=torch.int32, device=dev)
    W = torch.randn((H, E), device=dev).to(dtype)
    gate = L.Gate(score="sigmoid")
    for T in (0, 3, 0, 70):
        x = torch.randn((T, H), device=dev).to(dtype)
        logits = torch.randn((T, E), device=dev)
        ws = torch.empty(max(L.moe_route_workspace_size(T, H, E, 1), L.moe_select_workspace_size(T, E, 1)),
                         dtype=torch.uint8, device=dev)
        out = lambda: [torch.full((T, 1), -7, **i32), torch.full((T, 1), -7.0, device=dev)]  # noqa: E731
        rest = lambda: [torch.full((E,), -7, **i32), torch.full((E + 1,), -7, **i32),  # noqa: E731
                        torch.full((T + 1,), -7, **i32), torch.full((T, 1), -7, **i32)]
        for call in (lambda o, r: L.moe_route(x, W, None, 1, *o, None, *r, ws),
                     lambda o, r: L.moe_route_noalloc(x, W, None, 1, *o, None, *r),
                     lambda o, r: L.moe_route_scored(x, W, None, gate, 1, *o, None, *r, ws),
                     lambda o, r: L.moe_select(logits, gate, 1, *o, *r, ws)):
            o, r = out(), rest()
            call(o, r)
            torch.cuda.synchronize()
            counts, offsets, src, pos = r
            assert int(counts.sum()) == T and int(offsets[0]) == 0 and int(offsets[E]) == T
            assert torch.equal(offsets[1:], counts.cumsum(0).int())
            assert int(src[T]) == -7
            if T:
                assert torch.equal(counts, torch.bincount(o[0].reshape(-1), minlength=E).int())
