"""Resizing the cache of a decoder of int8 experts."""
import numpy as np
import pytest
import torch

import oracle
from tests import int8_cases as ic
from tests.parity import np64, npi
from tests.test_gpu_int8 import expected, int8_config
from workloads import gen

pytestmark = pytest.mark.gpu
dev = "cuda"


@pytest.mark.parametrize("kind", ["host", "device"])
def test_resize_refuses_unaligned_slots(kind):
    """A slot buffer off 16 bytes is refused before the cache changes; steps go on from the old slots, and a resize to an
    aligned buffer follows."""
    from routed_expert_layer_amd import _lib as L
    from routed_expert_layer_amd.runtime import DecodeLayer, DeviceDecodeLayer, ExpertStore
    cfg = int8_config(L=1, S=8)
    E, H, I, k, T = cfg.E, cfg.H, cfg.I, cfg.k, cfg.T
    store = ExpertStore(1, E, H, I, "int8")
    try:
        ex = [ic.expert(H, I, e, dev) for e in range(E)]
        store.pack_layer(0, lambda e: ex[e], device=dev)
        host = kind == "host"
        dl = (DecodeLayer if host else DeviceDecodeLayer)(store, cfg.S, T, k, "bf16", dev, keep_logits=True)
        W = gen.router_weight(cfg, 0, dev)

        def step(i):
            x, b = gen.tokens(cfg, i, 0, dev), gen.router_bias(cfg, 0, i, dev)
            out = dl.step(i, 0, x, W, b) if host else dl.step(0, x, W, b)
            torch.cuda.synchronize()
            l64 = np64(dl.rb.logits)
            idx = npi(dl.rb.topk_idx)
            assert np.array_equal(idx, oracle.topk_select(l64, k))
            counts, off, pos, src = oracle.permute(idx, E)
            rt = dict(idx=idx, w=oracle.topk_weights(l64, idx), counts=counts, offsets=off, pos=pos, src=src)
            ref, tol = expected(x, ex, rt, range(E), E)
            # moe_route's weights carry fp32 exponentials: 1e-5, as the routing tests allow
            ic.check(np64(out), ref, tol + 1e-5 * k * np.abs(ref).max(), f"{kind} step {i}")

        for i in range(3):
            step(i)
        new = torch.empty(13 * store.stride + 16, dtype=torch.uint8, device=dev)
        resize = L.moe_decoder_resize if host else L.moe_device_decoder_resize
        for n in (8, 7, 12):
            with pytest.raises(L.MoEError, match="16-byte") as ei:
                resize(dl.dec, n, new[8:], torch.cuda.current_stream())
            assert ei.value.code == L.MOE_EINVAL
        for i in range(3, 6):
            step(i)
        dl.resize(12)
        for i in range(6, 9):
            step(i)
    finally:
        store.close()
