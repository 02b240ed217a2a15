"""Refusals of moe_select, moe_route_scored, moe_experts and the int8 format: every call here is turned away before
anything is launched (no GPU is needed)."""
import ctypes

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def gate(L, **kw):
    return L.Gate(**dict(dict(score="sigmoid", n_group=4, topk_group=2, group_top=2), **kw))


BAD_GATES = [dict(score=2), dict(score=-1), dict(n_group=0), dict(n_group=3), dict(n_group=16, topk_group=17),
             dict(topk_group=0), dict(topk_group=5), dict(group_top=0), dict(group_top=3), dict(scale=float("inf")),
             dict(scale=float("nan")), dict(n_group=8, topk_group=1)]


@pytest.mark.parametrize("kw", BAD_GATES, ids=lambda d: "-".join(f"{k}={v}" for k, v in d.items()))
def test_bad_gates(L, kw):
    E, k, ws = 16, 4, 1 << 20
    g = ctypes.byref(gate(L, **kw))
    assert L._lib.moe_select(16, g, 4, E, k, 16, 16, 16, 16, 16, 16, 16, ws, None) == L.MOE_EINVAL
    assert L.moe_last_error().startswith("moe_select: ")
    assert L._lib.moe_route_scored(16, 1, 16, None, g, 4, 64, E, k, 16, 16, None, 16, 16, 16, 16, 16, ws, None) \
        == L.MOE_EINVAL
    assert L._lib.moe_prefill_layer_scored(16, 1, 16, None, g, 4, 256, E, k, 256, L.MOE_W_BF16, 16, 1 << 20,
                                           ctypes.byref(L.DecoderBuffers()), 16, 1, None) == L.MOE_EINVAL


def test_select_refusals(L):
    g = ctypes.byref(gate(L))
    call = lambda **o: L._lib.moe_select(*[dict(dict(  # noqa: E731
        l=16, g=g, T=4, E=16, k=4, i=16, w=16, c=16, o=16, s=16, p=16, ws=16, n=1 << 20, st=None), **o)[n]
        for n in ("l", "g", "T", "E", "k", "i", "w", "c", "o", "s", "p", "ws", "n", "st")])
    for o in (dict(g=None), dict(T=-1), dict(E=0), dict(E=1028), dict(k=0), dict(k=17, E=64), dict(k=17), dict(l=None),
              dict(i=None), dict(w=None), dict(c=None), dict(o=None), dict(s=None), dict(p=None), dict(ws=None),
              dict(ws=8), dict(n=16), dict(T=1 << 30)):
        assert call(**o) == L.MOE_EINVAL, o
    assert L.moe_select_workspace_size(-1, 16, 4) == 0 and L.moe_select_workspace_size(4, 1025, 4) == 0
    assert L.moe_select_workspace_size(65, 256, 8) >= 2 * 256 * 12


def test_experts_refusals(L):
    H, I, T, k, E = 256, 128, 4, 2, 8
    need = L.moe_experts_workspace_size(T, k, E, H, I, L.MOE_W_INT8)
    blob = L.moe_expert_bytes(L.MOE_W_INT8, H, I)
    names = ("x", "dt", "i", "w", "s", "p", "c", "o", "so", "T", "k", "E", "n", "b", "st", "f", "H", "I", "out", "odt",
             "ws", "wn", "stream")
    base = dict(x=16, dt=L.MOE_DT_BF16, i=16, w=16, s=16, p=16, c=16, o=16, so=None, T=T, k=k, E=E, n=E, b=16, st=blob,
                f=L.MOE_W_INT8, H=H, I=I, out=16, odt=L.MOE_DT_BF16, ws=16, wn=need, stream=None)
    call = lambda **o: L._lib.moe_experts(*[dict(base, **o)[n] for n in names])  # noqa: E731
    for o in (dict(x=None), dict(x=8), dict(dt=L.MOE_DT_F32), dict(i=None), dict(w=None), dict(s=None), dict(p=None),
              dict(c=None), dict(o=None), dict(T=-1), dict(k=0), dict(k=9), dict(E=0), dict(E=1025), dict(n=0),
              dict(n=E - 1), dict(b=None), dict(b=8), dict(st=blob - 16), dict(st=blob + 8), dict(f=L.MOE_W_BF16),
              dict(H=100), dict(I=100), dict(H=16448), dict(I=8256), dict(out=None), dict(out=8), dict(odt=2),
              dict(ws=None), dict(ws=8), dict(wn=need - 1), dict(T=1 << 21, H=4096, wn=1 << 60, st=1 << 30)):
        assert call(**o) == L.MOE_EINVAL, o
        assert L.moe_last_error().startswith("moe_experts: ")
    assert call(T=0) == L.MOE_OK  # nothing to do
    assert L.moe_experts_workspace_size(T, k, E, H, I, L.MOE_W_INT4) == 0
    assert L.moe_experts_workspace_size(T, k, E, 100, I, L.MOE_W_INT8) == 0


def test_int8_format_refusals(L):
    f = L.MOE_W_INT8
    least = 3 * 4096 * 2048 + 4 * (2 * 2048 + 4096 + 1)  # codes, scales and one word more
    assert least <= L.moe_expert_bytes(f, 4096, 2048) < least + 4 * 256
    for H, I in ((32, 64), (64, 32), (16448, 64), (64, 8256), (0, 64)):
        assert L.moe_expert_bytes(f, H, I) == 0
    lib = L._lib
    assert lib.moe_pack_expert(f, 64, 64, 16, 16, 16, None, 16, 16, 16, None) == L.MOE_EINVAL
    assert lib.moe_pack_expert(f, 64, 64, 16, 16, 16, 16, 16, 16, 8, None) == L.MOE_EINVAL
    w = np.array([[0, 0, 0, 1]], np.int32)
    ok = dict(x=16, dt=L.MOE_DT_BF16, y=16, b=16, st=1 << 20, H=256, I=128, mode=0)
    call = lambda **o: (lambda a: lib.moe_ffn(  # noqa: E731
        a["x"], a["dt"], 16, w.ctypes.data, 1, a["b"], a["st"], f, a["H"], a["I"], a["y"], 16, 1 << 30, a["mode"],
        None))(dict(ok, **o))
    for o in (dict(dt=L.MOE_DT_F32), dict(x=8), dict(y=8), dict(b=8), dict(st=(1 << 20) + 8), dict(st=1024), dict(H=96),
              dict(H=320, mode=L.MOE_FFN_PREFILL), dict(I=192, mode=L.MOE_FFN_PREFILL)):
        assert call(**o) == L.MOE_EINVAL, o
    # the host's expert kernel and the grouped call name the formats that they take
    x = np.zeros((1, 64), np.uint16)
    y = np.zeros((1, 64), np.float32)
    assert lib.moe_cpu_ffn(16, f, 64, 64, x.ctypes.data, 1, y.ctypes.data, 1) == L.MOE_EINVAL
    assert lib.moe_ffn_grouped(16, L.MOE_DT_BF16, 16, 16, 16, None, 4, 4, 8, 16, 1 << 20, f, 256, 128, 16, 16, 1 << 30,
                               None) == L.MOE_EINVAL
    # a decoder of int8 experts needs bf16 activations
    c = L.MoeCache(1, 8, 4)
    st = ctypes.c_int(0)
    b = L.DecoderBuffers(*([16] * 9), 1 << 30, 16, 1 << 30)
    lp = L.layer_table([4096])
    assert not lib.moe_decoder_create(c.h, 1, 256, 128, 8, 2, L.MOE_DT_F32, f, lp.ctypes.data, 1 << 20, 16, 1 << 20,
                                      ctypes.byref(b), ctypes.byref(st))
    assert st.value == L.MOE_EINVAL and "bf16" in L.moe_last_error()
    assert lib.moe_decoder_set_gate(None, None) == L.MOE_EINVAL
    assert lib.moe_device_decoder_set_gate(None, None) == L.MOE_EINVAL


def test_binding_checks_types(L):
    """The binding refuses wrong element types, sizes and host tensors before the call."""
    with pytest.raises(ValueError):
        L.Gate(score="relu")
    with pytest.raises(ValueError):
        L.Gate(balance=torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        L.Gate(balance=torch.zeros(8))  # a host tensor
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    out = [i(4, 2), torch.zeros(4, 2), i(8), i(9), i(8), i(4, 2)]
    for n, bad in ((0, i(4, 3)), (1, torch.zeros(4, 2, dtype=torch.float64)), (2, i(7)), (3, i(8)), (4, i(7)),
                   (5, i(4, 2).long())):
        args = list(out)
        args[n] = bad
        with pytest.raises(ValueError):
            L.moe_select(torch.zeros(4, 8), L.Gate(), 2, *args, torch.zeros(1 << 16, dtype=torch.uint8), stream=0)
