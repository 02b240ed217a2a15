"""Refusals of the training operators: every call here is turned away before anything is launched (no GPU is needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from routed_expert_layer_amd import _lib
    return _lib


def caller(fn, names, base):
    return lambda **o: fn(*[dict(base, **o)[n] for n in names])


def refused(L, call, cases):
    for o in cases:
        assert call(**o) == L.MOE_EINVAL, o
        assert L.moe_last_error()


def test_group(L):
    names = ("i", "T", "k", "E", "c", "o", "s", "p", "ws", "n", "st")
    call = caller(L._lib.moe_group, names, dict(i=16, T=4, k=4, E=16, c=16, o=16, s=16, p=16, ws=None, n=0, st=None))
    refused(L, call, [dict(T=-1), dict(k=0), dict(k=17), dict(E=0), dict(E=1025), dict(T=1 << 30), dict(i=None),
                      dict(c=None), dict(o=None), dict(s=None), dict(p=None), dict(i=18), dict(c=17), dict(o=18),
                      dict(s=18), dict(p=18), dict(T=100000), dict(T=100000, ws=16, n=64)])
    need = L.moe_group_workspace_size(100000, 4, 16)
    assert need > 0 and call(T=100000, ws=18, n=need) == L.MOE_EINVAL
    assert L.moe_group_workspace_size(100000, 4, 1024) >= need and L.moe_group_workspace_size(1, 1, 1) == 0
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 17, 1), (1, 1, 0), (1, 1, 1025), (1 << 30, 2, 1)):
        assert L.moe_group_workspace_size(*bad) == 0


SIZES = [dict(T=-1), dict(k=0), dict(k=17), dict(T=1 << 24), dict(H=0), dict(H=(1 << 20) + 1), dict(n=-1), dict(dt=2),
         dict(dt=-1)]


def test_dispatch(L):
    names = ("x", "dt", "p", "T", "k", "H", "n", "out", "st")
    call = caller(L._lib.moe_dispatch, names, dict(x=16, dt=1, p=16, T=4, k=2, H=64, n=8, out=16, st=None))
    refused(L, call, SIZES + [dict(x=None), dict(p=None), dict(out=None), dict(x=17), dict(out=17), dict(p=18),
                              dict(dt=0, x=18), dict(dt=0, out=18)])
    assert call(T=0, x=None, p=None, out=None) == L.MOE_OK and call(n=0, out=None) == L.MOE_OK


def test_collect(L):
    names = ("r", "dt", "p", "w", "T", "k", "H", "n", "out", "odt", "st")
    call = caller(L._lib.moe_collect, names, dict(r=16, dt=1, p=16, w=16, T=4, k=2, H=64, n=8, out=16, odt=0, st=None))
    refused(L, call, SIZES + [dict(odt=2), dict(r=None), dict(p=None), dict(out=None), dict(r=17), dict(dt=0, r=18),
                              dict(out=18), dict(odt=1, out=17), dict(w=18), dict(p=18)])
    assert call(T=0, r=None, p=None, w=None, out=None) == L.MOE_OK


def test_collect_backward(L):
    names = ("d", "odt", "r", "dt", "p", "w", "T", "k", "H", "n", "dr", "dw", "st")
    call = caller(L._lib.moe_collect_backward, names, dict(d=16, odt=1, r=16, dt=1, p=16, w=16, T=4, k=2, H=64, n=8,
                                                           dr=16, dw=16, st=None))
    refused(L, call, SIZES + [dict(odt=2), dict(d=None), dict(r=None), dict(p=None), dict(dr=None, dw=None),
                              dict(d=17), dict(r=17), dict(dr=17), dict(dw=18), dict(w=18), dict(p=18),
                              dict(odt=0, d=18), dict(dt=0, dr=18)])
    assert call(T=0, d=None, r=None, p=None, w=None) == L.MOE_OK


def test_swiglu(L):
    names = ("g", "dt", "n", "nr", "I", "h", "c", "s", "st")
    save = caller(L._lib.moe_swiglu_save, names, dict(g=16, dt=1, n=4, nr=None, I=64, h=16, c=16, s=16, st=None))
    sizes = [dict(dt=2), dict(n=-1), dict(n=(1 << 27) + 1), dict(I=0), dict(I=(1 << 20) + 1),
             dict(n=1 << 30, I=1 << 20), dict(nr=18), dict(s=18), dict(s=None), dict(h=17)]
    refused(L, save, sizes + [dict(g=None), dict(h=None), dict(c=None), dict(g=17), dict(dt=0, g=18)])
    assert save(n=0, g=None, h=None, c=None, s=None) == L.MOE_OK
    names = ("c", "s", "d", "dt", "n", "nr", "I", "dg", "h", "st")
    back = caller(L._lib.moe_swiglu_backward, names, dict(c=16, s=16, d=16, dt=1, n=4, nr=None, I=64, dg=16, h=16,
                                                          st=None))
    refused(L, back, sizes + [dict(c=None), dict(d=None), dict(dg=None), dict(d=17), dict(dg=17), dict(dt=0, h=18)])
    assert back(n=0, c=None, s=None, d=None, dg=None) == L.MOE_OK


def test_matmul(L):
    names = ("a", "w", "c", "o", "E", "n", "K", "N", "t", "out", "odt", "st")
    call = caller(L._lib.moe_matmul_grouped, names, dict(a=16, w=16, c=16, o=16, E=4, n=8, K=64, N=64, t=0, out=16,
                                                         odt=1, st=None))
    sizes = [dict(E=0), dict(E=1025), dict(n=-1), dict(n=(1 << 30) + 1), dict(K=0), dict(K=4), dict(K=12), dict(N=0),
             dict(N=20), dict(K=65544), dict(N=65544), dict(K=65536, N=16392), dict(odt=2), dict(a=None), dict(c=None),
             dict(o=None), dict(out=None), dict(a=24), dict(out=24), dict(c=18), dict(o=18)]
    refused(L, call, sizes + [dict(w=None), dict(w=8)])
    assert call(n=0, a=None, w=None, out=None) == L.MOE_OK
    names = ("a", "d", "c", "o", "E", "n", "K", "N", "out", "odt", "st")
    call = caller(L._lib.moe_matmul_grouped_dw, names, dict(a=16, d=16, c=16, o=16, E=4, n=8, K=64, N=64, out=16,
                                                            odt=0, st=None))
    refused(L, call, sizes + [dict(d=None), dict(d=8), dict(n=0, out=None)])


def test_binding_refuses_host_tensors(L):
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    n = torch.zeros(8, dtype=torch.int32)
    for call in (lambda: L.moe_group(i, 4, n, n, n, i), lambda: L.moe_dispatch(f, i, f),
                 lambda: L.moe_collect(f, i, None, f), lambda: L.moe_collect_backward(f, f, i, None, f, f),
                 lambda: L.moe_swiglu_save(f, f, f, f), lambda: L.moe_swiglu_backward(f, f, f, f),
                 lambda: L.moe_matmul_grouped(f, f[None], n, n, f), lambda: L.moe_matmul_grouped_dw(f, f, n, n, f[None]),
                 lambda: L.moe_dispatch(f[0], i, f), lambda: L.moe_collect_backward(f, None, i, None, None, None),
                 lambda: L.moe_swiglu_save(f[:, :7], f, f, f), lambda: L.moe_matmul_grouped(f, f, n, n, f),
                 lambda: L.moe_matmul_grouped_dw(f, f, n, n, f)):
        with pytest.raises(ValueError):
            call()
