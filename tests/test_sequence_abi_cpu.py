"""Layer norm, causal convolution and selective scan on the CPU: descriptors, workspace sizes and
every refusal, by status, before any device work (the addresses are never dereferenced)."""
import ctypes as C

import pytest

import convolution_layer_amd as cm

INV, UNS, WS, MIS = cm.ERR_INVALID_ARG, cm.ERR_UNSUPPORTED, cm.ERR_WORKSPACE, cm.ERR_MISALIGNED


def B(i):
    return 0x7F0000000000 + i * 0x1000000  # fake device addresses, far apart


def status(fn, *args):
    s = fn(*args)
    if s != cm.OK:
        assert cm.lib.convmi_last_error().decode()
    return s


# ------------------------------------------------------------------ layer norm
def norm(**kw):
    return cm.make_layer_norm_desc(kw.get("rows", 4), kw.get("cols", 64), dtype=kw.get("dtype", 1),
                                   eps=kw.get("eps", 1e-5))


@pytest.mark.parametrize("kw,want", [(dict(rows=-1), INV), (dict(cols=0), INV), (dict(dtype=5), INV),
                                     (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
                                     (dict(cols=(1 << 24) + 1), UNS), (dict(rows=1 << 32, cols=1 << 10), UNS)])
def test_layer_norm_descriptors(kw, want):
    d, n = norm(**kw), C.c_size_t()
    assert status(cm.lib.layer_norm_workspace_size, C.byref(d), C.byref(n)) == want
    assert status(cm.lib.layer_norm_forward, C.byref(d), *[B(i) for i in range(10)], None) == want
    assert status(cm.lib.layer_norm_backward, C.byref(d), *[B(i) for i in range(9)], 0, B(11), 1 << 30, None) == want


def test_layer_norm_forward_refusals():
    d = norm()

    def call(x=B(0), res=B(1), gamma=B(2), beta=B(3), h=B(4), y=B(5), y8=B(6), sc=B(7), mean=B(8), inv=B(9)):
        return status(cm.lib.layer_norm_forward, C.byref(d), x, res, gamma, beta, h, y, y8, sc, mean, inv, None)

    assert call(x=None) == INV and call(gamma=None) == INV
    assert call(y=None, y8=None, sc=None) == INV
    assert call(y8=None) == INV and call(sc=None) == INV
    for k in ("x", "res", "h", "y", "y8", "sc"):
        assert call(**{k: B(12) + 4}) == MIS
    for k in ("gamma", "beta", "mean", "inv"):
        assert call(**{k: B(12) + 2}) == MIS
    for out in ("y", "y8", "sc", "mean", "inv"):
        for i in range(4):
            assert call(**{out: B(i)}) == INV, (out, i)
    assert call(h=B(0) + 16) == INV and call(h=B(1) + 32) == INV and call(h=B(2)) == INV
    assert call(y=B(4)) == INV and call(y8=B(5)) == INV and call(mean=B(7)) == INV and call(inv=B(8)) == INV
    assert status(cm.lib.layer_norm_forward, None, *[B(i) for i in range(10)], None) == INV


def test_layer_norm_backward_refusals():
    d = norm()
    need = cm.layer_norm_workspace_size(d)
    assert need > 0

    def call(h=B(0), gamma=B(1), mean=B(2), inv=B(3), dy=B(4), dh=B(5), dx=B(6), dg=B(7), db=B(8), acc=0, ws=B(9),
             n=need):
        return status(cm.lib.layer_norm_backward, C.byref(d), h, gamma, mean, inv, dy, dh, dx, dg, db, acc, ws, n, None)

    for k in ("h", "gamma", "mean", "inv", "dy", "dx"):
        assert call(**{k: None}) == INV
    assert call(acc=2) == INV
    assert call(dx=B(4) + 16) == INV and call(dx=B(5) + 16) == INV
    for i in (0, 1, 2, 3):
        assert call(dx=B(i)) == INV
    for out in ("dg", "db"):
        for i in range(7):
            assert call(**{out: B(i)}) == INV
    assert call(db=B(7)) == INV
    for kw in ({}, dict(dg=None), dict(db=None)):
        assert call(ws=None, **kw) == WS and call(n=need - 1, **kw) == WS and call(ws=B(9) + 16, **kw) == MIS
    assert call(dx=B(6) + 2) == MIS and call(dg=B(7) + 2) == MIS and call(db=B(8) + 2) == MIS
