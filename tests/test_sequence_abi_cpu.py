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


# ------------------------------------------------------------------ causal convolution
def conv(**kw):
    d = cm.make_causal_conv_desc(8, 64, 4, batch=2, dtype=1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def conv_calls(d):
    """Every entry point on one descriptor."""
    n = C.c_size_t()
    r = C.byref(d)
    return [status(cm.lib.causal_conv_workspace_size, r, C.byref(n)),
            status(cm.lib.causal_conv_forward, r, *[B(i) for i in range(7)], None),
            status(cm.lib.causal_conv_backward, r, *[B(i) for i in range(11)], 0, B(12), 1 << 30, None),
            status(cm.lib.causal_conv_step, r, B(0), B(1), B(2), B(3), 1 << 20, B(4), B(5), None)]


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(channels=0), INV), (dict(batch=-1), INV), (dict(batch=0), INV), (dict(taps=0), INV),
    (dict(taps=9), INV), (dict(activation=6), INV), (dict(activation=-1), INV), (dict(dtype=2), INV),
    (dict(x_pitch=63), INV), (dict(x_pitch=-1), INV), (dict(rows=(1 << 30) + 1), UNS), (dict(channels=(1 << 24) + 1), UNS),
    (dict(batch=(1 << 24) + 1), UNS), (dict(rows=1 << 20, x_pitch=1 << 21), UNS), (dict(rows=0, x_pitch=1 << 41), UNS),
    (dict(rows=1 << 20, channels=1 << 21), UNS), (dict(rows=0, batch=1 << 24, channels=1 << 20), UNS)])
def test_conv_descriptors(kw, want):
    assert conv_calls(conv(**kw)) == [want] * 4
    assert status(cm.lib.causal_conv_forward, None, *[B(i) for i in range(7)], None) == INV


def test_conv_forward_refusals():
    def call(d=conv(), x=B(0), st=None, w=B(1), b=B(2), i=B(3), y=B(4), f=B(5)):
        return status(cm.lib.causal_conv_forward, C.byref(d), x, st, w, b, i, y, f, None)

    assert call(x=None) == INV and call(w=None) == INV and call(y=None) == INV
    assert call(x=B(9) + 1) == MIS and call(st=B(9) + 2) == MIS and call(b=B(9) + 2) == MIS
    for k in ("w", "y", "i", "f"):
        assert call(**{k: B(9) + 8}) == MIS
    for out in ("y", "f"):
        for a in ("x", "w", "b"):
            assert call(**{out: B(8), a: B(8)}) == INV
        assert call(**{out: B(8), "st": B(8)}) == INV
    assert call(y=B(3)) == INV and call(y=B(5)) == INV and call(f=B(3) + 16) == INV
    assert call(d=conv(rows=9)) == INV  # not of equal length, and no starts


def test_conv_backward_refusals():
    d = conv()
    need = cm.causal_conv_workspace_size(d)
    assert need > 0 and cm.causal_conv_workspace_size(conv(rows=0)) == 0

    def call(d=d, x=B(0), st=None, w=B(1), b=B(2), i=B(3), dy=B(4), df=B(5), dx=B(6), di=B(7), dw=B(8), db=B(9), acc=0,
             ws=B(10), n=need):
        return status(cm.lib.causal_conv_backward, C.byref(d), x, st, w, b, i, dy, df, dx, di, dw, db, acc, ws, n, None)

    for k in ("x", "w", "dy", "dx"):
        assert call(**{k: None}) == INV
    assert call(acc=2) == INV and call(d=conv(rows=9)) == INV
    assert call(x=B(11) + 1) == MIS and call(dx=B(11) + 1) == MIS
    for k in ("w", "dy", "i", "df", "di", "dw"):
        assert call(**{k: B(11) + 8}) == MIS
    assert call(db=B(11) + 2) == MIS and call(b=B(11) + 2) == MIS
    for out in ("dx", "di", "dw", "db"):
        for i in range(6):
            assert call(**{out: B(i)}) == INV, (out, i)
    assert call(di=B(6)) == INV and call(dw=B(7)) == INV and call(db=B(8)) == INV
    for kw in ({}, dict(dw=None), dict(db=None)):
        assert call(ws=None, **kw) == WS and call(n=need - 1, **kw) == WS and call(ws=B(10) + 16, **kw) == MIS
    # columns of one matrix: side by side they are apart, one column further they meet
    p = conv(x_pitch=128)
    assert call(d=p, x=B(0), dx=B(0) + 2 * 63, ws=None) == INV
    assert call(d=p, x=B(0), dx=B(0) + 2 * 64, ws=None) == WS
    assert call(d=p, x=B(0) + 2 * 64, dx=B(0), ws=None) == WS
    assert call(d=p, x=B(0), dx=B(0) + 2 * 65, ws=None) == INV


def test_conv_step_refusals():
    def call(d=conv(), x=B(0), w=B(1), b=B(2), s=B(3), n=8, sl=B(4), y=B(5)):
        return status(cm.lib.causal_conv_step, C.byref(d), x, w, b, s, n, sl, y, None)

    for k in ("x", "w", "s", "y"):
        assert call(**{k: None}) == INV
    assert call(n=-1) == INV and call(n=7, sl=None) == INV and call(n=1 << 31) == UNS
    assert call(d=conv(rows=(1 << 16) + 1)) == UNS
    assert call(x=B(9) + 1) == MIS and call(sl=B(9) + 2) == MIS and call(b=B(9) + 1) == MIS
    for k in ("w", "s", "y"):
        assert call(**{k: B(9) + 8}) == MIS
    for out in ("s", "y"):
        for a in ("x", "w", "b", "sl"):
            assert call(**{out: B(8), a: B(8)}) == INV
    assert call(y=B(3) + 16) == INV


def test_silu_is_the_causal_convolutions_only():
    d = cm.make_linear_desc(4, 8, 8, activation=cm.ACT_SILU)
    n = C.c_size_t()
    assert status(cm.lib.linear_workspace_size, C.byref(d), 0, C.byref(n)) == INV
    c = cm.make_desc(1, 4, 4, 3, 3, 1, 1, activation=cm.ACT_SILU)
    assert status(cm.lib.convmi_workspace_size, C.byref(c), 0, C.byref(n)) == INV


# ------------------------------------------------------------------ selective scan
def scan(**kw):
    d = cm.make_scan_desc(8, 64, 16, batch=2, groups=2, dtype=1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BIG = 1 << 45


def scan_calls(d):
    n, r = C.c_size_t(), C.byref(d)
    return [status(cm.lib.selective_scan_workspace_size, r, 0, C.byref(n)),
            status(cm.lib.selective_scan_workspace_size, r, 1, C.byref(n)),
            status(cm.lib.selective_scan_saved_size, r, C.byref(n)),
            status(cm.lib.selective_scan_forward, r, *[B(i) for i in range(13)], B(20), BIG, None),
            status(cm.lib.selective_scan_backward, r, *[B(i) for i in range(21)], 0, B(22), BIG, None),
            status(cm.lib.selective_scan_step, r, *[B(i) for i in range(9)], 1 << 20, B(9), B(10), None)]


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(channels=0), INV), (dict(batch=-1), INV), (dict(batch=0), INV), (dict(states=0), INV),
    (dict(states=65), INV), (dict(groups=0), INV), (dict(groups=3), INV), (dict(dtype=2), INV), (dict(delta_softplus=2), INV),
    (dict(x_pitch=63), INV), (dict(dt_pitch=-1), INV), (dict(z_pitch=1), INV), (dict(bc_pitch=31), INV),
    (dict(rows=(1 << 30) + 1), UNS), (dict(channels=(1 << 24) + 2), UNS), (dict(batch=(1 << 24) + 1), UNS),
    (dict(rows=1 << 20, x_pitch=1 << 21), UNS), (dict(rows=0, batch=1 << 20, channels=1 << 20), UNS),
    (dict(rows=1 << 28, channels=1 << 10, groups=1 << 10, batch=1 << 24), UNS)])
def test_scan_descriptors(kw, want):
    assert scan_calls(scan(**kw)) == [want] * 6
    assert status(cm.lib.selective_scan_saved_size, C.byref(scan()), None) == INV
    assert status(cm.lib.selective_scan_workspace_size, C.byref(scan()), 2, C.byref(C.c_size_t())) == INV


def refuse(call, need, misaligned16, misaligned4, outs, ins):
    for k in need:
        assert call(**{k: None}) == INV, k
    for k in misaligned16:
        assert call(**{k: B(40) + 8}) == MIS, k
    for k in misaligned4:
        assert call(**{k: B(40) + 2}) == MIS, k
    for o in outs:
        for i in ins:
            assert call(**{o: B(41), i: B(41)}) == INV, (o, i)
        for p in outs:
            if p != o:
                assert call(**{o: B(41), p: B(41)}) == INV, (o, p)


SCAN_IN = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")


def test_scan_forward_refusals():
    need = cm.scan_workspace_size(scan(), cm.SCAN_FORWARD)

    def call(d=scan(), ws=B(30), n=None, **kw):
        names = SCAN_IN + ("st", "init", "y", "final", "saved")
        p = {k: B(i) for i, k in enumerate(names)} | {"st": None} | kw
        return status(cm.lib.selective_scan_forward, C.byref(d), *[p[k] for k in names], ws, BIG if n is None else n, None)

    refuse(call, ("x", "dt", "A", "B", "C", "y"), ("init", "y", "final", "saved"), ("dt_bias", "A", "D", "st"),
           ("y", "final", "saved"), SCAN_IN + ("st",))
    for k in ("x", "dt", "B", "C", "z"):
        assert call(**{k: B(40) + 1}) == MIS
    assert call(y=B(9)) == INV and call(saved=B(9)) == INV and call(final=B(9) + 16) == INV
    assert call(d=scan(rows=9)) == INV
    if need:
        assert call(ws=None) == WS and call(n=need - 1) == WS and call(ws=B(30) + 16) == MIS


def test_scan_backward_refusals():
    need = cm.scan_workspace_size(scan(), cm.SCAN_BACKWARD)
    assert need > 0

    def call(d=scan(), ws=B(30), n=need, acc=0, **kw):
        names = SCAN_IN + ("st", "saved", "dy", "df", "dx", "ddt", "dB", "dC", "dz", "db", "dA", "dD", "di")
        p = {k: B(i) for i, k in enumerate(names)} | {"st": None} | kw
        return status(cm.lib.selective_scan_backward, C.byref(d), *[p[k] for k in names], acc, ws, n, None)

    refuse(call, ("x", "dt", "A", "B", "C", "saved", "dy", "dx", "ddt", "dB", "dC", "dz"), ("saved", "dy", "df", "di"),
           ("dt_bias", "A", "D", "st", "db", "dA", "dD"), ("dx", "ddt", "dB", "dC", "dz", "db", "dA", "dD", "di"),
           SCAN_IN + ("st", "saved", "dy", "df"))
    for k in ("x", "dt", "B", "C", "z", "dx", "ddt", "dB", "dC", "dz"):
        assert call(**{k: B(40) + 1}) == MIS
    assert call(z=None) == INV and call(z=None, dz=None, ws=None) == WS
    assert call(acc=2) == INV and call(d=scan(rows=9)) == INV
    assert call(ws=None) == WS and call(n=need - 1) == WS and call(ws=B(30) + 16) == MIS
    # dB and dC as columns of one matrix
    p = scan(bc_pitch=64)
    assert call(d=p, dB=B(40), dC=B(40) + 2 * 32, ws=None) == WS
    assert call(d=p, dB=B(40), dC=B(40) + 2 * 31, ws=None) == INV
    assert call(d=p, dC=B(40), dB=B(40) + 2 * 33, ws=None) == INV


def test_scan_step_refusals():
    def call(d=scan(), n=8, **kw):
        names = SCAN_IN + ("s",)
        p = {k: B(i) for i, k in enumerate(names + ("sl", "y"))} | kw
        return status(cm.lib.selective_scan_step, C.byref(d), *[p[k] for k in names], n, p["sl"], p["y"], None)

    refuse(call, ("x", "dt", "A", "B", "C", "s", "y"), ("s", "y"), ("dt_bias", "A", "D", "sl"), ("s", "y"),
           SCAN_IN + ("sl",))
    assert call(n=-1) == INV and call(n=7, sl=None) == INV and call(n=1 << 31) == UNS
    assert call(d=scan(rows=(1 << 16) + 1)) == UNS


def test_scan_sizes():
    """Kept states: one every 16 rows (32 for 17 to 32 states) and one more a sequence."""
    for rows, batch, ch, N, seg in ((100, 3, 8, 16, 16), (64, 1, 5, 33, 16), (31, 2, 4, 1, 16), (99, 2, 4, 17, 32)):
        d = cm.make_scan_desc(rows, ch, N, batch=batch)
        assert cm.scan_saved_size(d) == (rows // seg + batch) * ch * N * 4
    # whole sequences in one pass need no workspace in the forward
    assert cm.scan_workspace_size(cm.make_scan_desc(64, 64, 16, batch=64), cm.SCAN_FORWARD) == 0


def test_launches_count_their_threads_in_32_bits():
    n = C.c_size_t()
    size = lambda d: status(cm.lib.causal_conv_workspace_size, C.byref(d), C.byref(n))  # noqa: E731
    assert size(conv(rows=0, batch=(1 << 24) - 2)) == 0 and size(conv(rows=0, batch=1 << 24)) == UNS
    step = lambda d: status(cm.lib.causal_conv_step, C.byref(d), B(0), B(1), B(2), B(3), 1 << 30, None, B(4), None)  # noqa: E731
    assert step(conv(rows=1 << 24, batch=1, channels=1)) == UNS
    size = lambda d: status(cm.lib.selective_scan_workspace_size, C.byref(d), 0, C.byref(n))  # noqa: E731
    assert size(scan(rows=0, groups=1, batch=(1 << 23) - 1)) == 0 and size(scan(rows=0, batch=1 << 23)) == UNS
    step = lambda d: status(cm.lib.selective_scan_step, C.byref(d), *[B(i) for i in range(8)], B(8), 1 << 26, None, B(10),  # noqa: E731
                            None)
    assert step(scan(rows=1 << 26, batch=1, channels=64, groups=1, states=1)) == UNS


def test_scan_of_many_rows():
    """Rows up to 2^30, as the header has it, forward and backward."""
    for rows, channels, batch in ((1 << 26, 64, 1), (1 << 27, 64, 3 << 20), ((1 << 30) - 1, 4, 1), (1 << 30, 1, 1 << 20)):
        d = cm.make_scan_desc(rows, channels, 1, batch=batch)
        sizes = [cm.scan_workspace_size(d, op) for op in (cm.SCAN_FORWARD, cm.SCAN_BACKWARD)]
        assert 0 <= sizes[0] <= sizes[1] and cm.scan_saved_size(d) == (rows // 16 + batch) * channels * 4


def test_scan_workspace_of_short_sequences():
    """Sequences of one chunk keep no state between chunks: thousands of them ask for little, however many."""
    one = cm.scan_workspace_size(cm.make_scan_desc(65536, 4096, 16, dtype=cm.BF16), cm.SCAN_FORWARD)
    many = cm.scan_workspace_size(cm.make_scan_desc(65536, 4096, 16, batch=8192, dtype=cm.BF16), cm.SCAN_FORWARD)
    assert 0 < one <= many <= 2 * one
    assert cm.scan_workspace_size(cm.make_scan_desc(65536, 64, 16, batch=1 << 20), cm.SCAN_FORWARD) < 1 << 25
