"""RMS norm, linear layer and MX8 on the CPU: descriptors, workspace sizes, kernel plans and
every refusal, by status, before any device work (the addresses are never dereferenced)."""
import ctypes as C

import pytest
import torch
from hypothesis import example, given, settings, strategies as st

import convolution_layer_amd as cm

A = 0x7F0000000000  # a fake device address; B(i) lie far apart
INV, UNS, WS, MIS = cm.ERR_INVALID_ARG, cm.ERR_UNSUPPORTED, cm.ERR_WORKSPACE, cm.ERR_MISALIGNED


def B(i):
    return A + i * 0x1000000


def status(fn, *args):
    s = fn(*args)
    if s != cm.OK:
        assert cm.lib.convmi_last_error().decode()
    return s


# ------------------------------------------------------------------ MX8
@pytest.mark.parametrize("fn", ["mx8_pack", "mx8_unpack"])
def test_mx8_refusals(fn):
    f = getattr(cm.lib, fn)

    def call(rows=4, cols=64, dtype=1, a=B(0), b=B(1), c=B(2)):
        return status(f, rows, cols, dtype, a, b, c, None)

    assert call(rows=-1) == INV and call(cols=0) == INV and call(dtype=2) == INV
    assert call(rows=1 << 30, cols=1 << 20) == UNS and call(cols=(1 << 31) - 16) == UNS
    for k in "abc":
        assert call(**{k: None}) == INV
        assert call(**{k: B(5) + 8}) == MIS
    assert call(c=B(0) + 64) == INV and call(c=B(1)) == INV  # an output over an input
    if fn == "mx8_pack":
        assert call(b=B(0)) == INV
    assert call(rows=0, a=None, b=None, c=None) == cm.OK  # nothing to do


# ------------------------------------------------------------------ RMS norm
def rms(**kw):
    return cm.make_rms_desc(kw.get("rows", 4), kw.get("cols", 64), dtype=kw.get("dtype", 1), eps=kw.get("eps", 1e-5))


@pytest.mark.parametrize("kw,want", [(dict(rows=-1), INV), (dict(cols=0), INV), (dict(dtype=5), INV),
                                     (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
                                     (dict(cols=(1 << 24) + 1), UNS), (dict(rows=1 << 32, cols=1 << 10), UNS)])
def test_rms_descriptors(kw, want):
    d = rms(**kw)
    n = C.c_size_t()
    assert status(cm.lib.rms_norm_workspace_size, C.byref(d), C.byref(n)) == want
    assert status(cm.lib.rms_norm_forward, C.byref(d), *[B(i) for i in range(8)], None) == want
    assert status(cm.lib.rms_norm_backward, C.byref(d), *[B(i) for i in range(7)], 0, B(9), 1 << 30, None) == want


def test_rms_forward_refusals():
    d = rms()

    def call(x=B(0), res=B(1), gamma=B(2), h=B(3), y=B(4), y8=B(5), sc=B(6), inv=B(7)):
        return status(cm.lib.rms_norm_forward, C.byref(d), x, res, gamma, h, y, y8, sc, inv, None)

    assert call(x=None) == INV and call(gamma=None) == INV
    assert call(y=None, y8=None, sc=None) == INV      # no output
    assert call(y8=None) == INV and call(sc=None) == INV  # codes and scales come together
    for k in ("x", "res", "h", "y", "y8", "sc"):
        assert call(**{k: B(9) + 4}) == MIS
    assert call(gamma=B(9) + 2) == MIS and call(inv=B(9) + 1) == MIS
    for out in ("y", "y8", "sc", "inv"):
        assert call(**{out: B(0)}) == INV and call(**{out: B(1) + 16}) == INV and call(**{out: B(2)}) == INV
    assert call(h=B(0) + 16) == INV and call(h=B(1) + 32) == INV  # h may be x or the residual, not a part of one
    assert call(y=B(3)) == INV and call(y8=B(4)) == INV and call(inv=B(6)) == INV  # two outputs in one place
    assert status(cm.lib.rms_norm_forward, None, *[B(i) for i in range(8)], None) == INV


def test_rms_backward_refusals():
    d = rms()
    need = cm.rms_workspace_size(d)
    assert need > 0

    def call(h=B(0), gamma=B(1), inv=B(2), dy=B(3), dh=B(4), dx=B(5), dg=B(6), acc=0, ws=B(7), n=need):
        return status(cm.lib.rms_norm_backward, C.byref(d), h, gamma, inv, dy, dh, dx, dg, acc, ws, n, None)

    for k in ("h", "gamma", "inv", "dy", "dx"):
        assert call(**{k: None}) == INV
    assert call(acc=2) == INV
    assert call(dx=B(0)) == INV and call(dx=B(3) + 16) == INV and call(dx=B(4) + 16) == INV and call(dx=B(1)) == INV
    assert call(dg=B(1)) == INV and call(dg=B(5) + 16) == INV
    assert call(dg=B(0)) == INV and call(dg=B(2)) == INV and call(dg=B(3)) == INV and call(dg=B(4) + 32) == INV
    assert call(ws=None) == WS and call(n=need - 1) == WS and call(ws=B(7) + 16) == MIS
    assert call(dx=B(5) + 2) == MIS and call(dg=B(6) + 2) == MIS


# ------------------------------------------------------------------ linear layer
def lin(**kw):
    return cm.make_linear_desc(kw.get("M", 32), kw.get("K", 64), kw.get("N", 48), activation=kw.get("activation", 0),
                               dtype=kw.get("dtype", 1), x_mx8=kw.get("x_mx8", 0), z_mx8=kw.get("z_mx8", 0))


BAD_LINEAR = [(dict(M=-1), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(activation=5), INV), (dict(dtype=2), INV),
              (dict(x_mx8=2), INV), (dict(z_mx8=-1), INV), (dict(K=(1 << 20) + 1), UNS), (dict(N=1 << 21), UNS),
              (dict(M=1 << 31), UNS), (dict(M=1 << 30, N=1 << 11), UNS)]


@pytest.mark.parametrize("kw,want", BAD_LINEAR)
def test_linear_descriptors(kw, want):
    d = lin()
    for k, v in kw.items():
        setattr(d, k, v)
    n, buf = C.c_size_t(), C.create_string_buffer(64)
    for op in range(3):
        assert status(cm.lib.linear_workspace_size, C.byref(d), op, C.byref(n)) == want
        assert status(cm.lib.linear_plan_name, C.byref(d), op, buf, 64) == want
    big = 1 << 40
    assert status(cm.lib.linear_forward, C.byref(d), *[B(i) for i in range(9)], B(9), big, None) == want
    assert status(cm.lib.linear_activation_backward, C.byref(d), *[B(i) for i in range(4)], None) == want
    assert status(cm.lib.linear_backward_data, C.byref(d), *[B(i) for i in range(3)], B(9), big, None) == want
    assert status(cm.lib.linear_backward_weight, C.byref(d), *[B(i) for i in range(5)], 0, B(9), big, None) == want


def test_linear_ops_and_pointers():
    d, n, buf = lin(), C.c_size_t(), C.create_string_buffer(64)
    for op in (-1, 3):
        assert status(cm.lib.linear_workspace_size, C.byref(d), op, C.byref(n)) == INV
        assert status(cm.lib.linear_plan_name, C.byref(d), op, buf, 64) == INV
    assert status(cm.lib.linear_workspace_size, C.byref(d), 0, None) == INV
    assert status(cm.lib.linear_plan_name, C.byref(d), 0, None, 64) == INV
    assert status(cm.lib.linear_plan_name, C.byref(d), 0, buf, 0) == INV
    f32 = lin(x_mx8=1, dtype=0)  # 8-bit operands have bf16 outputs; the gradients take float32 too
    assert status(cm.lib.linear_workspace_size, C.byref(f32), 0, C.byref(n)) == UNS
    assert status(cm.lib.linear_forward, C.byref(f32), *[B(i) for i in range(9)], B(9), 1 << 40, None) == UNS
    assert status(cm.lib.linear_workspace_size, C.byref(f32), 2, C.byref(n)) == cm.OK


def test_linear_forward_refusals():
    def call(d, x=B(0), xs=None, w=B(1), ws_=None, bias=B(2), res=B(3), z=B(4), zs=None, y=B(5), ws=B(9), n=1 << 40):
        return status(cm.lib.linear_forward, C.byref(d), x, xs, w, ws_, bias, res, z, zs, y, ws, n, None)

    d, d8, z8 = lin(), lin(x_mx8=1), lin(z_mx8=1)
    for k in ("x", "w", "y"):
        assert call(d, **{k: None}) == INV
    for k in ("x", "w", "res", "z", "y"):
        assert call(d, **{k: B(8) + 2}) == MIS
    assert call(d, bias=B(8) + 2) == MIS
    assert call(d, xs=B(6)) == INV and call(d, ws_=B(6)) == INV and call(d, zs=B(6)) == INV  # scales of dense tensors
    assert call(d8, xs=None, ws_=B(7)) == INV and call(d8, xs=B(6), ws_=None) == INV
    assert call(z8, zs=None) == INV and call(z8, z=None, zs=B(6)) == INV
    assert call(d, y=B(0)) == INV and call(d, y=B(1) + 64) == INV and call(d, y=B(2)) == INV
    assert call(d, y=B(3) + 16) == INV and call(d, z=B(3)) == INV and call(d, y=B(4)) == INV
    odd = lin(K=65)  # padded copies need a workspace
    need = cm.linear_workspace_size(odd, cm.LINEAR_FORWARD)
    assert need > 0
    assert call(odd, ws=None, n=0) == WS and call(odd, n=need - 1) == WS and call(odd, ws=B(9) + 16) == MIS


def test_linear_backward_refusals():
    d, d8 = lin(), lin(x_mx8=1)
    big = 1 << 40

    def act(d, z=B(0), zs=None, dy=B(1), dz=B(2)):
        return status(cm.lib.linear_activation_backward, C.byref(d), z, zs, dy, dz, None)

    for k in ("z", "dy", "dz"):
        assert act(d, **{k: None}) == INV and act(d, **{k: B(6) + 2}) == MIS
    assert act(d, zs=B(4)) == INV and act(lin(z_mx8=1)) == INV
    assert act(d, dz=B(0)) == INV and act(d, dz=B(1) + 16) == INV

    def data(dz=B(0), w=B(1), dx=B(2), ws=B(9), n=big):
        return status(cm.lib.linear_backward_data, C.byref(d), dz, w, dx, ws, n, None)

    for k in ("dz", "w", "dx"):
        assert data(**{k: None}) == INV and data(**{k: B(6) + 2}) == MIS
    assert data(dx=B(0)) == INV and data(dx=B(1) + 32) == INV

    def weight(d, x=B(0), xs=None, dz=B(1), dw=B(2), db=B(3), acc=0, ws=B(9), n=big):
        return status(cm.lib.linear_backward_weight, C.byref(d), x, xs, dz, dw, db, acc, ws, n, None)

    for k in ("x", "dz", "dw"):
        assert weight(d, **{k: None}) == INV and weight(d, **{k: B(6) + 2}) == MIS
    assert weight(d, db=B(6) + 2) == MIS and weight(d, acc=3) == INV
    assert weight(d, xs=B(5)) == INV and weight(d8) == INV
    assert weight(d, dw=B(0)) == INV and weight(d, dw=B(1)) == INV and weight(d, db=B(2) + 16) == INV
    assert weight(d, db=B(0)) == INV
    assert weight(d8, xs=B(5), ws=None, n=0) == WS  # x is unpacked into the workspace
    assert weight(lin(M=0), x=None, dz=None, dw=None) == INV  # an empty batch still has gradients


def test_conv_backward_mx8_refusals():
    d = cm.make_desc(2, 8, 8, 16, 16, 3, 3, pad=(1, 1), activation=cm.ACT_TANH, dtype=cm.BF16)
    need = cm.workspace_size(d, cm.OP_BACKWARD_FULL_MX8)
    assert need >= cm.workspace_size(d, cm.OP_BACKWARD_FULL) + 2 * 8 * 8 * 16 * 2 and need % 256 == 0

    def call(d=d, x=B(0), xs=B(1), w=B(2), y=B(3), ys=B(4), out=1, dy=B(5), dx=B(6), dw=B(7), db=B(8), acc=0, ws=B(9),
             n=need):
        return status(cm.lib.conv2d_backward_full_mx8, C.byref(d), x, xs, w, y, ys, out, dy, dx, dw, db, acc, ws, n,
                      None)

    for k in ("x", "w", "y", "dy", "dw"):
        assert call(**{k: None}) == INV
    assert call(xs=B(1) + 8) == MIS and call(ys=B(4) + 8) == MIS
    assert call(dx=B(0)) == INV and call(dx=B(1)) == INV and call(dx=B(4)) == INV
    assert call(out=2) == INV and call(acc=-1) == INV
    assert call(n=need - 1) == WS and call(ws=None) == WS and call(ws=B(9) + 64) == MIS
    gelu = cm.make_desc(2, 8, 8, 16, 16, 3, 3, pad=(1, 1), activation=cm.ACT_GELU, dtype=cm.BF16)
    assert call(d=gelu) == INV
    norm = cm.make_desc(2, 8, 8, 16, 16, 3, 3, pad=(1, 1), normalization=cm.NORM_BATCH, dtype=cm.BF16)
    assert call(d=norm) == UNS


# ------------------------------------------------------------------ plans and workspaces
SIZES = st.one_of(st.integers(1, 40), st.integers(41, 3000), st.sampled_from([64, 128, 256, 512, 1024, 4096, 8192]))


@settings(max_examples=300, deadline=None)
@given(st.integers(0, 1 << 17), SIZES, SIZES, st.integers(0, 1), st.integers(0, 1), st.integers(0, 2))
def test_linear_plans(M, K, N, dtype, x8, op):
    """Every valid size has a plan and a workspace that covers what the plan copies."""
    d = cm.make_linear_desc(M, K, N, dtype=dtype, x_mx8=x8)
    if op == 0 and x8 and dtype == cm.F32:
        return
    es = 1 if (op == 0 and x8) else (2 if dtype else 4)
    name, n = cm.linear_plan_name(d, op), cm.linear_workspace_size(d, op)
    assert n % 256 == 0
    if M == 0:
        assert name == "empty" and n == 0
        return
    if op == 0 and M <= 16:
        assert name.startswith("rows ") and n == 0
        return
    assert name.startswith("tiles ")
    splits = int(name.split(" split ")[1].split()[0])
    I, J = (M, N) if op == 0 else (M, K) if op == 1 else (N, K)
    least = splits * I * J * 4 if splits > 1 else 0
    up = lambda v: -(-v * es // 16) * 16  # noqa: E731
    a, b = (K, K) if op == 0 else (N, K)
    ra, rb = M, (M if op == 2 else N)
    if a * es % 16:
        least += ra * up(a)
    if b * es % 16 or (op == 2 and x8):
        least += rb * up(b)
    assert name.endswith(" prep") == bool(a * es % 16 or b * es % 16 or (op == 2 and x8))
    assert n >= least


def test_gpu_shapes_reach_every_plan():
    """The sizes of the GPU tests reach the few-row kernel and every tile side, whole and split."""
    from tests.test_gpu_linear import LARGE, SHAPES
    seen = set()
    cases = [(*s, ty, op) for s in SHAPES for ty in ("bf16", "f32", "mx8") for op in range(3)] + LARGE
    for M, K, N, ty, op in cases:
        if ty == "mx8" and op:
            continue
        d = cm.make_linear_desc(M, K, N, dtype=cm.F32 if ty == "f32" else cm.BF16, x_mx8=ty == "mx8")
        w = cm.linear_plan_name(d, op).split()
        seen.add((ty, op, "rows") if w[0] == "rows" else (ty, op, int(w[2].split("x")[0])))
        if w[0] == "tiles":
            seen.add((ty, op, "split" if w[4] != "1" else "whole"))
    for ty, sides in (("bf16", (64, 128, 256)), ("f32", (64, 128)), ("mx8", (64, 128, 256))):
        for op in range(1 if ty == "mx8" else 3):
            for what in sides + ("whole", "split") + (("rows",) if op == 0 else ()):
                assert (ty, op, what) in seen, (ty, op, what)


@settings(max_examples=400, deadline=None)
@example(1, 44, 62, 12, 112, 7, 1, 0, 0)
@example(32, 5, 20, 12, 256, 5, 1, 0, 1)
@given(st.integers(1, 32), st.integers(1, 64), st.integers(1, 64), st.integers(1, 130), st.integers(1, 260),
       st.sampled_from([1, 2, 3, 5, 7]), st.integers(1, 2), st.integers(0, 1), st.sampled_from([0, 1, 4]))
def test_mx8_backward_workspace_covers_dense_tensors(N, H, W, IC, OC, k, stride, dtype, act):
    """conv2d_backward_full_mx8 without scales lays its buffers out as conv2d_backward_full does, on the
    layer's own channel counts, whose weight gradient may be split more often than the padded ones'."""
    d = cm.make_desc(N, H, W, IC, OC, k, k, stride=(stride, stride), pad=(k // 2, k // 2), activation=act, dtype=dtype)
    assert cm.workspace_size(d, cm.OP_BACKWARD_FULL_MX8) >= cm.workspace_size(d, cm.OP_BACKWARD_FULL)


@pytest.mark.parametrize("s,p", [((1, 44, 62, 12, 112, 7, 7), (3, 3)), ((32, 5, 20, 12, 256, 5, 5), (2, 2))])
def test_mx8_backward_of_dense_tensors_checks_its_own_layout(s, p):
    """Refused with less than conv2d_backward_full needs."""
    d = cm.make_desc(*s, pad=p, dtype=cm.F32)
    n = cm.workspace_size(d, cm.OP_BACKWARD_FULL) - 256
    at = lambda i: A + (i << 32)  # noqa: E731
    assert status(cm.lib.conv2d_backward_full_mx8, C.byref(d), at(0), None, at(1), at(2), None, 0, at(3), at(4), at(5),
                  at(6), 0, at(7), n, None) == WS


# ------------------------------------------------------------------ the binding's own checks
def test_binding_refuses_host_tensors_and_wrong_types():
    x, q, s = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        cm.mx8_pack(x, q, s)
    with pytest.raises(ValueError, match="device"):
        cm.mx8_unpack(q, s, x)
    with pytest.raises(ValueError, match="dtype"):
        cm.mx8_pack(x.half(), q, s)
    with pytest.raises(ValueError, match="axis"):
        cm.mx8_pack(torch.zeros(()), q, s)
    d = cm.make_rms_desc(4, 64)
    with pytest.raises(ValueError, match="device"):
        cm.rms_norm_forward(d, x, None, torch.ones(64), None, x, None)
    with pytest.raises(ValueError, match="None"):
        cm.rms_norm_forward(d, None, None, torch.ones(64), None, x, None)
    ld = cm.make_linear_desc(4, 64, 8)
    with pytest.raises(ValueError, match="device"):
        cm.linear_forward(ld, x, torch.zeros(8, 64), None, None, None, torch.zeros(4, 8))
    with pytest.raises(cm.ConvmiError):
        cm.linear_forward(cm.make_linear_desc(4, 64, 8, dtype=9), x, x, None, None, None, x)
    assert cm.mx8_blocks(1) == 1 and cm.mx8_blocks(32) == 1 and cm.mx8_blocks(33) == 2


def test_binding_refuses_turned_weights():
    """A contiguous [K, N] matrix has the elements of [N, K] in another order; other shapes are taken."""
    ld = cm.make_linear_desc(4, 64, 8)
    x, y = torch.zeros(4, 64), torch.zeros(4, 8)
    turned = torch.zeros(64, 8)
    with pytest.raises(ValueError, match=r"w has shape \(64, 8\)"):
        cm.linear_forward(ld, x, turned, None, None, None, y)
    with pytest.raises(ValueError, match="w has shape"):
        cm.linear_backward_data(ld, y, turned, x)
    with pytest.raises(ValueError, match="dw has shape"):
        cm.linear_backward_weight(ld, x, y, turned, None)
    for shape in ((8, 64), (512,), (8, 1, 1, 64), (16, 32)):  # these get as far as the device
        with pytest.raises(ValueError, match="device"):
            cm.linear_forward(ld, x, torch.zeros(shape), None, None, None, y)
    with pytest.raises(ValueError, match="device"):
        cm.linear_forward(cm.make_linear_desc(4, 8, 8), torch.zeros(4, 8), torch.zeros(8, 8), None, None, None, y)
    with pytest.raises(ValueError, match="device"):  # one row or one column: the same order
        cm.linear_forward(cm.make_linear_desc(4, 64, 1), x, torch.zeros(64, 1), None, None, None, torch.zeros(4, 1))
