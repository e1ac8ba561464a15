"""RMS norm with the residual's addition, forward and backward, against the 64-bit formulas.

Error counts behind the bounds (u = 2^-24): a row's sum of squares runs through at most 64
fp32 roundings per value (at most 40 per thread, 10 across lanes and waves), all terms
positive, so inv_rms is within (64/2 + 4) u < 2^-18 of itself and y, three roundings later,
within 2^-18 too, plus its rounding to the data type."""
import pytest
import torch

from tests import block_reference as R

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18
# around every change of the row layout: 16, 64, 256 and 1024 threads, 1 to 4 pieces, two passes
SHAPES = [(1, 1), (1, 4096), (3, 7), (17, 16), (5, 31), (40, 128), (33, 129), (9, 512), (6, 513), (5, 1024), (4, 1025),
          (7, 2048), (3, 2049), (5, 4096), (3, 4097), (2, 8192), (3, 8200), (2, 16384), (2, 16390), (2, 32768),
          (2, 32770), (1, 40003), (2500, 96), (9000, 24)]
DTYPES = [torch.bfloat16, torch.float32]


def cdt(dtype):
    import convolution_layer_amd as cm
    return cm.BF16 if dtype == torch.bfloat16 else cm.F32


def make(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 31 + cols)
    scale = torch.exp(0.5 * torch.randn(cols, generator=g))
    x, res = ((torch.randn(rows, cols, generator=g) * scale).to(dtype) for _ in range(2))
    gamma = 1 + 0.2 * torch.randn(cols, generator=g)
    dy, dh = (torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2))
    return x, res, gamma, dy, dh


def forward(d, x, res, gamma, dtype, y=True, y8=True, h=True, inv=True):
    import convolution_layer_amd as cm
    rows, cols = d.rows, d.cols
    new = lambda t, *s: torch.full(s, 3, dtype=t, device="cuda")  # noqa: E731
    o = {"h": new(dtype, rows + 1, cols) if h else None, "y": new(dtype, rows + 1, cols) if y else None,
         "inv": new(torch.float32, rows + 1) if inv else None,
         "y8": new(torch.uint8, rows + 1, cols) if y8 else None,
         "s": new(torch.uint8, rows + 1, cm.mx8_blocks(cols)) if y8 else None}
    v = {k: None if t is None else t[:rows] for k, t in o.items()}
    cm.rms_norm_forward(d, x, res, gamma, v["h"], v["y"], v["inv"], y8=v["y8"], y8_scales=v["s"])
    for k, t in o.items():
        assert t is None or bool((t[rows] == 3).all()), f"{k}: written behind the last row"
    return v


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, residual, dtype):
    import convolution_layer_amd as cm
    x, res, gamma, _, _ = make(rows, cols, dtype)
    res = res if residual else None
    d = cm.make_rms_desc(rows, cols, dtype=cdt(dtype), eps=1e-5)
    v = forward(d, x.cuda(), res.cuda() if residual else None, gamma.cuda(), dtype)
    h, inv, y = R.rms_forward(x, res, gamma, float(torch.tensor(1e-5)))
    half = R.HALF[dtype]
    R.within(v["h"], h, (half + 2.0 ** -24) * h.abs(), "h")
    R.within(v["inv"], inv, REL * inv, "inv_rms")
    R.within(v["y"], y, (REL + half) * y.abs(), "y")
    kept = torch.empty(rows, cols, device="cuda")
    cm.mx8_unpack(v["y8"], v["s"], kept)
    R.within(kept, y, R.kept_bound(y, REL), "y8")
    # the outputs do not depend on which of them are asked for
    only = forward(d, x.cuda(), res.cuda() if residual else None, gamma.cuda(), dtype, y8=False, h=False, inv=False)
    R.same(only["y"], v["y"], "y alone")
    only = forward(d, x.cuda(), res.cuda() if residual else None, gamma.cuda(), dtype, y=False, h=False, inv=False)
    R.same(only["y8"], v["y8"], "y8 alone")
    R.same(only["s"], v["s"], "y8 scales alone")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, residual, dtype):
    import convolution_layer_amd as cm
    h, _, gamma, dy, dh = make(rows, cols, dtype, 1)
    inv = (1 / torch.sqrt((h.double() ** 2).mean(-1) + 1e-5)).float()
    dh = dh if residual else None
    d = cm.make_rms_desc(rows, cols, dtype=cdt(dtype))
    ws = cm.rms_workspace(d)
    ws.fill_(255)  # what the workspace holds does not matter
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    dx = torch.full((rows + 1, cols), 3.0, dtype=dtype, device="cuda")
    dg = torch.full((cols,), 0.5, device="cuda")
    args = (d, h.cuda(), gamma.cuda(), inv.cuda(), dy.cuda(), dev(dh))
    cm.rms_norm_backward(*args, dx[:rows], dg, 0, ws)
    rx, rg = R.rms_backward(h, gamma, inv, dy, dh)
    hhat, g = h.double() * inv.double()[:, None], gamma.double() * dy.double()
    # the mean of g*hhat: at most 64 roundings of terms of either sign; then four operations
    mean_abs = (g * hhat).abs().mean(-1, keepdim=True)
    bound = inv.double()[:, None] * (2.0 ** -21 * (g.abs() + hhat.abs() * mean_abs) + REL * hhat.abs() * mean_abs)
    bound = bound + R.HALF[dtype] * rx.abs() + 2.0 ** -24 * (rx.abs() + (dh.double().abs() if residual else 0))
    R.within(dx[:rows], rx, bound * (1 + R.HALF[dtype]), "dx")
    assert bool((dx[rows] == 3.0).all())
    # dgamma: a term passes at most 32 additions in fp32 (rows per workgroup, row groups)
    gb = 2.0 ** -18 * (dy.double() * hhat).abs().sum(0) + 2.0 ** -24 * rg.abs()
    R.within(dg, rg, gb, "dgamma")
    cm.rms_norm_backward(*args, dx[:rows], dg, 1, ws)
    R.within(dg, 2 * rg, 2 * gb + 2.0 ** -23 * rg.abs(), "dgamma added")
    # without dgamma no workspace is needed; in place of dy and of dh
    for name in ("dy", "dh") if residual else ("dy",):
        a = [t.clone() if isinstance(t, torch.Tensor) else t for t in args]
        out = a[4] if name == "dy" else a[5]
        cm.rms_norm_backward(*a, out)
        R.same(out, dx[:rows].contiguous(), f"dx over {name}")


@pytest.mark.parametrize("cols", [100, 40000])
def test_dgamma_with_dx_over_dy(cols):
    """dgamma is taken before dx replaces dy, also where it has a pass of its own."""
    import convolution_layer_amd as cm
    h, _, gamma, dy, _ = make(6, cols, torch.float32, 2)
    inv = (1 / torch.sqrt((h.double() ** 2).mean(-1) + 1e-5)).float()
    d = cm.make_rms_desc(6, cols)
    ws = cm.rms_workspace(d)
    out = []
    for over in (False, True):
        y, dg = dy.cuda(), torch.empty(cols, device="cuda")
        dx = y if over else torch.empty_like(y)
        cm.rms_norm_backward(d, h.cuda(), gamma.cuda(), inv.cuda(), y, None, dx, dg, 0, ws)
        out.append((dx, dg))
    for a, b in zip(*out):
        R.same(a, b, "over dy")


@pytest.mark.parametrize("alias", ["x", "residual"])
@pytest.mark.parametrize("cols", [96, 1000, 40000])
def test_h_in_place(alias, cols):
    import convolution_layer_amd as cm
    x, res, gamma, _, _ = make(4, cols, torch.bfloat16, 3)
    d = cm.make_rms_desc(4, cols, dtype=cm.BF16)
    v = forward(d, x.cuda(), res.cuda(), gamma.cuda(), torch.bfloat16)
    a, b = x.cuda(), res.cuda()
    y = torch.empty_like(a)
    cm.rms_norm_forward(d, a, b, gamma.cuda(), a if alias == "x" else b, y, None)
    R.same(a if alias == "x" else b, v["h"].contiguous(), "h")
    R.same(y, v["y"].contiguous(), "y")


@pytest.mark.parametrize("cols", [64, 1003])
def test_special_values_stay_in_their_row(cols):
    """A row of zeros gives zeros and inv = 1/sqrt(eps); NaN, infinities and the type's lowest
    value touch their own row only."""
    import convolution_layer_amd as cm
    x, _, gamma, _, _ = make(6, cols, torch.float32, 4)
    clean = x.clone()
    x[1] = 0.0
    x[2, 3] = float("nan")
    x[3, 5] = float("inf")
    x[4, 7] = torch.finfo(torch.float32).min
    d = cm.make_rms_desc(6, cols, eps=1e-5)
    v = forward(d, x.cuda(), None, gamma.cuda(), torch.float32)
    w = forward(d, clean.cuda(), None, gamma.cuda(), torch.float32)
    for r in (0, 5):
        R.same(v["y"][r], w["y"][r], "clean row")
        R.same(v["y8"][r], w["y8"][r], "clean row, 8 bits")
    assert bool((v["y"][1] == 0).all())
    assert abs(float(v["inv"][1]) * 1e-5 ** 0.5 - 1) < 1e-6
    assert bool(torch.isnan(v["y"][2]).all())
    assert float(v["inv"][3]) == 0.0 and bool(torch.isnan(v["y"][3, 5])) and bool((v["y"][3, 6:] == 0).all())
    assert bool((v["y"][4] == 0).all())  # the square overflows: y = 0, as documented


def test_no_rows():
    import convolution_layer_amd as cm
    d = cm.make_rms_desc(0, 64)
    e, g = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    cm.rms_norm_forward(d, e, None, g, None, e, None)
    dg = torch.full((64,), 2.0, device="cuda")
    cm.rms_norm_backward(d, e, g, torch.empty(0, device="cuda"), e, None, e, dg, 1, cm.rms_workspace(d))
    assert bool((dg == 2).all())
    cm.rms_norm_backward(d, e, g, torch.empty(0, device="cuda"), e, None, e, dg, 0, cm.rms_workspace(d))
    assert bool((dg == 0).all())


def test_gradient_against_differences():
    """dx and dgamma against central differences of the 64-bit forward."""
    import convolution_layer_amd as cm
    rows, cols = 3, 37
    x, _, gamma, dy, _ = make(rows, cols, torch.float32, 5)
    d = cm.make_rms_desc(rows, cols, eps=1e-3)
    eps = float(torch.tensor(1e-3))
    f = lambda a, g: float((R.rms_forward(a, None, g, eps)[2] * dy.double()).sum())  # noqa: E731
    v = forward(d, x.cuda(), None, gamma.cuda(), torch.float32, y8=False)
    dx, dg = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda")
    cm.rms_norm_backward(d, v["h"], gamma.cuda(), v["inv"], dy.cuda(), None, dx, dg, 0, cm.rms_workspace(d))
    t = 1e-5
    for i in range(rows):
        for j in range(0, cols, 5):
            p = torch.zeros(rows, cols, dtype=torch.float64)
            p[i, j] = t
            num = (f(x.double() + p, gamma) - f(x.double() - p, gamma)) / (2 * t)
            assert abs(num - float(dx[i, j])) <= 1e-5 * (1 + abs(num))  # differences lose ~1e-6 at step 1e-5
    for j in range(0, cols, 5):
        p = torch.zeros(cols, dtype=torch.float64)
        p[j] = t
        num = (f(x, gamma.double() + p) - f(x, gamma.double() - p)) / (2 * t)
        assert abs(num - float(dg[j])) <= 1e-5 * (1 + abs(num))


def test_offsets_beyond_32_bits():
    import convolution_layer_amd as cm
    rows, cols = 70001, 32800
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail, _, gamma, _, _ = make(2, cols, torch.bfloat16, 6)
    x[-2:] = tail.cuda()
    y = torch.empty_like(x)
    cm.rms_norm_forward(cm.make_rms_desc(rows, cols, dtype=cm.BF16), x, None, gamma.cuda(), None, y, None)
    _, _, ref = R.rms_forward(tail, None, gamma, float(torch.tensor(1e-5)))
    R.within(y[-2:], ref, (REL + 2.0 ** -8) * ref.abs(), "last rows")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(100001, 100), (65537, 260), (30011, 1000), (50001, 2000), (20011, 5003),
                                       (9001, 16384), (9001, 16400), (7001, 40000)])
def test_dgamma_of_many_rows_keeps_its_bits(rows, cols, dtype):
    """Whole numbers under inv_rms = 1: sums of 20 bits and more, below 2^24 and so exact in fp32 in any
    order, off by hundreds where a partial sum is kept in 16 bits."""
    import convolution_layer_amd as cm
    g = torch.Generator(device="cuda").manual_seed(rows)
    top = 12 if rows > 50000 else 22 if rows > 20000 else 30
    assert rows * top * top < 1 << 24
    h, dy = (torch.randint(0, top + 1, (rows, cols), generator=g, device="cuda").to(dtype) for _ in range(2))
    ref = torch.zeros(cols, dtype=torch.float64, device="cuda")
    for a, b in zip(h.split(8192), dy.split(8192)):
        ref += (a.double() * b.double()).sum(0)
    assert float(ref.min()) > 1 << 20
    d = cm.make_rms_desc(rows, cols, dtype=cdt(dtype))
    ws = cm.rms_workspace(d)
    ws.fill_(255)
    dg, dx = torch.full((cols,), 3.0, device="cuda"), torch.empty_like(h)
    ones = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    for acc in (0, 1):
        cm.rms_norm_backward(d, h, ones(cols), ones(rows), dy, None, dx, dg, acc, ws)
        assert torch.equal(dg.double(), ref * (1 + acc)), f"accumulate {acc}"
