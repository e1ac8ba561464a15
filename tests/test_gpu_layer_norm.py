"""Layer norm with the residual's addition, forward and backward, against the 64-bit formulas.

Error counts behind the bounds (u = 2^-24): a row's sum runs through at most 62 fp32 roundings
(40 values a thread, 6 levels of lanes, 15 waves, one division), so the mean is within
M = 2^-18 mean|h| of itself.  Squares around a mean that is off by d add n d^2 to their sum, so
inv_std is within (62 + 6) / 2 u + (M inv_std)^2 < 2^-18 + (M inv_std)^2 of itself, relative.  y
= gamma c inv_std + beta: c is off by M and u |h|, then three roundings."""
import pytest
import torch

from tests import block_reference as R

pytestmark = pytest.mark.gpu

U, REL = 2.0 ** -24, 2.0 ** -18
# around every change of the row layout: 16, 64, 128, 256, 512 and 1024 threads, 1 to 4 pieces, several passes
SHAPES = [(1, 1), (1, 4096), (3, 7), (17, 16), (5, 31), (40, 128), (33, 129), (9, 512), (6, 513), (5, 1024), (4, 1025),
          (7, 2048), (3, 2049), (5, 4096), (3, 4097), (2, 8192), (3, 8200), (2, 16384), (2, 16390), (2, 32768),
          (2, 32770), (1, 40003), (2500, 96), (9000, 24)]
DTYPES = [torch.bfloat16, torch.float32]
EPS = 1e-5
EPS32 = float(torch.tensor(EPS))


def cdt(dtype):
    import convolution_layer_amd as cm
    return cm.BF16 if dtype == torch.bfloat16 else cm.F32


def make(rows, cols, dtype, seed=0, offset=0.7):
    g = torch.Generator().manual_seed(seed + rows * 31 + cols)
    scale = torch.exp(0.5 * torch.randn(cols, generator=g))
    x, res = ((offset + torch.randn(rows, cols, generator=g) * scale).to(dtype) for _ in range(2))
    gamma, beta = 1 + 0.2 * torch.randn(cols, generator=g), 0.3 * torch.randn(cols, generator=g)
    dy, dh = (torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2))
    return x, res, gamma, beta, dy, dh


def reference(x, res, gamma, beta, eps=EPS32):
    h = x.double() + (res.double() if res is not None else 0.0)
    mean = h.mean(-1)
    c = h - mean[:, None]
    inv = 1 / torch.sqrt((c * c).mean(-1) + eps)
    return h, mean, inv, gamma.double() * c * inv[:, None] + (beta.double() if beta is not None else 0.0)


def reference_backward(h, gamma, mean, inv, dy, dh):
    hhat, g = (h.double() - mean.double()[:, None]) * inv.double()[:, None], gamma.double() * dy.double()
    dx = g - g.mean(-1, keepdim=True) - hhat * (g * hhat).mean(-1, keepdim=True)
    dx = inv.double()[:, None] * dx + (dh.double() if dh is not None else 0.0)
    return dx, (dy.double() * hhat).sum(0), dy.double().sum(0)


def forward(d, x, res, gamma, beta, dtype, y=True, y8=True, h=True, stats=True):
    import convolution_layer_amd as cm
    rows, cols = d.rows, d.cols
    new = lambda t, *s: torch.full(s, 3, dtype=t, device="cuda")  # noqa: E731
    o = {"h": new(dtype, rows + 1, cols) if h else None, "y": new(dtype, rows + 1, cols) if y else None,
         "mean": new(torch.float32, rows + 1) if stats else None, "inv": new(torch.float32, rows + 1) if stats else None,
         "y8": new(torch.uint8, rows + 1, cols) if y8 else None,
         "s": new(torch.uint8, rows + 1, cm.mx8_blocks(cols)) if y8 else None}
    v = {k: None if t is None else t[:rows] for k, t in o.items()}
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    cm.layer_norm_forward(d, dev(x), dev(res), dev(gamma), dev(beta), v["h"], v["y"], v["mean"], v["inv"], y8=v["y8"],
                          y8_scales=v["s"])
    for k, t in o.items():
        assert t is None or bool((t[rows] == 3).all()), f"{k}: written behind the last row"
    return v


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual,affine", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, residual, affine, dtype):
    import convolution_layer_amd as cm
    x, res, gamma, beta, _, _ = make(rows, cols, dtype)
    res, beta = res if residual else None, beta if affine else None
    d = cm.make_layer_norm_desc(rows, cols, dtype=cdt(dtype), eps=EPS)
    v = forward(d, x, res, gamma, beta, dtype)
    h, mean, inv, y = reference(x, res, gamma, beta)
    half = R.HALF[dtype]
    R.within(v["h"], h, (half + U) * h.abs(), "h")
    off = REL * h.abs().mean(-1)
    R.within(v["mean"], mean, off, "mean")
    rel = REL + (off * inv) ** 2
    R.within(v["inv"], inv, rel * inv, "inv_std")
    gc = (gamma.double() * (h - mean[:, None]) * inv[:, None]).abs()
    bound = gamma.double().abs() * inv[:, None] * (off[:, None] + U * h.abs()) + (rel[:, None] + 3 * U) * gc
    bound = bound + 2 * U * (gc + (beta.double().abs() if affine else 0.0))
    R.within(v["y"], y, bound + half * (y.abs() + bound), "y")
    # the 8-bit output is the fp32 y, packed
    f = cm.make_layer_norm_desc(rows, cols, eps=EPS)
    dense = forward(f, x.float(), None if res is None else res.float(), gamma, beta, torch.float32, y8=False)["y"]
    codes, scales = torch.empty_like(v["y8"]), torch.empty_like(v["s"])
    cm.mx8_pack(dense.contiguous(), codes, scales)
    R.same(v["y8"], codes, "y8")
    R.same(v["s"], scales, "y8 scales")
    # the outputs do not depend on which of them are asked for
    only = forward(d, x, res, gamma, beta, dtype, y8=False, h=False, stats=False)
    R.same(only["y"], v["y"], "y alone")
    only = forward(d, x, res, gamma, beta, dtype, y=False, h=False, stats=False)
    R.same(only["y8"], v["y8"], "y8 alone")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, residual, dtype):
    import convolution_layer_amd as cm
    h, _, gamma, _, dy, dh = make(rows, cols, dtype, 1)
    dh = dh if residual else None
    _, mean, inv, _ = reference(h, None, gamma, None)
    mean, inv = mean.float(), inv.float()
    d = cm.make_layer_norm_desc(rows, cols, dtype=cdt(dtype))
    ws = cm.layer_norm_workspace(d)
    ws.fill_(255)  # what the workspace holds does not matter
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    dx = torch.full((rows + 1, cols), 3.0, dtype=dtype, device="cuda")
    dg, db = (torch.full((cols + 1,), 0.5, device="cuda") for _ in range(2))
    args = (d, h.cuda(), gamma.cuda(), mean.cuda(), inv.cuda(), dy.cuda(), dev(dh))
    cm.layer_norm_backward(*args, dx[:rows], dg[:cols], db[:cols], 0, ws)
    rx, rg, rb = reference_backward(h, gamma, mean, inv, dy, dh)
    hhat = (h.double() - mean.double()[:, None]) * inv.double()[:, None]
    g = gamma.double() * dy.double()
    # both means: at most 62 roundings of terms of either sign, each of three; then five operations
    m1, m2 = g.abs().mean(-1, keepdim=True), (g * hhat).abs().mean(-1, keepdim=True)
    bound = inv.double()[:, None] * ((REL + 8 * U) * (m1 + hhat.abs() * m2) + 8 * U * g.abs())
    bound = bound + U * (rx.abs() + (dh.double().abs() if residual else 0))
    R.within(dx[:rows], rx, bound + R.HALF[dtype] * (rx.abs() + bound), "dx")
    assert bool((dx[rows] == 3.0).all())
    # a term passes at most 32 additions in fp32 (rows per workgroup, row groups)
    gb = REL * (dy.double() * hhat).abs().sum(0) + U * rg.abs()
    bb = REL * dy.double().abs().sum(0) + U * rb.abs()
    R.within(dg[:cols], rg, gb, "dgamma")
    R.within(db[:cols], rb, bb, "dbeta")
    assert float(dg[cols]) == 0.5 and float(db[cols]) == 0.5
    first = [t.clone() for t in (dx, dg, db)]
    for which in ("dgamma", "dbeta"):  # each alone
        one = torch.full((cols,), 0.5, device="cuda")
        cm.layer_norm_backward(*args, dx[:rows], **{which: one}, workspace=ws)
        R.same(one, first[1 if which == "dgamma" else 2][:cols], which + " alone")
    cm.layer_norm_backward(*args, dx[:rows], dg[:cols], db[:cols], 1, ws)
    R.within(dg[:cols], 2 * rg, 2 * gb + 2 * U * rg.abs(), "dgamma added")
    R.within(db[:cols], 2 * rb, 2 * bb + 2 * U * rb.abs(), "dbeta added")
    # without the sums no workspace is needed; in place of dy and of dh
    for name in ("dy", "dh") if residual else ("dy",):
        a = [t.clone() if isinstance(t, torch.Tensor) else t for t in args]
        out = a[5] if name == "dy" else a[6]
        cm.layer_norm_backward(*a, out)
        R.same(out, first[0][:rows].contiguous(), f"dx over {name}")


@pytest.mark.parametrize("cols", [100, 4096, 40000])
def test_large_common_offset(cols):
    """Values far from zero: the squares are taken around the mean, so the spread keeps its bits."""
    import convolution_layer_amd as cm
    g = torch.Generator().manual_seed(cols)
    x = 1000.0 + torch.randint(-8, 9, (4, cols), generator=g).float()  # exact in fp32, mean within 2^-18 * 1008
    gamma = torch.ones(cols)
    v = forward(cm.make_layer_norm_desc(4, cols, eps=EPS), x, None, gamma, None, torch.float32)
    h, mean, inv, y = reference(x, None, gamma, None)
    off = REL * 1008.0
    R.within(v["inv"], inv, (REL + (off * inv) ** 2) * inv, "inv_std")
    R.within(v["y"], y, inv[:, None] * off + (REL + (off * inv[:, None]) ** 2 + 6 * U) * y.abs(), "y")


@pytest.mark.parametrize("alias", ["x", "residual"])
@pytest.mark.parametrize("cols", [96, 1000, 40000])
def test_h_in_place(alias, cols):
    import convolution_layer_amd as cm
    x, res, gamma, beta, _, _ = make(4, cols, torch.bfloat16, 3)
    d = cm.make_layer_norm_desc(4, cols, dtype=cm.BF16)
    v = forward(d, x, res, gamma, beta, torch.bfloat16)
    a, b = x.cuda(), res.cuda()
    y = torch.empty_like(a)
    cm.layer_norm_forward(d, a, b, gamma.cuda(), beta.cuda(), a if alias == "x" else b, y, None, None)
    R.same(a if alias == "x" else b, v["h"].contiguous(), "h")
    R.same(y, v["y"].contiguous(), "y")


@pytest.mark.parametrize("cols", [64, 1003])
def test_special_values_stay_in_their_row(cols):
    """A constant row gives beta and inv_std = 1/sqrt(eps); NaN, infinities and the type's lowest
    value touch their own row only."""
    import convolution_layer_amd as cm
    x, _, gamma, beta, _, _ = make(6, cols, torch.float32, 4)
    clean = x.clone()
    x[1] = 2.0
    x[2, 3] = float("nan")
    x[3, 5] = float("inf")
    x[4, 7] = torch.finfo(torch.float32).min
    d = cm.make_layer_norm_desc(6, cols, eps=EPS)
    v, w = (forward(d, t, None, gamma, beta, torch.float32) for t in (x, clean))
    for r in (0, 5):
        R.same(v["y"][r], w["y"][r], "clean row")
        R.same(v["y8"][r], w["y8"][r], "clean row, 8 bits")
    assert torch.equal(v["y"][1].cpu(), beta) and float(v["mean"][1]) == 2.0
    assert abs(float(v["inv"][1]) * EPS ** 0.5 - 1) < 1e-6
    for r in (2, 3):
        assert bool(torch.isnan(v["y"][r]).all())
    assert float(v["inv"][4]) == 0.0  # the square overflows, as documented for the RMS norm


def test_no_rows():
    import convolution_layer_amd as cm
    d = cm.make_layer_norm_desc(0, 64)
    e, g, n = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda"), torch.empty(0, device="cuda")
    cm.layer_norm_forward(d, e, None, g, g, None, e, None, None)
    dg, db = torch.full((64,), 2.0, device="cuda"), torch.full((64,), 2.0, device="cuda")
    cm.layer_norm_backward(d, e, g, n, n, e, None, e, dg, db, 1, cm.layer_norm_workspace(d))
    assert bool((dg == 2).all()) and bool((db == 2).all())
    cm.layer_norm_backward(d, e, g, n, n, e, None, e, dg, db, 0, cm.layer_norm_workspace(d))
    assert bool((dg == 0).all()) and bool((db == 0).all())


def test_gradient_against_differences():
    import convolution_layer_amd as cm
    rows, cols, eps = 3, 37, 1e-3
    x, _, gamma, beta, dy, _ = make(rows, cols, torch.float32, 5)
    d = cm.make_layer_norm_desc(rows, cols, eps=eps)
    e32 = float(torch.tensor(eps))
    f = lambda a, g, b: float((reference(a, None, g, b, e32)[3] * dy.double()).sum())  # noqa: E731
    v = forward(d, x, None, gamma, beta, torch.float32, y8=False)
    dx, dg, db = (torch.empty(s, device="cuda") for s in ((rows, cols), cols, cols))
    cm.layer_norm_backward(d, v["h"], gamma.cuda(), v["mean"], v["inv"], dy.cuda(), None, dx, dg, db, 0,
                           cm.layer_norm_workspace(d))
    t = 1e-5  # differences lose about 1e-6 at this step
    a, g, b = x.double(), gamma.double(), beta.double()
    for i in range(rows):
        for j in range(0, cols, 5):
            p = torch.zeros(rows, cols, dtype=torch.float64)
            p[i, j] = t
            num = (f(a + p, g, b) - f(a - p, g, b)) / (2 * t)
            assert abs(num - float(dx[i, j])) <= 1e-5 * (1 + abs(num))
    for j in range(0, cols, 5):
        p = torch.zeros(cols, dtype=torch.float64)
        p[j] = t
        for got, num in ((dg, f(a, g + p, b) - f(a, g - p, b)), (db, f(a, g, b + p) - f(a, g, b - p))):
            assert abs(num / (2 * t) - float(got[j])) <= 1e-5 * (1 + abs(num / (2 * t)))


@pytest.mark.parametrize("rows,cols", [(100001, 100), (30011, 1000), (20011, 5003), (9001, 16384), (7001, 40000)])
def test_sums_of_many_rows_keep_their_bits(rows, cols):
    """Whole numbers under mean 1 and inv_std 1: sums of 19 bits and more, below 2^24 and so exact in fp32
    in any order."""
    import convolution_layer_amd as cm
    g = torch.Generator(device="cuda").manual_seed(rows)
    top = 12 if rows > 50000 else 22 if rows > 20000 else 30
    assert rows * top * top < 1 << 24
    h = torch.randint(1, top + 2, (rows, cols), generator=g, device="cuda").float()
    dy = torch.randint(0, top + 1, (rows, cols), generator=g, device="cuda").float()
    rg, rb = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for a, b in zip(h.split(8192), dy.split(8192)):
        rg += ((a.double() - 1) * b.double()).sum(0)
        rb += b.double().sum(0)
    d = cm.make_layer_norm_desc(rows, cols)
    ws = cm.layer_norm_workspace(d)
    ws.fill_(255)
    dg, db, dx = torch.full((cols,), 3.0, device="cuda"), torch.full((cols,), 3.0, device="cuda"), torch.empty_like(h)
    ones = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    for acc in (0, 1):
        cm.layer_norm_backward(d, h, ones(cols), ones(rows), ones(rows), dy, None, dx, dg, db, acc, ws)
        assert torch.equal(dg.double(), rg * (1 + acc)) and torch.equal(db.double(), rb * (1 + acc)), acc
