"""The linear layer's products against 64-bit products, on every kernel plan.

Most cases use small integers: every product and partial sum is then a whole number below
2^24, exact in fp32 in any order, so results must equal the definition bit for bit (bf16
outputs: its one rounding).  Activations on random data are held to error counts: a sum of K
products accumulated in fp32 is within K * 2^-24 of the sum of magnitudes."""
import pytest
import torch

from tests import block_reference as R

pytestmark = pytest.mark.gpu

# ragged and whole tiles of every side, odd row lengths, splits, few rows
SHAPES = [(1, 1, 1), (1, 64, 16), (1, 4096, 40), (2, 130, 33), (3, 33, 7), (5, 1024, 64), (7, 257, 96), (16, 1003, 130),
          (17, 64, 64), (20, 130, 70), (33, 1000, 100), (64, 64, 64), (65, 129, 63), (128, 256, 128), (200, 72, 520),
          (257, 512, 129), (300, 1003, 517), (64, 8192, 64), (100, 5000, 130), (2100, 200, 2300), (2500, 136, 2600),
          (4100, 264, 3000)]
TYPES = ["bf16", "f32", "mx8"]


def ints(rows, cols, seed, top=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, (rows, cols), generator=g, device="cuda").double()


def tdt(ty):
    return torch.float32 if ty == "f32" else torch.bfloat16


def desc(M, K, N, ty, **kw):
    import convolution_layer_amd as cm
    return cm.make_linear_desc(M, K, N, dtype=cm.F32 if ty == "f32" else cm.BF16, x_mx8=ty == "mx8", **kw)


def operand(v, ty):
    """(tensor, scales): v as the operand type holds it (whole numbers up to 8 fit each)."""
    import convolution_layer_amd as cm
    if ty != "mx8":
        return v.to(tdt(ty)).contiguous(), None
    q = torch.empty(v.shape, dtype=torch.uint8, device="cuda")
    s = torch.empty(v.shape[0], cm.mx8_blocks(v.shape[1]), dtype=torch.uint8, device="cuda")
    cm.mx8_pack(v.bfloat16().contiguous(), q, s)
    return q, s


def poisoned(d, op):
    """The operation's workspace, filled with NaN bits."""
    import convolution_layer_amd as cm
    ws = cm.linear_workspace(d, op)
    if ws is not None:
        ws.fill_(255)
    return ws


def forward(d, x, w, bias=None, res=None, z=None, y=None, zs=None):
    import convolution_layer_amd as cm
    cm.linear_forward(d, x[0], w[0], bias, res, z, y, workspace=poisoned(d, cm.LINEAR_FORWARD), x_scales=x[1],
                      w_scales=w[1], z_scales=zs)


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward_exact(M, K, N, ty):
    import convolution_layer_amd as cm
    xi, wi, bi, ri = ints(M, K, 1), ints(N, K, 2), ints(1, N, 3)[0], ints(M, N, 4, 9)
    x, w, t = operand(xi, ty), operand(wi, ty), tdt(ty)
    plain = xi @ wi.T
    guard = torch.full((M + 2, N), 77.0, dtype=t, device="cuda")
    y = guard[:M]
    forward(desc(M, K, N, ty), x, w, y=y)
    assert torch.equal(y.double(), plain.to(t).double()), "product"
    assert bool((guard[M:] == 77).all()), "rows behind the last"
    z = torch.empty(M, N, dtype=t, device="cuda")
    d = desc(M, K, N, ty, activation=cm.ACT_RELU)
    forward(d, x, w, bi.float(), ri.to(t), z, y)
    zi = plain + bi
    assert torch.equal(z.double(), zi.to(t).double()), "z"
    assert torch.equal(y.double(), (zi.clamp(min=0) + ri).to(t).double()), "relu + residual"
    over = ri.to(t)
    forward(d, x, w, bi.float(), over, None, over)  # the residual's own place
    R.same(over, y.contiguous(), "in place of the residual")


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("M,K,N", [s for s in SHAPES if s[0] * s[2] < 1 << 19] + [(2100, 200, 2300)])
def test_forward_keeps_z_in_8_bits(M, K, N, ty):
    import convolution_layer_amd as cm
    xi, wi, bi = ints(M, K, 5), ints(N, K, 6), ints(1, N, 7)[0]
    x, w, t = operand(xi, ty), operand(wi, ty), tdt(ty)
    nb = cm.mx8_blocks(N)
    q = torch.full((M + 1, N), 99, dtype=torch.uint8, device="cuda")
    s = torch.full((M + 1, nb), 99, dtype=torch.uint8, device="cuda")
    y = torch.empty(M, N, dtype=t, device="cuda")
    forward(desc(M, K, N, ty, z_mx8=True), x, w, bi.float(), None, q[:M], y, s[:M])
    zi = xi @ wi.T + bi
    c, e, _ = R.keep(zi.cpu())
    assert torch.equal(s[:M].cpu().long(), e) and torch.equal(q[:M].cpu().long() & 127, c & 127)
    nz = zi.cpu() != 0
    assert torch.equal(q[:M].cpu().long()[nz], c[nz])
    assert torch.equal(y.double(), zi.to(t).double())
    assert bool((q[M] == 99).all()) and bool((s[M] == 99).all())


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("M,K,N", [(1, 256, 40), (6, 100, 64), (30, 200, 72), (140, 1003, 257)])
def test_forward_activations(M, K, N, act, ty):
    g = torch.Generator(device="cuda").manual_seed(act)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, t = operand(rnd(M, K), ty), operand(rnd(N, K) * (2.0 / K) ** 0.5, ty), tdt(ty)
    if ty == "mx8":
        xv, wv = (R.decode(q.cpu(), s.cpu()) for q, s in (x, w))
    else:
        xv, wv = x[0].double().cpu(), w[0].double().cpu()
    bias, res = rnd(N), rnd(M, N).to(t)
    y = torch.empty(M, N, dtype=t, device="cuda")
    forward(desc(M, K, N, ty, activation=act), x, w, bias, res, None, y)
    z = xv @ wv.T + bias.double().cpu()
    ref = R.act(z, act) + R.host(res)
    mag = xv.abs() @ wv.abs().T + bias.double().cpu().abs()
    # MX8: the instruction adds its 64 or 128 exact products with fewer kept bits (a few
    # times 2^-14 of the largest, measured); slopes are at most 1.13
    zb = (K + 2) * 2.0 ** -24 * mag + (2.0 ** -12 * mag if ty == "mx8" else 0)
    bound = 1.13 * zb + R.ACT_ABS * (1 + z.abs()) / 16 + 2.0 ** -23 * ref.abs() + R.HALF[t] * ref.abs()
    R.within(y, ref, bound * (1 + R.HALF[t]), "y")


def powers(codes):
    """Exponents of e4m3 codes, a subnormal's (and zero's) counted as -6."""
    return (codes.long() >> 3 & 15).clamp(min=1) - 7


@pytest.mark.parametrize("M,K,N", [(1, 128, 40), (7, 1003, 64), (40, 64, 64), (130, 1000, 70), (300, 2056, 257),
                                   (2600, 520, 3000)])
@pytest.mark.parametrize("spread", [0, 12])
def test_mx8_products_lose_only_what_the_header_says(M, K, N, spread):
    """Values and scales spread over many powers of two.  Of eight consecutive products each is
    cut to a multiple of 2^(E-13), E the largest power among them: it loses no more than that,
    nor more than itself.  Then K / 8 sums in fp32 (K * 2^-24 of the magnitudes allows for
    each product to be one) and the rounding to bf16."""
    import convolution_layer_amd as cm
    g = torch.Generator().manual_seed(K + spread)

    def wide(rows, cols):  # values over 2^12, each block of 32 over 2^spread more
        v = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, cols), generator=g).float())
        b = torch.exp2(torch.randint(-spread, spread + 1, (rows, cm.mx8_blocks(cols)), generator=g).float())
        return v * b.repeat_interleave(32, -1)[:, :cols]

    x, w = operand(wide(M, K).cuda(), "mx8"), operand(wide(N, K).cuda(), "mx8")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    forward(desc(M, K, N, "mx8"), x, w, y=y)
    rows = torch.unique(torch.cat([torch.arange(min(M, 40)), torch.arange(max(0, M - 40), M)]))
    xq, xs, wq, ws = (t.cpu() for t in (x[0][rows.cuda()], x[1][rows.cuda()], *w))
    xv, wv = R.decode(xq, xs), R.decode(wq, ws)
    top = lambda q, s: torch.where(q & 127 == 0, torch.tensor(-10 ** 6), powers(q)) + (  # noqa: E731
        s.long() - 127).repeat_interleave(32, -1)[:, : q.shape[1]]
    xe, we = top(xq, xs), top(wq, ws)
    lost = torch.zeros(len(rows), N, dtype=torch.float64)
    mag = torch.zeros_like(lost)
    for k in range(0, K, 8):
        p = (xv[:, None, k:k + 8] * wv[None, :, k:k + 8]).abs()
        E = (xe[:, None, k:k + 8] + we[None, :, k:k + 8]).amax(-1).clamp(min=-900)
        lost += torch.minimum(p, torch.ldexp(torch.ones(()).double(), E - 13)[..., None]).sum(-1)
        mag += p.sum(-1)
    ref = xv @ wv.T
    bound = lost + (K + 2) * 2.0 ** -24 * mag
    R.within(y[rows.cuda()], ref, (bound + 2.0 ** -8 * ref.abs()) * (1 + 2.0 ** -8), "y")


@pytest.mark.parametrize("M,N", [(1, 64), (40, 64)])
def test_mx8_groups_of_eight_follow_the_rule(M, N):
    """One group per output, the rest zero, codes of every size: the rule's own sum, taken away
    through the bias, leaves exactly zero."""
    import convolution_layer_amd as cm
    g = torch.Generator().manual_seed(M)
    K = 128
    x, w = torch.zeros(1, K, dtype=torch.uint8), torch.zeros(N, K, dtype=torch.uint8)
    code = lambda *s: (torch.randint(0, 127, s, generator=g) + 128 * torch.randint(0, 2, s, generator=g)).to(torch.uint8)  # noqa: E731
    at = 8 * torch.randint(0, K // 8, (N,), generator=g)
    x[:] = code(1, K)
    for n in range(N):
        w[n, at[n]:at[n] + 8] = code(8)
    ones = lambda r: torch.full((r, 4), 127, dtype=torch.uint8)  # noqa: E731
    xv, wv = R.decode(x, ones(1)), R.decode(w, ones(N))
    E = torch.where((w & 127 == 0) | (x & 127 == 0), torch.tensor(-900), powers(x) + powers(w))
    step = torch.ldexp(torch.ones(()).double(), E.amax(-1, keepdim=True) - 13)
    want = (torch.trunc(xv * wv / step) * step).sum(-1)  # at most 8 * 2^15.6 steps: exact in fp32
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    d = cm.make_linear_desc(M, K, N, dtype=cm.BF16, x_mx8=True)
    cm.linear_forward(d, x.repeat(M, 1).cuda(), w.cuda(), (-want).float().cuda(), None, None, y, poisoned(d, 0),
                      x_scales=ones(M).cuda(), w_scales=ones(N).cuda())
    assert bool((y == 0).all())


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_gradients_exact(M, K, N, ty):
    import convolution_layer_amd as cm
    t = tdt(ty)
    xi, wi, zi = ints(M, K, 8), ints(N, K, 9), ints(M, N, 10)
    x, w, dz = xi.to(t), wi.to(t), zi.to(t)
    d = desc(M, K, N, ty)
    dx = torch.full((M + 1, K), 55.0, dtype=t, device="cuda")
    cm.linear_backward_data(d, dz, w, dx[:M], poisoned(d, cm.LINEAR_BACKWARD_DATA))
    assert torch.equal(dx[:M].double(), (zi @ wi).to(t).double()), "dx"
    assert bool((dx[M] == 55).all())
    rw, rb = zi.T @ xi, zi.sum(0)
    dw, db = torch.full((N, K), 3.0, device="cuda"), torch.full((N,), 4.0, device="cuda")
    for acc in (0, 1):
        cm.linear_backward_weight(d, x, dz, dw, db, acc, poisoned(d, cm.LINEAR_BACKWARD_WEIGHT))
        assert torch.equal(dw.double(), rw * (1 + acc)), f"dw, accumulate {acc}"
        assert torch.equal(db.double(), rb * (1 + acc)), f"db, accumulate {acc}"
    cm.linear_backward_weight(d, x, dz, dw, None, 0, poisoned(d, cm.LINEAR_BACKWARD_WEIGHT))
    assert torch.equal(dw.double(), rw), "dw without db"
    d8 = cm.make_linear_desc(M, K, N, dtype=d.dtype, x_mx8=True)
    q, s = operand(xi, "mx8")
    cm.linear_backward_weight(d8, q, dz, dw, db, 0, poisoned(d8, cm.LINEAR_BACKWARD_WEIGHT), x_scales=s)
    assert torch.equal(dw.double(), rw) and torch.equal(db.double(), rb), "from 8-bit x"


# ragged edges of the large tiles and of the splits; tests/test_block_abi_cpu.py checks that
# these and SHAPES reach every tile side, with and without splits, for each type
LARGE = [(3100, 1000, 3200, "bf16", 0), (5000, 2056, 2100, "bf16", 1), (2500, 1300, 1300, "bf16", 1),
         (4200, 1100, 4100, "bf16", 2), (300, 4200, 4100, "bf16", 2), (2600, 3100, 3000, "mx8", 0),
         (700, 9000, 300, "bf16", 0), (300, 200, 9000, "bf16", 1), (9000, 200, 300, "bf16", 2),
         (9000, 100, 40, "f32", 2), (2500, 1032, 1100, "mx8", 0), (3000, 500, 3200, "f32", 0),
         (1000, 4104, 300, "mx8", 0), (3000, 3200, 200, "f32", 1), (100, 200, 5000, "f32", 1)]


@pytest.mark.parametrize("M,K,N,ty,op", LARGE)
def test_large_tiles_and_splits_exact(M, K, N, ty, op):
    import convolution_layer_amd as cm
    d = desc(M, K, N, ty)
    t = tdt(ty)
    xi, wi, zi = ints(M, K, 11), ints(N, K, 12), ints(M, N, 13)
    if op == 0:
        y = torch.empty(M, N, dtype=t, device="cuda")
        forward(d, operand(xi, ty), operand(wi, ty), ints(1, N, 3)[0].float(), None, None, y)
        assert torch.equal(y.double(), (xi @ wi.T + ints(1, N, 3)[0]).to(t).double())
    elif op == 1:
        dx = torch.empty(M, K, dtype=t, device="cuda")
        cm.linear_backward_data(d, zi.to(t), wi.to(t), dx, poisoned(d, op))
        assert torch.equal(dx.double(), (zi @ wi).to(t).double())
    else:
        dw, db = torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
        cm.linear_backward_weight(d, xi.to(t), zi.to(t), dw, db, 0, poisoned(d, op))
        assert torch.equal(dw.double(), zi.T @ xi) and torch.equal(db.double(), zi.sum(0))


@pytest.mark.parametrize("M,K,N", [(4, 72, 40), (40, 72, 40), (40, 65, 33), (300, 1000, 200)])
@pytest.mark.parametrize("ty", TYPES)
def test_special_values_stay_in_their_row_and_column(M, K, N, ty):
    """NaN and infinities in one row of x, one row of w and one column of dz reach only the
    outputs that use them: nothing leaks through padded tails or ragged tiles."""
    import convolution_layer_amd as cm
    t = tdt(ty)
    xi, wi = ints(M, K, 14), ints(N, K, 15)
    xi[2, K - 1], wi[5, 0], wi[N - 1, K - 1] = float("nan"), float("inf"), float("nan")
    y = torch.empty(M, N, dtype=t, device="cuda")
    forward(desc(M, K, N, ty), operand(xi, ty), operand(wi, ty), y=y)
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    rows[2], cols[5], cols[N - 1] = False, False, False
    ok = torch.outer(rows, cols).cuda()
    ref = torch.nan_to_num(xi, nan=0.0) @ torch.nan_to_num(wi, nan=0.0, posinf=0.0).T
    assert torch.equal(y.double()[ok], ref[ok].to(t).double())
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[:, N - 1]).all())
    assert not bool(torch.isfinite(y[:, 5]).any())
    if ty == "mx8":
        return
    zi, xi = ints(M, N, 16), ints(M, K, 17)
    zi[M - 1, N - 1] = float("nan")
    dw, db = torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    d = desc(M, K, N, ty)
    cm.linear_backward_weight(d, xi.to(t), zi.to(t), dw, db, 0, poisoned(d, 2))
    ref = torch.nan_to_num(zi, nan=0.0).T @ xi
    assert torch.equal(dw[: N - 1].double(), ref[: N - 1]) and bool(torch.isnan(dw[N - 1]).all())
    assert torch.equal(db[: N - 1].double(), zi[:, : N - 1].sum(0)) and bool(torch.isnan(db[N - 1]))
    dx = torch.empty(M, K, dtype=t, device="cuda")
    wi = ints(N, K, 18)
    cm.linear_backward_data(d, zi.to(t), wi.to(t), dx, poisoned(d, 1))
    assert torch.equal(dx[: M - 1].double(), (zi[: M - 1] @ wi).to(t).double()) and bool(torch.isnan(dx[M - 1]).all())


@pytest.mark.parametrize("act", range(5))
def test_activation_backward_from_dense_z(act):
    import convolution_layer_amd as cm
    for dtype in (torch.bfloat16, torch.float32):
        z, dy = (torch.randn(19, 77, generator=torch.Generator().manual_seed(i)).to(dtype) for i in (1, 2))
        d = cm.make_linear_desc(19, 5, 77, activation=act, dtype=cm.BF16 if dtype == torch.bfloat16 else cm.F32)
        dz = torch.empty(19, 77, dtype=dtype, device="cuda")
        cm.linear_activation_backward(d, z.cuda(), dy.cuda(), dz)
        ref = R.slope(z.double(), act) * dy.double()
        R.within(dz, ref, R.ACT_ABS * dy.double().abs() + R.HALF[dtype] * ref.abs(), "dz")


def test_empty_batch():
    import convolution_layer_amd as cm
    d = cm.make_linear_desc(0, 64, 32)
    e, w = torch.empty(0, 64, device="cuda"), torch.ones(32, 64, device="cuda")
    y = torch.empty(0, 32, device="cuda")
    cm.linear_forward(d, e, w, None, None, None, y)
    cm.linear_backward_data(d, y, w, e)
    dw, db = torch.full((32, 64), 2.0, device="cuda"), torch.full((32,), 2.0, device="cuda")
    cm.linear_backward_weight(d, e, y, dw, db, 1)
    assert bool((dw == 2).all()) and bool((db == 2).all())
    cm.linear_backward_weight(d, e, y, dw, db, 0)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_gradients_against_differences():
    """dx, dw, db of sum(c * act(x w^T + b)) against central differences in 64 bits."""
    import convolution_layer_amd as cm
    M, K, N = 5, 9, 7
    g = torch.Generator().manual_seed(4)
    x, w, b, c = (torch.randn(*s, generator=g) for s in ((M, K), (N, K), (N,), (M, N)))
    f = lambda x, w, b: float((R.act(x @ w.T + b, 4) * c.double()).sum())  # noqa: E731
    d = cm.make_linear_desc(M, K, N, activation=cm.ACT_GELU)
    z, y, dz, dx = (torch.empty(*s, device="cuda") for s in ((M, N), (M, N), (M, N), (M, K)))
    dw, db = torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    cm.linear_forward(d, x.cuda(), w.cuda(), b.cuda(), None, z, y)
    cm.linear_activation_backward(d, z, c.cuda(), dz)
    cm.linear_backward_data(d, dz, w.cuda(), dx, cm.linear_workspace(d, 1))
    cm.linear_backward_weight(d, x.cuda(), dz, dw, db, 0, cm.linear_workspace(d, 2))
    t = 1e-5
    for k, (v, grad) in enumerate(((x, dx), (w, dw), (b, db))):
        flat = grad.flatten().cpu()
        for i in range(v.numel()):
            p = torch.zeros(v.numel(), dtype=torch.float64)
            p[i] = t
            p = p.reshape(v.shape)
            args = [a.double() for a in (x, w, b)]
            lo, hi = list(args), list(args)
            hi[k], lo[k] = args[k] + p, args[k] - p
            num = (f(*hi) - f(*lo)) / (2 * t)
            assert abs(num - float(flat[i])) <= 2e-5 * (1 + abs(num)), (k, i)  # 6e-8 * ~30 sums, ~1e-6 of the differences


def test_misaligned_and_strided_tensors_are_refused():
    import convolution_layer_amd as cm
    d = cm.make_linear_desc(20, 64, 32, dtype=cm.BF16)
    buf = torch.zeros(20 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    w, y = torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(20, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(cm.ConvmiError) as e:
        cm.linear_forward(d, buf[1:1281].view(20, 64), w, None, None, None, y)
    assert e.value.status == cm.ERR_MISALIGNED
    cm.linear_forward(d, buf[8:1288].view(20, 64), w, None, None, None, y)  # 16 bytes in: aligned
    with pytest.raises(ValueError, match="contiguous"):
        cm.linear_forward(d, torch.zeros(64, 20, dtype=torch.bfloat16, device="cuda").t(), w, None, None, None, y)
    with pytest.raises(ValueError, match="dtype"):
        cm.linear_forward(d, buf[:1280].view(20, 64).float(), w, None, None, None, y)
    with pytest.raises(ValueError, match="elements"):
        cm.linear_forward(d, buf[:640].view(10, 64), w, None, None, None, y)
    with pytest.raises(ValueError, match="device"):
        cm.linear_forward(d, buf[:1280].view(20, 64), w.cpu(), None, None, None, y)
    odd = cm.make_linear_desc(20, 63, 32, dtype=cm.BF16)
    with pytest.raises(cm.ConvmiError) as e:
        cm.linear_forward(odd, buf[:1260], torch.zeros(32 * 63, dtype=torch.bfloat16, device="cuda"), None, None, None, y)
    assert e.value.status == cm.ERR_WORKSPACE


def test_offsets_beyond_32_bits():
    """Outputs of more than 2^31 values: the last rows and columns are right, forward and dX."""
    import convolution_layer_amd as cm
    M, K, N = 600001, 64, 4096
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    xi, wi = ints(3, K, 20), ints(N, K, 21)
    x[-3:] = xi.bfloat16()
    y = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
    d = cm.make_linear_desc(M, K, N, dtype=cm.BF16)
    cm.linear_forward(d, x, wi.bfloat16(), None, None, None, y, cm.linear_workspace(d, 0))
    assert torch.equal(y[-3:].double(), (xi @ wi.T).bfloat16().double())
    assert bool((y[:7] == 0).all()) and bool((y[M // 2] == 0).all())
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    zi = ints(2, N, 22)
    y.zero_()
    y[-2:] = zi.bfloat16()
    cm.linear_backward_data(d, y, wi.bfloat16(), dx, cm.linear_workspace(d, 1))
    assert torch.equal(dx[-2:].double(), (zi @ wi).bfloat16().double()) and bool((dx[:9] == 0).all())


def counts(rows, cols, seed, top):
    """Whole numbers 0..top: their sums grow with the length."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, top + 1, (rows, cols), generator=g, device="cuda").double()


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N,tx,tz,splits", [(100001, 72, 40, 16, 8, True), (100001, 72, 40, 1, 128, True),
                                                (30011, 200, 300, 16, 32, True), (9001, 4096, 4096, 16, 64, False),
                                                (9001, 4096, 4096, 1, 255, False)])
def test_long_sums_of_gradients_keep_their_bits(M, K, N, tx, tz, splits, ty):
    """dw and db whose sums need up to 23 bits, M * tx * tz < 2^24: exact in fp32 in any order, off by
    hundreds where a partial sum is kept in 16 bits.  From dense and from 8-bit x."""
    import convolution_layer_amd as cm
    assert M * tx * tz < 1 << 24
    t, xi, zi = tdt(ty), counts(M, K, 31, tx), counts(M, N, 32, tz)
    rw, rb = zi.T @ xi, zi.sum(0)
    assert max(float(rw.max()), float(rb.max())) > 1 << 20
    dz = zi.to(t)
    for x8 in (False, True):
        d = cm.make_linear_desc(M, K, N, dtype=cm.F32 if ty == "f32" else cm.BF16, x_mx8=x8)
        assert (int(cm.linear_plan_name(d, 2).split(" split ")[1].split()[0]) > 1) == splits
        x, sc = operand(xi, "mx8" if x8 else ty)
        dw, db = torch.full((N, K), 3.0, device="cuda"), torch.full((N,), 4.0, device="cuda")
        for acc in (0, 1):  # twice the sum is still exact
            cm.linear_backward_weight(d, x, dz, dw, db, acc, poisoned(d, 2), x_scales=sc)
            assert torch.equal(dw.double(), rw * (1 + acc)), f"dw, accumulate {acc}"
            assert torch.equal(db.double(), rb * (1 + acc)), f"db, accumulate {acc}"


@pytest.mark.parametrize("ty", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 100003, 48), (5, 65537, 64), (20, 65536, 64), (300, 20000, 300),
                                   (2600, 16400, 2500), (4100, 16384, 4100)])
def test_long_sums_of_the_forward_keep_their_bits(M, K, N, ty):
    """Sums of 22 bits and more, taken away again through the bias: what remains is small and whole, so
    that bf16 outputs show every bit of the sum.  All rows of x are one row."""
    t = tdt(ty)
    top = 16 if K < 30000 else 12
    xi, wi = counts(1, K, 33, top), counts(N, K, 34, top)
    assert K * top * top < 1 << 24
    z = (xi @ wi.T)[0]
    assert float(z.max()) > 1 << 20
    rest = ints(1, N, 35, 9)[0]
    y = torch.empty(M, N, dtype=t, device="cuda")
    forward(desc(M, K, N, ty), operand(xi.repeat(M, 1), ty), operand(wi, ty), (rest - z).float(), None, None, y)
    assert torch.equal(y.double(), rest.expand(M, N))


@pytest.mark.parametrize("M,K,N", [(300, 200, 100000), (2600, 2500, 16400)])
def test_long_sums_of_dx_keep_their_bits(M, K, N):
    import convolution_layer_amd as cm
    top = 12 if N > 30000 else 31
    zi, wi = counts(M, N, 36, top), counts(N, K, 37, top)
    assert N * top * top < 1 << 24
    ref = zi @ wi
    for ty in ("bf16", "f32"):
        t, d = tdt(ty), desc(M, K, N, ty)
        dx = torch.empty(M, K, dtype=t, device="cuda")
        cm.linear_backward_data(d, zi.to(t), wi.to(t), dx, poisoned(d, 1))
        assert torch.equal(dx.double(), ref.to(t).double())
