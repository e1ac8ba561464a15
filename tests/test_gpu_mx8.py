"""MX8 packing, unpacking, the activation derivative at kept values and the convolution's
backward pass from kept tensors, on the GPU.  Packing is exact: codes and scales must equal
the 64-bit definition's bit for bit."""
import pytest
import torch

from tests import block_reference as R

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (5, 7), (4, 8), (7, 64), (9, 100), (2, 4096), (33, 1003), (3, 9000),
          (513, 96), (1, 70001)]
DTYPES = [torch.bfloat16, torch.float32]


def pack(x):
    import convolution_layer_amd as cm
    q = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    s = torch.empty(x.shape[0], cm.mx8_blocks(x.shape[1]), dtype=torch.uint8, device="cuda")
    cm.mx8_pack(x, q, s)
    return q, s


def values(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, cols), generator=g).float())
    v[torch.rand(rows, cols, generator=g) < 0.05] = 0.0
    return v


def codes_equal(got, ref):
    """Equal codes; NaN codes may carry either sign."""
    got, ref = got.cpu().long(), ref.long()
    nan = (ref & 127) == 127
    assert torch.equal(got[~nan], ref[~nan]) and bool(((got[nan] & 127) == 127).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_pack_and_unpack_are_exact(rows, cols, dtype):
    import convolution_layer_amd as cm
    x = values(rows, cols, rows * 7 + cols).to(dtype)
    c, e, v = R.keep(x.double())
    q, s = pack(x.cuda())
    codes_equal(q, c)
    assert torch.equal(s.cpu().long(), e)
    for out in DTYPES:
        back = torch.full((rows, cols), 7.0, dtype=out, device="cuda")
        cm.mx8_unpack(q, s, back)
        assert torch.equal(back.double().cpu(), v)  # 4 significant bits fit both types


@pytest.mark.parametrize("dtype", DTYPES)
def test_pack_extremes(dtype):
    """Largest and smallest magnitudes, subnormals, ties, infinities and NaN."""
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).tiny
    rows = torch.zeros(9, 64, dtype=torch.float64)
    rows[0, :4] = torch.tensor([big, -big, 1.0, tiny])
    rows[1, :4] = torch.tensor([tiny, tiny / 4, -tiny / 2, 0.0])
    rows[2] = torch.arange(64) / 2.0                          # ties between e4m3 neighbours
    rows[3, :6] = torch.tensor([float("inf"), 1.0, -3.0, float("nan"), -float("inf"), 0.01])
    rows[4] = float("nan")
    rows[5, 32:] = 448.0
    rows[6, :2] = torch.tensor([452.0, 448.0])                # just beyond: the next scale
    rows[7] = -0.0
    rows[8] = 2.0 ** -130 if dtype == torch.float32 else 2.0 ** -126
    x = rows.to(dtype)
    c, e, v = R.keep(x.double())
    q, s = pack(x.cuda())
    assert torch.equal(s.cpu().long(), e)
    codes_equal(q, c)
    import convolution_layer_amd as cm
    back = torch.empty(9, 64, device="cuda")
    cm.mx8_unpack(q, s, back)
    assert torch.equal(torch.isnan(back.cpu()), torch.isnan(v))
    assert torch.equal(torch.nan_to_num(back.double().cpu()), torch.nan_to_num(v))


def test_unpack_takes_any_scale_byte():
    """All 256 codes under all 256 scale bytes: 0 is 2^-127, 255 is NaN."""
    import convolution_layer_amd as cm
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).reshape(256, 1).repeat(1, 8)
    ref = R.decode(codes, scales)
    ref = ref.float()  # beyond fp32's range only at the very top and bottom: rounded once
    got = torch.empty(256, 256, device="cuda")
    cm.mx8_unpack(codes.cuda(), scales.cuda(), got)
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(ref))
    assert torch.equal(torch.nan_to_num(got.cpu()), torch.nan_to_num(ref))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (16, 64), (5, 1003), (130, 256)])
def test_activation_backward_at_kept_values(rows, cols, act, dtype):
    import convolution_layer_amd as cm
    z = values(rows, cols, 11).to(dtype)
    dy = torch.randn(rows, cols, generator=torch.Generator().manual_seed(5)).to(dtype)
    _, _, kept = R.keep(z.double())
    q, s = pack(z.cuda())
    d = cm.make_linear_desc(rows, 1, cols, activation=act, dtype=cm.BF16 if dtype == torch.bfloat16 else cm.F32,
                            z_mx8=True)
    dz = torch.full((rows + 1, cols), 5.0, dtype=dtype, device="cuda")
    cm.linear_activation_backward(d, q, dy.cuda(), dz[:rows], z_scales=s)
    ref = R.slope(kept, act) * dy.double()
    R.within(dz[:rows], ref, R.ACT_ABS * dy.double().abs() + R.HALF[dtype] * ref.abs(), "dz")
    assert bool((dz[rows] == 5.0).all())
    inplace = dy.cuda()
    cm.linear_activation_backward(d, q, inplace, inplace, z_scales=s)
    R.same(inplace, dz[:rows].contiguous(), "in place")


CONV = [((2, 12, 20, 64, 64, 3, 3), (1, 1), (1, 1), torch.bfloat16, 2), ((1, 9, 7, 5, 9, 3, 2), (2, 1), (1, 0), torch.bfloat16, 3),
        ((2, 16, 16, 64, 64, 3, 3), (1, 1), (1, 1), torch.float32, 1), ((3, 10, 11, 24, 40, 1, 1), (1, 1), (0, 0), torch.bfloat16, 4),
        ((2, 8, 8, 3, 8, 3, 3), (1, 1), (1, 1), torch.float32, 0)]


@pytest.mark.parametrize("case", CONV)
@pytest.mark.parametrize("which", ["both", "x", "saved"])
def test_conv_backward_full_from_kept_tensors(case, which):
    """Bit for bit conv2d_backward_full on the unpacked tensors, with a poisoned workspace,
    from z and (where the activation allows it) from y, adding into existing gradients too."""
    import convolution_layer_amd as cm
    (N, H, W, IC, OC, KH, KW), stride, pad, dtype, act = case
    d = cm.make_desc(N, H, W, IC, OC, KH, KW, stride=stride, pad=pad, activation=act,
                     dtype=cm.BF16 if dtype == torch.bfloat16 else cm.F32)
    oh, ow = cm.output_dims(d)
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, w, dy = rnd(N * H * W, IC), rnd(OC, KH, KW, IC), rnd(N * oh * ow, OC)
    q, s = pack(x)
    xv = torch.empty_like(x)
    cm.mx8_unpack(q, s, xv)
    for from_y in ([0, 1] if act != cm.ACT_GELU else [0]):
        saved = torch.rand(N * oh * ow, OC, generator=g, device="cuda").to(dtype) if from_y else rnd(N * oh * ow, OC)
        sq, ss = pack(saved)
        sv = torch.empty_like(saved)
        cm.mx8_unpack(sq, ss, sv)
        xa, xsc = (x if which == "saved" else q), (None if which == "saved" else s)
        sa, ssc = (saved if which == "x" else sq), (None if which == "x" else ss)
        for acc in (0, 1):
            outs = []
            for mx in (False, True):
                dx = torch.empty(N * H * W, IC, dtype=dtype, device="cuda")
                dw, db = torch.ones(OC, KH, KW, IC, device="cuda"), torch.ones(OC, device="cuda")
                ws = cm.workspace(d, cm.OP_BACKWARD_FULL_MX8)
                ws.fill_(255)
                if mx:
                    cm.conv2d_backward_full_mx8(d, xa, xsc, w, sa, ssc, from_y, dy, dx, dw, db, acc, ws)
                else:
                    cm.conv2d_backward_full(d, x if which == "saved" else xv, w, saved if which == "x" else sv, from_y,
                                            dy, dx, dw, db, acc, ws)
                outs.append((dx, dw, db))
            for a, b, n in zip(*outs, ("dx", "dw", "db")):
                R.same(a, b, f"{n} from_y={from_y} acc={acc}")


PADDED = [((5, 42, 36, 55, 65, 1, 1), (1, 1), (0, 0), torch.bfloat16), ((6, 30, 11, 61, 103, 1, 1), (1, 1), (0, 0), torch.float32),
          ((3, 48, 32, 111, 8, 3, 3), (1, 1), (1, 1), torch.bfloat16), ((8, 33, 39, 4, 26, 3, 3), (2, 1), (1, 0), torch.float32),
          ((9, 15, 11, 64, 11, 3, 3), (1, 1), (1, 1), torch.bfloat16), ((4, 30, 31, 33, 47, 5, 2), (2, 3), (2, 1), torch.bfloat16)]


@pytest.mark.parametrize("case", PADDED)
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("which", ["both", "x", "saved"])
def test_conv_backward_on_padded_channels(case, act, which):
    """Channel counts that the tiled products do not take, with enough work to be padded.  Whole
    numbers: every sum is exact in any order, so the results equal conv2d_backward_full's bit for
    bit; the padding reads nothing behind the tensors' ends (NaN there) and writes nothing there."""
    import convolution_layer_amd as cm
    (N, H, W, IC, OC, KH, KW), stride, pad, dtype = case
    d = cm.make_desc(N, H, W, IC, OC, KH, KW, stride=stride, pad=pad, activation=act,
                     dtype=cm.BF16 if dtype == torch.bfloat16 else cm.F32)
    oh, ow = cm.output_dims(d)
    assert 2 * N * oh * ow * OC * KH * KW * IC > 6e6
    assert cm.workspace_size(d, cm.OP_BACKWARD_FULL_MX8) > cm.workspace_size(d, cm.OP_BACKWARD_FULL) + N * H * W * IC * (
        2 if dtype == torch.bfloat16 else 4) + 4096, "the padded path"
    g = torch.Generator(device="cuda").manual_seed(4)

    def ints(rows, cols):  # a row of NaN behind the last
        t = torch.randint(-2, 3, (rows + 1, cols), generator=g, device="cuda").to(dtype)
        t[rows] = float("nan")
        return t[:rows]

    x, w, dy = ints(N * H * W, IC), ints(OC * KH * KW, IC).reshape(OC, KH, KW, IC), ints(N * oh * ow, OC)
    saved = ints(N * oh * ow, OC).abs()
    q, s = pack(x)
    sq, ss = pack(saved)
    want, res = [], []
    for acc in (0, 1):
        for mx, out in ((False, want), (True, res)):
            dx = torch.full((N * H * W + 1, IC), 6.0, dtype=dtype, device="cuda")
            dw, db = torch.full((OC + 1, KH, KW, IC), 2.0, device="cuda"), torch.full((OC + 1,), 2.0, device="cuda")
            ws = cm.workspace(d, cm.OP_BACKWARD_FULL_MX8)
            ws.fill_(255)
            if mx:
                xa, xs = (x, None) if which == "saved" else (q, s)
                sa, sc = (saved, None) if which == "x" else (sq, ss)
                cm.conv2d_backward_full_mx8(d, xa, xs, w, sa, sc, 1, dy, dx[:-1], dw[:-1], db[:-1], acc, ws)
            else:
                cm.conv2d_backward_full(d, x, w, saved, 1, dy, dx[:-1], dw[:-1], db[:-1], acc, ws)
            assert bool((dx[-1] == 6).all()) and bool((dw[-1] == 2).all()) and float(db[-1]) == 2.0
            out.extend([dx, dw, db])
    for i, (a, b) in enumerate(zip(want, res)):
        R.same(a, b, f"output {i}")
    dw = torch.empty(OC, KH, KW, IC, device="cuda")  # neither dx nor db
    ws = cm.workspace(d, cm.OP_BACKWARD_FULL_MX8)
    cm.conv2d_backward_full_mx8(d, q, s, w, sq, ss, 1, dy, None, dw, None, 0, ws)
    R.same(dw, want[1][:-1].contiguous(), "dw alone")


DENSE = [((1, 44, 62, 12, 112, 7, 7), (3, 3), torch.float32), ((32, 5, 20, 12, 256, 5, 5), (2, 2), torch.float32),
         ((5, 42, 36, 55, 65, 1, 1), (0, 0), torch.bfloat16), ((2, 12, 20, 64, 64, 3, 3), (1, 1), torch.bfloat16)]


@pytest.mark.parametrize("case", DENSE)
@pytest.mark.parametrize("act", [0, 3])
def test_conv_backward_full_mx8_of_dense_tensors(case, act):
    """Neither tensor in 8 bits: bit for bit conv2d_backward_full, in a workspace of the size that the
    8-bit call asks for, with nothing written behind it."""
    import convolution_layer_amd as cm
    (N, H, W, IC, OC, KH, KW), pad, dtype = case
    d = cm.make_desc(N, H, W, IC, OC, KH, KW, pad=pad, activation=act,
                     dtype=cm.BF16 if dtype == torch.bfloat16 else cm.F32)
    oh, ow = cm.output_dims(d)
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, w, dy, z = rnd(N * H * W, IC), rnd(OC, KH, KW, IC), rnd(N * oh * ow, OC), rnd(N * oh * ow, OC)
    res = []
    for op in (cm.OP_BACKWARD_FULL, cm.OP_BACKWARD_FULL_MX8):
        n = cm.workspace_size(d, op)
        ws = torch.full((n + (4 << 20),), 255, dtype=torch.uint8, device="cuda")
        dx, dw, db = torch.empty_like(x), torch.empty(OC, KH, KW, IC, device="cuda"), torch.empty(OC, device="cuda")
        if op == cm.OP_BACKWARD_FULL:
            cm.conv2d_backward_full(d, x, w, z, 0, dy, dx, dw, db, 0, ws[:n])
        else:
            cm.conv2d_backward_full_mx8(d, x, None, w, z, None, 0, dy, dx, dw, db, 0, ws[:n])
        assert bool((ws[n:] == 255).all()), "behind the workspace"
        res.append((dx, dw, db))
    for a, b, what in zip(*res, ("dx", "dw", "db")):
        R.same(a, b, what)


@pytest.mark.parametrize("seed", range(24))
def test_conv_backward_of_random_layers_stays_in_its_buffers(seed):
    """Random layers, whole numbers, either tensor in 8 bits or dense: bit for bit conv2d_backward_full, NaN
    behind every input, and nothing written behind the workspace or an output."""
    import random
    import convolution_layer_amd as cm
    r = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for _ in range(6):
        N, H, W, k, st = r.randint(1, 5), r.randint(1, 40), r.randint(1, 40), r.choice([1, 2, 3, 5]), r.choice([1, 1, 2])
        IC, OC = (r.choice([r.randint(1, 140), 4 * r.randint(1, 35), 64]) for _ in range(2))
        if min(H, W) + 2 * (k // 2) < k:
            continue
        dtype, act = r.choice(DTYPES), r.choice([0, 1])
        d = cm.make_desc(N, H, W, IC, OC, k, k, stride=(st, st), pad=(k // 2, k // 2), activation=act,
                         dtype=cm.BF16 if dtype == torch.bfloat16 else cm.F32)
        oh, ow = cm.output_dims(d)
        behind = []

        def buf(n, t, fill):
            b = torch.full((n + 4096,), fill, dtype=t, device="cuda")
            behind.append((b[n:], b[n:].clone()))
            return b[:n]

        def ints(rows, cols):
            t = buf(rows * cols, dtype, float("nan"))
            t.copy_(torch.randint(-2, 3, (rows * cols,), generator=g, device="cuda"))
            return t.view(rows, cols)

        x, w, dy, saved = ints(N * H * W, IC), ints(OC * k * k, IC), ints(N * oh * ow, OC), ints(N * oh * ow, OC)
        res = []
        for op in (cm.OP_BACKWARD_FULL, cm.OP_BACKWARD_FULL_MX8):
            n = cm.workspace_size(d, op)
            ws = buf(n, torch.uint8, 255)
            out = (buf(x.numel(), dtype, 5), buf(w.numel(), torch.float32, 5), buf(OC, torch.float32, 5))
            if op == cm.OP_BACKWARD_FULL:
                cm.conv2d_backward_full(d, x, w, saved, 0, dy, *out, 0, ws if n else None)
            else:
                xa, xs = pack(x) if r.random() < 0.6 else (x, None)
                sa, ss = pack(saved) if r.random() < 0.6 else (saved, None)
                cm.conv2d_backward_full_mx8(d, xa, xs, w, sa, ss, 0, dy, *out, 0, ws)
            res.append(out)
        what = (N, H, W, IC, OC, k, st, act, dtype)
        for a, b in zip(*res):
            R.same(a, b, str(what))
        for now, then in behind:
            assert torch.equal(now.view(torch.uint8), then.view(torch.uint8)), what


@pytest.mark.parametrize("case", [((2, 12, 20, 64, 64, 3, 3), (1, 1), torch.bfloat16),   # dW on the second stream
                                  ((3, 48, 32, 111, 8, 3, 3), (1, 1), torch.bfloat16),   # padded
                                  ((9, 15, 11, 64, 11, 3, 3), (1, 1), torch.bfloat16),
                                  ((6, 30, 11, 61, 103, 1, 1), (0, 0), torch.float32)])
def test_conv_backward_replays_from_a_graph(case):
    """Captured once and replayed four times on new inputs, with outputs and workspace overwritten and
    eager calls of another layer in between: every replay equals the eager call."""
    import convolution_layer_amd as cm
    (N, H, W, IC, OC, KH, KW), pad, dtype = case
    d = cm.make_desc(N, H, W, IC, OC, KH, KW, pad=pad, activation=cm.ACT_RELU,
                     dtype=cm.BF16 if dtype == torch.bfloat16 else cm.F32)
    oh, ow = cm.output_dims(d)

    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
        q, s = pack(rnd(N * H * W, IC))
        sq, ss = pack(rnd(N * oh * ow, OC).relu())
        return [q, s, rnd(OC, KH, KW, IC), sq, ss, rnd(N * oh * ow, OC)]

    def outputs():
        return [torch.full((N * H * W, IC), 5.0, dtype=dtype, device="cuda"),
                torch.full((OC, KH, KW, IC), 5.0, device="cuda"), torch.full((OC,), 5.0, device="cuda")]

    def call(i, o, ws):
        q, s, w, sq, ss, dy = i
        cm.conv2d_backward_full_mx8(d, q, s, w, sq, ss, 1, dy, *o, 0, ws)

    mine, out, ws = inputs(0), outputs(), cm.workspace(d, cm.OP_BACKWARD_FULL_MX8)
    call(mine, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(mine, out, ws)
    for i in range(1, 5):
        fresh, want, other = inputs(i), outputs(), cm.workspace(d, cm.OP_BACKWARD_FULL_MX8)
        for a, b in zip(mine, fresh):
            a.copy_(b)
        for o in out:
            o.fill_(9)
        ws.fill_(255)
        graph.replay()
        call(fresh, want, other)
        torch.cuda.synchronize()
        for a, b, n in zip(out, want, ("dx", "dw", "db")):
            R.same(a, b, f"replay {i}: {n}")


def test_conv_backward_first_layer_has_no_dx():
    import convolution_layer_amd as cm
    d = cm.make_desc(2, 8, 8, 16, 16, 3, 3, pad=(1, 1), activation=cm.ACT_RELU, dtype=cm.BF16)
    x = torch.randn(128, 16, device="cuda").bfloat16()
    w, dy = torch.randn(16, 3, 3, 16, device="cuda").bfloat16(), torch.randn(128, 16, device="cuda").bfloat16()
    q, s = pack(x)
    xv = torch.empty_like(x)
    cm.mx8_unpack(q, s, xv)
    res = []
    for mx in (0, 1):
        dw = torch.empty(16, 3, 3, 16, device="cuda")
        ws = cm.workspace(d, cm.OP_BACKWARD_FULL_MX8)
        if mx:
            cm.conv2d_backward_full_mx8(d, q, s, w, q, s, 1, dy, None, dw, None, 0, ws)
        else:
            cm.conv2d_backward_full(d, xv, w, xv, 1, dy, None, dw, None, 0, ws)
        res.append(dw)
    R.same(*res, "dw")


def test_offsets_beyond_32_bits():
    """A tensor of more than 2^31 values and 2^32 bytes: its last rows come out right."""
    import convolution_layer_amd as cm
    rows, cols = 70001, 32800
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = values(3, cols, 8).bfloat16()
    x[-3:] = tail.cuda()
    q, s = pack(x)
    c, e, v = R.keep(tail.double())
    codes_equal(q[-3:], c)
    assert torch.equal(s[-3:].cpu().long(), e)
    x.fill_(9.0)
    cm.mx8_unpack(q, s, x)
    assert torch.equal(x[-3:].double().cpu(), v) and bool((x[:5] == 0).all())
