"""RMS norm, linear layer and MX8 at the edges of what their documentation allows: the largest
feature counts, very many rows, vectors at 4-byte addresses, every accepted torch type, and the
8-bit convolution backward pass replayed from graphs."""
import pytest
import torch

from tests import block_reference as R
from tests.test_gpu_linear import desc, ints, operand, poisoned, tdt
from tests.test_gpu_mx8 import pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ty", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("M", [3, 20])
def test_most_input_features(M, ty):
    """K = 2^20: whole numbers, sums below 2^24."""
    import convolution_layer_amd as cm
    K, N, t = 1 << 20, 24, tdt(ty)
    xi, wi, zi = ints(M, K, 1), ints(N, K, 2), ints(M, N, 3)
    d = desc(M, K, N, ty)
    x, w = operand(xi, ty), operand(wi, ty)
    y = torch.empty(M, N, dtype=t, device="cuda")
    cm.linear_forward(d, x[0], w[0], None, None, None, y, workspace=poisoned(d, 0), x_scales=x[1], w_scales=w[1])
    assert torch.equal(y.double(), (xi @ wi.T).to(t).double())
    if ty == "mx8":
        return
    dx = torch.empty(M, K, dtype=t, device="cuda")
    cm.linear_backward_data(d, zi.to(t), w[0], dx, poisoned(d, 1))
    assert torch.equal(dx.double(), (zi @ wi).to(t).double())
    dw, db = torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    cm.linear_backward_weight(d, x[0], zi.to(t), dw, db, 0, poisoned(d, 2))
    assert torch.equal(dw.double(), zi.T @ xi) and torch.equal(db.double(), zi.sum(0))


@pytest.mark.parametrize("M", [2, 33])
def test_most_output_features(M):
    """N = 2^20, z kept in 8 bits."""
    import convolution_layer_amd as cm
    K, N = 40, 1 << 20
    xi, wi, zi = ints(M, K, 4), ints(N, K, 5), ints(M, N, 6, 1)
    d = cm.make_linear_desc(M, K, N, dtype=cm.BF16, z_mx8=True)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(M, N, dtype=torch.uint8, device="cuda")
    s = torch.empty(M, N // 32, dtype=torch.uint8, device="cuda")
    cm.linear_forward(d, xi.bfloat16(), wi.bfloat16(), None, None, q, y, workspace=poisoned(d, 0), z_scales=s)
    ref = xi @ wi.T
    assert torch.equal(y.double(), ref.bfloat16().double())
    e = R.scale_bytes(ref[-1:].cpu())
    assert torch.equal(s[-1:].cpu().long(), e)
    dx, dw, db = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    cm.linear_backward_data(d, zi.bfloat16(), wi.bfloat16(), dx, poisoned(d, 1))
    assert torch.equal(dx.double(), (zi @ wi).bfloat16().double())
    cm.linear_backward_weight(d, xi.bfloat16(), zi.bfloat16(), dw, db, 0, poisoned(d, 2))
    assert torch.equal(dw.double(), zi.T @ xi) and torch.equal(db.double(), zi.sum(0))


@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_very_many_rows(ty):
    """2^25 + 3 rows, zero but for the last few: outputs, gradients and 8-bit x."""
    import convolution_layer_amd as cm
    M, K, N, t = (1 << 25) + 3, 8, 16, tdt(ty)
    xi, wi, zi = ints(5, K, 7), ints(N, K, 8), ints(5, N, 9)
    x, dz = torch.zeros(M, K, dtype=t, device="cuda"), torch.zeros(M, N, dtype=t, device="cuda")
    x[-5:], dz[-5:] = xi.to(t), zi.to(t)
    y, w = torch.full((M, N), 4.0, dtype=t, device="cuda"), wi.to(t)
    d = desc(M, K, N, ty)
    cm.linear_forward(d, x, w, None, None, None, y, workspace=poisoned(d, 0))
    assert torch.equal(y[-5:].double(), (xi @ wi.T).to(t).double()) and bool((y[:-5] == 0).all())
    dw, db = torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    cm.linear_backward_weight(d, x, dz, dw, db, 0, poisoned(d, 2))
    assert torch.equal(dw.double(), zi.T @ xi) and torch.equal(db.double(), zi.sum(0))
    q, s = pack(x)
    d8 = cm.make_linear_desc(M, K, N, dtype=d.dtype, x_mx8=True)
    cm.linear_backward_weight(d8, q, dz, dw, db, 0, poisoned(d8, 2), x_scales=s)
    assert torch.equal(dw.double(), zi.T @ xi)
    dx = torch.full((M, K), 4.0, dtype=t, device="cuda")
    cm.linear_backward_data(d, dz, w, dx, poisoned(d, 1))
    assert torch.equal(dx[-5:].double(), (zi @ wi).to(t).double()) and bool((dx[:-5] == 0).all())


def test_rms_of_very_many_short_rows():
    import convolution_layer_amd as cm
    rows, cols = (1 << 26) + 7, 3
    h = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(7, cols, generator=torch.Generator().manual_seed(1)).bfloat16()
    h[-7:] = tail.cuda()
    gamma = torch.tensor([1.0, 2.0, 0.5])
    d = cm.make_rms_desc(rows, cols, dtype=cm.BF16)
    y, inv = torch.empty_like(h), torch.empty(rows, device="cuda")
    cm.rms_norm_forward(d, h, None, gamma.cuda(), None, y, inv)
    _, ri, ry = R.rms_forward(tail, None, gamma, float(torch.tensor(1e-5)))
    R.within(y[-7:], ry, (2.0 ** -18 + 2.0 ** -8) * ry.abs(), "y")
    dy = torch.zeros_like(h)
    dy[-7:] = 1.0
    dx, dg = torch.empty_like(h), torch.empty(cols, device="cuda")
    cm.rms_norm_backward(d, h, gamma.cuda(), inv, dy, None, dx, dg, 0, cm.rms_workspace(d))
    _, rg = R.rms_backward(tail, gamma, R.host(inv[-7:]), torch.ones(7, cols), None)
    R.within(dg, rg, 2.0 ** -18 * (tail.double() * ri[:, None]).abs().sum(0), "dgamma")
    assert bool((dx[:-7] == 0).all())


def test_pieces_beyond_32_bits():
    """2^29 + 5 rows of one value: more than 2^31 pieces, split between rows by 64-bit division."""
    import convolution_layer_amd as cm
    rows = (1 << 29) + 5
    x = torch.zeros(rows, 1, dtype=torch.bfloat16, device="cuda")
    tail = torch.tensor([[1.0], [-3.0], [0.0], [448.0], [1e-3]], dtype=torch.bfloat16)
    x[-5:] = tail.cuda()
    q, s = pack(x)
    c, e, v = R.keep(tail.double())
    assert torch.equal(q[-5:].cpu().long(), c) and torch.equal(s[-5:].cpu().long(), e)
    cm.mx8_unpack(q, s, x)
    assert torch.equal(x[-5:].double().cpu(), v)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_vectors_at_four_byte_addresses(off):
    """bias, gamma, inv_rms, dgamma, db need only their element's alignment."""
    import convolution_layer_amd as cm
    M, K, N = 40, 64, 96

    def at(n, fill=None):
        t = torch.zeros(n + 4, device="cuda") if fill is None else torch.randn(n + 4, generator=fill, device="cuda")
        return t[off:off + n]

    g = torch.Generator(device="cuda").manual_seed(off)
    x, w = torch.randn(M, K, generator=g, device="cuda"), torch.randn(N, K, generator=g, device="cuda")
    bias, gamma = at(N, g), at(K, g)
    for rows in (M, 3):
        d = cm.make_linear_desc(rows, K, N)
        y, ref = torch.empty(rows, N, device="cuda"), torch.empty(rows, N, device="cuda")
        cm.linear_forward(d, x[:rows], w, bias, None, None, y, poisoned(d, 0))
        cm.linear_forward(d, x[:rows], w, bias.clone(), None, None, ref, poisoned(d, 0))
        R.same(y, ref, "y")
    dw, db, rb = torch.empty(N, K, device="cuda"), at(N), torch.empty(N, device="cuda")
    d = cm.make_linear_desc(M, K, N)
    cm.linear_backward_weight(d, x, y.new_ones(M, N), dw, db, 0, poisoned(d, 2))
    cm.linear_backward_weight(d, x, y.new_ones(M, N), dw, rb, 0, poisoned(d, 2))
    R.same(db.clone(), rb, "db")
    rd = cm.make_rms_desc(M, K)
    out = []
    for inv, dg, ga in ((at(M), at(K), gamma), (torch.empty(M, device="cuda"), torch.empty(K, device="cuda"), gamma.clone())):
        n, dx = torch.empty(M, K, device="cuda"), torch.empty(M, K, device="cuda")
        cm.rms_norm_forward(rd, x, None, ga, None, n, inv)
        cm.rms_norm_backward(rd, x, ga, inv, n, None, dx, dg, 0, cm.rms_workspace(rd))
        out.append([v.clone() for v in (n, dx, inv, dg)])
    for a, b in zip(*out):
        R.same(a, b, "norm")


def test_torchs_float8_types_are_taken():
    """float8_e4m3fn codes and float8_e8m0fnu scales are the same bytes as uint8 ones, and hold the
    values that torch gives them."""
    import convolution_layer_amd as cm
    x = torch.randn(20, 96, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    q, s = pack(x)
    q8 = torch.empty(20, 96, dtype=torch.float8_e4m3fn, device="cuda")
    s8 = torch.empty(20, 3, dtype=torch.float8_e8m0fnu, device="cuda")
    cm.mx8_pack(x, q8, s8)
    R.same(q8, q, "codes")
    R.same(s8, s, "scales")
    back = torch.empty(20, 96, device="cuda")
    cm.mx8_unpack(q8, s8, back)
    assert torch.equal(back, q8.float() * s8.float().repeat_interleave(32, 1))
    y, ref = (torch.empty(20, 20, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    d = cm.make_linear_desc(20, 96, 20, dtype=cm.BF16, x_mx8=True)
    cm.linear_forward(d, q8, q8, None, None, None, y, poisoned(d, 0), x_scales=s8, w_scales=s8)
    cm.linear_forward(d, q, q, None, None, None, ref, poisoned(d, 0), x_scales=s, w_scales=s)
    R.same(y, ref, "y")


@pytest.mark.parametrize("shape", [(2, 24, 40, 64, 64, 3, 3), (5, 42, 36, 55, 65, 1, 1), (4, 14, 16, 128, 128, 3, 3)])
def test_conv_backward_replays_from_a_graph(shape):
    """The forked (64 channels), the padded and the plain path: captured once, replayed three
    times on new inputs with eager calls in between, each replay equal to the eager call."""
    import convolution_layer_amd as cm
    N, H, W, IC, OC, KH, KW = shape
    d = cm.make_desc(N, H, W, IC, OC, KH, KW, pad=(KH // 2, KW // 2), activation=cm.ACT_TANH, dtype=cm.BF16)
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *n: torch.randn(*n, generator=g, device="cuda").bfloat16()  # noqa: E731
    P = N * H * W

    def fresh():
        q, s = pack(rnd(P, IC))
        yq, ys = pack(torch.rand(P, OC, generator=g, device="cuda").bfloat16())
        return [q, s, rnd(OC, KH, KW, IC), yq, ys, rnd(P, OC)]

    def outputs():
        return [torch.full((P, IC), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((OC, KH, KW, IC), 3.0, device="cuda"),
                torch.full((OC,), 3.0, device="cuda")]

    def call(i, o, ws):
        cm.conv2d_backward_full_mx8(d, i[0], i[1], i[2], i[3], i[4], 1, i[5], o[0], o[1], o[2], 0, ws)

    held, out, ws = fresh(), outputs(), cm.workspace(d, cm.OP_BACKWARD_FULL_MX8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(held, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held, out, ws)
    for _ in range(3):
        new, want = fresh(), outputs()
        for a, b in zip(held, new):
            a.copy_(b)
        for o in out:
            o.fill_(9.0)
        graph.replay()
        call(new, want, cm.workspace(d, cm.OP_BACKWARD_FULL_MX8))
        torch.cuda.synchronize()
        for a, b, n in zip(out, want, ("dx", "dw", "db")):
            R.same(a, b, n)
