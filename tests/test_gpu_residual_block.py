"""The operators as they are used together: a pre-norm residual block trained with its
activations kept in 8 bits, run eagerly, twice, on other streams and replayed from graphs."""
import pytest
import torch

from tests import block_reference as R

pytestmark = pytest.mark.gpu

M, D, F = 70, 96, 200  # tokens, model width, hidden width


class Block:
    """h = x + r;  n = rms_norm(h);  u = gelu(n w1^T + b1);  out = u w2^T + b2 + h.
    Kept for the backward pass: h (dense), inv_rms, n, z1 and u in 8 bits."""

    def __init__(self, seed, dtype=torch.bfloat16):
        import convolution_layer_amd as cm
        g = torch.Generator().manual_seed(seed)
        rnd = lambda s, *n: (torch.randn(*n, generator=g) * s)  # noqa: E731
        self.dtype = dtype
        dt = cm.BF16 if dtype == torch.bfloat16 else cm.F32
        self.src = {"x": rnd(1, M, D), "r": rnd(1, M, D), "gamma": 1 + rnd(0.1, D), "w1": rnd(D ** -0.5, F, D),
                    "b1": rnd(0.1, F), "w2": rnd(F ** -0.5, D, F), "b2": rnd(0.1, D), "dout": rnd(1, M, D)}
        for k in ("x", "r", "w1", "w2", "dout"):
            self.src[k] = self.src[k].to(dtype)
        self.t = {k: v.cuda() for k, v in self.src.items()}
        new = lambda n, t: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
        u8 = torch.uint8
        for k, s in (("h", (M, D)), ("n", (M, D)), ("u", (M, F)), ("out", (M, D)), ("du", (M, F)), ("dz", (M, F)),
                     ("dn", (M, D)), ("dx", (M, D))):
            self.t[k] = new(s, dtype)
        for k, s in (("n8", (M, D)), ("z8", (M, F)), ("u8", (M, F))):
            self.t[k], self.t[k + "s"] = new(s, u8), new((M, cm.mx8_blocks(s[1])), u8)
        for k, s in (("inv", (M,)), ("dw1", (F, D)), ("db1", (F,)), ("dw2", (D, F)), ("db2", (D,)), ("dgamma", (D,))):
            self.t[k] = new(s, torch.float32)
        self.norm = cm.make_rms_desc(M, D, dtype=dt)
        self.l1 = cm.make_linear_desc(M, D, F, activation=cm.ACT_GELU, dtype=dt, z_mx8=True)
        self.l2 = cm.make_linear_desc(M, F, D, dtype=dt)
        self.g1 = cm.make_linear_desc(M, D, F, dtype=dt, x_mx8=True)  # gradients read the kept inputs
        self.g2 = cm.make_linear_desc(M, F, D, dtype=dt, x_mx8=True)
        self.ws = {k: cm.linear_workspace(d, op) for k, d, op in (
            ("f1", self.l1, 0), ("f2", self.l2, 0), ("dx2", self.g2, 1), ("dw2", self.g2, 2), ("dx1", self.g1, 1),
            ("dw1", self.g1, 2))}
        self.ws["norm"] = cm.rms_workspace(self.norm)

    def step(self):
        import convolution_layer_amd as cm
        t, ws = self.t, self.ws
        cm.rms_norm_forward(self.norm, t["x"], t["r"], t["gamma"], t["h"], t["n"], t["inv"], y8=t["n8"],
                            y8_scales=t["n8s"])
        cm.linear_forward(self.l1, t["n"], t["w1"], t["b1"], None, t["z8"], t["u"], ws["f1"], z_scales=t["z8s"])
        cm.mx8_pack(t["u"], t["u8"], t["u8s"])
        cm.linear_forward(self.l2, t["u"], t["w2"], t["b2"], t["h"], None, t["out"], ws["f2"])
        cm.linear_backward_weight(self.g2, t["u8"], t["dout"], t["dw2"], t["db2"], 0, ws["dw2"], x_scales=t["u8s"])
        cm.linear_backward_data(self.g2, t["dout"], t["w2"], t["du"], ws["dx2"])
        cm.linear_activation_backward(self.l1, t["z8"], t["du"], t["dz"], z_scales=t["z8s"])
        cm.linear_backward_weight(self.g1, t["n8"], t["dz"], t["dw1"], t["db1"], 0, ws["dw1"], x_scales=t["n8s"])
        cm.linear_backward_data(self.g1, t["dz"], t["w1"], t["dn"], ws["dx1"])
        cm.rms_norm_backward(self.norm, t["h"], t["gamma"], t["inv"], t["dn"], t["dout"], t["dx"], t["dgamma"], 0,
                             ws["norm"])

    OUT = ("out", "dx", "dgamma", "dw1", "db1", "dw2", "db2")

    def results(self):
        return {k: self.t[k].clone() for k in self.OUT}

    def reference(self):
        """The same step in 64 bits, the kept tensors packed by their definition."""
        s = {k: v.double() for k, v in self.src.items()}
        h, inv, n = R.rms_forward(s["x"], s["r"], s["gamma"], float(torch.tensor(1e-5)))
        z = n @ s["w1"].T + s["b1"]
        u = R.act(z, 4)
        out = u @ s["w2"].T + s["b2"] + h
        n8, z8, u8 = (R.keep(v)[2] for v in (n, z, u))
        du = s["dout"] @ s["w2"]
        dz = R.slope(z8, 4) * du
        dx, dgamma = R.rms_backward(h, s["gamma"], inv, dz @ s["w1"], s["dout"])
        return {"out": out, "dx": dx, "dgamma": dgamma, "dw1": dz.T @ n8, "db1": dz.sum(0),
                "dw2": s["dout"].T @ u8, "db2": s["dout"].sum(0)}


@pytest.mark.parametrize("dtype,tol", [(torch.bfloat16, 2e-2), (torch.float32, 4e-3)])
def test_block_step_against_64_bits(dtype, tol):
    """Norm-wise.  bf16: about six chained roundings of 2^-8 at most, 2e-2 as for the layer's
    other bf16 checks.  fp32: a value at a rounding border of its 8-bit form may fall to the
    other side (a step of 2^-3 of one value in some 10^4): 2^-3 * 10^-2 with margin."""
    b = Block(1, dtype)
    b.step()
    for k, ref in b.reference().items():
        got = R.host(b.t[k])
        err = float((got - ref).norm() / ref.norm())
        assert err <= tol, (k, err)


def test_repeats_and_other_streams_agree_bit_for_bit():
    """The step again, on a second stream, and two blocks at once on two streams."""
    a, b = Block(2), Block(3)
    a.step()
    b.step()
    torch.cuda.synchronize()
    want = a.results(), b.results()
    for blk in (a, b):
        for k in blk.OUT:
            blk.t[k].fill_(7)
        for w in blk.ws.values():
            if w is not None:
                w.fill_(255)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s1):
            a.step()
        with torch.cuda.stream(s2):
            b.step()
    torch.cuda.synchronize()
    for blk, w in zip((a, b), want):
        for k, v in blk.results().items():
            R.same(v, w[k], k)


def test_explicit_stream_argument():
    import convolution_layer_amd as cm
    s = torch.cuda.Stream()
    x = torch.randn(50, 64, device="cuda")
    w, y = torch.randn(32, 64, device="cuda"), torch.empty(50, 32, device="cuda")
    ref = torch.empty_like(y)
    d = cm.make_linear_desc(50, 64, 32)
    cm.linear_forward(d, x, w, None, None, None, ref)
    s.wait_stream(torch.cuda.current_stream())
    cm.linear_forward(d, x, w, None, None, None, y, stream=s)
    s.synchronize()
    R.same(y, ref, "y")


def test_step_replays_from_a_graph():
    """Captured once, replayed four times on changed inputs with eager steps of another block
    and synchronizations in between; every replay equals the eager step."""
    a, other = Block(4), Block(5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a.step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for i in range(4):
        fresh = Block(10 + i)
        for k, v in fresh.src.items():
            a.t[k].copy_(v)
        for k in a.OUT:
            a.t[k].fill_(9)
        other.step()
        graph.replay()
        fresh.step()
        torch.cuda.synchronize()
        want = fresh.results()
        for k, v in a.results().items():
            R.same(v, want[k], f"replay {i}: {k}")


def test_two_graphs_with_their_own_workspaces():
    blocks = [Block(6), Block(7)]
    graphs = []
    for b in blocks:
        b.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.step()
        graphs.append((g, b.results()))
    want = []
    for b in blocks:
        b.step()
        torch.cuda.synchronize()
        want.append(b.results())
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for k, v in b.results().items():
            R.same(v, w[k], k)


def test_eight_bit_chain_norm_to_product():
    """The norm's 8-bit output feeds the product of 8-bit operands, with packed weights."""
    import convolution_layer_amd as cm
    g = torch.Generator().manual_seed(8)
    x, w = torch.randn(M, D, generator=g).bfloat16(), (torch.randn(F, D, generator=g) * D ** -0.5).bfloat16()
    gamma = 1 + 0.1 * torch.randn(D, generator=g)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    n8, ns, w8, wsc = u8(M, D), u8(M, cm.mx8_blocks(D)), u8(F, D), u8(F, cm.mx8_blocks(D))
    cm.mx8_pack(w.cuda(), w8, wsc)
    d = cm.make_rms_desc(M, D, dtype=cm.BF16)
    cm.rms_norm_forward(d, x.cuda(), None, gamma.cuda(), None, None, None, y8=n8, y8_scales=ns)
    for rows in (M, 5, 1):
        ld = cm.make_linear_desc(rows, D, F, dtype=cm.BF16, x_mx8=True)
        y = torch.empty(rows, F, dtype=torch.bfloat16, device="cuda")
        cm.linear_forward(ld, n8[:rows], w8, None, None, None, y, cm.linear_workspace(ld, 0), x_scales=ns[:rows],
                          w_scales=wsc)
        xv, wv = R.decode(n8[:rows].cpu(), ns[:rows].cpu()), R.decode(w8.cpu(), wsc.cpu())
        ref = xv @ wv.T
        bound = (2.0 ** -12 + D * 2.0 ** -24) * (xv.abs() @ wv.abs().T) + 2.0 ** -8 * ref.abs()
        R.within(y, ref, bound * (1 + 2.0 ** -8), f"{rows} rows")


def test_two_graphs_write_everything_on_every_replay():
    """Two captured steps replayed in turn, each on new inputs, every output and kept tensor and each
    workspace filled with other values before; compared with an eager step on the same inputs."""
    blocks, graphs = [Block(21), Block(22)], []
    for b in blocks:
        b.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.step()
        graphs.append(g)
    kept = ("h", "n", "u", "du", "dz", "dn", "inv", "n8", "n8s", "z8", "z8s", "u8", "u8s")
    for i in range(4):
        fresh = [Block(30 + 2 * i), Block(31 + 2 * i)]
        for b, f in zip(blocks, fresh):
            for k, v in f.src.items():
                b.t[k].copy_(v)
            for k in Block.OUT + kept:
                b.t[k].fill_(77 + i)
            for w in b.ws.values():
                if w is not None:
                    w.fill_(255)
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        for f in fresh:
            f.step()
        torch.cuda.synchronize()
        for b, f in zip(blocks, fresh):
            for k in Block.OUT + kept:
                R.same(b.t[k], f.t[k], f"replay {i}: {k}")
