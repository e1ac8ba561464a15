"""The operators along sequences as they are used together: a pre-norm block that mixes along ragged
sequences, trained, then run token by token from its prompts' states; eagerly, on other streams and
replayed from graphs.

    n = layer_norm(h);  (u | z) = n w_in^T;  c = silu(causal_conv(u));  dt = c w_dt^T
    (B | C) = c w_bc^T;  y = selective_scan(c, dt, B, C, z);  out = y w_out^T + h
"""
import pytest
import torch

from tests import block_reference as R

pytestmark = pytest.mark.gpu

M, D, E, N, W = 90, 40, 72, 16, 4  # tokens, model width, channels, states, taps
STARTS = (0, 33, 34, 90)
EPS = 1e-5


class Block:
    def __init__(self, seed, dtype=torch.float32, rows=M, starts=STARTS):
        import convolution_layer_amd as cm
        self.cm, self.dtype, self.rows, self.starts = cm, dtype, rows, starts
        dt = cm.BF16 if dtype == torch.bfloat16 else cm.F32
        g = torch.Generator().manual_seed(seed)
        rnd = lambda s, *n: torch.randn(*n, generator=g) * s  # noqa: E731
        self.src = {"h": rnd(1, rows, D), "gamma": 1 + rnd(0.1, D), "beta": rnd(0.1, D), "w_in": rnd(D ** -0.5, 2 * E, D),
                    "w_conv": rnd(0.5, E, W), "b_conv": rnd(0.1, E), "w_dt": rnd(E ** -0.5, E, E),
                    "w_bc": rnd(E ** -0.5, 2 * N, E), "dt_bias": rnd(1, E) - 2,
                    "A": -(0.5 + torch.rand(E, N, generator=g) * 3), "Dp": 1 + rnd(0.1, E),
                    "w_out": rnd(E ** -0.5, D, E), "dout": rnd(1, rows, D)}
        for k in ("h", "w_in", "w_conv", "w_dt", "w_bc", "w_out", "dout"):
            self.src[k] = self.src[k].to(dtype)
        self.t = {k: v.cuda() for k, v in self.src.items()}
        self.st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        b = self.batch = len(starts) - 1
        new = lambda s, t=dtype: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        f32 = torch.float32
        for k, s in (("n", (rows, D)), ("xz", (rows, 2 * E)), ("c", (rows, E)), ("dt", (rows, E)), ("bc", (rows, 2 * N)),
                     ("y", (rows, E)), ("out", (rows, D)), ("dy", (rows, E)), ("dxz", (rows, 2 * E)), ("dc", (rows, E)),
                     ("ddt", (rows, E)), ("dbc", (rows, 2 * N)), ("dc2", (rows, E)), ("dc3", (rows, E)), ("dn", (rows, D)),
                     ("dh", (rows, D)), ("conv_state", (b, W - 1, E))):
            self.t[k] = new(s)
        for k, s in (("mean", (rows,)), ("inv", (rows,)), ("state", (b, E, N))):
            self.t[k] = new(s, f32)
        self.grads = ("dh", "dw_in", "dw_conv", "db_conv", "dw_dt", "dw_bc", "d_dt_bias", "dA", "dDp", "dw_out", "dgamma",
                      "dbeta")
        for k in self.grads[1:]:
            like = {"d_dt_bias": "dt_bias"}.get(k, k[1:])
            self.t[k] = new(tuple(self.src[like].shape), f32)
        self.norm = cm.make_layer_norm_desc(rows, D, dtype=dt, eps=EPS)
        self.lin = {"in": (D, 2 * E), "dt": (E, E), "bc": (E, 2 * N), "out": (E, D)}
        self.lin = {k: cm.make_linear_desc(rows, i, o, dtype=dt) for k, (i, o) in self.lin.items()}
        self.conv = cm.make_causal_conv_desc(rows, E, W, batch=b, activation=cm.ACT_SILU, dtype=dt, x_pitch=2 * E)
        self.scan = cm.make_scan_desc(rows, E, N, batch=b, dtype=dt, z_pitch=2 * E, bc_pitch=2 * N)
        self.t["saved"] = cm.scan_saved_states(self.scan)
        self.ws = {}
        for k, d in self.lin.items():
            for op in range(3):
                self.ws[k, op] = cm.linear_workspace(d, op)
        self.ws["norm"], self.ws["conv"] = cm.layer_norm_workspace(self.norm), cm.causal_conv_workspace(self.conv)
        for op in range(2):
            self.ws["scan", op] = cm.scan_workspace(self.scan, op)

    def scan_args(self):
        t = self.t
        return (t["c"], t["dt"], t["dt_bias"], t["A"], t["bc"][:, :N], t["bc"][:, N:], t["Dp"], t["xz"][:, E:])

    def forward(self, stream=None):
        cm, t, lin = self.cm, self.t, self.lin
        kw = dict(stream=stream)
        cm.layer_norm_forward(self.norm, t["h"], None, t["gamma"], t["beta"], None, t["n"], t["mean"], t["inv"], **kw)
        cm.linear_forward(lin["in"], t["n"], t["w_in"], None, None, None, t["xz"], self.ws["in", 0], **kw)
        cm.causal_conv_forward(self.conv, t["xz"][:, :E], t["w_conv"], t["b_conv"], t["c"], seq_starts=self.st,
                               final_state=t["conv_state"], **kw)
        cm.linear_forward(lin["dt"], t["c"], t["w_dt"], None, None, None, t["dt"], self.ws["dt", 0], **kw)
        cm.linear_forward(lin["bc"], t["c"], t["w_bc"], None, None, None, t["bc"], self.ws["bc", 0], **kw)
        cm.selective_scan_forward(self.scan, *self.scan_args(), t["y"], seq_starts=self.st, final_state=t["state"],
                                  saved_states=t["saved"], workspace=self.ws["scan", 0], **kw)
        cm.linear_forward(lin["out"], t["y"], t["w_out"], None, t["h"], None, t["out"], self.ws["out", 0], **kw)

    def backward(self, stream=None):
        cm, t, lin = self.cm, self.t, self.lin
        kw = dict(stream=stream)

        def linear(name, dz, w, dx, x, dw):
            cm.linear_backward_data(lin[name], dz, w, dx, self.ws[name, 1], **kw)
            cm.linear_backward_weight(lin[name], x, dz, dw, None, 0, self.ws[name, 2], **kw)

        linear("out", t["dout"], t["w_out"], t["dy"], t["y"], t["dw_out"])
        cm.selective_scan_backward(self.scan, *self.scan_args(), t["saved"], t["dy"], t["dc"], t["ddt"], t["dbc"][:, :N],
                                   t["dbc"][:, N:], t["dxz"][:, E:], t["d_dt_bias"], t["dA"], t["dDp"], 0,
                                   self.ws["scan", 1], seq_starts=self.st, **kw)
        linear("dt", t["ddt"], t["w_dt"], t["dc2"], t["c"], t["dw_dt"])
        linear("bc", t["dbc"], t["w_bc"], t["dc3"], t["c"], t["dw_bc"])
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            t["dc"].add_(t["dc2"]).add_(t["dc3"])
        cm.causal_conv_backward(self.conv, t["xz"][:, :E], t["w_conv"], t["b_conv"], t["dc"], t["dxz"][:, :E], t["dw_conv"],
                                t["db_conv"], 0, self.ws["conv"], seq_starts=self.st, **kw)
        linear("in", t["dxz"], t["w_in"], t["dn"], t["n"], t["dw_in"])
        cm.layer_norm_backward(self.norm, t["h"], t["gamma"], t["mean"], t["inv"], t["dn"], t["dout"], t["dh"], t["dgamma"],
                               t["dbeta"], 0, self.ws["norm"], **kw)

    def results(self):
        return {k: self.t[k].clone() for k in ("out", "state", "conv_state") + self.grads}

    def spoil(self):
        for k, v in self.t.items():
            if k not in self.src:
                v.fill_(float("nan"))
        for v in self.ws.values():
            if v is not None:
                v.fill_(255)


def definition(src, noise=None):
    """Outputs and gradients in 64 bits; `noise` (a generator) puts a relative error of 2^-17 on every
    operator's output and on every gradient that passes it."""
    class Off(torch.autograd.Function):
        @staticmethod
        def forward(ctx, v):
            return v if noise is None else v * (1 + 2.0 ** -17 * torch.randn(v.shape, generator=noise, dtype=v.dtype))

        @staticmethod
        def backward(ctx, g):
            return Off.forward(None, g)

    p = {k: v.double().requires_grad_(k != "dout") for k, v in src.items()}
    off, h = Off.apply, p["h"]
    c = h - h.mean(-1, keepdim=True)
    n = off(p["gamma"] * c / torch.sqrt((c * c).mean(-1, keepdim=True) + float(torch.tensor(EPS))) + p["beta"])
    xz = off(n @ p["w_in"].t())
    u, z = xz[:, :E], xz[:, E:]
    cs, ys, states, tails = [], [], [], []
    for a, e in zip(STARTS, STARTS[1:]):
        x = torch.cat([torch.zeros(W - 1, E, dtype=torch.float64), u[a:e]])
        v = p["b_conv"] + sum(p["w_conv"][:, k] * x[k:k + e - a] for k in range(W))
        cs.append(off(v * torch.sigmoid(v)))
        tails.append(x[e - a:].detach())
    cc = torch.cat(cs)
    delta = torch.nn.functional.softplus(off(cc @ p["w_dt"].t()) + p["dt_bias"], threshold=100)
    bc = off(cc @ p["w_bc"].t())
    for a, e in zip(STARTS, STARTS[1:]):
        s = torch.zeros(E, N, dtype=torch.float64)
        for r in range(a, e):
            s = torch.exp(delta[r][:, None] * p["A"]) * s + (delta[r] * cc[r])[:, None] * bc[r, :N]
            ys.append((s * bc[r, N:]).sum(-1))
        states.append(s.detach())
    y = off((torch.stack(ys) + p["Dp"] * cc) * z * torch.sigmoid(z))
    out = off(y @ p["w_out"].t()) + h
    names = [k for k in p if k != "dout"]
    grads = torch.autograd.grad(out, [p[k] for k in names], p["dout"])
    o = {"out": out.detach(), "state": torch.stack(states), "conv_state": torch.stack(tails)}
    return o | {("d_" if k == "dt_bias" else "d") + k: g for k, g in zip(names, grads)}


def same(a, b, what):
    for k in a:
        R.same(a[k], b[k], f"{what}: {k}")


def test_block_against_the_definition():
    """Each operator is within 2^-17 of its exact result, relative to the values that meet in it; what such
    errors do together is taken from the definition itself, with four times the largest of three
    draws as the bound (of the largest value of each result)."""
    b = Block(1)
    b.forward()
    b.backward()
    ref = definition(b.src)
    off = {k: 0.0 for k in ref}
    for i in range(3):
        d = definition(b.src, torch.Generator().manual_seed(100 + i))
        off = {k: max(off[k], float((d[k] - ref[k]).abs().max())) for k in ref}
    for k, v in b.results().items():
        bound = 4 * off[k] + 2.0 ** -22 * float(ref[k].abs().max())
        err = float((R.host(v) - ref[k]).abs().max())
        assert err <= bound, (k, err, bound)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_repeats_streams_and_graphs(dtype):
    b = Block(2, dtype)
    b.forward()
    b.backward()
    first = b.results()
    b.spoil()
    b.forward()
    b.backward()
    same(b.results(), first, "again")
    b.spoil()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.forward(stream=s)
    b.backward(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    same(b.results(), first, "another stream")
    graphs = []
    for part in (b.forward, b.backward):  # two graphs on the same workspaces
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            part()
        graphs.append(g)
    other = Block(3, dtype)
    for i in range(4):
        b.spoil()
        for g in graphs:
            g.replay()
        other.forward()  # eager work between the replays
        other.backward()
        torch.cuda.synchronize()
        same(b.results(), first, f"replay {i}")


def test_tokens_follow_the_prompts():
    """Prompts, then single tokens from a pool of states in a captured graph with a padded batch, against the
    longer sequences at once."""
    import convolution_layer_amd as cm
    new, pad = 5, 2  # tokens each sequence grows by; rows of the batch that hold none
    long_starts, rows = [0], []
    for a, e in zip(STARTS, STARTS[1:]):
        long_starts.append(long_starts[-1] + e - a + new)
    whole = Block(4, rows=long_starts[-1], starts=tuple(long_starts))
    whole.forward()
    t = whole.t
    prompt = Block(4)
    for k in ("w_in", "w_conv", "w_dt", "w_bc", "w_out", "gamma", "beta", "b_conv", "dt_bias", "A", "Dp"):
        prompt.t[k] = t[k]
    seqs = list(zip(STARTS, STARTS[1:]))
    for (a, e), l in zip(seqs, long_starts):
        prompt.t["h"][a:e] = t["h"][l:l + e - a]
    prompt.forward()
    batch = len(seqs) + pad
    pool = {"conv": torch.zeros(6, W - 1, E, device="cuda"), "scan": torch.zeros(6, E, N, device="cuda")}
    where = [4, 1, 3]
    pool["conv"][where], pool["scan"][where] = prompt.t["conv_state"], prompt.t["state"]
    slots = torch.tensor([4, -1, 1, 3, -1], dtype=torch.int32, device="cuda")
    live = [0, 2, 3]
    one = Block(4, rows=batch, starts=tuple(range(batch + 1)))
    for k in prompt.src:
        if k not in ("h", "dout"):
            one.t[k] = t[k]
    o, lin = one.t, one.lin
    conv = cm.make_causal_conv_desc(batch, E, W, activation=cm.ACT_SILU, x_pitch=2 * E)
    scan = cm.make_scan_desc(batch, E, N, z_pitch=2 * E, bc_pitch=2 * N)

    def token():
        cm.layer_norm_forward(one.norm, o["h"], None, o["gamma"], o["beta"], None, o["n"], None, None)
        cm.linear_forward(lin["in"], o["n"], o["w_in"], None, None, None, o["xz"], one.ws["in", 0])
        cm.causal_conv_step(conv, o["xz"][:, :E], o["w_conv"], o["b_conv"], pool["conv"], o["c"], slots=slots)
        cm.linear_forward(lin["dt"], o["c"], o["w_dt"], None, None, None, o["dt"], one.ws["dt", 0])
        cm.linear_forward(lin["bc"], o["c"], o["w_bc"], None, None, None, o["bc"], one.ws["bc", 0])
        cm.selective_scan_step(scan, *one.scan_args(), pool["scan"], o["y"], slots=slots)
        cm.linear_forward(lin["out"], o["y"], o["w_out"], None, o["h"], None, o["out"], one.ws["out", 0])

    o["h"].zero_()
    o["c"].zero_()
    o["y"].zero_()
    kept = {k: v.clone() for k, v in pool.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        token()
    for k, v in kept.items():
        pool[k].copy_(v)
    for i in range(new):
        for r, (a, e), l in zip(live, seqs, long_starts):
            o["h"][r] = t["h"][l + e - a + i]
        g.replay()
        torch.cuda.synchronize()
        for r, (a, e), l in zip(live, seqs, long_starts):
            got, ref = R.host(o["out"][r]), R.host(t["out"][l + e - a + i])
            # two fp32 evaluations of one definition, each within 16 operators of 2^-17 at most
            assert float((got - ref).abs().max()) <= 2 * 16 * 2.0 ** -17 * float(ref.abs().max()), (i, r)
    assert bool((o["c"][[1, 4]] == 0).all()) and bool((o["y"][[1, 4]] == 0).all()), "padding rows"
    rest = [0, 2, 5]
    assert bool((pool["conv"][rest] == 0).all()) and bool((pool["scan"][rest] == 0).all()), "other states"
    for k, name in (("conv", "conv_state"), ("scan", "state")):
        ref = R.host(t[name])
        assert float((R.host(pool[k][where]) - ref).abs().max()) <= 32 * 2.0 ** -17 * float(ref.abs().max()), k
