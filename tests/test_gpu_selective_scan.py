"""Selective scan, forward, backward and by single tokens, against the 64-bit definition, with bounds
that sequence_reference carries along operation by operation."""
import pytest
import torch

from tests import block_reference as R
from tests import sequence_reference as Q

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
# rows, batch, channels, states, groups, starts (None: equal lengths), softplus
CASES = [
    (1, 1, 1, 1, 1, None, True), (1, 1, 64, 16, 1, None, True), (2, 1, 5, 3, 1, None, True), (33, 1, 70, 16, 1, None, True),
    (64, 2, 64, 16, 1, None, True), (31, 1, 16, 8, 2, None, True), (130, 2, 24, 5, 3, None, True),
    (65, 1, 66, 17, 1, None, True), (40, 1, 10, 64, 1, None, True), (50, 2, 12, 33, 2, None, True),
    (200, 1, 130, 4, 1, None, True), (200, 1, 65, 32, 1, None, True), (300, 1, 20, 2, 20, None, False),
    (150, 3, 40, 16, 1, (0, 1, 1, 150), True),                 # one of a single row, an empty one
    (150, 3, 33, 16, 1, (9, 40, 105, 141), True),              # rows before the first and behind the last
    (260, 4, 18, 6, 2, (0, 128, 192, 192, 260), True),         # ends on the borders of chunks and segments
    (20, 2, 16, 16, 1, (20, 20, 20), True),                    # all empty
    (140, 70, 9, 16, 1, tuple(2 * i for i in range(71)), True),  # more sequences than a wave has lanes
    (390, 1, 7, 20, 7, None, True), (129, 1, 6, 50, 1, None, False),
]


def cdt(dtype):
    import convolution_layer_amd as cm
    return cm.BF16 if dtype == torch.bfloat16 else cm.F32


def make(rows, batch, ch, N, G, dtype, plus=True, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + ch * 3 + N)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = {"x": rnd(rows, ch), "dt": rnd(rows, ch) if plus else rnd(rows, ch).abs() * 0.1, "B": rnd(rows, G * N),
         "C": rnd(rows, G * N), "z": rnd(rows, ch) * 2, "dy": rnd(rows, ch)}
    t = {k: v.to(dtype) for k, v in t.items()}
    t["dt_bias"] = rnd(ch) - 2 if plus else rnd(ch).abs() * 0.1
    t["A"] = -(0.2 + torch.rand(ch, N, generator=g) * 4)
    t["D"] = 1 + 0.2 * rnd(ch)
    t["initial"], t["dfinal"] = rnd(batch, ch, N), rnd(batch, ch, N)
    return t


def gaps(seqs, rows):
    m = torch.ones(rows, dtype=torch.bool)
    for a, e in seqs:
        m[a:e] = False
    return m


class Call:
    """One scan's tensors on the GPU, dense or as columns of wider matrices."""

    def __init__(self, t, rows, batch, ch, N, G, starts, plus, dtype, extras, state, wide):
        import convolution_layer_amd as cm
        self.cm, self.rows, self.ch, self.N, self.G, self.batch, self.wide = cm, rows, ch, N, G, batch, wide
        self.dtype, bc = dtype, G * N
        pitch = {"x": ch + 3, "dt": 2 * ch + 1, "z": 2 * ch, "bc": 2 * bc + 5} if wide else dict.fromkeys(("x", "dt", "z", "bc"), 0)
        self.d = cm.make_scan_desc(rows, ch, N, batch=batch, groups=G, dtype=cdt(dtype), delta_softplus=plus,
                                   x_pitch=pitch["x"], dt_pitch=pitch["dt"], z_pitch=pitch["z"], bc_pitch=pitch["bc"])
        self.cols = {"x": (pitch["x"], 3, ch), "dt": (pitch["dt"], 0, ch), "z": (pitch["z"], ch, ch),
                     "B": (pitch["bc"], 1, bc), "C": (pitch["bc"], 1 + bc, bc)}
        dev = lambda v: None if v is None else v.cuda()  # noqa: E731
        self.t = {k: self.put(k, t[k]) for k in ("x", "dt", "B", "C", "z")}
        if not extras:
            self.t["z"] = None
        self.t.update(A=dev(t["A"]), dt_bias=dev(t["dt_bias"]) if extras else None, D=dev(t["D"]) if extras else None)
        self.starts = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.initial, self.dfinal = (dev(t["initial"]), dev(t["dfinal"])) if state else (None, None)
        self.dy = dev(t["dy"])

    def put(self, name, v, matrix=None):
        pitch, at, n = self.cols[name]
        if not pitch:
            return v.cuda()
        m = torch.full((self.rows, pitch), 7.0, dtype=v.dtype, device="cuda") if matrix is None else matrix
        m[:, at:at + n] = v.cuda()
        return m[:, at:at + n]

    def args(self):
        return [self.t[k] for k in ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")]

    def ws(self, op):
        w = self.cm.scan_workspace(self.d, op)
        return w if w is None else w.fill_(255)

    def forward(self, saved=True):
        y = torch.full((self.rows + 1, self.ch), 3.0, dtype=self.dtype, device="cuda")
        final = torch.full((self.batch + 1, self.ch, self.N), 3.0, device="cuda")
        n = self.cm.scan_saved_size(self.d) // 4
        self.saved = torch.full((n + 16,), 3.0, device="cuda") if saved else None
        self.cm.selective_scan_forward(self.d, *self.args(), y[:self.rows], seq_starts=self.starts,
                                       initial_state=self.initial, final_state=final[:self.batch],
                                       saved_states=self.saved[:n] if saved else None, workspace=self.ws(self.cm.SCAN_FORWARD))
        assert bool((y[self.rows] == 3).all()) and bool((final[self.batch:] == 3).all())
        assert not saved or bool((self.saved[n:] == 3).all())
        return {"y": y[:self.rows], "final": final[:self.batch]}

    def backward(self, accumulate=0, sums=None, all_of_it=True):
        o, whole = {}, {}
        for name, like in (("dx", "x"), ("ddt", "dt"), ("dB", "B"), ("dC", "C"), ("dz", "z")):
            if self.t[like] is None:
                continue
            pitch, at, n = self.cols[like]
            key = "bc" if like in "BC" else like
            if pitch and key not in whole:
                whole[key] = torch.full((self.rows, pitch), 7.0, dtype=self.dtype, device="cuda")
            fill = torch.full((self.rows, n), 3.0, dtype=self.dtype, device="cuda")
            o[name] = self.put(like, fill, whole[key]) if pitch else fill
        sums = sums or {"ddt_bias": torch.full((self.ch,), 0.5, device="cuda"),
                        "dA": torch.full((self.ch, self.N), 0.5, device="cuda"),
                        "dD": torch.full((self.ch,), 0.5, device="cuda")}
        di = torch.full((self.batch + 1, self.ch, self.N), 3.0, device="cuda")
        n = self.cm.scan_saved_size(self.d) // 4
        ws = self.ws(self.cm.SCAN_BACKWARD)
        self.cm.selective_scan_backward(
            self.d, *self.args(), self.saved[:n], self.dy, o["dx"], o["ddt"], o["dB"], o["dC"], o.get("dz"),
            *([sums[k] for k in ("ddt_bias", "dA", "dD")] if all_of_it else [None] * 3), accumulate=accumulate, workspace=ws,
            seq_starts=self.starts, d_final_state=self.dfinal, d_initial_state=di[:self.batch] if all_of_it else None)
        assert bool((di[self.batch:] == 3).all())
        if self.wide:  # nothing beside the gradients' columns
            for key, m in whole.items():
                used = torch.zeros(m.shape[1], dtype=torch.bool)
                for like, (_, at, n) in self.cols.items():
                    if ("bc" if like in "BC" else like) == key:
                        used[at:at + n] = True
                assert bool((m[:, ~used.cuda()] == 7).all()), key
        return o | sums | ({"dinitial": di[:self.batch]} if all_of_it else {})


def check(got, ref, dtype, what, rows=None):
    half = R.HALF[dtype] if got.dtype == dtype else 0.0
    v, e = (ref.v, ref.e) if rows is None else (ref.v[rows], ref.e[rows])
    R.within(got if rows is None else got[rows.cuda()], v, e * (1 + half) + half * v.abs() + 1e-37, what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extras,state", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("rows,batch,ch,N,G,starts,plus", CASES)
def test_forward_and_backward(rows, batch, ch, N, G, starts, plus, extras, state, dtype):
    t = make(rows, batch, ch, N, G, dtype, plus)
    seqs = Q.bounds(starts, rows, batch)
    gap = gaps(seqs, rows)
    names = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")
    part = {k: t[k] if extras or k not in ("dt_bias", "D", "z") else None for k in names}
    ref = Q.scan(part, seqs, G, plus, t["initial"] if state else None, t["dy"], t["dfinal"] if state else None)
    for k in ("x", "dt", "B", "C", "z", "dy"):  # rows of no sequence are not looked at
        t[k] = t[k].clone()
        t[k][gap] = float("nan")
    c = Call(t, rows, batch, ch, N, G, starts, plus, dtype, extras, state, wide=False)
    f = c.forward()
    check(f["y"], ref["y"], dtype, "y", ~gap)
    assert bool((f["y"][gap.cuda()] == 3).all())
    check(f["final"], ref["final"], dtype, "final")
    b = c.backward()
    for k in ("dx", "ddt", "dB", "dC") + (("dz",) if extras else ()):
        check(b[k], ref[k], dtype, k, ~gap)
        assert bool((b[k][gap.cuda()] == 3).all()), k
    check(b["dinitial"], ref["dinitial"], dtype, "dinitial")
    for k in ("dA", "dD", "ddt_bias"):
        check(b[k], ref[k], dtype, k)
    # columns of wider matrices, without the kept states, with the final state in the initial one's place
    w = Call(t, rows, batch, ch, N, G, starts, plus, dtype, extras, state, wide=True)
    f2 = w.forward()
    for k in f:
        R.same(f2[k], f[k], k + " by pitch")
    b2 = w.backward()
    for k in b:
        R.same(b2[k].contiguous(), b[k].contiguous(), k + " by pitch")
    R.same(c.forward(saved=False)["y"], f["y"], "y without kept states")
    if state:
        c.cm.selective_scan_forward(c.d, *c.args(), f2["y"], seq_starts=c.starts, initial_state=c.initial,
                                    final_state=c.initial, workspace=c.ws(c.cm.SCAN_FORWARD))
        R.same(f2["y"], f["y"], "y, state in place")
        R.same(c.initial, f["final"].contiguous(), "state in place")
    # the sums added to what is there; without them
    twice = w.backward(1, {k: b2[k].clone() for k in ("ddt_bias", "dA", "dD")})
    for k in ("ddt_bias", "dA", "dD"):
        check(twice[k], Q.V(2 * ref[k].v, 2 * ref[k].e + 4 * Q.U * ref[k].v.abs()), dtype, k + " added")
    for k, v in w.backward(all_of_it=False).items():
        if k in ("dx", "ddt", "dB", "dC", "dz"):
            R.same(v.contiguous(), b[k].contiguous(), k + " alone")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extras", [False, True])
@pytest.mark.parametrize("rows,ch,N,G", [(1, 1, 1, 1), (1, 4096, 16, 1), (3, 70, 16, 1), (5, 12, 5, 3), (2, 66, 33, 2),
                                         (200, 8, 64, 8), (4, 130, 7, 1)])
def test_step(rows, ch, N, G, extras, dtype):
    import convolution_layer_amd as cm
    n = rows + 3
    t = make(rows, n, ch, N, G, dtype, seed=3)
    if not extras:
        t["dt_bias"] = t["D"] = t["z"] = None
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(rows))[:rows].to(torch.int32)
    names = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")
    d = cm.make_scan_desc(rows, ch, N, groups=G, dtype=cdt(dtype))
    dev = {k: None if t[k] is None else t[k].cuda() for k in names}
    for use in (None, slots):
        at = torch.arange(rows) if use is None else use.long()
        ref = Q.scan({k: t[k] for k in names}, [(i, i + 1) for i in range(rows)], G, True, t["initial"][at])
        state, y = t["initial"].cuda(), torch.full((rows + 1, ch), 3.0, dtype=dtype, device="cuda")
        cm.selective_scan_step(d, *dev.values(), state, y[:rows], slots=None if use is None else use.cuda())
        check(y[:rows], ref["y"], dtype, "y")
        assert bool((y[rows] == 3).all())
        check(state[at.cuda()], ref["final"], torch.float32, "state")
        rest = torch.ones(n, dtype=torch.bool)
        rest[at] = False
        assert torch.equal(state[rest.cuda()].cpu(), t["initial"][rest]), "other states"


def test_step_slots_out_of_order():
    """Padding rows keep their y; slots that do not exist or come twice give NaN and touch no state."""
    import convolution_layer_amd as cm
    rows, ch, N, n = 7, 40, 16, 5
    t = make(rows, n, ch, N, 1, torch.float32, seed=4)
    names = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")
    slots = torch.tensor([2, -1, 0, 2, 5, -7, 1 << 30], dtype=torch.int32)
    state, y = t["initial"].cuda(), torch.full((rows, ch), 3.0, device="cuda")
    cm.selective_scan_step(cm.make_scan_desc(rows, ch, N), *[t[k].cuda() for k in names], state, y, slots=slots.cuda())
    assert bool((y[[1, 5]] == 3).all()) and bool(torch.isnan(y[[3, 4, 6]]).all())
    pick = {k: t[k][[0, 2]] if t[k].shape[0] == rows else t[k] for k in names}
    ref = Q.scan(pick, [(0, 1), (1, 2)], 1, True, t["initial"][[2, 0]])
    check(y[[0, 2]], ref["y"], torch.float32, "y")
    check(state[[2, 0]], ref["final"], torch.float32, "state")
    assert torch.equal(state[[1, 3, 4]].cpu(), t["initial"][[1, 3, 4]])


def test_tokens_one_by_one_follow_the_prompt():
    """A prompt, then single tokens from its final state, against the whole sequence."""
    import convolution_layer_amd as cm
    rows, ch, N, cut = 45, 72, 16, 37
    t = make(rows, 1, ch, N, 1, torch.float32, seed=5)
    names = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")
    ref = Q.scan({k: t[k] for k in names}, [(0, rows)], 1, True)
    dev = {k: t[k].cuda() for k in names}
    part = lambda a, e: [v[a:e] if k in ("x", "dt", "B", "C", "z") else v for k, v in dev.items()]  # noqa: E731
    y, state = torch.empty(rows, ch, device="cuda"), torch.empty(1, ch, N, device="cuda")
    d = cm.make_scan_desc(cut, ch, N)
    cm.selective_scan_forward(d, *part(0, cut), y[:cut], final_state=state, workspace=cm.scan_workspace(d, cm.SCAN_FORWARD))
    for i in range(cut, rows):
        cm.selective_scan_step(cm.make_scan_desc(1, ch, N), *part(i, i + 1), state, y[i:i + 1])
    check(y, ref["y"], torch.float32, "y")
    check(state, ref["final"], torch.float32, "final")


@pytest.mark.parametrize("rows,ch,N,G", [(96, 40, 16, 1), (40, 6, 40, 2)])
def test_gradient_against_differences(rows, ch, N, G):
    import convolution_layer_amd as cm
    t = make(rows, 2, ch, N, G, torch.float32, seed=6)
    starts = (0, 30, rows)
    seqs = Q.bounds(starts, rows, 2)
    c = Call(t, rows, 2, ch, N, G, starts, True, torch.float32, True, True, wide=False)
    c.forward()
    got = c.backward()
    names = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")
    t = {k: v.double() for k, v in t.items()}

    def f(v):
        out, fin = 0.0, []
        delta = torch.nn.functional.softplus(v["dt"] + v["dt_bias"], threshold=100)
        for i, (a, e) in enumerate(seqs):
            h = v["initial"][i]
            for r in range(a, e):
                wide = lambda b: b.reshape(G, 1, N).expand(G, ch // G, N).reshape(ch, N)  # noqa: E731
                h = torch.exp(delta[r][:, None] * v["A"]) * h + (delta[r] * v["x"][r])[:, None] * wide(v["B"][r])
                y = ((h * wide(v["C"][r])).sum(-1) + v["D"] * v["x"][r]) * v["z"][r] * torch.sigmoid(v["z"][r])
                out = out + (y * t["dy"][r]).sum()
            fin.append(h)
        return float(out + (torch.stack(fin) * t["dfinal"]).sum())

    h = 1e-5  # differences lose about 1e-5 of a sum of this size
    called = {"dt": "ddt", "dt_bias": "ddt_bias", "initial": "dinitial"}
    g = torch.Generator().manual_seed(rows)
    for name in names + ("initial",):
        grad = got[called.get(name, "d" + name)].flatten()
        for i in torch.randint(0, grad.numel(), (4,), generator=g).tolist():
            p, m = dict(t), dict(t)
            for v, s in ((p, h), (m, -h)):
                v[name] = t[name].clone()
                v[name].view(-1)[i] += s
            num = (f(p) - f(m)) / (2 * h)
            assert abs(num - float(grad[i])) <= 2e-5 * (1 + abs(num)), (name, i, num, float(grad[i]))


def test_extreme_values():
    """Decays to nothing, steps of zero, large inputs of softplus and the gate; infinities stay in their channel."""
    import convolution_layer_amd as cm
    rows, ch, N = 40, 8, 16
    t = make(rows, 1, ch, N, 1, torch.float32, seed=7)
    t["dt"][:, 0] = 80.0      # delta about 80: every state forgets at once
    t["dt"][:, 1] = -90.0     # delta about 1e-39: flushes or stays, the state stands still
    t["z"][:, 2] = -100.0
    t["z"][:, 3] = 100.0
    t["A"][4] = 0.0           # sums without forgetting
    t["x"][5, 5] = float("inf")
    t["dt"][3, 6] = float("nan")
    clean = Q.scan({k: t[k][:, :5] if k in ("x", "dt", "z") else t[k][:5] if k in ("dt_bias", "A", "D") else t[k]
                    for k in ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")}, [(0, rows)], 1, True)
    c = Call(t, rows, 1, ch, N, 1, None, True, torch.float32, True, False, wide=False)
    f = c.forward()
    check(f["y"][:, :5], clean["y"], torch.float32, "y")
    assert bool(torch.isfinite(f["y"][:, 7]).all()) and bool(torch.isfinite(f["y"][:5, 5]).all())
    assert bool(torch.isnan(f["y"][3:, 6]).all()) and bool(torch.isfinite(f["y"][:3, 6]).all())
    b = c.backward()
    for k in ("dx", "ddt", "dz"):
        assert bool(torch.isfinite(b[k][:, :5]).all()) and bool(torch.isfinite(b[k][:, 7]).all()), k


def test_starts_out_of_range_stay_inside():
    import convolution_layer_amd as cm
    rows, ch, N = 200, 70, 16
    t = make(rows, 3, ch, N, 1, torch.float32, seed=8)
    for starts in ((-5, 10, 1 << 30, 2), (0, 130, 10, 200), (1 << 30, -1, 7, 1000)):
        c = Call(t, rows, 3, ch, N, 1, starts, True, torch.float32, True, True, wide=False)
        c.saved = torch.zeros(cm.scan_saved_size(c.d) // 4 + 16, device="cuda")
        f = c.forward()
        assert all(v is not None for v in f.values())
        c.saved.nan_to_num_(0.0)
        c.backward()


def test_long_sequences_in_chunks():
    """Few channels and many rows run in some hundred chunks: the end against the definition."""
    import convolution_layer_amd as cm
    rows, ch, N, tail = 20000, 16, 16, 2200
    t = make(rows, 1, ch, N, 1, torch.float32, seed=9)
    t["A"] -= 1.0
    t["dt_bias"] = t["dt_bias"].clamp(min=-3.0)
    names = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")
    d = cm.make_scan_desc(rows, ch, N)
    y, final = torch.empty(rows, ch, device="cuda"), torch.empty(1, ch, N, device="cuda")
    cm.selective_scan_forward(d, *[t[k].cuda() for k in names], y, final_state=final,
                              workspace=cm.scan_workspace(d, cm.SCAN_FORWARD))
    part = {k: t[k][-tail:] if t[k].shape[0] == rows else t[k] for k in names}
    # what lies 2000 rows back is forgotten: decays of at most exp(-1.2 sum of delta)
    past = torch.nn.functional.softplus(part["dt"].double() + part["dt_bias"]).abs()[:2000].sum(0).min()
    assert float(past) * 1.2 > 50
    ref = Q.scan(part, [(0, tail)], 1, True)
    R.within(y[-100:], ref["y"].v[-100:], ref["y"].e[-100:] + 1e-9, "y")
    R.within(final[0], ref["final"].v[0], ref["final"].e[0] + 1e-9, "final")


@pytest.mark.parametrize("ch", [128, 301])
@pytest.mark.parametrize("starts", [None, (0, 2, 3500, 6000)])
def test_state_in_place_with_many_chunks(starts, ch):
    """Every chunk of a sequence reads its initial state: the final one takes its place after all have."""
    import convolution_layer_amd as cm
    rows, batch, N = 6000, 3, 16
    t = make(rows, batch, ch, N, 1, torch.bfloat16, seed=12)
    c = Call(t, rows, batch, ch, N, 1, starts, True, torch.bfloat16, True, True, wide=False)
    f = c.forward(saved=False)
    for i in range(3):
        state, y = c.initial.clone(), torch.empty_like(f["y"])
        cm.selective_scan_forward(c.d, *c.args(), y, seq_starts=c.starts, initial_state=state, final_state=state,
                                  workspace=c.ws(cm.SCAN_FORWARD))
        R.same(y, f["y"].contiguous(), f"y, {i}")
        R.same(state, f["final"].contiguous(), f"state, {i}")


@pytest.mark.parametrize("rows,starts", [(45, None), (3001, None), (3001, (0, 700, 3000))])
def test_states_that_forget_everything(rows, starts):
    """A = -inf is a state without memory, in tiles that end inside and in chunks, as A = -1e38 is."""
    batch, ch, N = 1 if starts is None else 2, 5, 6
    t = make(rows, batch, ch, N, 1, torch.float32, seed=14)
    outs = []
    for lowest in (-1e38, -3e38, float("-inf")):
        t["A"][:, 1::2] = lowest
        c = Call(t, rows, batch, ch, N, 1, starts, True, torch.float32, True, True, wide=False)
        outs.append(c.forward() | c.backward())
    for o in outs[1:]:
        for k in o:
            if k == "ddt" or starts is None or k in ("final", "dinitial", "dA", "dD", "ddt_bias"):
                assert bool(torch.isfinite(o[k]).all()), k
            R.same(o[k].contiguous(), outs[0][k].contiguous(), k)


@pytest.mark.parametrize("ch", [3, 70])
def test_more_sequences_than_workgroups(ch):
    """Thousands of short sequences: a workgroup of the backward takes several."""
    rows, N = 2600, 2
    lens = [i % 3 for i in range(rows)]  # 0, 1, 2
    starts = [0]
    for n in lens:
        starts.append(min(rows - 5, starts[-1] + n))
    batch = len(lens)
    t = make(rows, batch, ch, N, 1, torch.float32, seed=13)
    seqs = Q.bounds(starts, rows, batch)
    names = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")
    ref = Q.scan({k: t[k] for k in names}, seqs, 1, True, t["initial"], t["dy"], t["dfinal"])
    c = Call(t, rows, batch, ch, N, 1, starts, True, torch.float32, True, True, wide=False)
    f = c.forward()
    inside = ~gaps(seqs, rows)
    check(f["y"], ref["y"], torch.float32, "y", inside)
    check(f["final"], ref["final"], torch.float32, "final")
    b = c.backward()
    for k in ("dx", "ddt", "dB", "dC", "dz"):
        check(b[k], ref[k], torch.float32, k, inside)
    for k in ("dA", "dD", "ddt_bias", "dinitial"):
        check(b[k], ref[k], torch.float32, k)


def test_offsets_beyond_32_bits():
    """The last rows of tensors of more than 2^32 bytes: equal lengths, so the last sequence starts afresh."""
    import convolution_layer_amd as cm
    n, ch, N, batch = 8, 64, 8, 5000
    pitch = 1 << 16
    rows = n * batch
    m = torch.zeros(rows, pitch, dtype=torch.bfloat16, device="cuda")
    t = make(n, 1, ch, N, 1, torch.bfloat16, seed=10)
    cols = {}
    for i, k in enumerate(("x", "dt", "z", "B", "C")):
        w = t[k].shape[1]
        cols[k] = m[:, -(i + 1) * 64:][:, :w]
        cols[k][-n:] = t[k].cuda()
    d = cm.make_scan_desc(rows, ch, N, batch=batch, dtype=cm.BF16, x_pitch=pitch, dt_pitch=pitch, z_pitch=pitch,
                          bc_pitch=pitch)
    y = torch.empty(rows, ch, dtype=torch.bfloat16, device="cuda")
    A, D, bias = t["A"].cuda(), t["D"].cuda(), t["dt_bias"].cuda()
    cm.selective_scan_forward(d, cols["x"], cols["dt"], bias, A, cols["B"], cols["C"], D, cols["z"], y,
                              workspace=cm.scan_workspace(d, cm.SCAN_FORWARD))
    ref = Q.scan({k: t[k] for k in ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")}, [(0, n)], 1, True)
    check(y[-n:], ref["y"], torch.bfloat16, "last rows")


def test_refusals_of_the_binding():
    import convolution_layer_amd as cm
    rows, ch, N = 6, 8, 16
    t = make(rows, 2, ch, N, 1, torch.float32, seed=11)
    c = Call(t, rows, 2, ch, N, 1, None, True, torch.float32, True, True, wide=False)
    y = torch.empty(rows, ch, device="cuda")
    order = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")

    def call(y=y, **kw):
        a = [kw.pop(k, c.t[k]) for k in order]
        cm.selective_scan_forward(kw.pop("desc", c.d), *a, y, workspace=c.ws(cm.SCAN_FORWARD), **kw)

    call()
    for kw in (dict(x=c.t["x"].cpu()), dict(dt=c.t["dt"].bfloat16()), dict(A=c.t["A"].t().contiguous()), dict(B=c.t["B"][:, :8]),
               dict(z=c.t["z"].t()), dict(D=c.t["D"].double()), dict(initial_state=c.initial[:1]), dict(y=y[:3]),
               dict(seq_starts=torch.zeros(3, dtype=torch.int64, device="cuda")),
               dict(saved_states=torch.empty(7, device="cuda")),
               dict(desc=cm.make_scan_desc(rows, ch, N, batch=2, bc_pitch=40))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        call(x=None)
    with pytest.raises(cm.ConvmiError) as e:
        call(A=None)
    assert e.value.status == cm.ERR_INVALID_ARG
