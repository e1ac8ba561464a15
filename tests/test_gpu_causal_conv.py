"""Causal convolution, forward, backward and by single tokens, against the 64-bit definition.

Bounds: z runs through W + 1 fp32 roundings of its terms, the activation as sequence_reference
counts it (its slope is at most 1.2), then the rounding to the data type."""
import pytest
import torch

from tests import block_reference as R
from tests import sequence_reference as Q

pytestmark = pytest.mark.gpu

U = Q.U
DTYPES = [torch.bfloat16, torch.float32]
# rows, batch, channels, taps, starts (None: equal lengths), activation
CASES = [
    (1, 1, 1, 1, None, 0), (1, 1, 8, 4, None, 5), (3, 1, 5, 4, None, 5), (64, 2, 64, 4, None, 5), (65, 5, 130, 3, None, 2),
    (200, 1, 513, 2, None, 3), (96, 3, 24, 8, None, 4), (33, 1, 1000, 5, None, 5), (70, 7, 31, 6, None, 0),
    (1030, 2, 16, 7, None, 5), (2500, 1, 3, 4, None, 5), (40, 40, 12, 4, None, 5),
    (100, 4, 70, 4, (0, 1, 1, 40, 100), 5),                # one of a single row, an empty one
    (57, 3, 40, 8, (0, 3, 8, 57), 5),                      # shorter than the taps reach
    (90, 3, 520, 4, (5, 20, 64, 83), 5),                   # rows before the first and behind the last
    (300, 6, 8, 4, (0, 0, 100, 100, 100, 299, 300), 4), (700, 2, 264, 3, (13, 500, 641), 2),
    (50, 3, 16, 4, (50, 50, 50, 50), 5),                   # all empty
    (129, 70, 9, 4, tuple(min(2 * i, 129) for i in range(71)), 5),  # more sequences than a wave has lanes
]


def cdt(dtype):
    import convolution_layer_amd as cm
    return cm.BF16 if dtype == torch.bfloat16 else cm.F32


def make(rows, batch, D, W, dtype, seed=0, whole=False):
    g = torch.Generator().manual_seed(seed + rows * 7 + D * 3 + W)
    rnd = (lambda *s: torch.randint(-3, 4, s, generator=g).float()) if whole else (
        lambda *s: torch.randn(*s, generator=g))
    t = {"x": rnd(rows, D), "w": rnd(D, W), "dy": rnd(rows, D), "initial": rnd(batch, W - 1, D),
         "dfinal": rnd(batch, W - 1, D)}
    t = {k: v.to(dtype) for k, v in t.items()}
    t["bias"] = rnd(D)
    return t


def gaps(seqs, rows):
    m = torch.ones(rows, dtype=torch.bool)
    for a, e in seqs:
        m[a:e] = False
    return m


def wide(t, pitch, at=0):
    """t as columns of a wider matrix of sevens, and the matrix."""
    m = torch.full((t.shape[0], pitch), 7.0, dtype=t.dtype, device="cuda")
    m[:, at:at + t.shape[1]] = t
    return m[:, at:at + t.shape[1]], m


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("rows,batch,D,W,starts,kind", CASES)
def test_forward(rows, batch, D, W, starts, kind, state, dtype):
    import convolution_layer_amd as cm
    t = make(rows, batch, D, W, dtype)
    seqs = Q.bounds(starts, rows, batch)
    gap = gaps(seqs, rows)
    t["x"][gap] = float("nan")  # rows of no sequence are not looked at
    init = t["initial"] if state else None
    bias = t["bias"] if not state else None
    x = t["x"].clone()
    x[gap] = 0
    z, mag, ext = Q.conv_z(x, t["w"], bias, seqs, init)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    dev = lambda v: None if v is None else v.cuda()  # noqa: E731
    outs = []
    for pitch, at in ((0, 0), (2 * D + 3, D + 1)):
        xs, whole = (t["x"].cuda(), None) if pitch == 0 else wide(t["x"].cuda(), pitch, at)
        d = cm.make_causal_conv_desc(rows, D, W, batch=batch, activation=kind, dtype=cdt(dtype), x_pitch=pitch)
        y = torch.full((rows + 1, D), 3.0, dtype=dtype, device="cuda")
        final = torch.full((batch + 1, W - 1, D), 3.0, dtype=dtype, device="cuda")
        cm.causal_conv_forward(d, xs, t["w"].cuda(), dev(bias), y[:rows], seq_starts=st, initial_state=dev(init),
                               final_state=final[:batch])
        outs.append((y, final))
    for a, b, what in zip(*outs, ("y", "final")):
        R.same(a, b, what + " by pitch")
    assert bool((y[rows] == 3).all()) and bool((y[:rows][gap.cuda()] == 3).all()) and bool((final[batch:] == 3).all())
    ref = Q.act(z, kind)
    err = 1.2 * (W + 1) * U * mag + Q.act_error(z, kind) + 2 * U * ref.abs()
    err = err + R.HALF[dtype] * (ref.abs() + err)
    R.within(y[:rows][~gap.cuda()], ref[~gap], err[~gap], "y")
    if W > 1:
        assert torch.equal(final[:batch].cpu().double(), torch.stack([e[len(e) - (W - 1):] for e in ext])), "final"
    # without the final state, and with it in the initial one's place
    y2 = torch.full((rows, D), 3.0, dtype=dtype, device="cuda")
    cm.causal_conv_forward(d, xs, t["w"].cuda(), dev(bias), y2, seq_starts=st, initial_state=dev(init))
    R.same(y2, y[:rows].contiguous(), "y alone")
    if state:
        s = init.cuda()
        cm.causal_conv_forward(d, xs, t["w"].cuda(), dev(bias), y2, seq_starts=st, initial_state=s, final_state=s)
        R.same(y2, y[:rows].contiguous(), "y, state in place")
        R.same(s, final[:batch].contiguous(), "state in place")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("rows,batch,D,W,starts,kind", CASES)
def test_backward(rows, batch, D, W, starts, kind, state, dtype):
    import convolution_layer_amd as cm
    t = make(rows, batch, D, W, dtype, 1)
    seqs = Q.bounds(starts, rows, batch)
    gap = gaps(seqs, rows)
    init, dfin = (t["initial"], t["dfinal"]) if state else (None, None)
    ref = Q.conv_backward(t["x"], t["w"], t["bias"], seqs, init, kind, t["dy"], dfin)
    t["x"][gap] = t["dy"][gap] = float("nan")
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    dev = lambda v: None if v is None else v.cuda()  # noqa: E731
    outs = []
    for pitch, at in ((0, 0), (2 * D + 3, D + 1)):
        x = t["x"].cuda()
        dx, whole = torch.full((rows, D), 3.0, dtype=dtype, device="cuda"), None
        if pitch:
            x, dx = wide(x, pitch, at)[0], wide(dx, pitch, at)
            dx, whole = dx
        d = cm.make_causal_conv_desc(rows, D, W, batch=batch, activation=kind, dtype=cdt(dtype), x_pitch=pitch)
        ws = cm.causal_conv_workspace(d)
        if ws is not None:
            ws.fill_(255)
        di = torch.full((batch + 1, W - 1, D), 3.0, dtype=dtype, device="cuda") if state else None
        dw, db = torch.full((D + 1, W), 0.5, device="cuda"), torch.full((D + 1,), 0.5, device="cuda")
        args = (d, x, t["w"].cuda(), t["bias"].cuda(), t["dy"].cuda(), dx)
        kw = dict(seq_starts=st, initial_state=dev(init), d_final_state=dev(dfin))
        cm.causal_conv_backward(*args, dw[:D], db[:D], 0, ws, d_initial_state=None if di is None else di[:batch], **kw)
        if whole is not None:
            assert bool((whole[:, :at] == 7).all()) and bool((whole[:, at + D:] == 7).all()), "beside dx"
        outs.append((dx.clone(), dw, db) + (() if di is None else (di,)))
    for a, b in zip(*outs):
        R.same(a, b, "by pitch")
    assert bool((dx[gap.cuda()] == 3).all())
    half = R.HALF[dtype]
    lim = lambda v, e: e + half * (v.abs() + e)  # noqa: E731
    R.within(dx[~gap.cuda()], ref["dx"][~gap], lim(ref["dx"], ref["dx_err"])[~gap], "dx")
    if state:
        R.within(di[:batch], ref["di"], lim(ref["di"], ref["di_err"]), "d_initial")
        assert bool((di[batch:] == 3).all())
    R.within(dw[:D], ref["dw"], ref["dw_err"] + U * ref["dw"].abs(), "dw")
    R.within(db[:D], ref["db"], ref["db_err"] + U * ref["db"].abs(), "db")
    assert bool((dw[D] == 0.5).all()) and float(db[D]) == 0.5
    first = [v.clone() for v in outs[1]]
    for name, i in (("dw", 1), ("db", 2)):  # each alone
        one = torch.full_like(first[i][:D], 0.5)
        cm.causal_conv_backward(*args, **{name: one}, workspace=ws, **kw)
        R.same(one, first[i][:D].contiguous(), name + " alone")
    cm.causal_conv_backward(*args, **kw)  # neither: no workspace
    R.same(dx.contiguous(), first[0].contiguous(), "dx alone")
    cm.causal_conv_backward(*args, dw[:D], db[:D], 1, ws, **kw)
    R.within(dw[:D], 2 * ref["dw"], 2 * ref["dw_err"] + 4 * U * ref["dw"].abs(), "dw added")
    R.within(db[:D], 2 * ref["db"], 2 * ref["db_err"] + 4 * U * ref["db"].abs(), "db added")


@pytest.mark.parametrize("rows,D,W", [(7, 20, 4), (1000, 130, 3), (5000, 513, 4), (300, 40, 8)])
def test_whole_numbers_to_the_last_bit(rows, D, W):
    """Small whole numbers through ReLU: every sum is exact in fp32, so every bit is known."""
    import convolution_layer_amd as cm
    t = make(rows, 1, D, W, torch.float32, 2, whole=True)
    d = cm.make_causal_conv_desc(rows, D, W, activation=cm.ACT_RELU)
    z, _, _ = Q.conv_z(t["x"], t["w"], t["bias"], [(0, rows)], None)
    y, dx = (torch.empty(rows, D, device="cuda") for _ in range(2))
    dw, db = torch.empty(D, W, device="cuda"), torch.empty(D, device="cuda")
    cm.causal_conv_forward(d, t["x"].cuda(), t["w"].cuda(), t["bias"].cuda(), y)
    assert torch.equal(y.cpu().double(), z.clamp(min=0))
    cm.causal_conv_backward(d, t["x"].cuda(), t["w"].cuda(), t["bias"].cuda(), t["dy"].cuda(), dx, dw, db, 0,
                            cm.causal_conv_workspace(d))
    ref = Q.conv_backward(t["x"], t["w"], t["bias"], [(0, rows)], None, 1, t["dy"], None)
    for got, name in ((dx, "dx"), (dw, "dw"), (db, "db")):
        assert torch.equal(got.cpu().double(), ref[name]), name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,D,W,kind", [(1, 1, 1, 0), (1, 4096, 4, 5), (3, 37, 4, 5), (9, 2050, 2, 4), (5, 64, 8, 5),
                                           (200, 8, 4, 2)])
def test_step(rows, D, W, kind, dtype):
    import convolution_layer_amd as cm
    t = make(rows, rows + 3, D, W, dtype, 3)
    pool = t["initial"]
    n = rows + 3
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(rows))[:rows].to(torch.int32)
    seqs = [(i, i + 1) for i in range(rows)]
    for use in (None, slots):
        at = torch.arange(rows) if use is None else use.long()
        z, mag, ext = Q.conv_z(t["x"], t["w"], t["bias"], seqs, pool[at])
        after = pool.clone()
        for i, e in enumerate(ext):
            after[at[i]] = e[1:].to(dtype) if W > 1 else after[at[i]]
        state, y = pool.cuda(), torch.full((rows + 1, D), 3.0, dtype=dtype, device="cuda")
        d = cm.make_causal_conv_desc(rows, D, W, activation=kind, dtype=cdt(dtype))
        cm.causal_conv_step(d, t["x"].cuda(), t["w"].cuda(), t["bias"].cuda(), state, y[:rows],
                            slots=None if use is None else use.cuda())
        ref = Q.act(z, kind)
        err = 1.2 * (W + 1) * U * mag + Q.act_error(z, kind) + 2 * U * ref.abs()
        R.within(y[:rows], ref, err + R.HALF[dtype] * (ref.abs() + err), "y")
        assert bool((y[rows] == 3).all())
        assert torch.equal(state.cpu(), after), "state"


def test_step_slots_out_of_order():
    """Padding rows keep their y; slots that do not exist or come twice give NaN and touch no state."""
    import convolution_layer_amd as cm
    rows, D, W, n = 7, 40, 4, 5
    t = make(rows, n, D, W, torch.float32, 4)
    slots = torch.tensor([2, -1, 0, 2, 5, -7, 1 << 30], dtype=torch.int32)
    d = cm.make_causal_conv_desc(rows, D, W)
    state, y = t["initial"].cuda(), torch.full((rows, D), 3.0, device="cuda")
    cm.causal_conv_step(d, t["x"].cuda(), t["w"].cuda(), None, state, y, slots=slots.cuda())
    assert bool((y[[1, 5]] == 3).all()) and bool(torch.isnan(y[[3, 4, 6]]).all())
    z, mag, ext = Q.conv_z(t["x"], t["w"], None, [(0, 1), (2, 3)], t["initial"][[2, 0]])
    R.within(y[[0, 2]], z[[0, 2]], 6 * U * mag[[0, 2]], "y")
    want = t["initial"].clone()
    want[2], want[0] = ext[0][1:].float(), ext[1][1:].float()
    assert torch.equal(state.cpu(), want)


def test_tokens_one_by_one_are_the_prompt():
    """A prompt, then single tokens from its final state, give what the whole sequence gives, bit for bit."""
    import convolution_layer_amd as cm
    rows, D, W, cut = 30, 72, 4, 17
    t = make(rows, 1, D, W, torch.bfloat16, 5)
    x, w, b = t["x"].cuda(), t["w"].cuda(), t["bias"].cuda()
    kw = dict(activation=cm.ACT_SILU, dtype=cm.BF16)
    y, parts = torch.empty_like(x), torch.empty_like(x)
    cm.causal_conv_forward(cm.make_causal_conv_desc(rows, D, W, **kw), x, w, b, y)
    state = torch.empty(1, W - 1, D, dtype=torch.bfloat16, device="cuda")
    cm.causal_conv_forward(cm.make_causal_conv_desc(cut, D, W, **kw), x[:cut], w, b, parts[:cut], final_state=state)
    for i in range(cut, rows):
        cm.causal_conv_step(cm.make_causal_conv_desc(1, D, W, **kw), x[i:i + 1], w, b, state, parts[i:i + 1])
    R.same(y, parts, "y")


def test_starts_out_of_range_stay_inside():
    """Starts are device data: wrong ones give wrong sequences, never an access outside."""
    import convolution_layer_amd as cm
    rows, D, W = 40, 16, 4
    t = make(rows, 3, D, W, torch.float32, 6)
    d = cm.make_causal_conv_desc(rows, D, W, batch=3)
    for starts in ((-5, 10, 1 << 30, 2), (0, 30, 10, 40), (1 << 30, -1, 7, 1000)):
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        y = torch.full((rows + 8, D), 3.0, device="cuda")
        final, di = (torch.full((5, W - 1, D), 3.0, device="cuda") for _ in range(2))
        cm.causal_conv_forward(d, t["x"].cuda(), t["w"].cuda(), None, y[4:rows + 4], seq_starts=st, final_state=final[1:4])
        for v, lo, hi in ((y, 4, rows + 4), (final, 1, 4)):
            assert bool((v[:lo] == 3).all()) and bool((v[hi:] == 3).all())
        dx = torch.full((rows + 8, D), 3.0, device="cuda")
        cm.causal_conv_backward(d, t["x"].cuda(), t["w"].cuda(), None, t["dy"].cuda(), dx[4:rows + 4], seq_starts=st,
                                d_final_state=t["dfinal"].cuda(), d_initial_state=di[1:4])
        for v, lo, hi in ((dx, 4, rows + 4), (di, 1, 4)):
            assert bool((v[:lo] == 3).all()) and bool((v[hi:] == 3).all())
        assert bool(torch.isfinite(dx).all())


@pytest.mark.parametrize("rows,starts", [(1000, None), (1000, (0, 400, 401, 1000))])
def test_infinities_reach_the_taps_that_meet_them(rows, starts):
    """An infinite x makes infinite the sums that its products are in, and no others NaN: rows that only help a
    neighbouring run or lie behind a sequence count for nothing."""
    import convolution_layer_amd as cm
    D, W, batch = 1000, 4, 1 if starts is None else len(starts) - 1
    t = make(rows, batch, D, W, torch.float32, 10)
    seqs = Q.bounds(starts, rows, batch)
    for c in range(D):  # one a channel, at every row; the last row of each sequence among them
        t["x"][c % rows, c] = float("inf")
    d = cm.make_causal_conv_desc(rows, D, W, batch=batch)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    dx, dw = torch.empty(rows, D, device="cuda"), torch.empty(D, W, device="cuda")
    cm.causal_conv_backward(d, t["x"].cuda(), t["w"].cuda(), None, t["dy"].cuda(), dx, dw, None, 0,
                            cm.causal_conv_workspace(d), seq_starts=st)
    want, size = torch.zeros(D, W, dtype=torch.float64), torch.zeros(D, W, dtype=torch.float64)
    for a, e in seqs:
        for k in range(W):
            back = W - 1 - k
            p = t["dy"][a + back:e].double() * t["x"][a:max(e - back, a)].double()
            want[:, k] += p.sum(0)
            size[:, k] += p.abs().sum(0)
    got, inf = dw.cpu().double(), want.isinf()
    assert not want.isnan().any() and 0 < int((~inf).sum())
    assert torch.equal(got[inf], want[inf])
    R.within(got[~inf], want[~inf], ((rows + 1) * U * size)[~inf], "finite sums")


def test_gradient_against_differences():
    import convolution_layer_amd as cm
    rows, D, W, starts = 9, 5, 3, (0, 4, 9)
    t = {k: v.float() for k, v in make(rows, 2, D, W, torch.float32, 7).items()}
    seqs = Q.bounds(starts, rows, 2)
    d = cm.make_causal_conv_desc(rows, D, W, batch=2, activation=cm.ACT_SILU)
    dx, dw, db = (torch.empty(s, device="cuda") for s in ((rows, D), (D, W), (D,)))
    di = torch.empty(2, W - 1, D, device="cuda")
    cm.causal_conv_backward(d, t["x"].cuda(), t["w"].cuda(), t["bias"].cuda(), t["dy"].cuda(), dx, dw, db, 0,
                            cm.causal_conv_workspace(d), seq_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                            initial_state=t["initial"].cuda(), d_final_state=t["dfinal"].cuda(), d_initial_state=di)
    t = {k: v.double() for k, v in t.items()}

    def f(v):
        z, _, ext = Q.conv_z(v["x"], v["w"], v["bias"], seqs, v["initial"])
        fin = torch.stack([e[len(e) - (W - 1):] for e in ext])
        return float((Q.act(z, Q.SILU) * t["dy"]).sum() + (fin * t["dfinal"]).sum())

    h = 1e-5  # differences lose about 1e-6 at this step
    for name, got in (("x", dx), ("w", dw), ("bias", db), ("initial", di)):
        for i in range(t[name].numel()):
            p, m = dict(t), dict(t)
            for v, s in ((p, h), (m, -h)):
                v[name] = t[name].clone()
                v[name].view(-1)[i] += s
            num = (f(p) - f(m)) / (2 * h)
            assert abs(num - float(got.flatten()[i])) <= 1e-5 * (1 + abs(num)), (name, i)


def test_refusals_of_the_binding():
    import convolution_layer_amd as cm
    t = {k: v.cuda() for k, v in make(6, 2, 8, 4, torch.float32, 8).items()}
    d, y = cm.make_causal_conv_desc(6, 8, 4, batch=2), torch.empty(6, 8, device="cuda")
    call = lambda **kw: cm.causal_conv_forward(**{**dict(desc=d, x=t["x"], w=t["w"], bias=t["bias"], y=y), **kw})  # noqa: E731
    call()
    wide_x = torch.empty(6, 20, device="cuda")
    for kw in (dict(x=t["x"].cpu()), dict(x=wide_x[:, :8]), dict(x=t["x"].bfloat16()), dict(x=t["x"][:5]),
               dict(w=t["w"].t().contiguous()), dict(y=y.t()), dict(seq_starts=torch.zeros(3, device="cuda")),
               dict(seq_starts=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(initial_state=t["initial"][:1]),
               dict(desc=cm.make_causal_conv_desc(6, 8, 4, batch=2, x_pitch=20)),
               dict(desc=cm.make_causal_conv_desc(6, 8, 4, batch=2, x_pitch=20), x=wide_x[:, :16:2]),
               dict(desc=cm.make_causal_conv_desc(6, 8, 4, batch=2, x_pitch=24), x=wide_x[:, :8])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(cm.ConvmiError) as e:  # 6 rows are not 4 equal sequences
        cm.causal_conv_forward(cm.make_causal_conv_desc(6, 8, 4, batch=4), t["x"], t["w"], None, y)
    assert e.value.status == cm.ERR_INVALID_ARG
    call(desc=cm.make_causal_conv_desc(6, 8, 4, batch=2, x_pitch=20), x=wide_x[:, 3:11])


@pytest.mark.parametrize("pitch", [0, 1 << 20])
def test_offsets_beyond_32_bits(pitch):
    """The last rows of a tensor of more than 2^32 bytes."""
    import convolution_layer_amd as cm
    rows, D, W = (2 ** 20 + 5, 2100, 4) if pitch == 0 else (2400, 16, 4)
    m = torch.zeros(rows, pitch or D, dtype=torch.bfloat16, device="cuda")
    x = m[:, -D:]
    t = make(8, 1, D, W, torch.bfloat16, 9)
    x[-8:] = t["x"].cuda()
    y = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda")
    d = cm.make_causal_conv_desc(rows, D, W, dtype=cm.BF16, x_pitch=pitch)
    cm.causal_conv_forward(d, x, t["w"].cuda(), None, y)
    z, mag, _ = Q.conv_z(t["x"], t["w"], None, [(0, 8)], None)
    R.within(y[-8:], z, 5 * U * mag + 2.0 ** -8 * (z.abs() + 5 * U * mag), "last rows")
    dy = torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    dy[-8:] = t["dy"].cuda()
    dx = y if pitch == 0 else torch.empty_like(m)[:, -D:]
    cm.causal_conv_backward(d, x, t["w"].cuda(), None, dy, dx)
    ref = Q.conv_backward(t["x"], t["w"], None, [(0, 8)], None, 0, t["dy"], None)
    R.within(dx[-8:], ref["dx"], ref["dx_err"] + 2.0 ** -8 * (ref["dx"].abs() + ref["dx_err"]), "last rows of dx")


@pytest.mark.parametrize("starts", [None, (5, 70, 71, 4000, 8190)])
def test_long_runs_to_the_last_bit(starts):
    """Runs of 64 rows and their sums over workgroups, as a training batch has them, in whole numbers."""
    import convolution_layer_amd as cm
    rows, D, W, batch = 8192, 4096, 4, 4
    t = make(rows, batch, D, W, torch.bfloat16, 11, whole=True)
    seqs = Q.bounds(starts, rows, batch)
    gap = gaps(seqs, rows)
    x, dy = t["x"].clone(), t["dy"].clone()
    x[gap] = dy[gap] = float("nan")
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    d = cm.make_causal_conv_desc(rows, D, W, batch=batch, activation=cm.ACT_RELU, dtype=cm.BF16)
    dx = torch.full((rows, D), 3.0, dtype=torch.bfloat16, device="cuda")
    dw, db = torch.empty(D, W, device="cuda"), torch.empty(D, device="cuda")
    di = torch.empty(batch, W - 1, D, dtype=torch.bfloat16, device="cuda")
    ws = cm.causal_conv_workspace(d)
    assert ws.numel() == 32 * D * (W + 1) * 4  # workgroups of four threads that walk 64 rows each
    cm.causal_conv_backward(d, x.cuda(), t["w"].cuda(), t["bias"].cuda(), dy.cuda(), dx, dw, db, 0, ws.fill_(255),
                            seq_starts=st, initial_state=t["initial"].cuda(), d_final_state=t["dfinal"].cuda(),
                            d_initial_state=di)
    assert bool((dx[gap.cuda()] == 3).all())
    for c in range(0, D, 512):  # the definition by channels, which do not meet
        at = slice(c, c + 512)
        ref = Q.conv_backward(t["x"][:, at], t["w"][at], t["bias"][at], seqs, t["initial"][..., at], 1, t["dy"][:, at],
                              t["dfinal"][..., at])
        assert torch.equal(dx[:, at].cpu().double()[~gap], ref["dx"][~gap])
        assert torch.equal(dw[at].cpu().double(), ref["dw"]) and torch.equal(db[at].cpu().double(), ref["db"])
        assert torch.equal(di[..., at].cpu().double(), ref["di"])


def test_step_of_one_tap_looks_at_the_pool():
    """With one tap the states are empty, but a slot that the pool does not have still gives NaN."""
    import convolution_layer_amd as cm
    rows, D = 4, 12
    t = make(rows, 2, D, 1, torch.float32, 12)
    d = cm.make_causal_conv_desc(rows, D, 1)
    slots = torch.tensor([1, 3, -1, 0], dtype=torch.int32, device="cuda")
    y = torch.full((rows, D), 3.0, device="cuda")
    cm.causal_conv_step(d, t["x"].cuda(), t["w"].cuda(), None, t["initial"].cuda(), y, slots=slots)
    assert bool(torch.isnan(y[1]).all()) and bool((y[2] == 3).all())
    want = t["x"] * t["w"][:, 0]
    assert torch.equal(y[[0, 3]].cpu(), want[[0, 3]])
    cm.causal_conv_step(d, t["x"].cuda(), t["w"].cuda(), None, None, y)  # without a pool: a state for each row
    assert torch.equal(y.cpu(), want)
