"""Selective scan in the shapes in which long prompts and batches run, against the 64-bit definition."""
import pytest
import torch

from tests import block_reference as R
from tests import sequence_reference as Q
from tests.test_gpu_selective_scan import Call, check, make

pytestmark = pytest.mark.gpu

NAMES = ("x", "dt", "dt_bias", "A", "B", "C", "D", "z")


@pytest.mark.parametrize("N", [3, 16, 40])
@pytest.mark.parametrize("batch,starts", [(1, None), (2, (0, 700, 1000))])
def test_states_that_grow_across_chunks(batch, starts, N):
    """Steps below zero: a chunk's factor exp(A sum of delta) leaves fp32 at both ends while the state (or the
    gradient) that it meets is zero, or small enough for the product to stay inside."""
    rows, ch = 1000, 8
    t = make(rows, batch, ch, N, 1, torch.float32, plus=False, seed=20)
    x, dt, dy, A = t["x"], t["dt"], t["dy"], t["A"]
    t["initial"].zero_()
    t["dfinal"].zero_()
    # channels 0, 1: nothing comes in before row 100, the states' factors are e^4 .. e^84 a row up to there
    x[:100, :2], dt[:100, :2] = 0.0, -20.0
    dy[:, :2] = 0.0
    # channels 2, 3: the same for the gradient, from the last rows on
    x[:, 2:4], dy[600:, 2:4], dt[600:, 2:4] = 0.0, 0.0, -20.0
    # channels 4, 5: a state of 1e-30 grows by 2^140 in rows 32 .. 63 and shrinks by as much in the next 32
    x[:96, 4:6], dy[:, 4:6], A[4:6] = 0.0, 0.0, -1.0
    dt[:32, 4:6], dt[32:64, 4:6], dt[64:96, 4:6] = 0.0, -3.03, 3.03
    t["initial"][0, 4:6] = 1e-30
    part = {k: t[k] if k in ("x", "dt", "A", "B", "C") else None for k in NAMES}
    seqs = Q.bounds(starts, rows, batch)
    ref = Q.scan(part, seqs, 1, False, t["initial"], dy, t["dfinal"])
    assert all(bool(torch.isfinite(ref[k].v).all()) and float(ref[k].v.abs().max()) < 1e30 for k in ref)
    c = Call(t, rows, batch, ch, N, 1, starts, False, torch.float32, False, True, wide=False)
    got = c.forward() | c.backward()
    for k in ("y", "final", "dx", "ddt", "dB", "dC", "dA", "dinitial"):
        check(got[k], ref[k], torch.float32, k)


@pytest.mark.parametrize("rows,starts", [(45, None), (3001, None), (3001, (0, 700, 3000))])
def test_highest_rates_with_steps_below_zero(rows, starts):
    """The mirror image of A = -inf: with steps below zero A = inf forgets everything, as A = 1e38 does, in tiles
    that end inside and in chunks."""
    batch, ch, N = 1 if starts is None else 2, 5, 6
    t = make(rows, batch, ch, N, 1, torch.float32, plus=False, seed=22)
    t["dt"] = -1 - t["dt"]
    outs = []
    for highest in (1e38, 3e38, float("inf")):
        t["A"][:] = highest
        c = Call(t, rows, batch, ch, N, 1, starts, False, torch.float32, False, True, wide=False)
        outs.append(c.forward() | c.backward())
    inside = torch.zeros(rows, dtype=torch.bool)
    for a, e in Q.bounds(starts, rows, batch):
        inside[a:e] = True
    for k, v in outs[0].items():
        per_row = k in ("y", "dx", "ddt", "dB", "dC")
        assert bool(torch.isfinite(v[inside.cuda()] if per_row else v).all()), k
    for o in outs[1:]:
        for k in o:
            R.same(o[k].contiguous(), outs[0][k].contiguous(), k)


def test_more_rows_than_waves_of_the_sums():
    """Beyond 2^22 rows a wave adds up dB and dC of several: thousands of like sequences, all checked."""
    import convolution_layer_amd as cm
    n, batch, ch, N = 64, (1 << 16) + 1, 2, 1
    t = make(n, 1, ch, N, 1, torch.float32, seed=23)
    ref = Q.scan({k: t[k] for k in NAMES}, [(0, n)], 1, True, t["initial"], t["dy"], t["dfinal"])
    all_of = lambda v: v.cuda().repeat(batch, *[1] * (v.dim() - 1))  # noqa: E731
    d = cm.make_scan_desc(n * batch, ch, N, batch=batch)
    args = [all_of(t[k]) if k in ("x", "dt", "B", "C", "z") else t[k].cuda() for k in NAMES]
    like = lambda k: torch.full((n * batch, t[k].shape[1]), 3.0, device="cuda")  # noqa: E731
    y, saved = like("x"), cm.scan_saved_states(d)
    cm.selective_scan_forward(d, *args, y, initial_state=all_of(t["initial"]), saved_states=saved,
                              workspace=cm.scan_workspace(d, cm.SCAN_FORWARD))
    out = {"dx": like("x"), "ddt": like("x"), "dB": like("B"), "dC": like("C"), "dz": like("x")}
    cm.selective_scan_backward(d, *args, saved, all_of(t["dy"]), *out.values(), d_final_state=all_of(t["dfinal"]),
                               workspace=cm.scan_workspace(d, cm.SCAN_BACKWARD))
    for k, v in ({"y": y} | out).items():
        v = v.view(batch, n, -1)
        check(v[0], ref[k], torch.float32, k)
        assert bool((v == v[0]).all()), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("edge", [0, 1])
def test_long_sequences_among_many_short_ones(edge, dtype):
    """Some sequences of many chunks of 32 rows, beginning and ending on a chunk's border and beside it, between
    short and empty ones: the states between chunks stay apart, and inside the workspace."""
    import convolution_layer_amd as cm
    ch, N = 5, 6
    lens = [i % 3 for i in range(90)] + [333 - edge] + [0] * 20 + [64 + edge] * 3 + [1] * (30 + edge) + [256] + [33] * 4
    lens += [32] * 3 + [700] + [2] * 15
    starts = [3]
    for n in lens:
        starts.append(starts[-1] + n)
    rows, batch = starts[-1], len(lens)
    t = make(rows, batch, ch, N, 1, dtype, seed=24)
    ref = Q.scan({k: t[k] for k in NAMES}, Q.bounds(starts, rows, batch), 1, True, t["initial"], t["dy"], t["dfinal"])
    c = Call(t, rows, batch, ch, N, 1, starts, True, dtype, True, True, wide=False)
    guarded = []

    def ws(op):
        n = cm.scan_workspace_size(c.d, op)
        guarded.append((torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda"), n))
        return guarded[-1][0][:n]

    c.ws = ws
    got = c.forward() | c.backward()
    for w, n in guarded:
        assert bool((w[n:] == 255).all())
    for k in ("y", "dx", "ddt", "dB", "dC", "dz"):
        check(got[k], ref[k], dtype, k, torch.arange(rows) >= 3)
    for k in ("final", "dinitial", "dA", "dD", "ddt_bias"):
        check(got[k], ref[k], dtype, k)
    state, y = c.initial.clone(), torch.empty_like(got["y"])
    cm.selective_scan_forward(c.d, *c.args(), y, seq_starts=c.starts, initial_state=state, final_state=state,
                              workspace=ws(cm.SCAN_FORWARD))
    R.same(y[3:], got["y"][3:].contiguous(), "y, state in place")
    R.same(state, got["final"].contiguous(), "state in place")


# rows, batch, channels, states, groups, starts, softplus, rows of a chunk (0: sequences run whole)
TILES = [
    (2000, 1, 64, 5, 64, None, True, 96), (2000, 3, 64, 16, 64, (3, 700, 760, 1990), True, 96),
    (2600, 2, 70, 20, 70, None, True, 128), (1200, 2, 150, 40, 150, (0, 1000, 1200), True, 128),
    (1300, 1, 2640, 4, 40, None, True, 96), (1300, 2, 64, 3, 64, (0, 65, 1300), False, 64),
    (200, 1, 160, 16, 160, None, True, 0), (200, 3, 160, 20, 160, (5, 60, 61, 190), True, 0),
    (230, 1, 160, 40, 160, None, True, 0), (230, 1, 320, 7, 160, None, False, 0), (2100, 1, 160, 2, 160, None, True, 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,batch,ch,N,G,starts,plus,chunk", TILES)
def test_several_tiles(rows, batch, ch, N, G, starts, plus, chunk, dtype):
    """Chunks of two to four tiles and whole sequences of seven and more, with states before and behind."""
    t = make(rows, batch, ch, N, G, dtype, plus, seed=21)
    seqs = Q.bounds(starts, rows, batch)
    inside = torch.zeros(rows, dtype=torch.bool)
    for a, e in seqs:
        inside[a:e] = True
    ref = Q.scan({k: t[k] for k in NAMES}, seqs, G, plus, t["initial"], t["dy"], t["dfinal"])
    c = Call(t, rows, batch, ch, N, G, starts, plus, dtype, True, True, wide=False)
    # a state and a sum for each chunk, up to 256 bytes each: the size tells how long the chunks are
    places = min(rows // chunk + batch, 2 * (rows // chunk)) if chunk else 0
    size = -(-places * ch * N * 4 // 256) * 256 + -(-places * ch * 4 // 256) * 256
    assert c.cm.scan_workspace_size(c.d, c.cm.SCAN_FORWARD) == size
    got = c.forward() | c.backward()
    for k in ("y", "dx", "ddt", "dB", "dC", "dz"):
        check(got[k], ref[k], dtype, k, inside)
    for k in ("final", "dinitial", "dA", "dD", "ddt_bias"):
        check(got[k], ref[k], dtype, k)


@pytest.mark.parametrize("starts", [(-5, 10, 1 << 30, 2), (0, 130, 10, 200), (1 << 30, -1, 7, 1000), (0, 200, 0, 200),
                                    (190, 5, -(1 << 31), (1 << 31) - 1)])
def test_wrong_starts_write_nothing_outside(starts):
    """Starts that decrease or lie outside give wrong sequences, but every output keeps what stands around it."""
    import convolution_layer_amd as cm
    rows, batch, ch, N = 200, 3, 70, 16
    t = make(rows, batch, ch, N, 1, torch.float32, seed=25)
    d = cm.make_scan_desc(rows, ch, N, batch=batch)
    whole = []

    def guarded(n, *shape, dtype=torch.float32):  # n rows between 64 others on either side
        whole.append(torch.full((n + 128, *shape), 3, dtype=dtype, device="cuda"))
        return whole[-1][64:64 + n]

    args = [t[k].cuda() for k in NAMES]
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    ws = [guarded(cm.scan_workspace_size(d, op) // 64, 64, dtype=torch.uint8) for op in (cm.SCAN_FORWARD, cm.SCAN_BACKWARD)]
    ws = [w.fill_(255).view(-1) for w in ws]
    y, final, saved = guarded(rows, ch), guarded(batch, ch, N), guarded(cm.scan_saved_size(d) // (4 * N), N)
    cm.selective_scan_forward(d, *args, y, seq_starts=st, initial_state=t["initial"].cuda(), final_state=final,
                              saved_states=saved, workspace=ws[0])
    dx, ddt, dB, dC, dz = (guarded(rows, n) for n in (ch, ch, N, N, ch))
    dbias, dA, dD, di = guarded(ch), guarded(ch, N), guarded(ch), guarded(batch, ch, N)
    cm.selective_scan_backward(d, *args, saved, t["dy"].cuda(), dx, ddt, dB, dC, dz, dbias, dA, dD, 0, ws[1], st,
                               t["dfinal"].cuda(), di)
    for v in whole:
        assert bool((v[:64] == 3).all()) and bool((v[-64:] == 3).all()), v.shape
