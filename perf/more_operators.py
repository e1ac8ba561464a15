"""Work lists of the sequence-mixing operators: layer norm, short causal convolution and
selective state space scan, for training batches, prompts and single tokens.

``run`` computes one pass of an operator on the state that ``prepare`` made: with the
module's ``own`` false in a plain form of elementary torch operations in 32 bits, with
``own`` true through convolution_layer_amd's entry points.  ``exact`` computes the same
outputs from the definitions in 64 bits.

The operators, for rows r or t, columns c, channels d, states n, taps k of W:

  layer norm    h = x + residual; y = gamma (h - mean) inv_std + beta
    backward    hhat = (h - mean) inv_std; g = gamma dy; dgamma = sum_r dy hhat; dbeta = sum_r dy
                dx = dh + inv_std (g - mean_c(g) - hhat mean_c(g hhat))
  causal conv   z_t = bias + sum_k w_k x_(t-W+1+k) within the row's sequence; y = act(z); what
                lies before a sequence comes from its initial state, the last W-1 inputs are
                its final one.  One token: the state is shifted in place.
  scan          delta = softplus(dt + dt_bias); h_t = exp(delta A) h_(t-1) + delta B_t x_t
                y_t = (sum_n C_t h_t + D x_t) silu(z_t)
                B and C are shared by the channels of a group; h before a sequence is its
                initial state.  One token: the state is updated in place.
Sequences lie one behind the other in the rows.
"""
import math
import random

import torch

own = False

EPS = 1e-5
BLOCK = 32


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token's hidden state, normalised before the next layer
        {"name": "norm_token", "kind": "norm_forward", "dtype": "bf16", "rows": 1, "cols": 4096, "residual": True,
         "y8": False},
        # a training batch's tokens, with the residual's addition
        {"name": "norm_batch", "kind": "norm_forward", "dtype": "bf16", "rows": 8192, "cols": 4096, "residual": True,
         "y8": False},
        # the same batch's backward pass, with the residual branch's gradient added
        {"name": "norm_backward_batch", "kind": "norm_backward", "dtype": "bf16", "rows": 8192, "cols": 4096,
         "residual": True},
        # a ragged float32 batch: odd width, odd number of rows
        {"name": "norm_backward_odd", "kind": "norm_backward", "dtype": "f32", "rows": 1733, "cols": 771,
         "residual": False},
        # one new token of each of 64 running sequences, their states in a pool of 96
        {"name": "conv_tokens", "kind": "conv_step", "dtype": "bf16", "rows": 64, "slots": 96, "channels": 4096,
         "taps": 4, "act": "silu"},
        # prompts of unequal length, one behind the other, read from one half of a projection
        {"name": "conv_prompts", "kind": "conv_forward", "dtype": "bf16", "rows": 6151, "batch": 7, "ragged": True,
         "channels": 4096, "taps": 4, "act": "silu", "initial": False, "pitched": True},
        # a training batch's backward pass, the gradient written into the projection's
        {"name": "conv_backward_batch", "kind": "conv_backward", "dtype": "bf16", "rows": 8192, "batch": 4,
         "ragged": False, "channels": 4096, "taps": 4, "act": "silu", "initial": False, "pitched": True},
        # sizes that divide nothing, in float32
        {"name": "conv_backward_odd", "kind": "conv_backward", "dtype": "f32", "rows": 1003, "batch": 5,
         "ragged": True, "channels": 517, "taps": 3, "act": "gelu", "initial": False, "pitched": False},
        # one new token of each of 64 running sequences
        {"name": "scan_tokens", "kind": "scan_step", "dtype": "bf16", "rows": 64, "slots": 96, "channels": 4096,
         "states": 16, "groups": 1, "gate": True},
        # prompts of unequal length that go on from kept states
        {"name": "scan_prompts", "kind": "scan_forward", "dtype": "bf16", "rows": 6151, "batch": 5, "ragged": True,
         "channels": 4096, "states": 16, "groups": 1, "gate": True, "initial": True},
        # a training batch, forward and backward
        {"name": "scan_train_batch", "kind": "scan_train", "dtype": "bf16", "rows": 8192, "batch": 4, "ragged": False,
         "channels": 4096, "states": 16, "groups": 1, "gate": True, "initial": False},
        # sizes that divide nothing, in float32, B and C of two groups
        {"name": "scan_train_odd", "kind": "scan_train", "dtype": "f32", "rows": 701, "batch": 3, "ragged": True,
         "channels": 134, "states": 5, "groups": 2, "gate": False, "initial": True},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; half of them as drawn (odd ones
    among them), the others rounded to a multiple of 64 where that stays in the range."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    kind = rng.choice(["norm_forward", "norm_backward", "conv_step", "conv_forward", "conv_backward", "scan_step",
                       "scan_forward", "scan_train", "scan_train"])
    case = {"kind": kind, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if kind in ("norm_forward", "norm_backward"):
        case["cols"] = _spread(rng, 16, 16384)
        case["rows"] = _spread(rng, 1, min(16384, (1 << 25) // case["cols"]))
        case["residual"] = rng.random() < 0.5
        if kind == "norm_forward":
            case["y8"] = rng.random() < 0.4
        return case
    scan = kind.startswith("scan")
    if scan:
        case["groups"] = rng.choice([1, 1, 1, 2, 4])
        case["states"] = rng.choice([16, 16, 8, rng.randint(1, 32)])
        case["channels"] = _spread(rng, 16, 2048) * case["groups"]
        case["gate"] = rng.random() < 0.7
        most = (1 << 28) // (case["channels"] * case["states"])
    else:
        case["channels"] = _spread(rng, 16, 8192)
        case["taps"] = rng.choice([4, 4, rng.randint(2, 8)])
        case["act"] = rng.choice(["silu", "silu", "identity", "relu", "gelu"])
        most = (1 << 25) // case["channels"]
    if kind.endswith("step"):
        case["rows"] = _spread(rng, 1, 256)
        case["slots"] = case["rows"] + rng.randint(0, 64)
        return case
    case["rows"] = _spread(rng, 1, max(1, min(16384, most)))
    case["batch"] = rng.randint(1, min(8, case["rows"]))
    case["ragged"] = rng.random() < 0.6
    if not case["ragged"]:
        case["rows"] -= case["rows"] % case["batch"]
    case["initial"] = kind != "conv_backward" and rng.random() < 0.4
    if not scan:
        case["pitched"] = rng.random() < 0.5
    return case


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    kind, r = case["kind"], case["rows"]
    if kind == "norm_forward":
        c, n = case["cols"], r * case["cols"]
        out = n + r * -(-c // BLOCK) if case["y8"] else n * es
        return {"bytes": n * es * (3 if case["residual"] else 1) + out + 8 * (r + c), "flops": 8 * n}
    if kind == "norm_backward":
        c, n = case["cols"], r * case["cols"]
        return {"bytes": n * es * (4 if case["residual"] else 3) + 8 * r + 12 * c, "flops": 15 * n}
    d, n = case["channels"], r * case["channels"]
    if kind.startswith("conv"):
        w = case["taps"]
        if kind == "conv_step":  # the state moves by one row: read and written
            return {"bytes": n * es * (2 * (w - 1) + 2) + d * (w * es + 4), "flops": n * (2 * w + 4)}
        state = case["batch"] * (w - 1) * d * es
        if kind == "conv_forward":
            return {"bytes": 2 * n * es + state * (2 if case["initial"] else 1) + d * (w * es + 4),
                    "flops": n * (2 * w + 4)}
        return {"bytes": 3 * n * es + d * (w * (es + 4) + 8), "flops": n * (6 * w + 8)}
    s, gn = case["states"], case["groups"] * case["states"]
    params = 4 * d * (s + 2)
    if kind == "scan_step":
        return {"bytes": n * es * (4 if case["gate"] else 3) + 2 * r * gn * es + 8 * n * s + params,
                "flops": n * (7 * s + 12)}
    state = 4 * case["batch"] * d * s
    forward = n * es * (4 if case["gate"] else 3) + 2 * r * gn * es + params
    if kind == "scan_forward":
        return {"bytes": forward + state * (2 if case["initial"] else 1), "flops": n * (7 * s + 12)}
    backward = n * es * (7 if case["gate"] else 5) + 4 * r * gn * es + 2 * params
    return {"bytes": forward + backward + state * (4 if case["initial"] else 1), "flops": n * (27 * s + 40)}


# ------------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, kind, r = _dtype(case), case["kind"], case["rows"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def hidden(rows, cols):  # channels of unequal size and mean, as hidden states have
        return (normal(rows, cols) + 0.3 * normal(cols)) * torch.exp(0.5 * normal(cols))

    s = {"case": case, "out": {}}
    if kind == "norm_forward":
        s["x"] = hidden(r, case["cols"]).to(dt)
        s["residual"] = hidden(r, case["cols"]).to(dt) if case["residual"] else None
        s["gamma"], s["beta"] = 1.0 + 0.2 * normal(case["cols"]), 0.1 * normal(case["cols"])
        return s
    if kind == "norm_backward":
        s["h"] = hidden(r, case["cols"]).to(dt)
        h = s["h"].double()
        s["mean"] = h.mean(-1).float()
        s["inv_std"] = (h.var(-1, unbiased=False) + EPS).rsqrt().float()
        s["gamma"] = 1.0 + 0.2 * normal(case["cols"])
        s["dy"] = normal(r, case["cols"], std=0.01).to(dt)
        s["dh"] = normal(r, case["cols"], std=0.01).to(dt) if case["residual"] else None
        return s
    D = case["channels"]
    if kind.endswith("step"):
        order = torch.randperm(case["slots"], generator=g, device="cuda")
        s["slots"] = order[:r].to(torch.int32)
    else:
        b = case["batch"]
        if case["ragged"]:
            cuts = sorted(random.Random(seed).sample(range(1, r), b - 1)) if b > 1 else []
        else:
            cuts = [r // b * i for i in range(1, b)]
        s["lens"] = [e - a for a, e in zip([0] + cuts, cuts + [r])]
        s["starts"] = torch.tensor([0] + cuts + [r], dtype=torch.int32, device="cuda")
    if kind.startswith("conv"):
        W = case["taps"]
        if kind != "conv_step" and case["pitched"]:  # the projection holds the gate beside the input
            s["xz"] = normal(r, 2 * D).to(dt)
            s["x"] = s["xz"][:, :D]
        else:
            s["x"] = normal(r, D).to(dt)
        s["w"] = normal(D, W, std=1.0 / math.sqrt(W)).to(dt)
        s["bias"] = 0.1 * normal(D)
        if kind == "conv_step":
            s["state"] = normal(case["slots"], W - 1, D).to(dt)
        elif case["initial"]:
            s["initial"] = normal(case["batch"], W - 1, D).to(dt)
        if kind == "conv_backward":
            s["dy"] = normal(r, D, std=0.01).to(dt)
        return s
    G, N = case["groups"], case["states"]
    x = normal(r, D)
    s["x"] = (x * torch.sigmoid(x)).to(dt)
    s["dt"] = normal(r, D, std=0.5).to(dt)
    step = torch.exp(uniform(D) * math.log(100.0) + math.log(0.001))  # 0.001 .. 0.1
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(1.0 + torch.arange(N, device="cuda")) * torch.exp(0.1 * normal(D, N))
    s["bc"] = normal(r, 2 * G * N).to(dt)  # one projection's output
    s["B"], s["C"] = s["bc"][:, :G * N], s["bc"][:, G * N:]
    s["D"] = 1.0 + 0.1 * normal(D)
    if case["gate"]:
        s["xz"] = normal(r, 2 * D).to(dt)
        s["z"] = s["xz"][:, D:]
    else:
        s["z"] = None
    if kind == "scan_step":
        s["state"] = normal(case["slots"], D, N)
    else:
        s["initial"] = normal(case["batch"], D, N) if case["initial"] else None
        if kind == "scan_train":
            s["dy"] = normal(r, D, std=0.01).to(dt)
    return s


# -------------------------------------------------------------------- plain form
def _values8(v):
    """The float32 values that the rows of v stand for once kept as e4m3 codes with one
    power of two per 32 values, the smallest that brings the largest to 448 or below."""
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    blocks = torch.nn.functional.pad(v, (0, nb * BLOCK - cols)).reshape(rows, nb, BLOCK)
    e = ((blocks.abs().amax(-1).view(torch.int32) + 0x1FFFFF) >> 23) - 8  # 448 = 1.75 * 2^8
    e = e.clamp_min(1)
    inv, scale = ((254 - e) << 23).view(torch.float32), (e << 23).view(torch.float32)
    codes = (blocks * inv.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return (codes.float() * scale.unsqueeze(-1)).reshape(rows, nb * BLOCK)[:, :cols]


def _silu(a):
    return a / (1.0 + torch.exp(-a))


def _silu_slope(a):
    s = 1.0 / (1.0 + torch.exp(-a))
    return s * (1.0 + a * (1.0 - s))


def _gelu_t(a):
    return torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a))


def _act(a, act):
    if act == "silu":
        return _silu(a)
    if act == "relu":
        return a.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * a * (1.0 + _gelu_t(a))
    return a


def _slope(a, act):
    if act == "silu":
        return _silu_slope(a)
    if act == "relu":
        return (a > 0).to(a.dtype)
    if act == "gelu":
        t = _gelu_t(a)
        return 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * a * a)
    return torch.ones_like(a)


def _softplus(v):
    return v.clamp_min(0.0) + torch.log1p(torch.exp(-v.abs()))


def _recurrence(a, b):
    """h_t = a_t h_(t-1) + b_t along the first axis, from zero: pairs of steps are joined
    into one, the half as long recurrence gives every second h, one step each the others."""
    n = a.shape[0]
    if n == 1:
        return b
    m = n // 2 * 2
    odd = _recurrence(a[1:m:2] * a[0:m:2], a[1:m:2] * b[0:m:2] + b[1:m:2])
    h = torch.empty_like(b)
    h[1:m:2] = odd
    h[0] = b[0]
    h[2::2] = a[2::2] * odd[: (n - 1) // 2] + b[2::2]
    return h


def _rows_of(s):
    """First row and sequence of every row."""
    n = s["starts"].diff().long()
    first = torch.repeat_interleave(s["starts"][:-1].long(), n, output_size=s["case"]["rows"])
    return first, torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=s["case"]["rows"])


def _taps(s, rows, first, seq):
    """x at `rows` [m, k] of sequences that begin at `first` [m, 1], float32 [m, k, channels]: rows
    before it come from the initial state, or are zero."""
    W, inside = s["case"]["taps"], rows >= first
    x = s["x"].float()[rows.clamp_min(0)]
    if s.get("initial") is not None:
        before = s["initial"].float()[seq.unsqueeze(-1), (rows - first + W - 1).clamp(0, W - 2)]
        return torch.where(inside.unsqueeze(-1), x, before)
    return x * inside.unsqueeze(-1)


def _plain_conv(s):
    case, dt = s["case"], _dtype(s["case"])
    W, w = case["taps"], s["w"].float()
    if case["kind"] == "conv_step":
        slots = s["slots"].long()
        xe = torch.cat([s["state"][slots], s["x"].unsqueeze(1)], 1).float()  # [rows, W, channels]
        y = _act((xe * w.t()).sum(1) + s["bias"], case["act"])
        s["state"][slots] = xe[:, 1:].to(dt)
        return {"y": y.to(dt), "state": s["state"]}
    first, seq = _rows_of(s)
    rows = torch.arange(case["rows"], device="cuda").unsqueeze(-1)
    k = torch.arange(W, device="cuda")
    xe = _taps(s, rows - (W - 1) + k, first.unsqueeze(-1), seq)
    z = (xe * w.t()).sum(1) + s["bias"]
    if case["kind"] == "conv_forward":
        ends = s["starts"][1:].long().unsqueeze(-1)
        final = _taps(s, ends - (W - 1) + k[:-1], s["starts"][:-1].long().unsqueeze(-1),
                      torch.arange(case["batch"], device="cuda"))
        return {"y": _act(z, case["act"]).to(dt), "final": final.to(dt)}
    dz = s["dy"].float() * _slope(z, case["act"])
    after = rows + (W - 1) - k  # the rows whose tap k reads this one
    end = s["starts"][1:].long()[seq].unsqueeze(-1)
    dx = (dz[after.clamp_max(case["rows"] - 1)] * (after < end).unsqueeze(-1) * w.t()).sum(1)
    return {"dx": dx.to(dt), "dw": (xe * dz.unsqueeze(1)).sum(0).t().contiguous(), "db": dz.sum(0)}


def _plain_scan(s):
    case, dt = s["case"], _dtype(s["case"])
    r, D, G, N = case["rows"], case["channels"], case["groups"], case["states"]
    x, v = s["x"].float(), s["dt"].float() + s["dt_bias"]
    delta = _softplus(v)
    A = s["A"]
    B = s["B"].float().reshape(r, G, 1, N).expand(r, G, D // G, N).reshape(r, D, N)
    C = s["C"].float().reshape(r, G, 1, N).expand(r, G, D // G, N).reshape(r, D, N)
    a = torch.exp(delta.unsqueeze(-1) * A)
    b = (delta * x).unsqueeze(-1) * B
    gate = _silu(s["z"].float()) if case["gate"] else torch.ones_like(x)
    if case["kind"] == "scan_step":
        slots = s["slots"].long()
        h = a * s["state"][slots] + b
        s["state"][slots] = h
        return {"y": (((h * C).sum(-1) + s["D"] * x) * gate).to(dt), "state": s["state"]}
    first, last = s["starts"][:-1].long(), s["starts"][1:].long() - 1
    start = s["initial"] if case["initial"] else torch.zeros(case["batch"], D, N, device="cuda")
    b[first] += a[first] * start
    a0 = a.clone()
    a0[first] = 0.0
    h = _recurrence(a0, b)
    y = (h * C).sum(-1) + s["D"] * x
    out = {"y": (y * gate).to(dt), "final": h[last]}
    if case["kind"] == "scan_forward":
        return out
    dy = s["dy"].float()
    if case["gate"]:
        out["dz"] = (dy * y * _silu_slope(s["z"].float())).to(dt)
        dy = dy * gate
    a_next = torch.cat([a[1:], torch.zeros_like(a[:1])])
    a_next[last] = 0.0
    g = _recurrence(a_next.flip(0), (C * dy.unsqueeze(-1)).flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = start
    if case["initial"]:
        out["dinitial"] = a[first] * g[first]
    q = g * a * before
    through = (g * B).sum(-1)
    out["dx"] = (delta * through + s["D"] * dy).to(dt)
    ddelta = x * through + (q * A).sum(-1)
    ddt = ddelta / (1.0 + torch.exp(-v))
    out["ddt"], out["ddt_bias"] = ddt.to(dt), ddt.sum(0)
    out["dA"], out["dD"] = (delta.unsqueeze(-1) * q).sum(0), (dy * x).sum(0)
    out["dB"] = ((delta * x).unsqueeze(-1) * g).reshape(r, G, D // G, N).sum(2).reshape(r, G * N).to(dt)
    out["dC"] = (dy.unsqueeze(-1) * h).reshape(r, G, D // G, N).sum(2).reshape(r, G * N).to(dt)
    return out


def _plain(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind.startswith("conv"):
        return _plain_conv(s)
    if kind.startswith("scan"):
        return _plain_scan(s)
    dt = _dtype(case)
    if kind == "norm_forward":
        h = s["x"].float()
        if case["residual"]:
            h = h + s["residual"].float()
        mean = h.mean(-1)
        c = h - mean.unsqueeze(-1)
        inv = 1.0 / torch.sqrt((c * c).mean(-1) + EPS)
        y = s["gamma"] * (c * inv.unsqueeze(-1)) + s["beta"]
        out = {"mean": mean, "inv_std": inv, "y": _values8(y).to(torch.bfloat16) if case["y8"] else y.to(dt)}
        if case["residual"]:
            out["h"] = h.to(dt)
        return out
    dy, inv = s["dy"].float(), s["inv_std"].unsqueeze(-1)
    hhat = (s["h"].float() - s["mean"].unsqueeze(-1)) * inv
    g = s["gamma"] * dy
    dx = inv * (g - g.mean(-1, keepdim=True) - hhat * (g * hhat).mean(-1, keepdim=True))
    if case["residual"]:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * hhat).sum(0), "dbeta": dy.sum(0)}


# ------------------------------------------------------------ the framework's calls
def _kept(s, name, make):
    """What a program makes once and keeps from call to call."""
    if name not in s["out"]:
        s["out"][name] = make()
    return s["out"][name]


def _buffer(s, name, shape, dtype):
    return _kept(s, name, lambda: torch.empty(shape, dtype=dtype, device="cuda"))


def _own_norm(s, cm, cdt):
    case, dt = s["case"], _dtype(s["case"])
    rows, cols, f32 = case["rows"], case["cols"], torch.float32
    desc = _kept(s, "desc", lambda: cm.make_layer_norm_desc(rows, cols, dtype=cdt, eps=EPS))
    if case["kind"] == "norm_backward":
        dx = _buffer(s, "dx", (rows, cols), dt)
        dgamma, dbeta = _buffer(s, "dgamma", (cols,), f32), _buffer(s, "dbeta", (cols,), f32)
        ws = _kept(s, "ws", lambda: cm.layer_norm_workspace(desc))
        cm.layer_norm_backward(desc, s["h"], s["gamma"], s["mean"], s["inv_std"], s["dy"], s["dh"], dx, dgamma, dbeta,
                               accumulate=0, workspace=ws)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    out = {"mean": _buffer(s, "mean", (rows,), f32), "inv_std": _buffer(s, "inv_std", (rows,), f32)}
    if case["residual"]:
        out["h"] = _buffer(s, "h", (rows, cols), dt)
    q = qs = y = None
    if case["y8"]:
        q = _buffer(s, "y8", (rows, cols), torch.uint8)
        qs = _buffer(s, "y8_scales", (rows, -(-cols // BLOCK)), torch.uint8)
        out["y"] = _buffer(s, "values", (rows, cols), torch.bfloat16)
    else:
        y = out["y"] = _buffer(s, "y", (rows, cols), dt)
    cm.layer_norm_forward(desc, s["x"], s["residual"], s["gamma"], s["beta"], out.get("h"), y, out["mean"],
                          out["inv_std"], y8=q, y8_scales=qs)
    if case["y8"]:
        cm.mx8_unpack(q, qs, out["y"])
    return out


def _own_conv(s, cm, cdt):
    case, dt, kind = s["case"], _dtype(s["case"]), s["case"]["kind"]
    rows, D, W = case["rows"], case["channels"], case["taps"]
    act = {"identity": cm.ACT_IDENTITY, "relu": cm.ACT_RELU, "gelu": cm.ACT_GELU, "silu": cm.ACT_SILU}[case["act"]]
    pitch = 2 * D if case.get("pitched") else 0
    desc = _kept(s, "desc", lambda: cm.make_causal_conv_desc(rows, D, W, batch=case.get("batch", rows),
                                                             activation=act, dtype=cdt, x_pitch=pitch))
    if kind == "conv_step":
        y = _buffer(s, "y", (rows, D), dt)
        cm.causal_conv_step(desc, s["x"], s["w"], s["bias"], s["state"], y, slots=s["slots"])
        return {"y": y, "state": s["state"]}
    starts = s["starts"] if case["ragged"] else None
    if kind == "conv_forward":
        out = {"y": _buffer(s, "y", (rows, D), dt), "final": _buffer(s, "final", (case["batch"], W - 1, D), dt)}
        cm.causal_conv_forward(desc, s["x"], s["w"], s["bias"], out["y"], seq_starts=starts,
                               initial_state=s.get("initial"), final_state=out["final"])
        return out
    # the gradient's rows lie as the input's do: beside the gate's gradient in the projection's
    dx = _kept(s, "dx", lambda: torch.empty((rows, pitch or D), dtype=dt, device="cuda")[:, :D])
    dw, db = _buffer(s, "dw", (D, W), torch.float32), _buffer(s, "db", (D,), torch.float32)
    ws = _kept(s, "ws", lambda: cm.causal_conv_workspace(desc))
    cm.causal_conv_backward(desc, s["x"], s["w"], s["bias"], s["dy"], dx, dw, db, accumulate=0, workspace=ws,
                            seq_starts=starts)
    return {"dx": dx, "dw": dw, "db": db}


def _own_scan(s, cm, cdt):
    case, dt, kind = s["case"], _dtype(s["case"]), s["case"]["kind"]
    rows, D, G, N, f32 = case["rows"], case["channels"], case["groups"], case["states"], torch.float32
    desc = _kept(s, "desc", lambda: cm.make_scan_desc(
        rows, D, N, batch=case.get("batch", rows), groups=G, dtype=cdt, delta_softplus=True,
        z_pitch=2 * D if case["gate"] else 0, bc_pitch=2 * G * N))
    y = _buffer(s, "y", (rows, D), dt)
    args = (s["x"], s["dt"], s["dt_bias"], s["A"], s["B"], s["C"], s["D"], s["z"])
    if kind == "scan_step":
        cm.selective_scan_step(desc, *args, s["state"], y, slots=s["slots"])
        return {"y": y, "state": s["state"]}
    starts = s["starts"] if case["ragged"] else None
    out = {"y": y, "final": _buffer(s, "final", (case["batch"], D, N), f32)}
    train = kind == "scan_train"
    saved = _kept(s, "saved", lambda: cm.scan_saved_states(desc)) if train else None
    cm.selective_scan_forward(desc, *args, y, seq_starts=starts, initial_state=s["initial"],
                              final_state=out["final"], saved_states=saved,
                              workspace=_kept(s, "ws", lambda: cm.scan_workspace(desc, cm.SCAN_FORWARD)))
    if not train:
        return out
    out["dx"], out["ddt"] = _buffer(s, "dx", (rows, D), dt), _buffer(s, "ddt", (rows, D), dt)
    out["ddt_bias"], out["dD"] = _buffer(s, "ddt_bias", (D,), f32), _buffer(s, "dD", (D,), f32)
    out["dA"] = _buffer(s, "dA", (D, N), f32)
    dbc = _buffer(s, "dbc", (rows, 2 * G * N), dt)
    out["dB"], out["dC"] = dbc[:, :G * N], dbc[:, G * N:]
    if case["gate"]:
        out["dz"] = _buffer(s, "dxz", (rows, 2 * D), dt)[:, D:]
    if case["initial"]:
        out["dinitial"] = _buffer(s, "dinitial", (case["batch"], D, N), f32)
    cm.selective_scan_backward(desc, *args, saved, s["dy"], out["dx"], out["ddt"], out["dB"], out["dC"],
                               out.get("dz"), out["ddt_bias"], out["dA"], out["dD"], accumulate=0,
                               workspace=_kept(s, "ws2", lambda: cm.scan_workspace(desc, cm.SCAN_BACKWARD)),
                               seq_starts=starts, d_initial_state=out.get("dinitial"))
    return out


def run(state):
    if own:
        import convolution_layer_amd as cm
        case = state["case"]
        cdt = cm.BF16 if case["dtype"] == "bf16" else cm.F32
        call = {"norm": _own_norm, "conv": _own_conv, "scan": _own_scan}[case["kind"].split("_")[0]]
        return call(state, cm, cdt)
    return _plain(state)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    kind, r = case["kind"], case["rows"]
    f64 = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}

    def act(z):
        if case["act"] == "gelu":
            return z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z.pow(3)))
        return {"identity": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()

    def kept8(v):
        # each block of 32 times a power of two, rounded to 4 significant bits (ties to
        # even), spacing 2^-9 below 2^-6
        rows, cols = v.shape
        b = torch.nn.functional.pad(v, (0, -cols % BLOCK)).reshape(rows, -1, BLOCK)
        top = b.abs().amax(-1, keepdim=True)
        _, e = torch.frexp(top / 448.0)
        e = torch.where(torch.ldexp(torch.full_like(top, 448.0), e - 1) >= top, e - 1, e).clamp_min(-126)
        u = torch.ldexp(b, -e)
        step = torch.ldexp(torch.ones_like(u), torch.clamp(torch.frexp(u)[1] - 4, min=-9))
        return torch.ldexp(torch.round(u / step) * step, e).reshape(rows, -1)[:, :cols]

    if kind == "norm_forward":
        h = f64["x"] + f64.get("residual", 0.0)
        mean, var = h.sum(-1) / case["cols"], h.var(-1, unbiased=False)
        y = (h - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * f64["gamma"] + f64["beta"]
        out = {"mean": mean, "inv_std": (var + EPS) ** -0.5, "y": kept8(y) if case["y8"] else y}
        return out | {"h": h} if case["residual"] else out
    if kind == "norm_backward":
        inv, dy = f64["inv_std"][:, None], f64["dy"]
        centred = f64["h"] - f64["mean"][:, None]
        g = dy * f64["gamma"] * inv
        dx = g - g.sum(-1, keepdim=True) / case["cols"]
        dx = dx - centred * inv.square() * (g * centred).sum(-1, keepdim=True) / case["cols"]
        return {"dx": dx + f64.get("dh", 0.0), "dgamma": (dy * centred * inv).sum(0), "dbeta": dy.sum(0)}

    D = case["channels"]
    if kind.startswith("conv"):
        W = case["taps"]
        if kind == "conv_step":
            at = s["slots"].long()
            old = f64["state"][at]
            z = f64["bias"] + f64["w"][:, W - 1] * f64["x"]
            for k in range(W - 1):
                z = z + f64["w"][:, k] * old[:, k]
            state = f64["state"]
            state[at] = torch.cat([old[:, 1:], f64["x"][:, None]], 1)
            return {"y": act(z), "state": state}
        leaves = {k: f64[k].clone().requires_grad_() for k in ("x", "w", "bias")}
        ys, finals, begin = [], [], 0
        for i, n in enumerate(s["lens"]):  # each sequence behind its state, tap by tap
            head = f64["initial"][i] if case["initial"] else torch.zeros(W - 1, D, dtype=torch.float64, device="cuda")
            xs = torch.cat([head, leaves["x"][begin:begin + n]])
            z = leaves["bias"].expand(n, D)
            for k in range(W):
                z = z + leaves["w"][:, k] * xs[k:k + n]
            ys.append(act(z))
            finals.append(xs[n:])
            begin += n
        y = torch.cat(ys)
        if kind == "conv_forward":
            return {"y": y.detach(), "final": torch.stack(finals).detach()}
        dx, dw, db = torch.autograd.grad(y, [leaves["x"], leaves["w"], leaves["bias"]], f64["dy"])
        return {"dx": dx, "dw": dw, "db": db}

    G, N = case["groups"], case["states"]

    def wide(v):  # [m, G*N] -> [m, D, N]
        return v.reshape(-1, G, 1, N).expand(-1, G, D // G, N).reshape(-1, D, N)

    if kind == "scan_step":
        at = s["slots"].long()
        delta = torch.nn.functional.softplus(f64["dt"] + f64["dt_bias"], threshold=100.0)
        h = torch.exp(delta[..., None] * f64["A"]) * f64["state"][at]
        h = h + wide(f64["B"]) * (delta * f64["x"])[..., None]
        y = torch.matmul(h.reshape(r, G, D // G, N), f64["C"].reshape(r, G, N, 1)).reshape(r, D)
        y = y + f64["D"] * f64["x"]
        state = f64["state"]
        state[at] = h
        return {"y": y * f64["z"] * torch.sigmoid(f64["z"]) if case["gate"] else y, "state": state}

    # step by step; the gradients by differentiating through the steps
    train = kind == "scan_train"
    names = ["x", "dt", "dt_bias", "A", "B", "C", "D"] + (["z"] if case["gate"] else [])
    names += ["initial"] if case["initial"] else []
    leaves = {k: f64[k].clone().requires_grad_(train) for k in names}
    ys, finals, begin = [], [], 0
    with torch.set_grad_enabled(train):
        delta = torch.nn.functional.softplus(leaves["dt"] + leaves["dt_bias"], threshold=100.0)
        force = delta * leaves["x"]
        for i, n in enumerate(s["lens"]):
            h = leaves["initial"][i] if case["initial"] else torch.zeros(D, N, dtype=torch.float64, device="cuda")
            cut = [v[begin:begin + n].unbind(0) for v in (delta, force, leaves["B"], leaves["C"])]
            for d_t, f_t, b_t, c_t in zip(*cut):
                b_t = b_t.reshape(G, 1, N).expand(G, D // G, N).reshape(D, N)
                h = torch.exp(d_t[:, None] * leaves["A"]) * h + f_t[:, None] * b_t
                ys.append(torch.matmul(h.reshape(G, D // G, N), c_t.reshape(G, N, 1)).reshape(D))
            finals.append(h)
            begin += n
        y = torch.stack(ys) + leaves["D"] * leaves["x"]
        if case["gate"]:
            y = y * leaves["z"] * torch.sigmoid(leaves["z"])
    out = {"y": y.detach(), "final": torch.stack(finals).detach()}
    if train:
        called = {"initial": "dinitial", "dt": "ddt", "dt_bias": "ddt_bias"}
        grads = torch.autograd.grad(y, [leaves[k] for k in names], f64["dy"])
        out.update({called.get(k, "d" + k): v for k, v in zip(names, grads)})
    return out
