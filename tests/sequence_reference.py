"""Plain 64-bit definitions of the operators along sequences (causal convolution, selective scan) on
CPU tensors, sequence by sequence and step by step; test infrastructure only, no library code."""
import torch

from tests import block_reference as R

U = 2.0 ** -24
SILU = 5


def act(a, kind):
    return a * torch.sigmoid(a) if kind == SILU else R.act(a, kind)


def slope(a, kind):
    if kind != SILU:
        return R.slope(a, kind)
    s = torch.sigmoid(a)
    return s + a * s * torch.sigmoid(-a)


def act_error(a, kind):
    """Bound on the fp32 evaluation of act and act' at a: for SiLU the exponential's argument is rounded
    to |a| u, the rest takes at most ten roundings; the others as block_reference counts them."""
    if kind == SILU:
        return (a.abs() + 10) * U * (1 + a.abs() * torch.sigmoid(-a.abs()))
    return torch.full_like(a, 0.0 if kind in (0, 1) else R.ACT_ABS)


def bounds(starts, rows, batch):
    """(first row, row behind the last) of every sequence."""
    if starts is None:
        n = rows // batch if batch else 0
        return [(i * n, (i + 1) * n) for i in range(batch)]
    s = [min(max(int(v), 0), rows) for v in starts]
    return [(s[i], max(s[i], s[i + 1])) for i in range(batch)]


# ------------------------------------------------------------------ causal convolution
def conv_z(x, w, bias, seqs, initial):
    """z, and sum_k |w_k x| + |bias| for the rounding bounds; rows of no sequence are 0."""
    D, W = w.shape
    z, mag = (torch.zeros(x.shape[0], D, dtype=torch.float64) for _ in range(2))
    ext = []
    for i, (a, e) in enumerate(seqs):
        head = initial[i].double() if initial is not None else torch.zeros(W - 1, D, dtype=torch.float64)
        xs = torch.cat([head, x[a:e].double()])
        ext.append(xs)
        for k in range(W):
            z[a:e] += w[:, k].double() * xs[k:k + e - a]
            mag[a:e] += (w[:, k].double() * xs[k:k + e - a]).abs()
        if bias is not None:
            z[a:e] += bias.double()
            mag[a:e] += bias.double().abs()
    return z, mag, ext


def conv_backward(x, w, bias, seqs, initial, kind, dy, dfinal):
    """dx, d_initial, dw, db and bounds on their fp32 evaluation."""
    D, W = w.shape
    z, mag, ext = conv_z(x, w, bias, seqs, initial)
    wd = w.double()
    o = {k: torch.zeros(x.shape[0], D, dtype=torch.float64) for k in ("dx", "dx_err")}
    o.update({k: torch.zeros(len(seqs), W - 1, D, dtype=torch.float64) for k in ("di", "di_err")})
    o.update({k: torch.zeros(D, W, dtype=torch.float64) for k in ("dw", "dw_err")})
    o.update({k: torch.zeros(D, dtype=torch.float64) for k in ("db", "db_err")})
    for i, (a, e) in enumerate(seqs):
        n = e - a
        s = slope(z[a:e], kind)
        g = dy[a:e].double()
        dz = s * g
        err = g.abs() * (act_error(z[a:e], kind) + (0 if kind in (0, 1) else 1) * (W + 1) * U * mag[a:e]) + 2 * U * dz.abs()
        d_ext, d_err = (torch.zeros(n + W - 1, D, dtype=torch.float64) for _ in range(2))
        for k in range(W):
            d_ext[k:k + n] += wd[:, k] * dz
            d_err[k:k + n] += wd[:, k].abs() * (err + (W + 2) * U * dz.abs())
            o["dw"][:, k] += (dz * ext[i][k:k + n]).sum(0)
            # at most 256 rows and 256 runs of rows are added in fp32
            o["dw_err"][:, k] += (ext[i][k:k + n].abs() * (err + 2.0 ** -15 * dz.abs())).sum(0)
        o["db"] += dz.sum(0)
        o["db_err"] += (err + 2.0 ** -15 * dz.abs()).sum(0)
        if dfinal is not None:
            d_ext[n:] += dfinal[i].double()
            d_err[n:] += U * dfinal[i].double().abs()
        d_err += U * d_ext.abs()
        o["di"][i], o["dx"][a:e] = d_ext[:W - 1], d_ext[W - 1:]
        o["di_err"][i], o["dx_err"][a:e] = d_err[:W - 1], d_err[W - 1:]
    return o


# ------------------------------------------------------------------ selective scan
class V:
    """A value with a bound on how far an fp32 evaluation may be from it: every operation passes on
    its operands' bounds and adds half a step of its own result."""

    def __init__(self, v, e=None):
        self.v = v.double() if isinstance(v, torch.Tensor) else torch.tensor(float(v), dtype=torch.float64)
        self.e = torch.zeros_like(self.v) if e is None else e

    def __getitem__(self, i):
        return V(self.v[i], self.e[i])

    def __add__(self, o):
        v = self.v + o.v
        return V(v, self.e + o.e + U * v.abs())

    def __mul__(self, o):
        v = self.v * o.v
        return V(v, self.v.abs() * o.e + o.v.abs() * self.e + self.e * o.e + U * v.abs())

    def map(self, f, slope, own):
        """f, whose derivative is at most `slope` around the value, evaluated to within `own` of itself."""
        v = f(self.v)
        return V(v, slope * self.e + own)

    def exp(self):  # the hardware's 2^x is off by at most one step (2 u)
        v = self.v.exp()
        return V(v, v * (torch.expm1(self.e) + 2 * U))

    def sum(self, dim, adds):
        """Sum in any order in which a term passes at most `adds` additions."""
        v = self.v.sum(dim)
        return V(v, self.e.sum(dim) + adds * U * (self.v.abs() + self.e).sum(dim))

    def view(self, *s):
        return V(self.v.reshape(*s), self.e.reshape(*s).clone())


def silu(z):
    s = torch.sigmoid(z.v)
    return z.map(lambda a: a * torch.sigmoid(a), 1.1, (z.v.abs() + 10) * U * (z.v * s).abs())


def silu_slope(z):
    return z.map(lambda a: slope(a, SILU), 0.6, act_error(z.v, SILU))


def softplus(v):
    """max(v, 0) + log(1 + exp(-|v|)): the exponential's argument is rounded to |v| u, the polynomial is off by
    3 u, four roundings."""
    f = lambda a: a.clamp(min=0) + torch.log1p(torch.exp(-a.abs()))  # noqa: E731
    return v.map(f, torch.sigmoid(v.v), (v.v.abs() + 8) * U * f(v.v))


CHUNK = 128  # the tests' sequences are cut at most this long, or not at all


def scan(t, seqs, groups, plus, initial=None, dy=None, dfinal=None):
    """Outputs of the scan of tensors t (x, dt, dt_bias, A, B, C, D, z; the last two and dt_bias may be None), with
    dy its gradients too: a dictionary of V; rows of no sequence are 0."""
    rows, ch = t["x"].shape
    N, per = t["A"].shape[1], ch // groups
    g = {k: None if v is None else V(v) for k, v in t.items()}
    v = g["dt"] if g["dt_bias"] is None else g["dt"] + g["dt_bias"]
    delta = softplus(v) if plus else v
    du = delta * g["x"]
    gate = silu(g["z"]) if g["z"] is not None else None
    wide = lambda b: V(b.v.reshape(rows, groups, 1, N).expand(rows, groups, per, N).reshape(rows, ch, N))  # noqa: E731
    B, Cm = wide(g["B"]), wide(g["C"])
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    o = {}

    def put(name, at, val, *shape):
        if name not in o:
            o[name] = V(zero(*shape))
        o[name].v[at], o[name].e[at] = val.v, val.e

    def add(name, val):
        o[name] = val if name not in o else o[name] + val

    dyp = None if dy is None else V(dy) * gate if gate is not None else V(dy)
    for name in ("dA", "dD", "ddt_bias") if dy is not None else ():
        o[name] = V(zero(ch, N) if name == "dA" else zero(ch))
    for i, (a, e) in enumerate(seqs):
        h = V(initial[i]) if initial is not None else V(zero(ch, N))
        hs, As = [h], []
        for r in range(a, e):
            x = delta[r].view(ch, 1) * g["A"]
            # scaled by log2 e (two roundings); a chunk's sum of delta takes up to CHUNK additions
            x = V(x.v, x.e + (2 + CHUNK) * U * x.v.abs())
            As.append(x.exp())
            h = As[-1] * h + du[r].view(ch, 1) * B[r]
            h = V(h.v, h.e + 2 * U * h.v.abs())  # a chunk's state from zero is added to what enters it
            hs.append(h)
        put("final", i, h, len(seqs), ch, N)
        ys = []
        for r in range(a, e):
            y = (Cm[r] * hs[r - a + 1]).sum(-1, N)
            if g["D"] is not None:
                y = y + g["D"] * g["x"][r]
            ys.append(y)
            put("y", r, y * gate[r] if gate is not None else y, rows, ch)
        if dy is None:
            continue
        G = V(dfinal[i]) if dfinal is not None else V(zero(ch, N))
        for r in range(e - 1, a - 1, -1):
            j = r - a
            gr = Cm[r] * dyp[r].view(ch, 1) + G
            s = (B[r] * gr).sum(-1, N)
            G = As[j] * gr
            G = V(G.v, G.e + 2 * U * G.v.abs())
            u = G * hs[j]
            w = (g["A"] * u).sum(-1, N + 2)
            dx = delta[r] * s
            if g["D"] is not None:
                dx = dx + g["D"] * dyp[r]
            put("dx", r, dx, rows, ch)
            dd = g["x"][r] * s + w
            ddt = dd * v[r].map(torch.sigmoid, 0.25, 8 * U * torch.sigmoid(v.v[r]) * (1 + v.v[r].abs())) if plus else dd
            put("ddt", r, ddt, rows, ch)
            if gate is not None:
                put("dz", r, V(dy[r]) * ys[j] * silu_slope(g["z"][r]), rows, ch)
            # over the channels of a group: 3 in a wave, 8 waves, one for every 64 channels
            adds = 11 + per // 64 + 1
            put("dB", r, (du[r].view(ch, 1) * gr).view(groups, per, N).sum(1, adds).view(-1), rows, groups * N)
            put("dC", r, (dyp[r].view(ch, 1) * hs[j + 1]).view(groups, per, N).sum(1, adds).view(-1), rows, groups * N)
            # `add` counts one rounding for every row, in any order
            add("dA", delta[r].view(ch, 1) * u)
            add("dD", dyp[r] * g["x"][r])
            add("ddt_bias", ddt)
        put("dinitial", i, G, len(seqs), ch, N)
    if dy is not None:
        for name in ("dx", "ddt", "dz"):
            o.setdefault(name, V(zero(rows, ch)))
        for name in ("dB", "dC"):
            o.setdefault(name, V(zero(rows, groups * N)))
        o.setdefault("dinitial", V(zero(len(seqs), ch, N)))
    o.setdefault("y", V(zero(rows, ch)))
    return o
