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
