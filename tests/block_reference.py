"""Plain 64-bit definitions of the residual-block operators (RMS norm, linear layer, MX8),
element formulas on CPU tensors; test infrastructure only, no library code.

Roundings counted by the tolerances (half a step, relative): bf16 2^-8, fp32 2^-24, e4m3
2^-4 (or 2^-10 of the block's scale below its smallest normal)."""
import math

import torch

BLOCK = 32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# fp32 evaluations of the activations and their slopes with the hardware exponential and
# reciprocal (1 ulp each): |t error| <= 6 * 2^-24, so |1 - t^2| is off by <= 13 * 2^-24; the
# GELU slope multiplies that by at most 0.5 |a| du/da <= 6.3 (beyond |a| = 4.4 t rounds to
# 1 and the term is 0), 82 * 2^-24, plus the argument's own rounding: within 2^-16.
ACT_ABS = 2.0 ** -16


def act(a, kind):
    if kind == 1:
        return torch.where(a > 0, a, torch.zeros_like(a))
    if kind == 2:
        return torch.tanh(a)
    if kind == 3:
        return 1 / (1 + torch.exp(-a))
    if kind == 4:
        return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    return a.clone()


def slope(a, kind):
    if kind == 1:
        return (a > 0).double()
    if kind == 2:
        return 1 - torch.tanh(a) ** 2
    if kind == 3:
        s = 1 / (1 + torch.exp(-a))
        return s * (1 - s)
    if kind == 4:
        t = torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))
        return 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * a ** 2)
    return torch.ones_like(a)


def slope_of_output(y, kind):
    return {0: torch.ones_like(y), 1: (y > 0).double(), 2: 1 - y * y, 3: y * (1 - y)}[kind]


def blocks(v):
    """[rows, cols] -> [rows, nb, 32], zeros behind the row."""
    rows, cols = v.shape
    return torch.nn.functional.pad(v, (0, -cols % BLOCK)).reshape(rows, -1, BLOCK)


def scale_bytes(v):
    """Smallest e >= 1 with largest finite magnitude <= 448 * 2^(e-127), per block."""
    b = blocks(v.double().abs())
    top = torch.where(torch.isfinite(b), b, torch.zeros_like(b)).amax(-1)
    e = torch.ones_like(top, dtype=torch.int64)
    for k in range(2, 254):  # count the powers that are too small
        e += (top > 448.0 * 2.0 ** (k - 1 - 127)).long()
    return e


E4M3 = torch.tensor([math.ldexp(m, -9) if ex == 0 else math.ldexp(8 + m, ex - 10)
                     for ex in range(16) for m in range(8)][:127], dtype=torch.float64)


def encode(v, e):
    """Codes of v under scale bytes e: the nearest e4m3 magnitude, ties to the even code; at
    most 240 under 2^120 (byte 247), where 256 would be beyond fp32."""
    u = torch.ldexp(blocks(v.double()), (127 - e).unsqueeze(-1))
    mag = u.abs()
    mag = torch.where((e.unsqueeze(-1) == 247) & torch.isfinite(mag), mag.clamp(max=240.0), mag)
    hi = torch.searchsorted(E4M3, torch.nan_to_num(mag, nan=0.0, posinf=0.0).contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = mag - E4M3[lo], E4M3[hi] - mag
    code = torch.where(dl < dh, lo, torch.where(dl > dh, hi, torch.where(lo % 2 == 0, lo, hi)))
    code = torch.where(torch.isfinite(u), code, torch.full_like(code, 127))
    neg = torch.signbit(u) & torch.isfinite(u)
    return (code + 128 * neg.long()).reshape(v.shape[0], -1)[:, : v.shape[1]]


def decode(codes, e):
    c = codes.long()
    mag = torch.cat([E4M3, torch.tensor([float("nan")], dtype=torch.float64)])[c & 127]
    sign = 1.0 - 2.0 * (c >> 7).double()
    s = torch.ldexp(torch.ones((), dtype=torch.float64), e.long() - 127)
    s = torch.where(e.long() == 255, torch.full_like(s, float("nan")), s)
    return sign * mag * s.repeat_interleave(BLOCK, -1)[:, : codes.shape[1]]


def keep(v):
    """(codes, scale bytes, values) of v."""
    e = scale_bytes(v)
    c = encode(v, e)
    return c, e, decode(c, e)


def kept_bound(ref, rel):
    """How far a kept value may be from ref when what was packed is within `rel` of ref:
    half an e4m3 step under the largest scale that its block can then have, and that."""
    e = scale_bytes(ref * (1 + rel))
    s = torch.ldexp(torch.ones((), dtype=torch.float64), e - 127).repeat_interleave(BLOCK, -1)[:, : ref.shape[1]]
    return torch.maximum(2.0 ** -4 * ref.abs() * (1 + rel), 2.0 ** -10 * s) + rel * ref.abs()


def rms_forward(x, res, gamma, eps):
    h = x.double() + (res.double() if res is not None else 0.0)
    inv = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h, inv, gamma.double() * (h * inv[:, None])


def rms_backward(h, gamma, inv, dy, dh):
    hhat, g = h.double() * inv.double()[:, None], gamma.double() * dy.double()
    dx = inv.double()[:, None] * (g - hhat * (g * hhat).mean(-1, keepdim=True))
    return dx + (dh.double() if dh is not None else 0.0), (dy.double() * hhat).sum(0)


def dev(t, dtype):
    return t.to(dtype).cuda().contiguous()


def host(t):
    return t.detach().double().cpu()


def within(got, ref, bound, what):
    """Elementwise |got - ref| <= bound, both finite in the same places."""
    got = host(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    ok = torch.isnan(ref) | ((got - ref).abs() <= bound) | (got == ref)
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        b = bound.expand_as(ref).flatten()[i]
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} beyond, first at {i}: got "
                             f"{got.flatten()[i]:.9g} ref {ref.flatten()[i]:.9g} bound {b:.3g}")


def same(a, b, what):
    assert torch.equal(a.view(torch.uint8) if a.dtype.itemsize == 1 else a, b.view(torch.uint8)
                       if b.dtype.itemsize == 1 else b), f"{what}: not equal bit for bit"
