"""The 64-bit definitions that the residual-block tests compare with, pinned on the CPU
against torch's float8 conversion and autograd."""
import pytest
import torch

from tests import block_reference as R


def test_e4m3_codes_match_torchs_conversion():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double()
    got = R.decode(codes.reshape(1, -1), torch.full((1, 8), 127))[0]
    assert torch.equal(torch.isnan(ref), torch.isnan(got))
    ok = ~torch.isnan(ref)
    assert torch.equal(ref[ok], got[ok])


def test_rounding_matches_torchs_conversion():
    g = torch.Generator().manual_seed(1)
    v = torch.randn(64, 64, generator=g) * torch.exp2(torch.randint(-12, 8, (64, 64), generator=g).float())
    v = v.clamp(-448, 448)
    e = torch.full((64, 2), 127)
    assert torch.equal(R.encode(v, e).to(torch.uint8), v.to(torch.float8_e4m3fn).view(torch.uint8).to(torch.uint8))
    mid = (R.E4M3[1:] + R.E4M3[:-1]) / 2  # ties
    mid = torch.nn.functional.pad(mid, (0, 2)).reshape(1, -1).float()
    assert torch.equal(R.encode(mid, torch.full((1, 4), 127)).to(torch.uint8),
                       mid.to(torch.float8_e4m3fn).view(torch.uint8))


def test_scale_is_the_smallest_that_holds_the_block():
    g = torch.Generator().manual_seed(2)
    v = torch.randn(50, 96, generator=g).double() * torch.exp2(torch.randint(-100, 100, (50, 1), generator=g).double())
    v[0] = 448.0
    v[1] = 448.0000001
    v[2] = 0.0
    e = R.scale_bytes(v)
    top = R.blocks(v.abs()).amax(-1)
    assert bool((top <= 448 * 2.0 ** (e - 127).double()).all())
    assert bool(((top > 448 * 2.0 ** (e - 128).double()) | (e == 1)).all())
    assert int(e[0, 0]) == 127 and int(e[1, 0]) == 128 and int(e[2, 0]) == 1


@pytest.mark.parametrize("kind", range(5))
def test_slopes_against_autograd(kind):
    a = torch.linspace(-6, 6, 401, dtype=torch.float64).requires_grad_()
    a.data[200] = 0.01
    (gr,) = torch.autograd.grad(R.act(a, kind).sum(), a)
    assert float((gr - R.slope(a.detach(), kind)).abs().max()) < 1e-12
    if kind != 4:
        y = R.act(a.detach(), kind)
        assert float((R.slope_of_output(y, kind) - gr).abs().max()) < 1e-12


def test_rms_backward_against_autograd():
    g = torch.Generator().manual_seed(3)
    x, res = (torch.randn(5, 37, generator=g, dtype=torch.float64).requires_grad_() for _ in range(2))
    gamma = torch.randn(37, generator=g, dtype=torch.float64).requires_grad_()
    dy, dh = (torch.randn(5, 37, generator=g, dtype=torch.float64) for _ in range(2))
    h, inv, y = R.rms_forward(x, res, gamma, 1e-5)
    gx, gr, gg = torch.autograd.grad((y * dy).sum() + (h * dh).sum(), (x, res, gamma))
    dx, dgamma = R.rms_backward(h.detach(), gamma.detach(), inv.detach(), dy, dh)
    assert float((gx - dx).abs().max()) < 1e-12 and float((gr - dx).abs().max()) < 1e-12
    assert float((gg - dgamma).abs().max()) < 1e-12
