"""GELU's derivative where |z| is so large that z (1 + 3c z^2) overflows fp32: it is 1 or 0 there."""
import pytest
import torch

from tests.test_gpu_mx8 import pack

pytestmark = pytest.mark.gpu

BIG = [1e11, 1e13, 1e14, 1e19, 1e20, 3e37]


@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_slope_of_large_values(ty, mx8):
    import convolution_layer_amd as cm
    t, dt = (torch.bfloat16, cm.BF16) if ty == "bf16" else (torch.float32, cm.F32)
    z = torch.zeros(len(BIG) + 2, 32, dtype=t)  # a block per magnitude
    for i, v in enumerate(BIG):
        z[i] = v
        z[i, 1::2] = -v
    z[len(BIG)] = float("nan")
    if not mx8:  # 8-bit blocks hold no infinity
        z[len(BIG) + 1] = float("inf")
        z[len(BIG) + 1, 1::2] = -float("inf")
    M, N = z.shape
    dy = torch.arange(1, M * N + 1, dtype=torch.float32).reshape(M, N).remainder(100).to(t).cuda()
    dz = torch.empty(M, N, dtype=t, device="cuda")
    d = cm.make_linear_desc(M, 8, N, activation=cm.ACT_GELU, dtype=dt, z_mx8=mx8)
    keep = pack(z.cuda()) if mx8 else (z.cuda(), None)
    cm.linear_activation_backward(d, keep[0], dy, dz, z_scales=keep[1])
    ref = torch.where(z > 0, dy.cpu(), torch.zeros_like(z))
    if mx8:
        ref[-1] = dy[-1].cpu() * 0.5  # z = 0
    got = dz.cpu()
    assert bool(torch.isnan(got[len(BIG)]).all())
    keep_rows = [i for i in range(M) if i != len(BIG)]
    assert torch.equal(got[keep_rows].float(), ref[keep_rows].float())
