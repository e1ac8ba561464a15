"""A linear layer with more rows than 64 x 64 tiles can cover in one launch."""
import pytest
import torch

from tests.test_gpu_linear import ints

pytestmark = pytest.mark.gpu


def test_a_billion_rows():
    """2^30 + 7 rows, zero but for the last few; one output feature, so dz is padded as well."""
    import convolution_layer_amd as cm
    M, K, N = (1 << 30) + 7, 8, 1
    xi, wi, zi = ints(5, K, 7), ints(N, K, 8), ints(5, N, 9)
    d = cm.make_linear_desc(M, K, N, dtype=cm.BF16)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    dz = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    x[-5:], dz[-5:] = xi.bfloat16(), zi.bfloat16()
    w, y = wi.bfloat16(), torch.full((M, N), 4.0, dtype=torch.bfloat16, device="cuda")
    cm.linear_forward(d, x, w, None, None, None, y, cm.linear_workspace(d, cm.LINEAR_FORWARD))
    assert torch.equal(y[-5:].double(), (xi @ wi.T).bfloat16().double()) and int((y[:-5] != 0).sum()) == 0
    dw, db = torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    cm.linear_backward_weight(d, x, dz, dw, db, 0, cm.linear_workspace(d, cm.LINEAR_BACKWARD_WEIGHT))
    assert torch.equal(dw.double(), zi.T @ xi) and torch.equal(db.double(), zi.sum(0))
    x.fill_(4.0)
    cm.linear_backward_data(d, dz, w, x, cm.linear_workspace(d, cm.LINEAR_BACKWARD_DATA))
    assert torch.equal(x[-5:].double(), (zi @ wi).bfloat16().double()) and bool((x[:-5].amax(1) == 0).all())
    assert bool((x[:-5].amin(1) == 0).all())
