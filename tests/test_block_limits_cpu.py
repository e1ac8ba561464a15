"""Largest sizes of a linear layer, on the host: every size that is accepted has a plan whose
launch holds fewer than 2^32 threads along its first axis."""
import re

import pytest

import convolution_layer_amd as cm

LARGE = [(1, 1 << 30), (1, (1 << 30) + 7), (8, (1 << 30) + 77), (128, (1 << 31) - 128), (129, (1 << 30) - 128),
         (1024, (1 << 27) - 128)]


@pytest.mark.parametrize("dtype", [cm.BF16, cm.F32])
@pytest.mark.parametrize("N,M", LARGE)
def test_grids_of_accepted_sizes(N, M, dtype):
    for K in (1, 100):
        for op, (i, j) in enumerate([(M, N), (M, K), (N, K)]):
            name = cm.linear_plan_name(cm.make_linear_desc(M, K, N, dtype=dtype), op)
            side = int(re.search(r"(\d+)x", name).group(1))
            assert -(-i // side) * -(-j // side) * (512 if side == 256 else 256) < 1 << 32, name


@pytest.mark.parametrize("M,K,N", [((1 << 31) - 1, 1, 1), ((1 << 31) - 1, 1, 128), (1 << 30, 1, 129), (1 << 30, 129, 1),
                                   (1, 1 << 20, 1 << 20)])
def test_more_tiles_than_a_launch_holds_are_refused(M, K, N):
    for op in range(3):
        with pytest.raises(cm.ConvmiError) as e:
            cm.linear_workspace_size(cm.make_linear_desc(M, K, N), op)
        assert e.value.status == cm.ERR_UNSUPPORTED
