"""The 8-bit operators where a rare value, size or division of the work decides: against the plain
64-bit references of q8_ref, with its bounds."""

import math

import pytest
import torch

import q8_ref as R
import qwen2_decode_step_b200 as q2
from test_gpu_q8 import DT, both, empty_cache, filled_cache, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield
    torch.cuda.synchronize()
    q2.q2_check_device_error()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("M,N,K", [(3, 130, 8960), (3, 131, 384), (20, 5, 640), (70, 130, 4096), (129, 333, 2048),
                                   (66, 201, 384)])
def test_linear_split_over_a_cluster_with_remainder_tiles(dt, M, N, K):
    """Lanes of one warp that have an output next to lanes that have none, between two barriers of
    the cluster; many launches behind one another."""
    xq, xs = R.quantise(randn(300, M, K), 1)
    wq, ws = R.quantise(0.02 * randn(301, N, K), 128)
    bias = randn(302, N).to(DT[dt])
    d = both(xq, xs, wq, ws, bias)
    outs = torch.full((40, M, N), 9.0, dtype=DT[dt], device="cuda")
    for o in outs:
        q2.q2_linear_q8(o, *d)
    ref, bound = R.linear(xq, xs, wq, ws, bias, DT[dt])
    R.within(outs[0], ref, bound, "linear")
    assert torch.equal(outs, outs[:1].expand_as(outs))
