"""Products with 4-bit weights whose CTAs go round their stages many times, the weights out of L2."""
import pytest
import torch

import warp_specialized_tensor_gb300 as wst
from test_gpu_w4 import check, inputs, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,group", [(5, 1000, 65536, 128), (16, 6000, 16384, 64), (29, 1500, 25600, 32)])
def test_stages_used_many_times(M, N, K, group):
    A, W, S, _ = inputs(M + N, M, N, K, group)
    C = torch.empty(M, N, device="cuda")
    ws = wst.gemm_w4_workspace()
    y, tol = want(A, W, S, K, group)
    first = None
    for _ in range(4):
        torch.randn(1 << 27, device="cuda")
        C.fill_(3.0)
        wst.wst_gemm_w4(A, W, S, C, group=group, workspace=ws)
        assert wst.wst_sync_status(ws) == 0
        check(C, y, tol)
        first = C.clone() if first is None else first
        assert torch.equal(C, first)
