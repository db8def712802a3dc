"""Every form of the products with 4-bit weights (tiles of 8, 16 and 32 rows, each group size), and tiles that outnumber
the SMs and are cut all the same, so that a CTA's share spans tiles and both its ends are pieces."""
import pytest
import torch

import warp_specialized_tensor_gb300 as wst
from test_gpu_w4 import check, inputs, rows, want

pytestmark = pytest.mark.gpu

DENSE = [  # M, N, K, group, epi, type, whole workspace, rows of a tile
    (16, 8192, 8192, 128, "bias_silu", torch.bfloat16, True, 16),
    (15, 8190, 8191, 32, "none", torch.float32, True, 16),
    (9, 4500, 8100, 64, "bias", torch.bfloat16, True, 16),
    (29, 4090, 8192, 32, "none", torch.bfloat16, False, 16),
    (64, 4096, 8192, 128, "none", torch.bfloat16, True, 32),
    (61, 4001, 8190, 32, "bias", torch.float32, True, 32),
    (33, 4100, 8130, 64, "bias_gelu", torch.bfloat16, True, 32),
    (97, 4097, 8191, 128, "none", torch.float32, False, 32),
    (5, 20700, 1100, 32, "none", torch.bfloat16, True, 8),
    (8, 20601, 2100, 64, "bias", torch.float32, True, 8),
    (3, 20700, 2101, 128, "none", torch.float32, True, 8),
    (16, 20700, 2100, 128, "none", torch.float32, True, 16),
    (13, 20601, 1900, 64, "bias_silu", torch.bfloat16, True, 16),
    (32, 20700, 2100, 32, "none", torch.bfloat16, True, 32),
    (61, 20601, 1100, 64, "bias", torch.float32, True, 32),
]
GROUPS = [  # rows of the groups, rows behind, N, K, group, type, whole workspace, rows of a tile
    ([1] * 40 + [0] * 20 + [6] * 4, 3, 1500, 2000, 128, torch.bfloat16, True, 8),
    ([0, 17, 3, 0, 1, 9, 8, 16, 0, 2] * 2, 0, 2040, 2000, 64, torch.float32, True, 16),
    ([5, 0, 7, 1, 9, 16, 3, 8, 4, 7] * 2, 1, 2048, 1900, 32, torch.bfloat16, True, 16),
    ([40, 0, 1, 9, 32, 33, 3, 0, 8, 7] * 2 + [5], 2, 2040, 2001, 128, torch.bfloat16, True, 32),
    ([64, 5, 0, 31] * 3, 0, 2048, 2100, 32, torch.float32, False, 32),
]


@pytest.mark.parametrize("M,N,K,group,epi,dtype,whole,tile", DENSE)
def test_dense(M, N, K, group, epi, dtype, whole, tile):
    assert wst.wst_gemm_w4_tile_rows(M, N, K) == tile
    A, W, S, bias = inputs(M * 7 + N, M, N, K, group)
    C = rows(torch.full((M, N), 3.0, dtype=dtype, device="cuda"))
    ws = wst.gemm_w4_workspace() if whole else wst.workspace()
    y, tol = want(A, W, S, K, group, bias, epi)
    for _ in range(2):  # (the second on a workspace that has been used)
        wst.wst_gemm_w4(A, W, S, C, group=group, bias=bias, epi=epi, workspace=ws)
        assert wst.wst_sync_status(ws) == 0
        check(C, y, tol)


@pytest.mark.parametrize("sizes,behind,N,K,group,dtype,whole,tile", GROUPS)
def test_grouped(sizes, behind, N, K, group, dtype, whole, tile):
    G, M = len(sizes), sum(sizes) + behind
    assert wst.wst_gemm_w4_tile_rows(M, N, K, groups=G) == tile
    A, W, S, bias = inputs(G * 5 + N, M, N, K, group, (G,))
    off = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
    C = rows(torch.full((M, N), 3.0, dtype=dtype, device="cuda"))
    ws = wst.gemm_w4_workspace() if whole else wst.workspace()
    for _ in range(2):
        wst.wst_grouped_gemm_w4(A, W, S, off, C, group=group, bias=bias, epi="bias", workspace=ws)
        assert wst.wst_sync_status(ws) == 0
    o = off.tolist()
    for e in range(G):
        if o[e + 1] > o[e]:
            check(C[o[e]:o[e + 1]], *want(A[o[e]:o[e + 1]], W[e], S[e], K, group, bias[e], "bias"))
    assert bool((C[o[-1]:] == 3.0).all())


@pytest.mark.parametrize("sizes,N,K,group", [([3, 0, 9, 1], 260, 515, 64), ([20, 33], 1500, 2000, 128)])
def test_groups_that_share_weights(sizes, N, K, group):
    """One matrix for all groups, a stride of 0."""
    G, M = len(sizes), sum(sizes)
    A, W, S, _ = inputs(M + N, M, N, K, group)
    off = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
    C = rows(torch.full((M, N), 3.0, device="cuda"))
    ws = wst.gemm_w4_workspace()
    wst.wst_grouped_gemm_w4(A, W[None].expand(G, *W.shape), S[None].expand(G, *S.shape), off, C, group=group, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    check(C, *want(A, W, S, K, group))
