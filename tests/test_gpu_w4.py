"""Products with 4-bit weights and group scales against the definition in 64 bits."""
import math

import pytest
import torch

import warp_specialized_tensor_gb300 as wst

pytestmark = pytest.mark.gpu


def rows(x):
    """The same values in rows that begin on 16 bytes, the rest of each row filled with a value that shows."""
    per = 16 // x.element_size()
    n = -(-x.shape[-1] // per) * per
    out = torch.full((*x.shape[:-1], n), 255 if x.dtype is torch.uint8 else float("nan"), dtype=x.dtype, device=x.device)[..., :x.shape[-1]]
    return out.copy_(x)


def inputs(seed, M, N, K, group, lead=()):
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = rows(torch.randn(M, K, generator=g, device="cuda").bfloat16())
    W = rows(torch.randint(0, 256, (*lead, N, -(-K // 2)), generator=g, device="cuda", dtype=torch.uint8))
    S = rows((torch.randn(*lead, -(-K // group), N, generator=g, device="cuda") * 0.05).bfloat16())
    bias = torch.randn(*lead, N, generator=g, device="cuda").bfloat16()
    return A, W, S, bias


def weights(W, S, K, group):
    q = torch.stack((W & 15, W >> 4), dim=-1).flatten(-2)[..., :K].double() - 8
    return q * S.double().transpose(-1, -2).repeat_interleave(group, dim=-1)[..., :K]


def want(A, W, S, K, group, bias=None, epi="none"):
    """The result in 64 bits and the bound of fp32's part of the error: an mma adds 16 products to its accumulator and
    is off by at most 2^-22 of the sum of their sizes, a group takes group/16 of them; a group's sum is scaled and
    added with half a last bit each, and so are at most 160 pieces of a tile.  The activations' slopes stay below 1.13
    and their own evaluation below 2^-20."""
    w = weights(W, S, K, group)
    y, size = A.double() @ w.T, A.double().abs() @ w.abs().T
    tol = size * (group / 16 * 2.0 ** -22 + (math.ceil(K / group) + 160) * 2.0 ** -24)
    if epi != "none":
        y = y + bias.double()
        tol = tol + y.abs() * 2.0 ** -24
    if epi == "bias_silu":
        y = y * torch.sigmoid(y)
    if epi == "bias_gelu":
        y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
    return y, 1.13 * tol + y.abs() * 2.0 ** -20 + 2.0 ** -126


def check(got, y, tol):
    half = 2.0 ** -8 if got.dtype is torch.bfloat16 else 2.0 ** -24
    err = (got.double() - y).abs()
    assert bool((err <= tol + half * (y.abs() + tol)).all()), float((err - tol - half * y.abs()).max())


CASES = [  # M, N, K, group, epi, type, whole workspace
    (1, 4096, 4096, 128, "none", torch.bfloat16, True),
    (1, 128, 128, 128, "none", torch.float32, True),
    (1, 1, 1, 32, "none", torch.float32, True),
    (2, 7, 31, 32, "bias", torch.bfloat16, True),
    (3, 130, 257, 64, "bias_silu", torch.float32, False),
    (8, 64, 8192, 128, "bias_gelu", torch.bfloat16, True),
    (9, 1000, 1000, 32, "none", torch.float32, True),
    (16, 2048, 640, 64, "bias", torch.bfloat16, True),
    (17, 513, 2744, 32, "bias_silu", torch.bfloat16, True),
    (32, 300, 4096, 128, "none", torch.float32, False),
    (61, 1531, 2744, 32, "bias", torch.float32, True),
    (64, 640, 384, 64, "none", torch.bfloat16, True),
    (65, 257, 1032, 128, "bias_gelu", torch.float32, True),
    (200, 384, 513, 64, "none", torch.bfloat16, True),
]


@pytest.mark.parametrize("M,N,K,group,epi,dtype,whole", CASES)
def test_dense(M, N, K, group, epi, dtype, whole):
    A, W, S, bias = inputs(M * 7 + N, M, N, K, group)
    C = rows(torch.full((M, N), 3.0, dtype=dtype, device="cuda"))
    ws = wst.gemm_w4_workspace() if whole else wst.workspace()
    wst.wst_gemm_w4(A, W, S, C, group=group, bias=bias, epi=epi, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    check(C, *want(A, W, S, K, group, bias, epi))


GROUPS = [  # rows of the groups, rows behind, N, K, group, type, whole workspace
    ([1, 0, 3, 0, 0, 2, 1], 0, 256, 512, 128, torch.bfloat16, True),
    ([0, 0, 5], 4, 100, 100, 32, torch.float32, True),
    ([0, 0, 0], 3, 64, 64, 64, torch.float32, True),
    ([40, 1, 9, 100, 7], 0, 384, 1000, 64, torch.bfloat16, True),
    ([2] * 70, 1, 136, 256, 128, torch.float32, False),
    ([1] * 600 + [0] * 50 + [3] * 7, 2, 32, 96, 32, torch.float32, True),
    ([129], 0, 130, 2050, 128, torch.bfloat16, True),
]


@pytest.mark.parametrize("sizes,behind,N,K,group,dtype,whole", GROUPS)
@pytest.mark.parametrize("epi", ["none", "bias_silu"])
def test_grouped(sizes, behind, N, K, group, dtype, whole, epi):
    G, M = len(sizes), sum(sizes) + behind
    A, W, S, bias = inputs(G * 5 + N, M, N, K, group, (G,))
    off = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
    C = rows(torch.full((M, N), 3.0, dtype=dtype, device="cuda"))
    ws = wst.gemm_w4_workspace() if whole else wst.workspace()
    wst.wst_grouped_gemm_w4(A, W, S, off, C, group=group, bias=bias, epi=epi, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    o = off.tolist()
    for e in range(G):
        if o[e + 1] > o[e]:
            check(C[o[e]:o[e + 1]], *want(A[o[e]:o[e + 1]], W[e], S[e], K, group, bias[e], epi))
    assert bool((C[o[-1]:] == 3.0).all())


def test_whole_numbers_are_exact_and_runs_are_alike():
    """Whole numbers and scales that are powers of two: every sum is exact, in any order; and random numbers give the
    same bits every time, on a workspace that another operation has used."""
    M, N, K = 5, 384, 2048
    g = torch.Generator(device="cuda").manual_seed(5)
    A = torch.randint(-8, 9, (M, K), generator=g, device="cuda").bfloat16()
    W = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    S = torch.pow(2.0, torch.randint(-2, 3, (K // 64, N), generator=g, device="cuda").float()).bfloat16()
    C = torch.empty(M, N, device="cuda")
    ws = torch.zeros(max(wst.wst_gemm_w4_workspace_size(), wst.wst_gemm_fp8_workspace_size()), dtype=torch.uint8, device="cuda")
    wst.wst_gemm_w4(A, W, S, C, group=64, workspace=ws)
    assert torch.equal(C.double(), A.double() @ weights(W, S, K, 64).T)
    A, W, S, _ = inputs(9, 12, 1111, 4096, 128)
    first = rows(torch.empty(12, 1111, device="cuda"))
    wst.wst_gemm_w4(A, W, S, first, workspace=ws)
    for _ in range(5):
        ws[256:].random_(0, 256)      # what other operations leave behind the header
        again = rows(torch.empty(12, 1111, device="cuda"))
        wst.wst_gemm_w4(A, W, S, again, workspace=ws)
        assert torch.equal(first, again)
    assert wst.wst_sync_status(ws) == 0


def test_neighbours_values_and_bad_offsets():
    """Infinities in another group's rows stay there; offsets that break the rule are clamped and reported."""
    N, K = 128, 256
    A, W, S, _ = inputs(3, 10, N, K, 128, (3,))
    A[4:7] = float("inf")
    off = torch.tensor([0, 4, 7, 10], dtype=torch.int32, device="cuda")
    C = torch.zeros(10, N, device="cuda")
    ws = wst.gemm_w4_workspace()
    wst.wst_grouped_gemm_w4(A, W, S, off, C, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    for e, (i, j) in enumerate(((0, 4), (7, 10))):
        check(C[i:j], *want(A[i:j], W[2 * e], S[2 * e], K, 128))
    for bad in ([0, 4, 2, 10], [0, 4, 7, 11], [1, 4, 7, 10], [0, -5, 7, 10]):
        wst.wst_grouped_gemm_w4(A, W, S, torch.tensor(bad, dtype=torch.int32, device="cuda"), C, workspace=ws)
        assert wst.wst_sync_status(ws) == wst.WST_ERR_BAD_OFFSETS
    wst.wst_grouped_gemm_w4(A, W, S, off, C, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
