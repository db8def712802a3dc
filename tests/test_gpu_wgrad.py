"""GPU: the grouped GEMM's weight gradient against the product in 64 bits."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from test_gpu_fp8 import rows16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wst():
    import warp_specialized_tensor_gb300 as w
    w.load_library()
    return w


def run(wst, dC, A, off, dtype, start=None):
    G, N, K = len(off) - 1, dC.shape[1], A.shape[1]
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((G, N, (-(-K // per) + 1) * per), float("nan"), dtype=dtype, device="cuda")
    out = buf[..., :K]
    if start is not None:
        out.copy_(start)
    ws = wst.workspace()
    wst.wst_grouped_gemm_wgrad_bf16(rows16(dC), rows16(A), torch.from_numpy(np.asarray(off)).int().cuda(), out,
                                    accumulate=start is not None, workspace=ws)
    status = wst.wst_sync_status(ws)
    assert torch.isnan(buf[..., K:].float()).all()
    return out, status


def check(wst, sizes, N, K, dtype, behind=0, start=False, poison=True):
    off = np.concatenate([[0], np.cumsum(sizes)])
    M = int(off[-1]) + behind
    g = torch.Generator().manual_seed(N + K + M)
    dC, A = torch.randn(M, N, generator=g).bfloat16(), torch.randn(M, K, generator=g).bfloat16()
    if behind and poison:                      # rows of no group, whatever they hold
        dC[off[-1]:], A[off[-1]:] = torch.nan, torch.inf
    before = torch.randn(len(sizes), N, K, generator=g).to(dtype) if start else None
    out, status = run(wst, dC, A, off, dtype, before)
    assert status == 0
    d, a = ref.f64(dC), ref.f64(A)
    for i in range(len(sizes)):
        r = slice(off[i], off[i + 1])
        want, size = d[r].T @ a[r], abs(d[r]).T @ abs(a[r])
        # one fp32 rounding (cut off: 2u) per token; the sum with what was there
        # rounds the gradient to the type first, then the sum
        err = 2 * ref.U * sizes[i] * size
        if start:
            err = err + ref.half(dtype) * (abs(want) + err)
            want = want + ref.f64(before[i])
        err = err + ref.half(dtype) * (abs(want) + err)
        assert (abs(ref.f64(out[i]) - want) <= err).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[1], [64], [65, 0, 3], [0, 0, 130, 0], [16, 48, 15, 17, 33, 63], [300, 1, 257], [0]])
@pytest.mark.parametrize("N,K", [(8, 8), (256, 256), (300, 520), (100, 1000), (1, 3)])
def test_wgrad(wst, sizes, N, K, dtype):
    check(wst, sizes, N, K, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[37, 0, 64], [129, 5]])
@pytest.mark.parametrize("N,K", [(200, 328), (33, 70), (130, 333)])
def test_wgrad_accumulates(wst, sizes, N, K, dtype):
    check(wst, sizes, N, K, dtype, start=True)


@pytest.mark.parametrize("sizes", [[37, 21], [5], [0, 0]])
def test_rows_of_no_group_do_not_count(wst, sizes):
    check(wst, sizes, 264, 136, torch.float32, behind=70)


def test_neighbours_not_finite(wst):
    # a group full of NaN next to one that ends inside a block of tokens
    off = [0, 21, 45, 60]
    g = torch.Generator().manual_seed(1)
    dC, A = torch.randn(60, 96, generator=g).bfloat16(), torch.randn(60, 160, generator=g).bfloat16()
    dC[21:45], A[21:45] = torch.nan, torch.inf
    out, status = run(wst, dC, A, off, torch.float32)
    assert status == 0 and torch.isnan(out[1]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()


def test_many_groups_every_output(wst):
    rng = np.random.default_rng(2)
    sizes = rng.integers(0, 90, 300)
    sizes[rng.choice(300, 60, replace=False)] = 0
    check(wst, sizes.tolist(), 264, 264, torch.bfloat16)


def test_no_rows(wst):
    out, status = run(wst, torch.empty(0, 40).bfloat16(), torch.empty(0, 24).bfloat16(), [0, 0, 0], torch.float32)
    assert status == 0 and (out == 0).all()


def test_bad_offsets_latched(wst):
    dC, A = torch.ones(300, 64).bfloat16(), torch.ones(300, 64).bfloat16()
    _, status = run(wst, dC, A, [0, 250, 120, 300], torch.float32)
    assert status == wst.WST_ERR_BAD_OFFSETS
    _, status = run(wst, dC, A, [3, 100, 120, 300], torch.float32)
    assert status == wst.WST_ERR_BAD_OFFSETS


@pytest.mark.parametrize("N,K", [(16, 24), (200, 328), (33, 70), (300, 333), (264, 520), (1, 3)])
def test_bf16_accumulation_rounds_once(wst, N, K):
    # dB holds the negative of the gradient in bf16, so what is left is the part that
    # a gradient rounded to bf16 first would have lost; and an ordinary dB.
    sizes = [40, 0, 129, 7]
    off = np.concatenate([[0], np.cumsum(sizes)])
    g = torch.Generator().manual_seed(N * K)
    dC, A = torch.randn(int(off[-1]), N, generator=g).bfloat16(), torch.randn(int(off[-1]), K, generator=g).bfloat16()
    d, a = ref.f64(dC), ref.f64(A)
    parts = [slice(off[i], off[i + 1]) for i in range(len(sizes))]
    want = np.stack([d[r].T @ a[r] for r in parts])
    size = np.stack([abs(d[r]).T @ abs(a[r]) for r in parts])
    for before in (-torch.from_numpy(want).bfloat16(), torch.randn(len(sizes), N, K, generator=g).bfloat16() * 8):
        out, status = run(wst, dC, A, off, torch.bfloat16, before)
        assert status == 0
        b = ref.f64(before)
        # one fp32 rounding (cut off: 2u) per token, one of the sum in fp32, one to bf16
        err = 2 * ref.U * np.array(sizes)[:, None, None] * size
        err = err + ref.U * (abs(want + b) + err)
        assert (abs(ref.f64(out) - (want + b)) <= err + ref.half(torch.bfloat16) * (abs(want + b) + err)).all()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_and_gradients_behind_32_bits(wst, dtype, accumulate):
    # the last group's rows lie more than 2^31 elements into A, and so does its gradient
    G, N, K = 130, 4096, 4104
    M = 530000
    off = torch.tensor([0] * (G - 1) + [M - 40, M], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(8)
    dC, A = torch.zeros(M, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    d, a = torch.randn(40, 64, generator=g).bfloat16(), torch.randn(40, K, generator=g).bfloat16()
    dC[-40:], A[-40:] = d.cuda(), a.cuda()
    dB = torch.full((G, N, K), 1.0, dtype=dtype, device="cuda")[:, :64]     # (64 of every 4096 rows)
    ws = wst.workspace()
    wst.wst_grouped_gemm_wgrad_bf16(dC, A, off, dB, accumulate=accumulate, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    want, size = ref.f64(d).T @ ref.f64(a) + accumulate, abs(ref.f64(d)).T @ abs(ref.f64(a)) + accumulate
    err = 2 * ref.U * 41 * size
    assert (abs(ref.f64(dB[-1]) - want) <= err + ref.half(dtype) * (abs(want) + err)).all()
    assert (dB[:-1] == (1 if accumulate else 0)).all()
