"""wst_tree_attention_bf16 against attention in 64 bits: lengths around the blocks,
trees, chains and arbitrary masks, head groups, page sizes and layouts, what lies in
masked places, and the limits that the device checks."""
import math

import numpy as np
import pytest
import torch

import warp_specialized_tensor_gb300 as wst
from tree_ref import Paged

pytestmark = pytest.mark.gpu


def run(c, dtype=torch.float32, scale=None, ws=None, whole=True, mask="own"):
    out = torch.full((c.T, c.H, c.Dh), 3.0, dtype=dtype, device="cuda")
    ws = ws if ws is not None else (wst.tree_attention_workspace() if whole else wst.workspace())
    wst.wst_tree_attention_bf16(c.q, c.offsets, c.context, c.k_cache, c.v_cache, c.table, out,
                                mask=c.mask if isinstance(mask, str) else mask, scale=scale, workspace=ws)
    return out, wst.wst_sync_status(ws)


def check(c, dtype=torch.float32, scale=None, **kw):
    out, status = run(c, dtype, scale, **kw)
    assert status == 0
    want, size, most = c.want(1.0 / math.sqrt(c.Dh) if scale is None else scale)
    n = c.starts[-1]
    err = (out[:n].double() - want).abs()
    tol = c.tolerance(want, size, most, dtype)
    assert bool((err <= tol).all()), (float(err.max()), float((err / tol.clamp_min(1e-30)).max()))
    assert bool((out[n:] == 3.0).all())
    return out


CASES = [  # lens, H, Hkv, Dh, page, mask, type, layout, whole workspace
    ([(0, 1)], 1, 1, 128, 16, "chain", torch.float32, "plain", True),
    ([(1, 1)], 1, 1, 64, 16, "chain", torch.bfloat16, "plain", True),
    ([(126, 1), (127, 1), (128, 1), (255, 1), (256, 1)], 8, 2, 128, 64, "chain", torch.float32, "plain", True),
    ([(126, 2), (127, 2), (128, 3), (0, 5), (300, 0), (1, 7)], 4, 4, 64, 32, "tree", torch.float32, "heads", True),
    ([(0, 0), (40, 3), (0, 0), (0, 0), (700, 1), (0, 0)], 6, 2, 128, 128, "tree", torch.float32, "plain", True),
    ([(500, 7)], 12, 4, 64, 16, "tree", torch.float32, "plain", True),
    ([(1000, 64), (70, 33), (0, 64)], 32, 8, 128, 64, "tree", torch.bfloat16, "plain", True),
    ([(1000, 64), (70, 33), (0, 64)], 32, 8, 128, 64, "any", torch.float32, "both", True),
    ([(1000, 64), (70, 33), (0, 64)], 32, 8, 128, 64, "any", torch.float32, "both", False),
    ([(300, 96), (5, 70)], 5, 1, 64, 256, "any", torch.float32, "heads", True),
    ([(333, 40)], 14, 2, 128, 8, "tree", torch.float32, "plain", True),
    ([(10, 3), (2000, 2)], 128, 1, 128, 64, "tree", torch.float32, "plain", True),
    ([(100, 5)], 100, 1, 64, 32, "chain", torch.bfloat16, "plain", True),
    ([(0, 300), (129, 257), (1000, 131)], 8, 2, 128, 32, "chain", torch.float32, "plain", True),
    ([(0, 300), (129, 257), (1000, 131)], 3, 3, 64, 64, "chain", torch.float32, "both", False),
    ([(7, 500)], 28, 4, 128, 32, "chain", torch.bfloat16, "heads", True),
    ([(20000, 1)], 8, 1, 128, 128, "chain", torch.float32, "plain", True),
    ([(20000, 30)], 16, 2, 64, 384, "tree", torch.float32, "plain", True),
    ([(i * 7 % 600, 1 + i % 3) for i in range(300)], 4, 2, 64, 16, "tree", torch.float32, "plain", True),
    ([(i * 37 % 900, 1) for i in range(64)], 16, 2, 128, 16, "chain", torch.bfloat16, "plain", False),
]


@pytest.mark.parametrize("lens,H,Hkv,Dh,page,mask,dtype,layout,whole", CASES, ids=["case%d" % i for i in range(len(CASES))])
def test_attention(lens, H, Hkv, Dh, page, mask, dtype, layout, whole):
    check(Paged(lens, H, Hkv, Dh, page, mask, seed=len(lens) + H, layout=layout, behind=len(lens) % 3), dtype, whole=whole)


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("size,scale", [(30.0, None), (1.0, -0.3), (1.0, 0.0), (6.0, 2.5)])
def test_scores_of_every_size(size, scale, Dh):
    """Sharp rows (the maximum moves block after block), scales below and at zero."""
    c = Paged([(1500, 9), (3000, 1)], 8, 2, Dh, 64, "tree", seed=4, size=size)
    # scores that grow along the context: every block rescales
    for b, (n, _) in enumerate(c.lens):
        c.K[b][:n] = (c.K[b][:n].float() * torch.linspace(0.05, 1.0, n, device="cuda")[:, None, None]).bfloat16()
    c.fill()
    check(c, scale=scale)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("Dh", [64, 128])
def test_keys_that_come_from_far_memory(page, Dh):
    """Sequences of many blocks with the caches out of L2, so that V arrives long after its scores: blocks that are
    cleaned behind a sequence's end while the ones before them are still read."""
    c = Paged([(2048 + 66 * i, 1 + i % 3) for i in range(32)], 32, 8, Dh, page, "chain", seed=2)
    want, size, most = c.want(1.0 / math.sqrt(Dh))
    tol = c.tolerance(want, size, most, torch.float32)
    for _ in range(3):
        torch.randn(1 << 27, device="cuda")
        out, status = run(c)
        assert status == 0 and bool(((out.double() - want).abs() <= tol).all())


def test_rows_that_see_nothing():
    c = Paged([(0, 40), (200, 5), (0, 3)], 4, 2, 128, 16, "any", seed=1)
    c.seen[0][::3] = False
    c.seen[2][:] = False
    mask = c.mask.clone()
    mask[0:40:3] = 0
    mask[45:] = 0
    out, status = run(c, mask=mask)
    assert status == 0
    want, size, most = c.want(1.0 / math.sqrt(128))
    assert bool(((out.double() - want).abs() <= c.tolerance(want, size, most, torch.float32)).all())
    assert bool((out[0:40:3] == 0).all()) and bool((out[45:] == 0).all())


@pytest.mark.parametrize("Dh,whole", [(128, True), (64, False)])
def test_what_lies_in_masked_places(Dh, whole):
    """NaN and infinities in new tokens reach the rows that see them and no others."""
    lens = [(250, 30), (0, 20), (3000, 64)]
    c = Paged(lens, 8, 2, Dh, 16, "tree", seed=8)
    clean, status = run(c, whole=whole)
    assert status == 0
    seen_by = []
    for b, (ctx, n) in enumerate(lens):
        for new, value in ((n // 2, float("nan")), (n - 2, float("inf"))):
            c.K[b][ctx + new] = value
            c.V[b][ctx + new] = value
        seen_by.append(torch.from_numpy(c.seen[b][:, [n // 2, n - 2]].any(axis=1)).cuda())
    touched = torch.cat(seen_by)
    c.fill()
    out, status = run(c, whole=whole)
    assert status == 0
    assert torch.equal(out[~touched], clean[~touched])
    assert not bool(out[touched].isfinite().any())
    # a value alone: infinity where it is seen, the other components as they were
    c = Paged(lens, 8, 2, Dh, 16, "tree", seed=8)
    for b, (ctx, n) in enumerate(lens):
        c.V[b][ctx + 3, :, 5] = -float("inf")
    c.fill()
    out, status = run(c, whole=whole)
    assert status == 0
    touched = torch.cat([torch.from_numpy(s[:, 3]).cuda() for s in c.seen])
    assert bool((out[touched][..., 5] == -float("inf")).all())
    out[touched, :, 5] = clean[touched, :, 5]
    assert torch.equal(out, clean)


def test_lowest_and_infinite_scores():
    """Keys of the type's largest size: weights of exactly 0 and 1."""
    c = Paged([(300, 4)], 2, 1, 64, 32, "chain", seed=2)
    c.q[:] = 1.0
    c.K[0][:] = -1e30
    c.K[0][7] = 1e30
    c.fill()
    out, status = run(c)
    assert status == 0
    assert bool((out == c.V[0][7].float()).all())


def test_same_bits_every_time_and_on_a_used_workspace():
    c = Paged([(5000, 20), (100, 3), (2500, 64)], 16, 4, 128, 64, "tree", seed=3)
    ws = wst.tree_attention_workspace()
    first, status = run(c, ws=ws)
    assert status == 0
    for _ in range(4):
        ws[256:].random_(0, 256)
        again, status = run(c, ws=ws)
        assert status == 0 and torch.equal(first, again)


def test_graphs_and_streams():
    """Captured once, replayed with other lengths; a captured call and an eager one on one workspace; a side stream."""
    lens = [(700, 5), (33, 64), (1500, 1)]
    c = Paged(lens, 8, 2, 128, 32, "tree", seed=6)
    ws = wst.tree_attention_workspace()
    want, _ = run(c, ws=ws)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        wst.wst_tree_attention_bf16(c.q, c.offsets, c.context, c.k_cache, c.v_cache, c.table, out, mask=c.mask, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    full = c.context.clone()
    c.context[:] = torch.tensor([400, 0, 1490], dtype=torch.int32, device="cuda")
    again, _ = run(c, ws=ws)      # (the masks now end at other keys)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again) and not torch.equal(out, want)
    c.context[:] = full
    with torch.cuda.stream(side):
        out.zero_()
        wst.wst_tree_attention_bf16(c.q, c.offsets, c.context, c.k_cache, c.v_cache, c.table, out, mask=c.mask, workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and wst.wst_sync_status(ws) == 0


def test_what_the_device_refuses():
    c = Paged([(100, 5), (30, 4)], 4, 2, 64, 16, "tree", seed=5)
    good, status = run(c)
    assert status == 0
    BAD, INVALID = wst.WST_ERR_BAD_OFFSETS, wst.WST_ERR_INVALID_ARG
    for name, value, code in (("offsets", [0, 5, 10], BAD), ("offsets", [1, 5, 9], BAD), ("offsets", [0, 7, 5], BAD),
                              ("offsets", [0, -3, 9], BAD), ("context", [-1, 30], BAD), ("context", [100, 2 ** 31 - 1], BAD),
                              ("context", [c.max_pages * 16 - 4, 30], BAD)):
        old = getattr(c, name).clone()
        getattr(c, name)[:] = torch.tensor(value, dtype=torch.int32, device="cuda")
        # (lengths that grow into the rubbish behind the table's pages may report that first)
        assert run(c)[1] in (code, INVALID), (name, value)
        getattr(c, name)[:] = old
    for page in (-1, c.pages, 2 ** 31 - 1):
        old = int(c.table[0, 1])
        c.table[0, 1] = page
        assert run(c)[1] == INVALID
        c.table[0, 1] = old
    assert run(c, mask=c.mask[:, :0].new_zeros(9, 1))[1] == 0
    out, status = run(c)
    assert status == 0 and torch.equal(out, good)
    many = Paged([(3, 40)], 2, 2, 64, 16, "tree", seed=5)
    assert run(many, mask=many.mask[:, :1].contiguous())[1] == BAD


def test_strided_operands_and_nothing_to_do():
    """Queries and outputs that are parts of wider rows, a mask and a page table with spare columns."""
    c = Paged([(90, 6), (11, 3)], 6, 3, 64, 32, "tree", seed=7, spare_words=1)
    want, _ = run(c)
    wide = torch.randn(c.T, 10, 64, device="cuda").bfloat16()
    wide[:, 2:8] = c.q
    out = torch.full((c.T, 9, 64), 5.0, device="cuda")
    ws = wst.tree_attention_workspace()
    wst.wst_tree_attention_bf16(wide[:, 2:8], c.offsets, c.context, c.k_cache, c.v_cache, c.table, out[:, 3:], mask=c.mask, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    assert torch.equal(out[:, 3:], want) and bool((out[:, :3] == 5.0).all())
    empty = torch.zeros(0, 6, 64, device="cuda")
    wst.wst_tree_attention_bf16(empty.bfloat16(), torch.zeros(3, dtype=torch.int32, device="cuda"), c.context, c.k_cache, c.v_cache, c.table,
                                empty, workspace=ws)
    out = torch.full((4, 6, 64), 5.0, device="cuda")
    wst.wst_tree_attention_bf16(c.q[:4], torch.zeros(3, dtype=torch.int32, device="cuda"), c.context, c.k_cache, c.v_cache, c.table, out,
                                workspace=ws)
    assert wst.wst_sync_status(ws) == 0 and bool((out == 5.0).all())


def test_keys_behind_two_to_the_31_elements():
    """A cache of more than 2^31 elements whose last page holds the sequence."""
    pages, page, Hkv, Dh = 17000, 128, 8, 128
    k = torch.zeros(pages, page, Hkv, Dh, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    k[-1] = torch.randn(page, Hkv, Dh, generator=g, device="cuda").bfloat16()
    v[-1] = torch.randn(page, Hkv, Dh, generator=g, device="cuda").bfloat16()
    v[-1, 100:, :, 3] = float("inf")
    q = torch.randn(1, 8, Dh, generator=g, device="cuda").bfloat16()
    out = torch.zeros(1, 8, Dh, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = wst.tree_attention_workspace()
    wst.wst_tree_attention_bf16(q, torch.tensor([0, 1], **i32), torch.tensor([99], **i32), k, v, torch.tensor([[pages - 1]], **i32), out, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    p = torch.softmax(torch.einsum("hd,jhd->hj", q[0].double(), k[-1, :100].double()) / math.sqrt(Dh), dim=1)
    want = torch.einsum("hj,jhd->hd", p, v[-1, :100].double())
    assert float((out[0].double() - want).abs().max()) <= 2.0 ** -7 * 4
