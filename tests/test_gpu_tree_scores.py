"""wst_tree_attention_bf16 with scores that fp32 holds exactly, so that what is left of the error is the probabilities':
maxima that grow in the middle of a block, and the parts in which fp32 output takes P."""
import math

import numpy as np
import pytest
import torch

import warp_specialized_tensor_gb300 as wst
from tree_ref import Paged

pytestmark = pytest.mark.gpu

LN2 = float(np.float32(math.log(2.0)))  # times log2(e), rounded to fp32, it is 1: a score is an exponent of 2
                                        # (off by less than 2^-28 of it)


def run(c, dtype, scale, whole=True):
    out = torch.full((c.T, c.H, c.Dh), 3.0, dtype=dtype, device="cuda")
    ws = wst.tree_attention_workspace() if whole else wst.workspace()
    wst.wst_tree_attention_bf16(c.q, c.offsets, c.context, c.k_cache, c.v_cache, c.table, out, mask=c.mask, scale=scale, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    return out


def exact_scores(lens, H, Hkv, Dh, page, mask, seed, every, rise):
    """Row (t, h) scores fine + rise * (how often its maximum has grown): two products of bf16 numbers whose sum 24 bits
    hold.  It grows at four of every `every`-th key (not the same ones for each head); `fine` lies in (-4, 0] in 64ths.
    A component of V is 1 for one key of the sequence and 0 for the others, so an output is that key's probability."""
    c = Paged(lens, H, Hkv, Dh, page, mask, seed=seed)
    rng = np.random.default_rng(seed)
    group = H // Hkv
    assert 2 * group <= Dh
    c.q.zero_()
    for h in range(H):
        c.q[:, h, 2 * (h % group)] = 1.0
        c.q[:, h, 2 * (h % group) + 1] = 1.0
    for b, (ctx, n) in enumerate(lens):
        N = ctx + n
        steps = -(-N // every)
        K, V = np.zeros((N, Hkv, Dh)), np.zeros((N, Hkv, Dh))
        for h in range(H):
            grows = np.zeros(steps, dtype=bool)
            grows[1 + rng.permutation(steps - 1)[:4]] = True  # (no more: below 2^-126 there is no P)
            K[:, h // group, 2 * (h % group)] = rise * np.cumsum(grows)[np.arange(N) // every]
            K[:, h // group, 2 * (h % group) + 1] = -rng.integers(0, 256, N) / 64.0
        for h in range(Hkv):
            keys = rng.permutation(N)[:Dh]
            V[keys, h, np.arange(keys.size)] = 1.0
        c.K[b] = torch.from_numpy(K).cuda().bfloat16()
        c.V[b] = torch.from_numpy(V).cuda().bfloat16()
        assert torch.equal(c.K[b].double().cpu(), torch.from_numpy(K))
    c.fill()
    return c


CASES = [  # lens, H, Hkv, Dh, page, mask, whole workspace
    ([(508, 5), (130, 3), (64, 1)], 8, 2, 128, 64, "chain", True),
    ([(508, 5), (130, 3), (64, 1)], 8, 2, 64, 16, "chain", False),
    ([(250, 70), (0, 64)], 16, 2, 128, 32, "tree", True),
    ([(900, 9)], 4, 1, 64, 128, "any", True),
    ([(0, 200), (96, 33)], 2, 1, 128, 16, "chain", True),
]


@pytest.mark.parametrize("every,rise", [(32, 10.0), (64, 20.0), (96, 12.0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,H,Hkv,Dh,page,mask,whole", CASES, ids=["case%d" % i for i in range(len(CASES))])
def test_probabilities_of_exact_scores(lens, H, Hkv, Dh, page, mask, whole, dtype, every, rise):
    """The whole relative error of an output, which is one probability p / l, in units of 2^-24:
    2^x is good to 2^-22, for p and for the terms of l: 8; l adds the terms of one size (what came before a growth counts
    2^-10 and less) in chains of 8 and their sums (7 + 2), over the 4 steps of a block and up to 8 blocks, a rounding each:
    21; the scale, 2^-28 of an exponent below 128 times ln 2: 6; 1 / l, its product, the join of two pieces: 6; the three
    bf16 of p: 1, their products with 1, added with 2^-22 each: 8.  That is 50 or 2^-18.3; two parts of p would be off by
    up to 2^-16, 256.  bf16 output: P and the result are each off by 2^-8, l adds 8 terms more in a chain."""
    c = exact_scores(lens, H, Hkv, Dh, page, mask, len(lens) + Dh + int(rise), every, rise)
    out = run(c, dtype, LN2, whole)
    want, _, _ = c.want(LN2)
    bound = 50 * 2.0 ** -24 if dtype is torch.float32 else 2.0 ** -8 + (1 + 2.0 ** -8) * 2.0 ** -8 + 60 * 2.0 ** -24
    err = (out.double() - want).abs()
    assert bool((err <= want * bound).all()), float((err / want.clamp_min(1e-300)).max())
    assert float(want[want > 0].min()) > 2.0 ** -100


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Dh,whole", [(128, True), (64, False)])
@pytest.mark.parametrize("first,last,value", [(0, 32, -float("inf")), (0, 64, -float("inf")), (0, 128, -float("inf")), (0, 900, -float("inf")),
                                              (0, 200, -3e38), (1000, 1500, -3e38)])
def test_context_whose_scores_are_infinite(first, last, value, Dh, whole, dtype):
    """Keys [first, last) of the context score -inf (held so, or beyond fp32: -3e38 * 4): they weigh nothing, wherever a
    block or a share begins."""
    lens = [(700, 3), (2500, 1), (1023, 2), (128, 1), (40, 5)]
    c = Paged(lens, 8, 2, Dh, 16, "chain", seed=last)
    c.q[:, :, 0] = 4.0

    def keys(x):
        for b, (n, _) in enumerate(lens):
            c.K[b][first:min(last, n), :, 0] = x
    keys(0.0)
    _, _, most = c.want(1.0 / math.sqrt(Dh))
    keys(-1e30)  # (whose weight 64 bits do not hold either)
    want, size, _ = c.want(1.0 / math.sqrt(Dh))
    keys(value)
    c.fill()
    out = run(c, dtype, 1.0 / math.sqrt(Dh), whole)
    tol = c.tolerance(want, size, most, dtype)
    assert bool(((out.double() - want).abs() <= tol).all())


def test_rows_whose_scores_are_all_infinite():
    """Nothing of weight: zeros, as where a row sees nothing; the sequences beside it as they were."""
    lens = [(300, 2), (127, 1), (255, 1), (0, 3)]
    c = Paged(lens, 4, 2, 128, 32, "chain", seed=1)
    c.q[:, :, 0] = 1.0
    clean = run(c, torch.float32, None)
    for b in (1, 2, 3):
        c.K[b][..., 0] = -float("inf")
    c.fill()
    out = run(c, torch.float32, None)
    assert torch.equal(out[:2], clean[:2]) and bool((out[2:] == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Dh,whole", [(128, True), (64, False)])
@pytest.mark.parametrize("value", [1e30, 2e7, float("inf")])
def test_large_scores_leave_the_other_rows_bits_alone(value, Dh, whole, dtype):
    """One component of a new token's key is large, so the rows that see it have large scores, of either sign: those that
    do not see it keep their bits, though they share warps with them."""
    lens = [(250, 30), (0, 20), (3000, 64)]
    c = Paged(lens, 8, 2, Dh, 16, "tree", seed=9)
    clean = run(c, dtype, None, whole)
    new = [next(i for i in range(1, n) if 2 <= c.seen[b][:, i].sum() <= n // 2) for b, (_, n) in enumerate(lens)]
    touched = torch.cat([torch.from_numpy(c.seen[b][:, i]).cuda() for b, i in enumerate(new)])
    for b, (ctx, _) in enumerate(lens):
        c.K[b][ctx + new[b], :, 3] = value
    c.fill()
    out = run(c, dtype, None, whole)
    assert torch.equal(out[~touched], clean[~touched]) and not torch.equal(out[touched], clean[touched])


def test_a_mask_without_words_is_refused():
    """No words hold no tokens' bits (and an empty tensor's address is NULL, which would mean a chain)."""
    c = Paged([(20, 3)], 2, 1, 64, 16, "tree", seed=1)
    out = torch.full((c.T, c.H, c.Dh), 3.0, device="cuda")
    with pytest.raises((ValueError, wst.WstError)):
        wst.wst_tree_attention_bf16(c.q, c.offsets, c.context, c.k_cache, c.v_cache, c.table, out, mask=c.mask[:, :0],
                                    workspace=wst.workspace())
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_last_page_behind_two_to_the_31_elements(dtype):
    """A cache of more than 2^31 elements, the sequence on its last page and its first: the bounds of the other tests."""
    pages, page, H, Hkv, Dh = 17000, 128, 8, 8, 128
    c = Paged([(150, 3)], H, Hkv, Dh, page, "chain", seed=3)
    k = torch.zeros(pages, page, Hkv, Dh, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c.k_cache, c.v_cache = k, v
    c.table[0, :2] = torch.tensor([pages - 1, 0], dtype=torch.int32, device="cuda")
    c.fill()
    k[0, 25:], v[0, 25:] = float("nan"), float("inf")
    out = run(c, dtype, 1.0 / math.sqrt(Dh))
    want, size, most = c.want(1.0 / math.sqrt(Dh))
    assert bool(((out.double() - want).abs() <= c.tolerance(want, size, most, dtype)).all())


def long_sums(lens, H, Hkv, Dh, dtype, seed):
    """Scores of whole numbers for bf16 output (P is a power of two, exact in bf16), in 64ths for fp32; V of one sign."""
    c = Paged(lens, H, Hkv, Dh, 128, "chain", seed=seed)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.q[:, :, 1] = 1.0
    g = torch.Generator(device="cuda").manual_seed(seed)
    for b, (ctx, n) in enumerate(lens):
        N = ctx + n
        c.K[b].zero_()
        if dtype is torch.bfloat16:
            c.K[b][..., 0] = -torch.randint(0, 12, (N, Hkv), generator=g, device="cuda").bfloat16()
        else:
            c.K[b][..., 0] = (-torch.randint(0, 256, (N, Hkv), generator=g, device="cuda") / 64.0).bfloat16()
        c.V[b] = (1.0 + torch.rand(N, Hkv, Dh, generator=g, device="cuda")).bfloat16()
    c.fill()
    return c


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("lens,H,Hkv,Dh", [([(2000, 1)], 4, 1, 128), ([(8000, 2), (3, 1), (129, 5)], 8, 2, 64), ([(70000, 1)], 8, 2, 128),
                                           ([(70000, 40)], 8, 1, 64), ([(262143, 1)], 2, 1, 64)])
def test_long_sums_fp32(lens, H, Hkv, Dh, whole):
    """In units of 2^-24, everything of one sign: 42 for P and l of a block (the test above), a block's last 8 products
    with V, each cut off by up to 2 (the two smaller parts' are 2^-8 of that): 17, and a rounding for every block in each
    of the two sums.  (Cut off with every product over the whole length it is 40 for a block.)"""
    c = long_sums(lens, H, Hkv, Dh, torch.float32, sum(lens[0]))
    out = run(c, torch.float32, LN2, whole)
    want, _, _ = c.want(LN2)
    blocks = max(-(-(ctx + n) // 128) for ctx, n in lens)
    bound = (42 + 17 + 2 * blocks) * 2.0 ** -24
    err = ((out.double() - want) / want).abs()
    assert float(err.max()) <= bound, float(err.max()) / bound
    # where nothing adds up, these are a walk's steps: the mean, which cutting off would move with every block
    assert abs(float(((out.double() - want) / want).mean())) <= (42 + 17 + 8) * 2.0 ** -24


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("lens,H,Hkv,Dh", [([(8000, 1)], 8, 2, 128), ([(600000, 1)], 4, 1, 64), ([(300000, 3)], 4, 1, 128), ([(33000, 33)], 8, 2, 64),
                                           ([(70000, 2), (100, 40), (131072, 1), (0, 5), (65535, 1)], 8, 2, 128)])
def test_long_sums_bf16(lens, H, Hkv, Dh, whole):
    """P and l are exact but for the scale (2^-22) and fp32's sums; what is left before the result's own rounding, half a
    step of the bf16 at hand: the 8 products of up to 512 blocks, each cut off by up to 2^-23, 2^-11 in all, and the
    roundings of the runs, of l and at the end, 2^-20.  (Cut off with every product, 300,000 keys are off by 2^-9.6.)"""
    c = long_sums(lens, H, Hkv, Dh, torch.bfloat16, sum(lens[0]))
    out = run(c, torch.bfloat16, LN2, whole)
    want, _, _ = c.want(LN2)
    half = torch.exp2(want.log2().floor()) * 2.0 ** -8
    over = ((out.double() - want).abs() - half) / want
    assert float(over.max()) <= 2.0 ** -11 + 2.0 ** -20, float(over.max()) * 2 ** 11


def test_sharp_rows_over_several_runs():
    """Maxima that grow in later runs, and rows that see nothing for a while: what was added up before is scaled."""
    c = Paged([(140000, 3)], 4, 2, 128, 64, "any", seed=5, size=2.0)
    n = c.lens[0][0]
    c.K[0][:n] = (c.K[0][:n].float() * torch.linspace(0.05, 1.0, n, device="cuda")[:, None, None]).bfloat16()
    c.q[:, :, 0] = 2.0
    c.K[0][:66000, :, 0] = -3e38 * 4  # (rounds to -inf)
    c.K[0][:1000, 1, 0] = 1.0
    c.fill()
    assert bool(c.K[0][:1000, 0, 0].isinf().all())
    for dtype in (torch.bfloat16, torch.float32):
        for whole in (True, False):
            out = run(c, dtype, 0.05, whole)
            K = c.K[0]
            c.K[0] = torch.where(K.isinf(), -1e30, K)
            want, size, _ = c.want(0.05)
            c.K[0] = torch.where(K.isinf(), 0.0, K)
            _, _, most = c.want(0.05)
            c.K[0] = K
            assert bool(((out.double() - want).abs() <= c.tolerance(want, size, most, dtype)).all())
