"""wst_cache_append_bf16 against the rotation in 64 bits: both pairings, partial
rotations, cache layouts, skipped tokens, far positions."""
import pytest
import torch

import warp_specialized_tensor_gb300 as wst

pytestmark = pytest.mark.gpu


def rotated(x, positions, inv_freq, style):
    """fp64 [T, heads, Dh], and |a| + |b| of each component's pair (0 where it is copied)."""
    x = x.double()
    y, size = x.clone(), torch.zeros_like(x)
    if inv_freq is None:
        return y, size
    half = inv_freq.numel()
    lo = torch.arange(half, device=x.device) * (1 if style == "halves" else 2)
    hi = lo + (half if style == "halves" else 1)
    angle = positions.double()[:, None, None] * inv_freq.double()
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
    size[..., lo] = size[..., hi] = a.abs() + b.abs()
    return y, size


def cache(layout, pages, page, heads, Dh):
    """k and v caches [pages, page, heads, Dh] of one layout, filled with a number that no test stores."""
    if layout == "plain":
        return tuple(torch.full((pages, page, heads, Dh), 7.75, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    if layout == "heads":       # heads before tokens
        return tuple(torch.full((pages, heads, page, Dh), 7.75, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in "kv")
    both = torch.full((pages, 2, page, heads, Dh + 16), 7.75, dtype=torch.bfloat16, device="cuda")[..., :Dh]
    return both[:, 0], both[:, 1]


def check(got, want, size):
    """A bf16 rounding, and fp32's: an angle in half turns is off by 2^-25 (2^-23.3 radians), sine and cosine by two
    of their last bits, two products and a sum by half a bit each; together below 2^-20 of |a| + |b|."""
    err = (got.double() - want).abs()
    assert bool((err <= want.abs() * 2.0 ** -8 + size * 2.0 ** -20).all()), float(err.max())


CASES = [  # T, H, Hkv, Dh, rot, style, page, layout, type
    (1, 8, 8, 128, 128, "halves", 64, "plain", torch.bfloat16),
    (5, 4, 1, 64, 64, "pairs", 16, "plain", torch.bfloat16),
    (33, 12, 4, 128, 32, "halves", 32, "heads", torch.bfloat16),
    (70, 7, 1, 64, 16, "pairs", 1, "both", torch.float32),
    (19, 3, 3, 256, 256, "halves", 7, "both", torch.float32),
    (19, 3, 3, 256, 256, "pairs", 128, "heads", torch.bfloat16),
    (300, 64, 8, 128, 128, "halves", 64, "plain", torch.float32),
    (2000, 2, 2, 16, 0, "halves", 16, "plain", torch.bfloat16),
    (9, 5, 5, 48, 32, "pairs", 3, "heads", torch.bfloat16),
    # several tokens to a step of a block, also with angles for eight only, and a last step of fewer
    (4001, 2, 1, 64, 32, "pairs", 16, "plain", torch.float32),
    (12347, 1, 1, 256, 256, "halves", 16, "heads", torch.bfloat16),
    (20011, 1, 1, 48, 48, "pairs", 8, "both", torch.bfloat16),
]


@pytest.mark.parametrize("T,H,Hkv,Dh,rot,style,page,layout,dtype", CASES)
def test_append(T, H, Hkv, Dh, rot, style, page, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(T * 131 + Dh)
    qkv = torch.randn(T, (H + 2 * Hkv) * Dh, generator=g, device="cuda").to(dtype)
    q, k, v = (x.view(T, -1, Dh) for x in qkv.split([H * Dh, Hkv * Dh, Hkv * Dh], dim=1))
    pages = T // page + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    slots[T // 2:T // 2 + T // 8] = -1
    positions = torch.randint(0, 4000000, (T,), generator=g, device="cuda", dtype=torch.int32)
    positions[-1] = 2 ** 31 - 1
    inv = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float().cuda() if rot else None
    k_cache, v_cache = cache(layout, pages, page, Hkv, Dh)
    q_out = torch.full((T, H, Dh), 7.75, dtype=torch.bfloat16, device="cuda")
    ws = wst.workspace()
    wst.wst_cache_append_bf16(k, v, positions, slots, k_cache, v_cache, inv_freq=inv, style=style, q=q, q_out=q_out, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    live = slots >= 0
    at = slots[live].long()
    want, size = rotated(q[live], positions[live], inv, style)
    check(q_out[live], want, size)
    assert bool((q_out[~live] == 7.75).all())
    want, size = rotated(k[live], positions[live], inv, style)
    check(k_cache[at // page, at % page], want, size)
    assert torch.equal(v_cache[at // page, at % page], v[live].to(torch.bfloat16))
    rest = torch.ones(pages, page, dtype=torch.bool, device="cuda")
    rest[at // page, at % page] = False
    for c in (k_cache, v_cache):
        assert bool((c[rest] == 7.75).all())


def test_position_times_frequency_is_exact():
    """One pair a token, (1, 0): the cache holds cos and sin of position * inv_freq, for positions of either sign and
    frequencies above one, against Python's integers and 60 digits of 2 pi."""
    from fractions import Fraction
    turn = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)
    positions = [0, 1, 77, 4095, 1000003, 2 ** 24 + 1, 2 ** 31 - 1, -1, -65537, -2 ** 31]
    freqs = [1.0, 0.7311, 3e-5, 2.5, 1e-9, -0.25, 0.0, 6.2831854820251465]
    T, rot = len(positions), 16
    x = torch.zeros(T, 1, 16, device="cuda")
    x[..., :8] = 1.0
    inv = torch.tensor(freqs, dtype=torch.float32, device="cuda")
    k_cache, v_cache = cache("plain", 1, T, 1, 16)
    ws = wst.workspace()
    wst.wst_cache_append_bf16(x, x, torch.tensor(positions, dtype=torch.int32, device="cuda"),
                              torch.arange(T, dtype=torch.int32, device="cuda"), k_cache, v_cache, inv_freq=inv, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    angle = torch.empty(T, 8, dtype=torch.float64)
    for i, p in enumerate(positions):
        for j, f in enumerate(inv.tolist()):
            part = Fraction(p) * Fraction(f) / turn
            angle[i, j] = float((part - (part.numerator // part.denominator)) * turn)
    got = k_cache[0, :, 0].double().cpu()
    # (the fraction of a turn is rounded to 2^-52: 2^31 positions make 2^-20 of it)
    for g, want in ((got[:, :8], angle.cos()), (got[:, 8:], angle.sin())):
        assert float((g - want).abs().max()) <= 2.0 ** -8 + 2.0 ** -18
        assert bool(((g - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -18).all())


def test_in_place_without_queries_and_bad_slots():
    T, H, Dh = 6, 2, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(T, H, Dh, generator=g, device="cuda").bfloat16() for _ in range(3))
    inv = torch.rand(32, generator=g, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    ws = wst.workspace()
    slots = torch.tensor([0, 15, -7, 16, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")  # 16 slots
    one, two = cache("plain", 2, 8, H, Dh), cache("plain", 2, 8, H, Dh)
    out = torch.full_like(q, 7.75)
    wst.wst_cache_append_bf16(k, v, pos, slots, *one, inv_freq=inv, q=q, q_out=out, workspace=ws)
    assert wst.wst_sync_status(ws) == wst.WST_ERR_INVALID_ARG
    assert wst.wst_sync_status(ws) == 0
    assert bool((out[[2, 3, 5]] == 7.75).all()) and not bool((out[[0, 1, 4]] == 7.75).all())
    good = torch.where(slots < 16, slots, -1)
    same = q.clone()
    wst.wst_cache_append_bf16(k, v, pos, good, *two, inv_freq=inv, q=same, q_out=same, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    live = good >= 0
    assert torch.equal(same[live], out[live]) and torch.equal(same[~live], q[~live])
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    three = cache("plain", 2, 8, H, Dh)
    wst.wst_cache_append_bf16(k, v, pos, good, *three, inv_freq=inv, workspace=ws)
    assert torch.equal(three[0], two[0]) and torch.equal(three[1], two[1])
    empty = k[:0]
    wst.wst_cache_append_bf16(empty, empty, pos[:0], good[:0], *three, inv_freq=inv, workspace=ws)
    assert wst.wst_sync_status(ws) == 0


def test_slots_behind_two_to_the_31_elements():
    """A cache of more than 2^31 elements: the last slot is found."""
    pages, page, H, Dh = 4300, 512, 8, 128
    k_cache = torch.zeros(pages, page, H, Dh, dtype=torch.bfloat16, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    x = torch.ones(2, H, Dh, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([pages * page - 1, 5], dtype=torch.int32, device="cuda")
    ws = wst.workspace()
    wst.wst_cache_append_bf16(x, 2 * x, slots, slots, k_cache, v_cache, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    assert bool((k_cache[-1, -1] == 1).all()) and bool((v_cache[-1, -1] == 2).all()) and bool((k_cache[0, 5] == 1).all())
    assert float(k_cache[-1].float().sum()) == H * Dh and float(v_cache[0].float().sum()) == 2 * H * Dh
