"""GPU: routing, the plan of the rows, combine and their gradients against plain
64-bit implementations, at the sizes, masks and ties where they can go wrong."""
import numpy as np
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wst():
    import warp_specialized_tensor_gb300 as w
    w.load_library()
    return w


def padded(x, extra=0):
    """x on the GPU in rows that begin on 16 bytes, NaN behind them."""
    per = 16 // x.element_size()
    buf = torch.full((*x.shape[:-1], -(-x.shape[-1] // per) * per + extra * per), float("nan"), dtype=x.dtype, device="cuda")
    out = buf[..., :x.shape[-1]]
    out.copy_(x)
    return out


def route(wst, x, k, **kw):
    T = x.shape[0]
    experts = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((T, k), float("nan"), device="cuda")
    bias = kw.pop("bias", None)
    wst.wst_moe_route(x, experts, weights, bias=None if bias is None else bias.cuda(), **kw)
    return experts.cpu().numpy(), weights


def check_route(wst, x, k, score, bias=None, **kw):
    got_e, got_w = route(wst, padded(x, 1), k, score=score, bias=bias, **kw)
    want_e, want_w = ref.route(ref.f64(x), k, score, bias=None if bias is None else ref.f64(bias), **kw)
    assert np.array_equal(got_e, want_e)
    # exp of a difference of at most 32 in size, a sum of at most 1024 terms and a quotient: below 2^-17 relative
    assert np.allclose(ref.f64(got_w), want_w, rtol=2.0 ** -17, atol=1e-30, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 7, 3), (5, 32, 2), (33, 60, 6), (9, 64, 16), (130, 100, 8), (257, 256, 8),
                                   (6, 384, 10), (3, 1000, 4), (4, 1024, 16)])
def test_route(wst, dtype, score, T, E, k):
    g = torch.Generator().manual_seed(T * 1000 + E)
    x = (torch.randn(T, E, generator=g) * 1.5).to(dtype)
    bias = torch.randn(E, generator=g) * 0.1
    check_route(wst, x, k, score, renorm=True)
    check_route(wst, x, k, score, renorm=False, scale=2.5)
    check_route(wst, x, k, score, bias=bias, renorm=True, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,best,k", [(256, 8, 4, 2, 8), (256, 8, 3, 1, 8), (60, 4, 2, 2, 6), (96, 32, 5, 2, 15),
                                                        (35, 5, 1, 2, 7), (512, 16, 16, 2, 4), (1024, 2, 1, 1, 16), (8, 8, 3, 2, 3)])
def test_route_groups(wst, score, E, groups, top_groups, best, k):
    g = torch.Generator().manual_seed(E + groups)
    x = torch.randn(200, E, generator=g) * 1.5
    x[::3] = torch.where(torch.rand(67, E, generator=g) < 0.6, -torch.inf, x[::3])  # many experts off, some groups empty
    for bias in (None, torch.randn(E, generator=g) * 0.2):
        check_route(wst, x, k, score, bias=bias, groups=groups, top_groups=top_groups, group_best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks_and_ties(wst, score):
    lowest = torch.finfo(torch.float32).min
    x = torch.tensor([[-torch.inf] * 8,                                    # nothing to choose
                      [-torch.inf] * 5 + [0.5] + [-torch.inf] * 2,          # one expert for three slots
                      [lowest] * 6 + [1.0, -200.0],                         # the lowest value masks too
                      [1.0] * 8,                                            # all equal: the lowest indices
                      [0.0, -0.0, 0.0, -0.0, -1.0, 2.0, 2.0, -1.0],          # -0 equals 0
                      [-100.0, -101.0, -120.0] + [-torch.inf] * 5])          # scores far below 1
    check_route(wst, x, 3, score)
    check_route(wst, x.bfloat16(), 3, score)
    bias = torch.tensor([5.0, 0.0, 0.0, -torch.inf, 0.0, 0.0, 0.0, 3.0])     # a bias does not bring back an expert that is off
    check_route(wst, x, 3, score, bias=bias)
    check_route(wst, x, 3, score, bias=bias, groups=4, top_groups=2, group_best=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_nan_and_infinite_logits(wst, score):
    x = torch.randn(4, 40, generator=torch.Generator().manual_seed(3))
    x[0, 17] = torch.nan
    x[1, 30] = torch.inf
    x[2, :] = torch.nan
    x[3, ::2] = -torch.inf
    x[3, 5] = torch.nan
    check_route(wst, x, 4, score)
    check_route(wst, x, 4, score, bias=torch.zeros(40))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scores_closer_than_fp32(wst, score):
    # Biases that nearly cancel the scores: all sums within about 2^-25 of each
    # other, so the order is decided by digits that fp32 does not have.
    g = torch.Generator().manual_seed(11)
    row = torch.randn(1, 128, generator=g)
    s = torch.from_numpy(ref.scores(ref.f64(row), score))[0]
    bias = (1.0 - s).float()
    check_route(wst, row.repeat(3, 1), 12, score, bias=bias)
    check_route(wst, row.repeat(3, 1), 12, score, bias=bias, groups=8, top_groups=3, group_best=2)


@pytest.mark.parametrize("place", ["inside", "border", "group"])
def test_route_one_close_pair(wst, place):
    # In every row two experts' sums differ by a few 2^-26: among the chosen, at the
    # border of the chosen ones, or in two groups of which one is kept.
    g = torch.Generator().manual_seed(17)
    T, E, k = 400, 64, 6
    x = torch.randn(T, E, generator=g) * 0.5 - 2.0
    x[:, [3, 11, 20]] = torch.randn(T, 3, generator=g) * 0.1 + 2.0     # certainly chosen
    bias = torch.randn(E, generator=g) * 0.02
    if place == "border":
        x[:, [30, 31]] = 1.0                                            # chosen too: five in front of the pair
    sum5 = 1.0 / (1.0 + np.exp(-0.2 * np.random.default_rng(1).random(T))) + float(bias[5])
    for e in (5, 37):
        s = sum5 - float(bias[e])
        x[:, e] = torch.from_numpy(np.log(s / (1 - s))).float()         # rounded: the sums are no longer equal
    kw = dict(groups=2, top_groups=1, group_best=1) if place == "group" else {}
    if place == "group":
        x[:, [3, 11, 20]] -= 6.0
    check_route(wst, x, k, "sigmoid", bias=bias, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("row", [[18.0, 18.0, 20.0, 1.0], [18.0, 18.0, 18.0, 18.0, 18.0, 19.0], [0.0, 0.0, 1e-8, -1.0],
                                 [20.0, 18.0, 18.0, 19.0], [20.0, 19.0, 18.0, 18.0, 18.5, 18.0], [3.0, 17.0, 17.0, 17.0]])
def test_route_equals_at_the_border_and_one_behind(wst, row, k, dtype):
    # The last chosen expert has an exact equal just outside, and behind the two
    # lies one that is larger by less than fp32 tells apart.
    x = torch.tensor([row, row[::-1]]).to(dtype)
    check_route(wst, x, k, "sigmoid", bias=torch.zeros(len(row)))
    check_route(wst, x, k, "softmax", bias=torch.zeros(len(row)))
    check_route(wst, x, k, "sigmoid", bias=torch.full((len(row),), 0.25), renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_equals_at_the_border_in_groups(wst, score):
    x = torch.tensor([[0.0, 0.0, 0.0, 0.0, 1e-8, 1e-8, 0.0, 0.0], [18.0, 1.0, 18.0, 1.0, 19.0, 1.0, 18.0, 1.0]])
    check_route(wst, x, 1, score, groups=4, top_groups=3, group_best=2)
    check_route(wst, x, 2, score, groups=4, top_groups=3, group_best=2)


def test_route_many_equal_logits(wst):
    # few different values, most of them where the sigmoid of fp32 is 1
    g = torch.Generator().manual_seed(23)
    x = torch.randint(30, 44, (300, 64), generator=g) / 2.0
    for bias in (torch.zeros(64), torch.randint(0, 3, (64,), generator=g) * 0.001):
        check_route(wst, x, 4, "sigmoid", bias=bias)
        check_route(wst, x.bfloat16(), 8, "sigmoid", bias=bias, groups=8, top_groups=4, group_best=2)


def test_route_is_the_same_on_every_call_and_stream(wst):
    x = torch.randn(3000, 256, device="cuda")
    bias = torch.randn(256) * 0.05
    a = route(wst, x, 8, score="sigmoid", bias=bias, groups=8, top_groups=4, group_best=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = route(wst, x, 8, score="sigmoid", bias=bias, groups=8, top_groups=4, group_best=2)
    s.synchronize()
    assert np.array_equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 7, 7), (50, 60, 6), (40, 256, 8), (5, 1000, 16)])
def test_route_backward(wst, dtype, renorm, score, T, E, k):
    g = torch.Generator().manual_seed(T + E)
    x = (torch.randn(T, E, generator=g) * 1.5).to(dtype)
    x[:, E // 2 + 1:] = -torch.inf if E > 16 else x[:, E // 2 + 1:]
    e, _ = ref.route(ref.f64(x), k, score)
    e[0, -1] = -1 if k > 1 else e[0, -1]        # a slot without an expert
    if T > 2 and k > 1:
        e[1, 1] = e[1, 0]                       # an expert in two slots
        e[2, 0] = 4000                          # an id out of range counts as none
    dw = torch.randn(T, k, generator=g)
    dx = padded(torch.full((T, E), float("nan"), dtype=dtype))
    wst.wst_moe_route_backward(padded(x), torch.from_numpy(e).to(torch.int32).cuda(), dw.cuda(), dx, score=score, renorm=renorm,
                               scale=1.5)
    want, size = ref.route_backward(ref.f64(x), e, ref.f64(dw), score, renorm, 1.5)
    # scores and shares are off by at most 2^-17, the sums over slots by less
    bound = 2.0 ** -16 * size + ref.half(dtype) * abs(want) * 1.01 + 1e-37
    assert (abs(ref.f64(dx) - want) <= bound).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_against_differences(wst, score, renorm):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 12, generator=g).double().numpy()
    dw = torch.randn(2, 4, generator=g)
    e, _ = ref.route(x.astype(np.float32).astype(np.float64), 4, score)
    xs = torch.from_numpy(x).float()
    dx = torch.empty(2, 12, device="cuda")
    wst.wst_moe_route_backward(xs.cuda(), torch.from_numpy(e).int().cuda(), dw.cuda(), dx, score=score, renorm=renorm, scale=0.7)

    def loss(z):
        s = np.take_along_axis(ref.scores(z, score), e, 1)
        return 0.7 * (ref.f64(dw) * (s / s.sum(1, keepdims=True) if renorm else s)).sum()
    z, h = ref.f64(xs), 1e-5
    for t in range(2):
        for j in range(12):
            d = np.zeros_like(z)
            d[t, j] = h
            # central differences in 64 bits: error h^2 + 1e-16 / h, below 1e-9
            assert abs((loss(z + d) - loss(z - d)) / (2 * h) - float(dx[t, j])) < 1e-5


@pytest.mark.parametrize("T,k,E", [(0, 2, 5), (1, 1, 1), (7, 3, 10), (512, 8, 256), (513, 8, 256), (4096, 1, 3), (4097, 1, 3),
                                   (5000, 4, 1024), (40000, 8, 60), (1, 4096, 7), (70000, 5, 1000)])
def test_plan(wst, T, k, E):
    rng = np.random.default_rng(T + E)
    e = rng.integers(0, E, (T, k))
    e[rng.random((T, k)) < 0.1] = -1
    if E > 4:
        e[e == 2] = 3                       # an expert without a row
    _check_plan(wst, e, E)


def _check_plan(wst, e, E, status=0):
    T, k = e.shape
    out = [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((E + 1,), (T * k,), (T * k,), (T, k))]
    ws = wst.moe_plan_workspace(T * k, E)
    wst.wst_moe_plan(torch.from_numpy(e.astype(np.int32)).cuda(), E, *out, workspace=ws)
    assert wst.wst_sync_status(ws) == status
    for got, want in zip(out, ref.plan(e, E)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_plan_one_expert_and_none(wst):
    _check_plan(wst, np.full((3000, 4), 5), 64)
    _check_plan(wst, np.full((3000, 4), -1), 64)


def test_plan_bad_ids_latched(wst):
    e = np.array([[0, 1], [2, 9], [1, -3], [0, 2]])
    _check_plan(wst, e, 3, status=wst.WST_ERR_INVALID_ARG)


def _rows_case(T, k, N, dtype, seed, drop=0.2):
    rng = np.random.default_rng(seed)
    _, _, _, pos = ref.plan(np.where(rng.random((T, k)) < drop, -1, rng.integers(0, 9, (T, k))), 9)
    rows = int(pos.max()) + 1 if pos.size else 0
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, N, generator=g).to(dtype), pos, torch.randn(T, k, generator=g)


SIZES = [(1, 1, 8), (1, 2, 1), (3, 5, 37), (40, 4, 256), (17, 8, 1531), (9, 10, 2048), (5, 32, 4104), (300, 2, 96)]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,N", SIZES)
def test_combine(wst, T, k, N, dtype, out_dtype):
    y, pos, w = _rows_case(T, k, N, dtype, T + k + N)
    for weights in (w, None):
        out = padded(torch.full((T, N), float("nan"), dtype=out_dtype), 1)
        ws = wst.workspace()
        wst.wst_moe_combine(padded(y, 2), torch.from_numpy(pos).int().cuda(), out, weights=None if weights is None else w.cuda(),
                            workspace=ws)
        assert wst.wst_sync_status(ws) == 0
        want, size = ref.combine(ref.f64(y), pos, ref.f64(w) if weights is not None else np.ones((T, k)))
        # k roundings of a fused multiply and add, one of the output
        assert (abs(ref.f64(out) - want) <= k * ref.U * size * 1.01 + ref.half(out_dtype) * (abs(want) + k * ref.U * size)).all()
        assert torch.isnan(out._base[:, N:].float()).all()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,N", SIZES)
def test_combine_backward(wst, T, k, N, dtype, out_dtype):
    y, pos, w = _rows_case(T, k, N, dtype, T + k + N)
    dout = torch.randn(T, N, generator=torch.Generator().manual_seed(9)).to(out_dtype)
    rows = y.shape[0]
    dy = padded(torch.full((rows + 3, N), float("nan"), dtype=dtype), 1)
    dw = torch.full((T, k), float("nan"), device="cuda")
    yy = padded(torch.cat([y, torch.zeros(3, N, dtype=dtype)]))
    ws = wst.workspace()
    wst.wst_moe_combine_backward(padded(dout), torch.from_numpy(pos).int().cuda(), y=yy, weights=w.cuda(), dy=dy, dweights=dw,
                                 workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    d, yv, wv = ref.f64(dout), ref.f64(y), ref.f64(w)
    want = np.full((rows + 3, N), np.nan)
    want_w, size_w = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for i in range(k):
            if pos[t, i] >= 0:
                want[pos[t, i]] = wv[t, i] * d[t]
                want_w[t, i], size_w[t, i] = (d[t] * yv[pos[t, i]]).sum(), abs(d[t] * yv[pos[t, i]]).sum()
    got = ref.f64(dy)
    assert np.isnan(got[rows:]).all()                  # rows that no pair names are left as they were
    assert (abs(got[:rows] - want[:rows]) <= (ref.U + ref.half(dtype)) * 1.01 * abs(want[:rows])).all()
    assert torch.isnan(dy._base[:, N:].float()).all()
    # a thread adds at most 8 ceil(N / 256) products (N / 8 threads up to 256 share a token), then 5 + 8 sums
    assert (abs(ref.f64(dw) - want_w) <= (8 * -(-N // 256) + 14) * ref.U * size_w).all()
    # either alone, and without weights
    dw2 = torch.empty_like(dw)
    wst.wst_moe_combine_backward(padded(dout), torch.from_numpy(pos).int().cuda(), y=yy, dweights=dw2, workspace=ws)
    assert torch.equal(dw, dw2)
    dy2 = padded(torch.full((rows + 3, N), float("nan"), dtype=dtype), 1)
    wst.wst_moe_combine_backward(padded(dout), torch.from_numpy(pos).int().cuda(), dy=dy2, workspace=ws)
    live = pos >= 0
    assert np.array_equal(ref.f64(dy2)[pos[live]], d[np.nonzero(live)[0]].astype(np.float32).astype(np.float64)
                          if dtype == torch.float32 else ref.f64(dout.to(dtype))[np.nonzero(live)[0]])


def test_combine_bad_positions_latched(wst):
    y = torch.ones(4, 16, device="cuda")
    pos = torch.tensor([[0, 4], [3, -5]], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 16, device="cuda")
    ws = wst.workspace()
    wst.wst_moe_combine(y, pos, out, workspace=ws)
    assert wst.wst_sync_status(ws) == wst.WST_ERR_INVALID_ARG
    assert (out == 1).all()                             # what is in range is added
    dy, dw = torch.zeros(4, 16, device="cuda"), torch.full((2, 2), 7.0, device="cuda")
    wst.wst_moe_combine_backward(out, pos, y=y, dy=dy, dweights=dw, workspace=ws)
    assert wst.wst_sync_status(ws) == wst.WST_ERR_INVALID_ARG
    assert dw.tolist() == [[16.0, 0.0], [16.0, 0.0]] and dy[1:3].abs().sum() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q_dtype", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("mode", ["rows", "cols", "blocks", "blocks_t"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (128, 1), (7, 130), (128, 256), (129, 255), (300, 1000)])
def test_quantise(wst, M, K, mode, dtype, q_dtype, pow2):
    g = torch.Generator().manual_seed(M + K)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-20, 12, (M, 1), generator=g).float())
    x[M // 2] = 0.0                                    # blocks of zeros
    x[:, K // 3] = 1.75 * 2.0 ** 9                     # exactly the border of a power of two
    _check_quantise(wst, x.to(dtype), mode, q_dtype, pow2)


def _check_quantise(wst, x, mode, q_dtype, pow2):
    want_q, want_s = ref.quantise(x, mode, q_dtype, pow2)
    q = torch.full((want_q.shape[0], -(-want_q.shape[1] // 16) * 16 + 16), 0.5).to(q_dtype).cuda()
    s = torch.full((want_s.shape[0], want_s.shape[1] + 3), -1.0, device="cuda")
    wst.wst_quantize_fp8(padded(x), q[:, :want_q.shape[1]], s[:, :want_s.shape[1]], mode=mode, pow2=pow2)
    assert np.array_equal(s[:, :want_s.shape[1]].cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(ref.f64(q[:, :want_q.shape[1]]), ref.f64(want_q), equal_nan=True)
    assert (q[:, want_q.shape[1]:].float() == 0.5).all() and (s[:, want_s.shape[1]:] == -1).all()


@pytest.mark.parametrize("mode", ["rows", "cols", "blocks", "blocks_t"])
def test_quantise_not_finite_and_tiny(wst, mode):
    x = torch.randn(300, 300, generator=torch.Generator().manual_seed(1))
    x[5, 7], x[200, 5], x[140, 290] = torch.nan, torch.inf, -torch.inf
    _check_quantise(wst, x, mode, torch.float8_e4m3fn, False)
    x = torch.randn(40, 200, generator=torch.Generator().manual_seed(2)) * 2.0 ** -110   # below the floor of a block's largest
    _check_quantise(wst, x, mode, torch.float8_e4m3fn, False)
    _check_quantise(wst, x, mode, torch.float8_e5m2, True)


@pytest.mark.parametrize("q_dtype,smallest", [(torch.float8_e4m3fn, 2.0 ** -9), (torch.float8_e5m2, 2.0 ** -16)])
def test_quantise_half_a_step(wst, q_dtype, smallest):
    x = torch.randn(256, 512, generator=torch.Generator().manual_seed(4)).cuda()
    q, s = torch.empty(256, 512, dtype=q_dtype, device="cuda"), torch.empty(4, 256, device="cuda")
    wst.wst_quantize_fp8(x, q, s)
    back = ref.values(q, s.cpu().numpy(), "rows")
    step = np.maximum(ref.half(q_dtype) * abs(ref.f64(x)), 0.5 * smallest * np.repeat(ref.f64(s).T, 128, axis=1))
    # three roundings in fp32 before the one to 8 bits
    assert (abs(back - ref.f64(x)) <= step * (1 + 2.0 ** -10)).all()


def test_quantise_batch(wst):
    x = torch.randn(3, 70, 200, generator=torch.Generator().manual_seed(8)).bfloat16()
    for mode in ("rows", "cols", "blocks", "blocks_t"):
        ref_q = [ref.quantise(x[i], mode, torch.float8_e4m3fn) for i in range(3)]
        qs, ss = ref_q[0][0].shape, ref_q[0][1].shape
        q = torch.empty(3, qs[0], -(-qs[1] // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")[..., :qs[1]]
        s = torch.empty(3, *ss, device="cuda")
        wst.wst_quantize_fp8(x.cuda(), q, s, mode=mode)
        for i in range(3):
            assert np.array_equal(ref.f64(q[i]), ref.f64(ref_q[i][0])) and np.array_equal(s[i].cpu().numpy(), ref_q[i][1])


@pytest.mark.parametrize("T,k,K", [(1, 1, 16), (5, 3, 200), (40, 8, 513), (300, 2, 1024)])
def test_quantise_dispatch(wst, T, k, K):
    rng = np.random.default_rng(T)
    _, _, row_token, pos = ref.plan(np.where(rng.random((T, k)) < 0.2, -1, rng.integers(0, 9, (T, k))), 9)
    rows = int((row_token >= 0).sum())
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).bfloat16()
    q = torch.full((rows + 2, -(-K // 16) * 16), 0.5).to(torch.float8_e4m3fn).cuda()[:, :K]
    s = torch.full((-(-K // 128), rows + 2), -1.0, device="cuda")
    ws = wst.workspace()
    wst.wst_quantize_fp8_dispatch(padded(x), torch.from_numpy(pos).int().cuda(), q, s, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    want_q, want_s = ref.quantise(x, "rows", torch.float8_e4m3fn)
    token = row_token[:rows]
    assert np.array_equal(ref.f64(q)[:rows], ref.f64(want_q)[token]) and np.array_equal(s.cpu().numpy()[:, :rows], want_s[:, token])
    assert (q[rows:].float() == 0.5).all() and (s[:, rows:] == -1).all()
    bad = torch.full((T, k), rows + 2, dtype=torch.int32, device="cuda")
    wst.wst_quantize_fp8_dispatch(padded(x), bad, q, s, workspace=ws)
    assert wst.wst_sync_status(ws) == wst.WST_ERR_INVALID_ARG


@pytest.mark.parametrize("K", [64, 256])
def test_quantise_dispatch_to_no_rows(wst, K):
    # a batch of which no token has an expert
    x, ws = torch.randn(5, K, device="cuda"), wst.workspace()
    q, s = torch.empty(0, K, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(-(-K // 128), 0, device="cuda")
    wst.wst_quantize_fp8_dispatch(x, torch.full((5, 2), -1, dtype=torch.int32, device="cuda"), q, s, workspace=ws)
    assert wst.wst_sync_status(ws) == 0
    wst.wst_quantize_fp8_dispatch(x, torch.zeros(5, 2, dtype=torch.int32, device="cuda"), q, s, workspace=ws)
    assert wst.wst_sync_status(ws) == wst.WST_ERR_INVALID_ARG        # a row that is not there


def test_combine_backward_to_no_rows(wst):
    # a batch of which no token has an expert
    ws, dout, dy = wst.workspace(), torch.randn(5, 32, device="cuda"), torch.empty(0, 32, device="cuda")
    none = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    wst.wst_moe_combine_backward(dout, none, dy=dy, workspace=ws)
    dw = torch.full((5, 2), 3.0, device="cuda")
    wst.wst_moe_combine_backward(dout, none, y=torch.empty(0, 32, device="cuda"), dy=dy, dweights=dw, workspace=ws)
    assert wst.wst_sync_status(ws) == 0 and (dw == 0).all()
    wst.wst_moe_combine_backward(dout, torch.zeros_like(none), dy=dy, workspace=ws)
    assert wst.wst_sync_status(ws) == wst.WST_ERR_INVALID_ARG        # a row that is not there


@pytest.mark.parametrize("lead", [(), (2,)])
@pytest.mark.parametrize("mode", ["rows", "cols", "blocks", "blocks_t"])
def test_quantise_no_rows(wst, mode, lead):
    q = {"rows": (0, 256), "cols": (256, 0), "blocks": (0, 256), "blocks_t": (256, 0)}[mode]
    s = {"rows": (2, 0), "cols": (0, 256), "blocks": (0, 2), "blocks_t": (2, 0)}[mode]
    wst.wst_quantize_fp8(torch.empty(*lead, 0, 256, device="cuda"), torch.empty(*lead, *q, dtype=torch.float8_e4m3fn, device="cuda"),
                         torch.empty(*lead, *s, device="cuda"), mode=mode)
    with pytest.raises(wst.WstError):
        wst.wst_quantize_fp8(torch.empty(4, 0, device="cuda"), torch.empty(4, 0, dtype=torch.float8_e4m3fn, device="cuda"),
                             torch.empty(0, 4, device="cuda"))       # blocks of no column


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_into_the_logits(wst, score, renorm, dtype):
    g = torch.Generator().manual_seed(6)
    x = torch.randn(300, 40, generator=g).to(dtype).cuda()
    e = torch.stack([torch.randperm(40, generator=g)[:4] for _ in range(300)]).int().cuda()
    dw, want = torch.randn(300, 4, generator=g).cuda(), torch.empty(300, 40, dtype=dtype, device="cuda")
    wst.wst_moe_route_backward(x, e, dw, want, score=score, renorm=renorm)
    wst.wst_moe_route_backward(x, e, dw, x, score=score, renorm=renorm)
    assert torch.equal(x, want)


def test_rows_behind_32_bits(wst):
    # y, dy and the rows of a dispatch whose last elements lie more than 2^31 elements in
    rows, N, T = 530000, 4096, 3
    ws = wst.workspace()
    y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    y[-2:] = torch.randn(2, N, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    pos = torch.tensor([[rows - 1, 5], [-1, rows - 2], [7, 9]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 1.0], [1.0, 2.0], [1.0, 1.0]], device="cuda")
    out = torch.empty(T, N, device="cuda")
    wst.wst_moe_combine(y, pos, out, weights=w, workspace=ws)
    assert torch.equal(out, torch.stack([0.5 * y[-1].float(), 2 * y[-2].float(), torch.zeros(N, device="cuda")]))
    dout, dw = torch.randn(T, N, generator=torch.Generator().manual_seed(3)).bfloat16().cuda(), torch.empty(T, 2, device="cuda")
    want = (dout[0].double() * y[-1].double()).sum()
    dy = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    wst.wst_moe_combine_backward(dout, pos, y=y, weights=w, dy=dy, dweights=dw, workspace=ws)
    # at most 8 ceil(N / 256) products a thread, then 5 + 8 sums
    assert abs(float(dw[0, 0]) - float(want)) <= (8 * 16 + 14) * ref.U * float((dout[0].double() * y[-1].double()).abs().sum())
    assert torch.equal(dy[-1], (0.5 * dout[0].float()).bfloat16()) and torch.equal(dy[-2], (2 * dout[1].float()).bfloat16())
    assert torch.equal(dy[9], dout[2]) and (dy[10:1000] == 0).all()
    del y, dy
    q, s = torch.zeros(rows, N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), torch.zeros(32, rows, device="cuda")
    wst.wst_quantize_fp8_dispatch(dout, pos, q, s, workspace=ws)
    want_q, want_s = ref.quantise(dout.cpu(), "rows", torch.float8_e4m3fn)
    assert np.array_equal(ref.f64(q[-2:]), ref.f64(want_q)[[1, 0]]) and np.array_equal(s[:, -2:].cpu().numpy(), want_s[:, [1, 0]])
    assert wst.wst_sync_status(ws) == 0
