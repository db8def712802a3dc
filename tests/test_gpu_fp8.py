"""GPU: 8-bit products with block scales, dense and grouped, against the 64-bit
product of the numbers that the 8-bit values and their scales stand for."""
import numpy as np
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


@pytest.fixture(scope="module")
def wst():
    import warp_specialized_tensor_gb300 as w
    w.load_library()
    return w


@pytest.fixture(scope="module")
def big_ws(wst):
    return wst.gemm_fp8_workspace()


def rows16(t):
    """t on the GPU in rows that begin on 16 bytes, the bits 0x7f (a NaN in 8 bits) behind them."""
    per = 16 // t.element_size()
    buf = torch.full((*t.shape[:-1], (-(-t.shape[-1] // per) + 1) * per * t.element_size()), 0x7f, dtype=torch.uint8, device="cuda")
    out = buf.view(t.dtype)[..., :t.shape[-1]]
    out.copy_(t)
    return out


def operand(M, K, mode, dtype, seed, lead=()):
    """Random 8-bit values and scales of very different sizes."""
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(*lead, M, K, generator=g) * 40).clamp(-440, 440).to(dtype)
    shape = (-(-K // 128), M) if mode == "rows" else (-(-M // 128), -(-K // 128))
    s = torch.exp2(torch.randn(*lead, *shape, generator=g) * 2) * 0.01
    return q, s


def product(qa, sa, qb, sb, scaling):
    a, b = ref.values(qa, sa, "rows"), ref.values(qb, sb, scaling)
    return a @ b.T, abs(a) @ abs(b).T


def bound(want, size, K, out_dtype):
    # 128 sums of a block in the tensor core, each cut off at one unit of the
    # sum (2u), three roundings for the scales and the sum of the blocks
    err = (128 * 2 + -(-K // 128) + 3) * ref.U * size
    return err + ref.half(out_dtype) * (abs(want) + err)


def out_buffer(M, N, dtype):
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.full((M + 2, (-(-N // per) + 1) * per), float("nan"), dtype=dtype, device="cuda")


SIZES = [(1, 1, 1), (1, 128, 128), (3, 256, 130), (16, 300, 1024), (17, 64, 4096), (33, 4096, 512), (128, 128, 16), (129, 129, 129),
         (256, 256, 256), (257, 500, 1000), (300, 700, 2100), (1030, 513, 640)]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("scaling", ["blocks", "rows"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_dense(wst, big_ws, M, N, K, scaling, split):
    qa, sa = operand(M, K, "rows", E4, 1)
    qb, sb = operand(N, K, scaling, E4, 2)
    ws = big_ws if split else wst.workspace()
    want, size = product(qa, sa, qb, sb, scaling)
    for dtype in (torch.float32, torch.bfloat16):
        buf = out_buffer(M, N, dtype)
        wst.wst_gemm_fp8(rows16(qa), sa.cuda(), rows16(qb), sb.cuda(), buf[:M, :N], scaling=scaling, workspace=ws)
        assert wst.wst_sync_status(ws) == 0
        assert (abs(ref.f64(buf[:M, :N]) - want) <= bound(want, size, K, dtype)).all()
        assert torch.isnan(buf[M:].float()).all() and torch.isnan(buf[:, N:].float()).all()


@pytest.mark.parametrize("ta,tb", [(E4, E5), (E5, E4), (E5, E5)])
def test_types(wst, big_ws, ta, tb):
    qa, sa = operand(70, 500, "rows", ta, 3)
    qb, sb = operand(200, 500, "blocks", tb, 4)
    want, size = product(qa, sa, qb, sb, "blocks")
    C = torch.empty(70, 200, device="cuda")
    wst.wst_gemm_fp8(rows16(qa), sa.cuda(), rows16(qb), sb.cuda(), C, workspace=big_ws)
    assert (abs(ref.f64(C) - want) <= bound(want, size, 500, torch.float32)).all()


@pytest.mark.parametrize("M,N,K", [(5, 300, 2048), (200, 260, 384)])
def test_whole_numbers_are_exact(wst, big_ws, M, N, K):
    # small whole numbers and scales that are powers of two: every partial sum is exact
    g = torch.Generator().manual_seed(M)
    qa, qb = torch.randint(-8, 9, (M, K), generator=g).to(E4), torch.randint(-8, 9, (N, K), generator=g).to(E4)
    sa = torch.exp2(torch.randint(0, 3, (-(-K // 128), M), generator=g).float())
    sb = torch.exp2(torch.randint(0, 3, (-(-N // 128), -(-K // 128)), generator=g).float())
    C = torch.empty(M, N, device="cuda")
    wst.wst_gemm_fp8(rows16(qa), sa.cuda(), rows16(qb), sb.cuda(), C, workspace=big_ws)
    assert np.array_equal(ref.f64(C), product(qa, sa, qb, sb, "blocks")[0])


@pytest.mark.parametrize("epi", ["bias", "bias_silu", "bias_gelu"])
def test_epilogues(wst, big_ws, epi):
    M, N, K = 37, 200, 384
    qa, sa = operand(M, K, "rows", E4, 5)
    qb, sb = operand(N, K, "blocks", E4, 6)
    sa, sb = sa * 0.1, sb * 0.1
    bias = torch.randn(N, generator=torch.Generator().manual_seed(1)).bfloat16()
    want, size = product(qa, sa, qb, sb, "blocks")
    x = want + ref.f64(bias)
    t = torch.from_numpy(x)
    y = {"bias": t, "bias_silu": t * torch.sigmoid(t), "bias_gelu": t * torch.special.ndtr(t)}[epi].numpy()
    C = torch.empty(M, N, device="cuda")
    wst.wst_gemm_fp8(rows16(qa), sa.cuda(), rows16(qb), sb.cuda(), C, bias=bias.cuda(), epi=epi, workspace=big_ws)
    # slopes are below 1.13; the approximate tanh behind SiLU is off by 2^-11, its half by 2^-12 of |x|
    tol = 1.13 * (bound(want, size, K, torch.float32) + ref.U * abs(x)) + abs(x) * (2.0 ** -12 if epi == "bias_silu" else 2.0 ** -21)
    assert (abs(ref.f64(C) - y) <= tol).all()


GROUPS = [[5], [0, 200, 0, 0, 77, 0], [513, 0], [1, 1, 1, 1, 127, 129, 128, 256], [0, 0, 0, 130], [16, 16, 300, 15, 17]]


@pytest.mark.parametrize("scaling", ["blocks", "rows"])
@pytest.mark.parametrize("sizes", GROUPS)
def test_grouped(wst, big_ws, sizes, scaling):
    N, K, G = 300, 400, len(sizes)
    off = np.concatenate([[0], np.cumsum(sizes)])
    M = int(off[-1]) + 7                                   # rows behind the last group
    qa, sa = operand(M, K, "rows", E4, 7)
    qb, sb = operand(N, K, scaling, E4, 8, (G,))
    bias = torch.randn(G, N).bfloat16()
    for dtype, ws, epi in ((torch.float32, big_ws, "none"), (torch.bfloat16, wst.workspace(), "bias")):
        buf = out_buffer(M, N, dtype)
        wst.wst_grouped_gemm_fp8(rows16(qa), sa.cuda(), rows16(qb), sb.cuda(), torch.from_numpy(off).int().cuda(), buf[:M, :N],
                                 scaling=scaling, bias=bias.cuda(), epi=epi, workspace=ws)
        assert wst.wst_sync_status(ws) == 0
        for g in range(G):
            r = slice(off[g], off[g + 1])
            want, size = product(qa[r], sa[:, r], qb[g], sb[g], scaling)
            err = bound(want, size, K, dtype)
            if epi == "bias":
                want = want + ref.f64(bias[g])
                err = err + ref.half(dtype) * abs(ref.f64(bias[g])) + ref.U * abs(want)
            assert (abs(ref.f64(buf[r, :N]) - want) <= err).all()
        assert torch.isnan(buf[off[-1]:].float()).all() and torch.isnan(buf[:, N:].float()).all()


def test_grouped_many_groups(wst, big_ws):
    rng = np.random.default_rng(1)
    sizes = rng.integers(0, 30, 300)
    sizes[rng.choice(300, 100, replace=False)] = 0
    off = np.concatenate([[0], np.cumsum(sizes)])
    M, N, K = int(off[-1]), 128, 256
    qa, sa = operand(M, K, "rows", E4, 9)
    qb, sb = operand(N, K, "blocks", E4, 10, (300,))
    C = torch.full((M, N), float("nan"), device="cuda")
    wst.wst_grouped_gemm_fp8(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), torch.from_numpy(off).int().cuda(), C, workspace=big_ws)
    assert wst.wst_sync_status(big_ws) == 0
    for g in range(300):
        r = slice(off[g], off[g + 1])
        want, size = product(qa[r], sa[:, r], qb[g], sb[g], "blocks")
        assert (abs(ref.f64(C[r]) - want) <= bound(want, size, K, torch.float32)).all()


def test_grouped_bad_offsets_latched(wst, big_ws):
    qa, sa = operand(300, 128, "rows", E4, 11)
    qb, sb = operand(256, 128, "blocks", E4, 12, (3,))
    buf = out_buffer(300, 256, torch.bfloat16)
    off = torch.tensor([0, 250, 120, 300], dtype=torch.int32, device="cuda")
    wst.wst_grouped_gemm_fp8(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), off, buf[:300, :256], workspace=big_ws)
    assert wst.wst_sync_status(big_ws) == wst.WST_ERR_BAD_OFFSETS
    assert torch.isnan(buf[300:].float()).all()


def test_nan_rows_stay_their_own(wst, big_ws):
    # a NaN scale or value shows in its row only, also inside a shared token tile
    qa, sa = operand(20, 256, "rows", E4, 13)
    qb, sb = operand(128, 256, "blocks", E4, 14)
    sa[1, 3] = torch.nan
    u = qa.view(torch.uint8)
    u[7, 9] = 0x7f
    C = torch.empty(20, 128, device="cuda")
    wst.wst_gemm_fp8(qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), C, workspace=big_ws)
    nan = torch.isnan(C).all(1).cpu()
    assert nan.nonzero().ravel().tolist() == [3, 7] and not torch.isnan(C[~nan]).any()


def test_replayed_graphs_share_a_workspace(wst, big_ws):
    # two captured split products with one workspace, replayed in turn, and the same bits every time
    cases = []
    for seed, (M, N, K) in enumerate([(16, 512, 4096), (7, 1024, 2048)]):
        qa, sa = operand(M, K, "rows", E4, 20 + seed)
        qb, sb = operand(N, K, "blocks", E4, 30 + seed)
        args = (qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), torch.empty(M, N, device="cuda"))
        wst.wst_gemm_fp8(*args, workspace=big_ws)
        first = args[4].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            wst.wst_gemm_fp8(*args, workspace=big_ws)
        cases.append((graph, args, first))  # (the graph reads the inputs where they are)
    for _ in range(20):
        for graph, (*_, out), first in cases:
            out.fill_(float("nan"))
            graph.replay()
            assert torch.equal(out, first)
    assert wst.wst_sync_status(big_ws) == 0


def test_two_streams_with_their_own_workspaces(wst):
    # split products on two streams at once, each with a workspace of its own
    cases = []
    for seed, (M, N, K) in enumerate([(16, 1024, 4096), (9, 768, 8192)]):
        qa, sa = operand(M, K, "rows", E4, 40 + seed)
        qb, sb = operand(N, K, "blocks", E4, 50 + seed)
        ws = wst.gemm_fp8_workspace()
        args = (qa.cuda(), sa.cuda(), qb.cuda(), sb.cuda(), torch.empty(M, N, device="cuda"))
        wst.wst_gemm_fp8(*args, workspace=ws)
        cases.append((args, ws, args[4].clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(30):
        for args, ws, _, stream in cases:
            wst.wst_gemm_fp8(*args, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for args, ws, first, stream in cases:
        assert wst.wst_sync_status(ws, stream) == 0 and torch.equal(args[4], first)


def test_training_products(wst, big_ws):
    # forward, gradient of the inputs and of the weights, each by quantise and product
    g = torch.Generator().manual_seed(3)
    X, W, dY = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((200, 320), (256, 320), (200, 256)))

    def quant(x, mode, dtype=E4):
        r, c = x.shape if mode in ("rows", "blocks") else x.shape[::-1]
        q = torch.empty(r, -(-c // 16) * 16, dtype=dtype, device="cuda")[:, :c]
        kb, rb = -(-c // 128), -(-r // 128)
        s = torch.empty(*((kb, r) if mode in ("rows", "cols") else (rb, kb)), device="cuda")
        wst.wst_quantize_fp8(x, q, s, mode=mode)
        return q, s

    for (a, ma), (b, mb), scaling in (((X, "rows"), (W, "blocks"), "blocks"), ((dY, "rows"), (W, "blocks_t"), "blocks"),
                                      ((dY, "cols"), (X, "cols"), "rows")):
        (qa, sa), (qb, sb) = quant(a, ma, E5 if a is dY else E4), quant(b, mb)
        C = torch.empty(qa.shape[0], qb.shape[0], device="cuda")
        wst.wst_gemm_fp8(qa, sa, qb, sb, C, scaling=scaling, workspace=big_ws)
        want, size = product(qa, sa.cpu(), qb, sb.cpu(), scaling)
        assert (abs(ref.f64(C) - want) <= bound(want, size, qa.shape[1], torch.float32)).all()
        # against the unquantised product: half a step of each operand's 8 bits, value by value
        va = ref.f64(a) if ma == "rows" else ref.f64(a).T
        vb = ref.f64(b) if mb in ("rows", "blocks") else ref.f64(b).T
        half = ref.half(qa.dtype) + ref.half(E4)
        full = abs(va) @ abs(vb).T
        assert (abs(ref.f64(C) - va @ vb.T) <= half * 1.1 * full + 2.0 ** -8 * full).all()


@pytest.mark.parametrize("K", [384, 130, 640, 900])
def test_odd_numbers_of_blocks_are_exact(wst, K):
    # Many units a pair, each of an odd number of K blocks (three at 384): whole
    # numbers and scales that are powers of two, so that every bit counts.
    M, N = 4096, 4100
    g = torch.Generator().manual_seed(K)
    qa, qb = torch.randint(-8, 9, (M, K), generator=g), torch.randint(-8, 9, (N, K), generator=g)
    sa = torch.exp2(torch.randint(0, 3, (-(-K // 128), M), generator=g).float())
    sb = torch.exp2(torch.randint(0, 3, (-(-N // 128), -(-K // 128)), generator=g).float())
    va, vb = torch.from_numpy(ref.values(qa, sa, "rows")).cuda(), torch.from_numpy(ref.values(qb, sb, "blocks")).cuda()
    want = (va @ vb.T).float()
    A, B, C = rows16(qa.to(E4)), rows16(qb.to(E4)), torch.empty(M, N, device="cuda")
    for _ in range(10):
        C.fill_(float("nan"))
        wst.wst_gemm_fp8(A, sa.cuda(), B, sb.cuda(), C, workspace=wst.workspace())
        assert torch.equal(C, want)


def test_bad_offsets_of_split_products(wst, big_ws):
    # Overlapping groups: more units of a split loop than pairs; clamped, latched,
    # and the workspace is as good as before.
    G, M, N, K = 60, 2, 256, 2048
    qa, sa = operand(M, K, "rows", E4, 60)
    qb, sb = operand(N, K, "blocks", E4, 61, (G,))
    C = torch.zeros(M, N, device="cuda")
    off = torch.tensor([0, 2] * 30 + [0], dtype=torch.int32, device="cuda")
    args = (rows16(qa), sa.cuda(), rows16(qb), sb.cuda())
    wst.wst_grouped_gemm_fp8(*args, off, C, workspace=big_ws)
    assert wst.wst_sync_status(big_ws) == wst.WST_ERR_BAD_OFFSETS
    off = torch.tensor([0, 1] + [1] * 58 + [2], dtype=torch.int32, device="cuda")
    wst.wst_grouped_gemm_fp8(*args, off, C, workspace=big_ws)
    assert wst.wst_sync_status(big_ws) == 0
    for row, g in ((0, 0), (1, G - 1)):
        want, size = product(qa[row:row + 1], sa[:, row:row + 1], qb[g], sb[g], "blocks")
        assert (abs(ref.f64(C[row:row + 1]) - want) <= bound(want, size, K, torch.float32)).all()


# Sizes whose K loops are split (tests/test_fp8_schedule_host.py holds the rule
# to that): one token tile and several, at most 64 tokens and more, ragged ends.
SPLIT_DENSE = [(7, 1030, 1800), (64, 512, 4096), (65, 520, 2100), (128, 1024, 8192), (200, 300, 4096), (300, 512, 4096),
               (520, 260, 8197)]
SPLIT_GROUPED = [([5, 0, 130, 0, 17], 300, 4096), ([300, 0, 70], 260, 4000), ([0, 16, 0, 33, 1, 0], 700, 2560), ([257], 128, 6000)]


def activated(x, epi):
    t = torch.from_numpy(x)
    return {"none": t, "bias": t, "bias_silu": t * torch.sigmoid(t), "bias_gelu": t * torch.special.ndtr(t)}[epi].numpy()


def activated_bound(x, err, y, epi, dtype):
    # slopes are below 1.13; the approximate tanh behind SiLU is off by 2^-11, its half by 2^-12 of |x|
    tol = 1.13 * (err + ref.U * abs(x)) + abs(x) * {"none": 0.0, "bias": 0.0, "bias_silu": 2.0 ** -12, "bias_gelu": 2.0 ** -21}[epi]
    return tol + ref.half(dtype) * (abs(y) + tol)


@pytest.mark.parametrize("scaling", ["blocks", "rows"])
@pytest.mark.parametrize("M,N,K", SPLIT_DENSE)
def test_split_dense(wst, big_ws, M, N, K, scaling):
    qa, sa = operand(M, K, "rows", E4, 70)
    qb, sb = operand(N, K, scaling, E4, 71)
    sb = sb * 0.01
    want, size = product(qa, sa, qb, sb, scaling)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(2)).bfloat16()
    args = (rows16(qa), sa.cuda(), rows16(qb), sb.cuda())
    for dtype in (torch.float32, torch.bfloat16):
        for epi in ("none", "bias", "bias_silu", "bias_gelu"):
            x = want if epi == "none" else want + ref.f64(bias)
            y = activated(x, epi)
            tol = activated_bound(x, bound(want, size, K, torch.float32), y, epi, dtype)
            buf = out_buffer(M, N, dtype)
            outs = []
            for _ in range(2):
                buf[:M, :N] = float("nan")
                wst.wst_gemm_fp8(*args, buf[:M, :N], scaling=scaling, bias=bias.cuda(), epi=epi, workspace=big_ws)
                outs.append(buf[:M, :N].clone())
            assert wst.wst_sync_status(big_ws) == 0
            assert torch.equal(*outs)
            assert (abs(ref.f64(outs[0]) - y) <= tol).all()
            assert torch.isnan(buf[M:].float()).all() and torch.isnan(buf[:, N:].float()).all()


@pytest.mark.parametrize("scaling", ["blocks", "rows"])
@pytest.mark.parametrize("sizes,N,K", SPLIT_GROUPED)
def test_split_grouped(wst, big_ws, sizes, N, K, scaling):
    G, off = len(sizes), np.concatenate([[0], np.cumsum(sizes)])
    M = int(off[-1]) + 7                                   # rows behind the last group
    qa, sa = operand(M, K, "rows", E4, 72)
    qb, sb = operand(N, K, scaling, E4, 73, (G,))
    sb = sb * 0.01
    bias = torch.randn(G, N, generator=torch.Generator().manual_seed(3)).bfloat16()
    args = (rows16(qa), sa.cuda(), rows16(qb), sb.cuda(), torch.from_numpy(off).int().cuda())
    for dtype in (torch.float32, torch.bfloat16):
        for epi in ("none", "bias", "bias_silu", "bias_gelu"):
            buf = out_buffer(M, N, dtype)
            wst.wst_grouped_gemm_fp8(*args, buf[:M, :N], scaling=scaling, bias=bias.cuda(), epi=epi, workspace=big_ws)
            assert wst.wst_sync_status(big_ws) == 0
            for g in range(G):
                r = slice(off[g], off[g + 1])
                want, size = product(qa[r], sa[:, r], qb[g], sb[g], scaling)
                x = want if epi == "none" else want + ref.f64(bias[g])
                y = activated(x, epi)
                tol = activated_bound(x, bound(want, size, K, torch.float32), y, epi, dtype)
                assert (abs(ref.f64(buf[r, :N]) - y) <= tol).all()
            assert torch.isnan(buf[off[-1]:].float()).all() and torch.isnan(buf[:, N:].float()).all()


def test_split_exact_and_in_graphs(wst, big_ws):
    # whole numbers, several token tiles: every bit, eagerly and replayed
    M, N, K = 300, 512, 4096
    g = torch.Generator().manual_seed(9)
    qa, qb = torch.randint(-8, 9, (M, K), generator=g), torch.randint(-8, 9, (N, K), generator=g)
    sa, sb = torch.ones(32, M), torch.full((4, 32), 0.5)
    want = torch.from_numpy((qa.double() @ qb.double().T * 0.5).numpy()).float()
    args = (qa.to(E4).cuda(), sa.cuda(), qb.to(E4).cuda(), sb.cuda(), torch.empty(M, N, device="cuda"))
    wst.wst_gemm_fp8(*args, workspace=big_ws)
    assert torch.equal(args[4].cpu(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wst.wst_gemm_fp8(*args, workspace=big_ws)
    for _ in range(5):
        args[4].fill_(float("nan"))
        graph.replay()
        assert torch.equal(args[4].cpu(), want)
    assert wst.wst_sync_status(big_ws) == 0


@pytest.mark.parametrize("N,K", [(1, 100), (3, 200)])
def test_one_group_whatever_its_stride(wst, big_ws, N, K):
    qa, sa = operand(9, K, "rows", E4, 80)
    qb, sb = operand(N, K, "blocks", E4, 81, (1,))
    store = torch.zeros(N * 208 + 100, dtype=torch.uint8, device="cuda").view(E4)
    B = store.as_strided((1, N, K), (100, 208, 1))           # a group stride of no multiple of 16 bytes
    B.copy_(qb)
    C = torch.full((9, 4), float("nan"), device="cuda")
    off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    wst.wst_grouped_gemm_fp8(rows16(qa), sa.cuda(), B, sb.cuda(), off, C[:, :N], workspace=big_ws)
    want, size = product(qa, sa, qb[0], sb[0], "blocks")
    assert (abs(ref.f64(C[:, :N]) - want) <= bound(want, size, K, torch.float32)).all()


@pytest.mark.parametrize("scaling", ["blocks", "rows"])
def test_groups_that_share_their_weights(wst, big_ws, scaling):
    # group strides of 0, and scales in rows of a larger array
    sizes, N, K = [20, 0, 300, 5], 200, 520
    off = np.concatenate([[0], np.cumsum(sizes)])
    M, G = int(off[-1]), len(sizes)
    qa, sa = operand(M, K, "rows", E4, 82)
    qb, sb = operand(N, K, scaling, E4, 83)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(4)).bfloat16()
    wide = [torch.full((t.shape[0], t.shape[1] + 5), float("nan"), device="cuda") for t in (sa, sb)]
    ka, kb = wide[0][:, :M], wide[1][:, :sb.shape[1]]
    ka.copy_(sa), kb.copy_(sb)
    C = torch.full((M, N), float("nan"), device="cuda")
    wst.wst_grouped_gemm_fp8(rows16(qa), ka, rows16(qb).expand(G, N, K), kb.expand(G, *kb.shape), torch.from_numpy(off).int().cuda(), C,
                             scaling=scaling, bias=bias.cuda().expand(G, N), epi="bias", workspace=big_ws)
    assert wst.wst_sync_status(big_ws) == 0
    want, size = product(qa, sa, qb, sb, scaling)
    err = bound(want, size, K, torch.float32)
    want = want + ref.f64(bias)
    assert (abs(ref.f64(C) - want) <= err + 2 * ref.U * (abs(want) + err)).all()


def test_grouped_rows_behind_32_bits(wst, big_ws):
    # the last group's rows lie more than 2^31 elements into A and C
    sizes, N, K = [529900, 100], 4100, 4096
    M = sum(sizes)
    qa, sa = operand(100, K, "rows", E4, 84)
    qb, sb = operand(N, K, "blocks", E4, 85)
    A = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    A[-100:] = qa.view(torch.uint8).cuda()
    scale = torch.ones(32, M, device="cuda")
    scale[:, -100:] = sa.cuda()
    buf = torch.full((M, 4104), float("nan"), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, sizes[0], M], dtype=torch.int32, device="cuda")
    wst.wst_grouped_gemm_fp8(A.view(E4), scale, rows16(qb).expand(2, N, K), sb.cuda().expand(2, *sb.shape), off, buf[:, :N],
                             workspace=big_ws)
    assert wst.wst_sync_status(big_ws) == 0
    want, size = product(qa, sa, qb, sb, "blocks")
    assert (abs(ref.f64(buf[-100:, :N]) - want) <= bound(want, size, K, torch.bfloat16)).all()
    assert (buf[:-100, :N] == 0).all() and torch.isnan(buf[:, N:].float()).all()
