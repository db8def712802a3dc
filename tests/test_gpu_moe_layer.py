"""GPU: the operators run together, as a mixture-of-experts layer uses them: routing,
plan, rows to experts, grouped product, combine, and all the gradients; in bf16
and in 8 bits, eagerly and as a replayed CUDA graph."""
import numpy as np
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8  # half a step of bf16


@pytest.fixture(scope="module")
def wst():
    import warp_specialized_tensor_gb300 as w
    w.load_library()
    return w


class Layer:
    """Buffers of one layer: T tokens of K features, E experts of N outputs, k per token."""

    def __init__(self, wst, T, E, k, K, N):
        self.wst, self.shape = wst, (T, E, k, K, N)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.experts, self.position = torch.empty(T, k, **i32), torch.empty(T, k, **i32)
        self.weights = torch.empty(T, k, device="cuda")
        self.offsets, self.row_pair, self.row_token = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T * k, **i32)
        self.plan_ws, self.ws, self.ws8 = wst.moe_plan_workspace(T * k, E), wst.workspace(), wst.gemm_fp8_workspace()
        self.rows = torch.empty(T * k, K, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(T * k, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        self.scales = torch.zeros(-(-K // 128), T * k, device="cuda")
        self.y = torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")

    def route(self, logits):
        w = self.wst
        w.wst_moe_route(logits, self.experts, self.weights, score="sigmoid", renorm=True, scale=1.5)
        w.wst_moe_plan(self.experts, self.shape[1], self.offsets, self.row_pair, self.row_token, self.position, workspace=self.plan_ws)

    def forward(self, logits, x, B):
        w = self.wst
        self.route(logits)
        w.wst_permute_rows(x, self.rows, src_index=self.row_token, workspace=self.ws)
        w.wst_grouped_gemm_bf16(self.rows, B, self.offsets, self.y, workspace=self.ws)
        w.wst_moe_combine(self.y, self.position, self.out, weights=self.weights, workspace=self.ws)

    def forward_fp8(self, logits, x, Bq, Bs):
        w = self.wst
        self.route(logits)
        w.wst_quantize_fp8_dispatch(x, self.position, self.q, self.scales, workspace=self.ws)
        w.wst_grouped_gemm_fp8(self.q, self.scales, Bq, Bs, self.offsets, self.y, workspace=self.ws8)
        w.wst_moe_combine(self.y, self.position, self.out, weights=self.weights, workspace=self.ws)

    def status(self):
        return [self.wst.wst_sync_status(s) for s in (self.plan_ws, self.ws, self.ws8)]


def inputs(T, E, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g), torch.randn(T, K, generator=g).bfloat16(),
            (torch.randn(E, N, K, generator=g) * K ** -0.5).bfloat16())


def experts_of(layer, logits, k):
    e, w = ref.route(ref.f64(logits), k, "sigmoid", renorm=True, scale=1.5)
    assert np.array_equal(layer.experts.cpu().numpy(), e)
    return e, w


@pytest.mark.parametrize("T,E,k,K,N", [(1, 8, 2, 128, 96), (50, 8, 2, 256, 384), (333, 16, 3, 200, 264)])
def test_layer_and_its_gradients(wst, T, E, k, K, N):
    logits, x, B = inputs(T, E, K, N, T)
    layer = Layer(wst, T, E, k, K, N)
    dl, dx_, dB_ = logits.cuda(), x.cuda(), B.cuda()
    layer.forward(dl, dx_, dB_)
    assert layer.status() == [0, 0, 0]
    e, w = experts_of(layer, logits, k)
    X, W = ref.f64(x), ref.f64(B)
    y = np.einsum("tk,tink->tin", X, W[e])                        # each pair's row
    ysize = np.einsum("tk,tink->tin", abs(X), abs(W[e]))
    out, size = np.einsum("ti,tin->tn", w, y), np.einsum("ti,tin->tn", abs(w), ysize)
    # y is rounded to bf16, the sum once more; the rest is fp32
    assert (abs(ref.f64(layer.out) - out) <= 2.02 * BF * size).all()

    # gradients for a random dout
    dout = torch.randn(T, N, generator=torch.Generator().manual_seed(1)).bfloat16()
    D = ref.f64(dout)
    dy = torch.empty_like(layer.y)
    dweights = torch.empty(T, k, device="cuda")
    wst.wst_moe_combine_backward(dout.cuda(), layer.position, y=layer.y, weights=layer.weights, dy=dy, dweights=dweights,
                                 workspace=layer.ws)
    dlogits = torch.empty(T, E, device="cuda")
    wst.wst_moe_route_backward(dl, layer.experts, dweights, dlogits, score="sigmoid", renorm=True, scale=1.5)
    drows = torch.empty(T * k, K, dtype=torch.bfloat16, device="cuda")
    wst.wst_grouped_gemm_bf16(dy, dB_.transpose(1, 2).contiguous(), layer.offsets, drows, workspace=layer.ws)
    dx = torch.empty(T, K, device="cuda")
    wst.wst_moe_combine(drows, layer.position, dx, workspace=layer.ws)
    dB = torch.empty(E, N, K, device="cuda")
    wst.wst_grouped_gemm_wgrad_bf16(dy, layer.rows, layer.offsets, dB, workspace=layer.ws)
    assert layer.status() == [0, 0, 0]

    # the same by the chain rule in 64 bits, and its terms' sizes
    want_dw, size_dw = np.einsum("tn,tin->ti", D, y), np.einsum("tn,tin->ti", abs(D), ysize)
    assert (abs(ref.f64(dweights) - want_dw) <= 1.01 * BF * size_dw).all()                 # y's rounding
    want_dl, _ = ref.route_backward(ref.f64(logits), e, want_dw, "sigmoid", True, 1.5)
    # (the size of an entry of the gradient is linear in |dweights|)
    size_dl = ref.route_backward(ref.f64(logits), e, size_dw, "sigmoid", True, 1.5)[1]
    assert (abs(ref.f64(dlogits) - want_dl) <= 1.02 * BF * size_dl).all()
    want_dx = np.einsum("ti,tn,tink->tk", w, D, W[e])
    size_dx = np.einsum("ti,tn,tink->tk", abs(w), abs(D), abs(W[e]))
    assert (abs(ref.f64(dx) - want_dx) <= 2.02 * BF * size_dx).all()                       # dy's and the rows' rounding
    want_dB, size_dB = np.zeros((E, N, K)), np.zeros((E, N, K))
    for t in range(T):
        for i in range(k):
            want_dB[e[t, i]] += w[t, i] * np.outer(D[t], X[t])
            size_dB[e[t, i]] += abs(w[t, i]) * np.outer(abs(D[t]), abs(X[t]))
    assert (abs(ref.f64(dB) - want_dB) <= 1.01 * BF * size_dB).all()                       # dy's rounding


def quantised(wst, B):
    E, N, K = B.shape
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(E, -(-N // 128), -(-K // 128), device="cuda")
    wst.wst_quantize_fp8(B.cuda(), q, s, mode="blocks")
    return q, s


def test_layer_in_8_bits_with_padding_tokens(wst):
    # the last tokens of the batch are padding: no expert, no row, a zero in the output
    T, E, k, K, N = 120, 8, 2, 384, 256
    logits, x, B = inputs(T, E, K, N, 3)
    logits[100:] = -torch.inf
    x[100:] = torch.nan
    layer = Layer(wst, T, E, k, K, N)
    layer.y.fill_(7.0)
    q, s = quantised(wst, B)
    layer.forward_fp8(logits.cuda(), x.cuda(), q, s)
    assert layer.status() == [0, 0, 0]
    e, w = experts_of(layer, logits, k)
    assert int(layer.offsets[-1]) == 200 and (layer.y[200:] == 7.0).all() and (layer.out[100:] == 0).all()
    X, W = ref.f64(x[:100]), ref.f64(B)
    want = np.einsum("ti,tk,tink->tn", w[:100], X, W[e[:100]])
    size = np.einsum("ti,tk,tink->tn", w[:100], abs(X), abs(W[e[:100]]))
    # 8-bit values of x and the weights: half a step each (2^-4), and both; a value
    # below 2^-6 / 448 of its block's largest is off by half of e4m3's smallest step
    tiny = 2.0 ** -10 / 448 * np.einsum("ti,tin->tn", w[:100], (abs(X).max(1)[:, None, None] * abs(W[e[:100]]).sum(3))
                                        + abs(X).sum(1)[:, None, None] * abs(W).max())
    assert (abs(ref.f64(layer.out[:100]) - want) <= (2 * 2.0 ** -4 + 2.0 ** -8 + 2.1 * BF) * size + 1.1 * tiny).all()


def test_layer_as_a_replayed_graph(wst):
    T, E, k, K, N = 64, 16, 4, 512, 256
    layer = Layer(wst, T, E, k, K, N)
    q, s = quantised(wst, inputs(T, E, K, N, 5)[2])
    logits, x = torch.empty(T, E, device="cuda"), torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward_fp8(logits.normal_(), x.normal_(), q, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward_fp8(logits, x, q, s)
    for seed in range(4):
        a, b, _ = inputs(T, E, K, N, 10 + seed)
        if seed == 2:
            a[40:] = -torch.inf          # fewer rows than the graph was captured with
        logits.copy_(a)
        x.copy_(b)
        layer.y.zero_()
        layer.forward_fp8(logits, x, q, s)
        want = [t.clone() for t in (layer.out, layer.weights, layer.position, layer.offsets)]
        layer.out.fill_(float("nan"))
        layer.y.zero_()
        graph.replay()
        for got, w in zip((layer.out, layer.weights, layer.position, layer.offsets), want):
            assert torch.equal(got, w)
    assert layer.status() == [0, 0, 0]


def test_gradient_from_a_graph(wst):
    # a captured backward pass of the weights and the logits gives the bits of the eager one
    T, E, k, K, N = 96, 8, 2, 256, 136
    logits, x, B = inputs(T, E, K, N, 7)
    layer = Layer(wst, T, E, k, K, N)
    dl = logits.cuda()
    layer.forward(dl, x.cuda(), B.cuda())
    dout = torch.randn(T, N, device="cuda").bfloat16()
    dy, dw, dlog = torch.empty_like(layer.y), torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    dB = torch.empty(E, N, K, device="cuda")

    def backward():
        wst.wst_moe_combine_backward(dout, layer.position, y=layer.y, weights=layer.weights, dy=dy, dweights=dw, workspace=layer.ws)
        wst.wst_moe_route_backward(dl, layer.experts, dw, dlog, score="sigmoid", renorm=True, scale=1.5)
        wst.wst_grouped_gemm_wgrad_bf16(dy, layer.rows, layer.offsets, dB, workspace=layer.ws)

    backward()
    want = [t.clone() for t in (dy, dw, dlog, dB)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        backward()
    for t in (dy, dw, dlog, dB):
        t.fill_(float("nan"))
    graph.replay()
    for got, w in zip((dy, dw, dlog, dB), want):
        assert torch.equal(got, w)
    assert layer.status() == [0, 0, 0]


SHARED_WORKSPACE = r'''
import sys, torch
sys.path.insert(0, %r); sys.path.insert(0, %r)
import synthetic
import warp_specialized_tensor_gb300 as wst
wst.load_library()
ws = wst.gemm_fp8_workspace()
# counts of 1 for experts 0 .. 63 of the first chunk, behind the header: where the
# first IKBO call of the process keeps the flags of 64 users
e = torch.full((4096,), 64, dtype=torch.int32)
e[:64] = torch.arange(64)
i32 = dict(dtype=torch.int32, device="cuda")
wst.wst_moe_plan(e.view(1024, 4).cuda(), 65, torch.empty(66, **i32), torch.empty(4096, **i32), torch.empty(4096, **i32),
                 torch.empty(1024, 4, **i32), workspace=ws)
d = {k: v.cuda() for k, v in synthetic.ikbo(users=64, cand_per_user=40, seed=5).items()}
O, D = d["W"].shape[0], d["U"].shape[2]
assert ws.numel() >= wst.wst_workspace_size(64, O, D)
def ikbo(ws):
    Y = torch.full((d["C"].shape[0], O, D), float("nan"), device="cuda")
    wst.wst_ikbo_linear_compress(d["U"], d["C"], d["W"], d["user_offsets"], Y, ws)
    assert wst.wst_sync_status(ws) == 0
    return Y
first = ikbo(ws)
want = ikbo(wst.workspace(64, O, D))
assert torch.equal(first, want)
# the sums of a split product in the same place
f8 = torch.float8_e4m3fn
q, qb = torch.ones(16, 8192, device="cuda").to(f8), torch.ones(512, 8192, device="cuda").to(f8)
C = torch.empty(16, 512, device="cuda")
for _ in range(3):
    wst.wst_gemm_fp8(q, torch.ones(64, 16, device="cuda"), qb, torch.ones(4, 64, device="cuda"), C, workspace=ws)
    assert (C == 8192).all()
    assert torch.equal(ikbo(ws), want)
print("ok")
'''


def test_other_operations_on_the_same_workspace():
    # in a process of its own: the flags' values count its calls
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SHARED_WORKSPACE % (root, os.path.join(root, "tests"))], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.rstrip().endswith("ok"), r.stdout + r.stderr


@pytest.mark.parametrize("live", [100, 1, 0])
@pytest.mark.parametrize("schedule", ["SCHED_STATIC", "SCHED_CLC"])
def test_layer_in_bf16_with_padding_tokens(wst, live, schedule):
    # Padding tokens have no expert: no row, no error, a zero in the output and in
    # the gradients; rows behind the last group stay as they were.
    T, E, k, K, N = 120, 8, 2, 256, 264
    logits, x, B = inputs(T, E, K, N, 11)
    logits[live:] = -torch.inf
    x[live:] = torch.nan
    layer = Layer(wst, T, E, k, K, N)
    layer.rows.fill_(float("nan"))
    layer.y.fill_(7.0)
    dl, dB_ = logits.cuda(), B.cuda()
    wst.wst_set_option(wst.OPT_GROUPED_SCHEDULE, getattr(wst, schedule))
    try:
        layer.forward(dl, x.cuda(), dB_)
        assert layer.status() == [0, 0, 0]
        e, w = experts_of(layer, logits, k)
        rows = live * k
        assert int(layer.offsets[-1]) == rows and (layer.y[rows:] == 7.0).all() and torch.isnan(layer.rows[rows:].float()).all()
        assert (layer.out[live:] == 0).all()
        X, W = ref.f64(x[:live]), ref.f64(B)
        want = np.einsum("ti,tk,tink->tn", w[:live], X, W[e[:live]])
        size = np.einsum("ti,tk,tink->tn", abs(w[:live]), abs(X), abs(W[e[:live]]))
        assert (abs(ref.f64(layer.out[:live]) - want) <= 2.02 * BF * size).all()

        dout = torch.randn(T, N, generator=torch.Generator().manual_seed(1)).bfloat16()
        D = ref.f64(dout[:live])
        dy, dweights, dlogits = torch.full_like(layer.y, float("nan")), torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
        drows = torch.full((T * k, K), float("nan"), dtype=torch.bfloat16, device="cuda")
        dx, dB = torch.empty(T, K, device="cuda"), torch.empty(E, N, K, device="cuda")
        wst.wst_moe_combine_backward(dout.cuda(), layer.position, y=layer.y, weights=layer.weights, dy=dy, dweights=dweights,
                                     workspace=layer.ws)
        wst.wst_moe_route_backward(dl, layer.experts, dweights, dlogits, score="sigmoid", renorm=True, scale=1.5)
        wst.wst_grouped_gemm_bf16(dy, dB_.transpose(1, 2).contiguous(), layer.offsets, drows, workspace=layer.ws)
        wst.wst_moe_combine(drows, layer.position, dx, workspace=layer.ws)
        wst.wst_grouped_gemm_wgrad_bf16(dy, layer.rows, layer.offsets, dB, workspace=layer.ws)
        assert layer.status() == [0, 0, 0]
    finally:
        wst.wst_set_option(wst.OPT_GROUPED_SCHEDULE, wst.SCHED_STATIC)
    assert (dweights[live:] == 0).all() and (dlogits[live:] == 0).all() and (dx[live:] == 0).all()
    assert torch.isnan(drows[rows:].float()).all()
    want_dx = np.einsum("ti,tn,tink->tk", w[:live], D, W[e[:live]])
    size_dx = np.einsum("ti,tn,tink->tk", abs(w[:live]), abs(D), abs(W[e[:live]]))
    assert (abs(ref.f64(dx[:live]) - want_dx) <= 2.02 * BF * size_dx).all()                # dy's and the rows' rounding
    want_dB, size_dB = np.zeros((E, N, K)), np.zeros((E, N, K))
    for t in range(live):
        for i in range(k):
            want_dB[e[t, i]] += w[t, i] * np.outer(D[t], X[t])
            size_dB[e[t, i]] += abs(w[t, i]) * np.outer(abs(D[t]), abs(X[t]))
    assert (abs(ref.f64(dB) - want_dB) <= 1.01 * BF * size_dB).all()                       # dy's rounding


def test_other_bad_rows_and_offsets_are_still_latched(wst):
    ws = wst.workspace()
    src, dst = torch.randn(4, 8, device="cuda").bfloat16(), torch.zeros(3, 8, device="cuda").bfloat16()
    for bad in (-2, 4):
        idx = torch.tensor([1, bad, -1], dtype=torch.int32, device="cuda")
        wst.wst_permute_rows(src, dst, src_index=idx, workspace=ws)
        assert wst.wst_sync_status(ws) == wst.WST_ERR_INVALID_ARG
        assert torch.equal(dst[0], src[1]) and (dst[1:] == 0).all()
    A, B, C = torch.randn(8, 64).bfloat16().cuda(), torch.randn(2, 64, 64).bfloat16().cuda(), torch.zeros(8, 64, device="cuda")
    for off in ([1, 2, 8], [0, 5, 4], [0, 5, 9]):
        wst.wst_grouped_gemm_bf16(A, B, torch.tensor(off, dtype=torch.int32, device="cuda"), C, workspace=ws)
        assert wst.wst_sync_status(ws) == wst.WST_ERR_BAD_OFFSETS
