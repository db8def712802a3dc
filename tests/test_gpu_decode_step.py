"""A decoding step as it is used: 4-bit projections, the append, attention of drafted
trees, 4-bit experts behind the router, the accepted tokens moved together, the next
step; eager, on another stream, and as two graphs that share a workspace."""
import math

import pytest
import torch

import warp_specialized_tensor_gb300 as wst
from test_gpu_cache_append import check as check_append
from test_gpu_cache_append import rotated
from test_gpu_w4 import check as check_product
from test_gpu_w4 import inputs, want
from tree_ref import Paged

pytestmark = pytest.mark.gpu

H, HKV, DH, HID, EXPERTS, TOP, PAGE, GROUP = 8, 2, 64, 256, 6, 2, 16, 64


class Layer:
    """Weights, and the arrays of a step of T tokens; one workspace for all of its calls."""

    def __init__(self, T, seed=0):
        self.T = T
        _, self.wqkv, self.sqkv, _ = inputs(seed + 1, 1, (H + 2 * HKV) * DH, HID, GROUP)
        _, self.wo, self.so, self.bo = inputs(seed + 2, 1, HID, H * DH, GROUP)
        _, self.wr, self.sr, _ = inputs(seed + 3, 1, EXPERTS, HID, GROUP)
        _, self.we, self.se, self.be = inputs(seed + 4, 1, HID, HID, GROUP, (EXPERTS,))
        self.inv = (10000.0 ** (-torch.arange(DH // 2, dtype=torch.float64) * 2 / DH)).float().cuda()
        new = lambda *s, t=torch.bfloat16: torch.full(s, 3.0, device="cuda").to(t)  # noqa: E731
        self.x = new(T, HID)
        self.qkv, self.o, self.y = new(T, (H + 2 * HKV) * DH), new(T, H, DH), new(T, HID)
        self.q = new(T, H, DH)
        self.logits = new(T, 8, t=torch.float32)[:, :EXPERTS]
        self.experts, self.weights = new(T, TOP, t=torch.int32), new(T, TOP, t=torch.float32)
        self.plan = [new(*s, t=torch.int32) for s in ((EXPERTS + 1,), (T * TOP,), (T * TOP,), (T, TOP))]
        self.rows, self.products, self.out = new(T * TOP, HID), new(T * TOP, HID, t=torch.float32), new(T, HID)
        size = max(wst.gemm_w4_workspace().numel(), wst.wst_tree_attention_workspace_size(), wst.moe_plan_workspace(T * TOP, EXPERTS).numel())
        self.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def split(self):
        return (x.view(self.T, -1, DH) for x in self.qkv.split([H * DH, HKV * DH, HKV * DH], dim=1))

    def run(self, c, positions, slots, **kw):
        kw["workspace"] = self.ws
        wst.wst_gemm_w4(self.x, self.wqkv, self.sqkv, self.qkv, group=GROUP, **kw)
        q, k, v = self.split()
        wst.wst_cache_append_bf16(k, v, positions, slots, c.k_cache, c.v_cache, inv_freq=self.inv, q=q, q_out=self.q, **kw)
        wst.wst_tree_attention_bf16(self.q, c.offsets, c.context, c.k_cache, c.v_cache, c.table, self.o, mask=c.mask, **kw)
        wst.wst_gemm_w4(self.o.view(self.T, H * DH), self.wo, self.so, self.y, group=GROUP, bias=self.bo, epi="bias", **kw)
        wst.wst_gemm_w4(self.y, self.wr, self.sr, self.logits, group=GROUP, **kw)
        stream = {n: kw[n] for n in kw if n == "stream"}
        wst.wst_moe_route(self.logits, self.experts, self.weights, **stream)
        wst.wst_moe_plan(self.experts, EXPERTS, *self.plan, **kw)
        offsets, _, row_token, position = self.plan
        wst.wst_permute_rows(self.y, self.rows, src_index=row_token, **kw)
        wst.wst_grouped_gemm_w4(self.rows, self.we, self.se, offsets, self.products, group=GROUP, bias=self.be, epi="bias_silu", **kw)
        wst.wst_moe_combine(self.products, position, self.out, weights=self.weights, **kw)

    def check(self, c, positions, slots):
        """Each call's output against the definition of what the call before it has left."""
        assert wst.wst_sync_status(self.ws) == 0
        check_product(self.qkv, *want(self.x, self.wqkv, self.sqkv, HID, GROUP))
        q, k, v = self.split()
        check_append(self.q, *rotated(q, positions, self.inv, "halves"))
        at = slots.long()
        keys, values = c.k_cache[at // PAGE, at % PAGE], c.v_cache[at // PAGE, at % PAGE]
        check_append(keys, *rotated(k, positions, self.inv, "halves"))
        assert torch.equal(values, v)
        c.q = self.q
        for b, (ctx, n) in enumerate(c.lens):
            rows = slice(c.starts[b], c.starts[b] + n)
            c.K[b][ctx:], c.V[b][ctx:] = keys[rows], values[rows]
        o, size, most = c.want(1.0 / math.sqrt(DH))
        assert bool(((self.o.double() - o).abs() <= c.tolerance(o, size, most, torch.bfloat16)).all())
        check_product(self.y, *want(self.o.view(self.T, -1), self.wo, self.so, H * DH, GROUP, self.bo, "bias"))
        check_product(self.logits, *want(self.y, self.wr, self.sr, HID, GROUP))
        offsets, position = self.plan[0].tolist(), self.plan[3].long()
        for e in range(EXPERTS):
            rows = slice(offsets[e], offsets[e + 1])
            if offsets[e + 1] > offsets[e]:
                check_product(self.products[rows], *want(self.rows[rows], self.we[e], self.se[e], HID, GROUP, self.be[e], "bias_silu"))
        token = torch.arange(self.T, device="cuda")[:, None].expand(-1, TOP)
        assert torch.equal(self.rows[position], self.y[token])
        parts = self.weights.double()[..., None] * self.products.double()[position]
        # two products and a sum of fp32, then the rounding; below 2^-126 (SiLU of large negative sums) a bf16's steps are
        # 2^-133 whatever the value, half of one is 2^-134, and fp32's far smaller ones fit into the other half
        sums, size = parts.sum(dim=1), parts.abs().sum(dim=1)
        err, tol = (self.out.double() - sums).abs(), size * 2.0 ** -22 + (sums.abs() + size * 2.0 ** -22) * 2.0 ** -8 + 2.0 ** -133
        assert bool((err <= tol).all()), (sums[err > tol][:4], err[err > tol][:4])


def step(lens, seed):
    """A cache that holds the contexts only, and where the new tokens go: their depths in the trees are their positions."""
    c = Paged(lens, H, HKV, DH, PAGE, "tree", seed=seed)
    place(c)
    c.k_cache[c.slots // PAGE, c.slots % PAGE] = float("nan")
    c.v_cache[c.slots // PAGE, c.slots % PAGE] = float("nan")
    return c, c.positions, c.slots.to(torch.int32)


def place(c):
    slots, positions = [], []
    for b, (ctx, n) in enumerate(c.lens):
        key = torch.arange(ctx, ctx + n, device="cuda")
        slots.append(c.table[b].long()[key // PAGE] * PAGE + key % PAGE)
        positions += [ctx + int(s.sum()) - 1 for s in c.seen[b]]
    c.slots = torch.cat(slots)
    c.positions = torch.tensor(positions, dtype=torch.int32, device="cuda")


def test_step_accept_and_the_next_step():
    lens = [(37, 9), (130, 20), (0, 5), (14, 1), (250, 33)]
    c, positions, slots = step(lens, 1)
    layer = Layer(c.T)
    layer.x.copy_(torch.randn(c.T, HID, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)))
    layer.run(c, positions, slots)
    layer.check(c, positions, slots)
    # The accepted path of each tree: what its last token sees.  Its rows move behind the context, by way of an array of
    # their own, because they may trade places.
    source, target, accepted = [], [], []
    for b, (ctx, n) in enumerate(lens):
        path = [int(i) for i in c.seen[b][n - 1].nonzero()[0]]
        accepted.append(path)
        mine = slots[c.starts[b]:c.starts[b] + n].tolist()
        source += [mine[i] for i in path]
        target += mine[:len(path)]
    source, target = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (source, target))
    moved = torch.empty(source.numel(), HKV * DH, dtype=torch.bfloat16, device="cuda")
    for cache in (c.k_cache, c.v_cache):
        rows = cache.view(-1, HKV * DH)
        wst.wst_permute_rows(rows, moved, src_index=source, workspace=layer.ws)
        wst.wst_permute_rows(moved, rows, dst_index=target, workspace=layer.ws)
    assert wst.wst_sync_status(layer.ws) == 0
    # The next step: one token for each sequence, behind what was accepted.
    after = [(ctx + len(path), 1) for (ctx, _), path in zip(lens, accepted)]
    d = Paged(after, H, HKV, DH, PAGE, "chain", seed=2)
    d.k_cache, d.v_cache, d.table = c.k_cache, c.v_cache, c.table
    for b, ((ctx, _), path) in enumerate(zip(lens, accepted)):
        keep = list(range(ctx)) + [ctx + i for i in path]
        d.K[b][:-1], d.V[b][:-1] = c.K[b][keep], c.V[b][keep]
    place(d)
    layer = Layer(d.T, seed=10)
    layer.x.copy_(torch.randn(d.T, HID, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)))
    layer.run(d, d.positions, d.slots.to(torch.int32))
    layer.check(d, d.positions, d.slots.to(torch.int32))


def test_streams_and_two_graphs_on_one_workspace():
    steps = [step([(37, 9), (130, 20), (0, 5)], 3), step([(300, 1), (0, 1), (15, 1), (16, 1)], 4)]
    layers = [Layer(c.T, seed=20 + i) for i, (c, _, _) in enumerate(steps)]
    layers[1].ws = layers[0].ws
    g = torch.Generator(device="cuda").manual_seed(7)
    for layer in layers:
        layer.x.copy_(torch.randn(layer.T, HID, device="cuda", generator=g))
    outputs = ("qkv", "q", "o", "y", "experts", "products", "out")
    eager = []
    for layer, s in zip(layers, steps):
        layer.run(*s)
        torch.cuda.synchronize()
        layer.check(*s)
        eager.append([getattr(layer, n).clone() for n in outputs])

    def same(i):
        torch.cuda.synchronize()
        return all(torch.equal(getattr(layers[i], n), e) for n, e in zip(outputs, eager[i]))

    def wipe(i):
        for n in outputs:
            getattr(layers[i], n).zero_()

    side = torch.cuda.Stream()
    for i in (0, 1):
        wipe(i)
    side.wait_stream(torch.cuda.current_stream())
    for i in (0, 1):
        layers[i].run(*steps[i], stream=side)
    assert same(0) and same(1)
    graphs = []
    for i in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=side):
            layers[i].run(*steps[i])
    for i in (0, 1, 1, 0):
        wipe(i)
        graphs[i].replay()
        assert same(i)
    # other inputs in the same places
    layers[0].x.mul_(-1.5)
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    layers[0].check(*steps[0])
    assert same(1) and wst.wst_sync_status(layers[0].ws) == 0
