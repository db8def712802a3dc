"""The mixture-of-experts operators next to the grouped GEMM, as measured cases.

Four operators: routing (scores, top-k experts, weights, the device-side plan of
the rows, and the gradient of the logits), combine (the weighted sum of the
experts' rows, and its gradients), the 8-bit product with a scale for each
block of 128 (quantisation, dense and grouped product) and the grouped weight
gradient in bf16.  `run` with `own` false computes them by elementary torch
operations; with `own` true it calls the library's entry points.
"""
import math

import numpy as np
import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
FLOOR = 2.0 ** -100      # a block's largest value counts as at least this
OFF = -3.0e38            # a logit at or below it marks an expert as off
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3, "e5m2": E5M2}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _route(T, E, k, score, logits, bias, groups=1, top_groups=1, group_best=1, renorm=True, scale=1.0, off=0.0):
    return {"op": "route", "T": T, "E": E, "k": k, "score": score, "logits": logits, "bias": bias, "groups": groups,
            "top_groups": top_groups, "group_best": group_best, "renorm": renorm, "scale": scale, "off": off}


def listed():
    return [
        # one step of a serving batch: 32 sequences, 256 experts in 8 groups of which 4 are kept
        dict(_route(32, 256, 8, "sigmoid", "f32", True, 8, 4, 2, True, 2.5), name="route_step"),
        # the router of a training batch or a long prompt
        dict(_route(16384, 256, 8, "sigmoid", "f32", True, 8, 4, 2, True, 2.5), name="route_batch"),
        # the gradient of that router's logits, for softmax scores that are not renormalised
        {"op": "route_backward", "T": 16384, "E": 64, "k": 2, "score": "softmax", "logits": "bf16", "renorm": False, "scale": 1.0,
         "name": "route_grad"},
        # the experts' outputs of the benchmark's layer (64 experts, two for each of 16384 tokens) added up
        {"op": "combine", "T": 16384, "k": 2, "N": 4096, "y": "bf16", "out": "bf16", "weighted": True, "drop": 0.0, "name": "combine_batch"},
        # its gradients at an odd width, four experts a token, some pairs dropped (tokens behind the last sequence)
        {"op": "combine_backward", "T": 5003, "k": 4, "N": 1531, "y": "bf16", "out": "bf16", "drop": 0.05, "name": "combine_grad"},
        # the layer's tokens quantised and written to their experts' rows
        {"op": "quantise_dispatch", "T": 16384, "k": 2, "K": 4096, "x": "bf16", "q": "e4m3", "pow2": False, "name": "quantise_tokens"},
        # weights quantised for the gradient of the inputs: 128 x 128 blocks, transposed
        {"op": "quantise", "mode": "blocks_t", "batch": 16, "M": 1536, "K": 4096, "x": "bf16", "q": "e4m3", "pow2": False, "name": "quantise_weights"},
        # a projection for one step of 16 sequences: the weights are read once
        {"op": "product", "M": 16, "N": 4096, "K": 8192, "a": "e4m3", "b": "e4m3", "scaling": "blocks", "c": "bf16", "name": "product_step"},
        # the benchmark's dense size
        {"op": "product", "M": 8192, "N": 8192, "K": 8192, "a": "e4m3", "b": "e4m3", "scaling": "blocks", "c": "bf16", "name": "product_dense"},
        # the benchmark's grouped size
        {"op": "grouped", "G": 64, "P": 32768, "N": 1536, "K": 4096, "a": "e4m3", "b": "e4m3", "c": "bf16", "empty": 0, "name": "product_experts"},
        # the gradient of the benchmark's expert weights, kept in 32 bits
        {"op": "wgrad", "G": 64, "P": 32768, "N": 1536, "K": 4096, "out": "f32", "empty": 0, "name": "wgrad_experts"},
        # small ragged experts, some without a token
        {"op": "wgrad", "G": 13, "P": 1777, "N": 520, "K": 712, "out": "bf16", "empty": 3, "name": "wgrad_ragged"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "combine", "combine_backward", "quantise_dispatch", "quantise", "product",
                     "product", "grouped", "grouped", "wgrad"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, 6, 384 // groups)
        top_groups = groups if groups == 1 else rng.randint(1, groups)
        k = rng.randint(1, min(10, top_groups * (E // groups)))
        return _route(_log(rng, 1, 16384), E, k, rng.choice(["softmax", "sigmoid"]), rng.choice(["f32", "bf16"]), rng.random() < 0.5,
                      groups, top_groups, rng.choice([1, 2]), rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.choice([0.0, 0.05]))
    if op == "route_backward":
        E = _log(rng, 6, 256)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(10, E)), "score": rng.choice(["softmax", "sigmoid"]),
                "logits": rng.choice(["f32", "bf16"]), "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5])}
    if op in ("combine", "combine_backward"):
        k = rng.randint(1, 8)
        N = _log(rng, 8, 5120)
        T = _log(rng, 1, min(16384, max(1, 16384 * 2 * 4096 // (2 * k * N))))
        case = {"op": op, "T": T, "k": k, "N": N, "y": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
                "drop": rng.choice([0.0, 0.1])}
        return dict(case, weighted=rng.random() < 0.7) if op == "combine" else case
    if op == "quantise_dispatch":
        K, k = _log(rng, 16, 7168), rng.randint(1, 8)
        return {"op": op, "T": _log(rng, 1, min(16384, 16384 * 4096 * 2 // (K * k))), "k": k, "K": K, "x": rng.choice(["bf16", "bf16", "f32"]),
                "q": rng.choice(["e4m3", "e4m3", "e5m2"]), "pow2": rng.random() < 0.4}
    if op == "quantise":
        M, K = _log(rng, 1, 8192), _log(rng, 16, 8192)
        return {"op": op, "mode": rng.choice(["rows", "cols", "blocks", "blocks_t"]), "batch": rng.choice([1, 1, 2, 5]) if M * K < 2 ** 24 else 1,
                "M": M, "K": K, "x": rng.choice(["bf16", "bf16", "f32"]), "q": rng.choice(["e4m3", "e4m3", "e5m2"]), "pow2": rng.random() < 0.4}
    if op == "product":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 8192), "K": _log(rng, 64, 8192), "a": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "b": "e4m3", "scaling": rng.choice(["blocks", "blocks", "rows"]), "c": rng.choice(["bf16", "bf16", "f32"])}
    G = _log(rng, 1, 64)
    case = {"op": op, "G": G, "P": _log(rng, 1, 32768), "N": _log(rng, 64, 2048 if G > 16 else 4096), "K": _log(rng, 64, 4096),
            "empty": rng.randint(0, G // 3)}
    if op == "grouped":
        return dict(case, a=rng.choice(["e4m3", "e4m3", "e5m2"]), b="e4m3", c=rng.choice(["bf16", "bf16", "f32"]))
    return dict(case, P=_log(rng, 1, 16384), N=_log(rng, 64, 1536), out=rng.choice(["bf16", "f32"]))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _up(n, m):
    return -(-n // m) * m


def _empty(rows, cols, dtype, lead=()):
    """[*lead, rows, cols] whose rows begin on 16 bytes."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty(*lead, rows, _up(cols, per), dtype=dtype, device="cuda")[..., :cols]


def _padded(x):
    """The same values in rows that begin on 16 bytes."""
    out = _empty(x.shape[-2], x.shape[-1], x.dtype, tuple(x.shape[:-2]))
    out.copy_(x)
    return out


def _features(g, rows, cols, dtype, lead=()):
    """Activations: normal, with a few channels much larger than the rest."""
    x = torch.randn(*lead, rows, cols, generator=g, device="cuda")
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 12.0, 1.0)
    return _padded(x.to(dtype))


def _routing(g, T, k, E):
    """k distinct experts of each token, some experts liked better than others."""
    liked = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    return liked.argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()


def _plan(experts, E):
    """offsets, the pair and the token of each row, the row of each pair; expert -1: no row."""
    flat = experts.reshape(-1).long()
    P, k = flat.numel(), experts.shape[1]
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=flat.device)).to(torch.int32)
    live = torch.arange(P, device=flat.device) < offsets[E]
    row_pair = torch.where(live, order, -1)
    row_token = torch.where(live, order // k, -1)
    position = torch.empty_like(order).scatter_(0, order, torch.where(live, torch.arange(P, device=flat.device), -1))
    return offsets, row_pair.to(torch.int32), row_token.to(torch.int32), position.reshape(experts.shape).to(torch.int32)


def _groups(rng, G, P, empty):
    """int32 offsets of G groups of P rows, `empty` of them without a row."""
    share = rng.uniform(0.5, 1.5, G)
    share[rng.choice(G, empty, replace=False)] = 0.0
    sizes = rng.multinomial(P, share / share.sum())
    return torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).cuda(), int(sizes.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(case)
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = torch.randn(T, E, generator=g, device="cuda") * 1.5
        if case["off"]:
            x = torch.where(torch.rand(T, E, generator=g, device="cuda") < case["off"], -math.inf, x)
            x[T - T // 8:] = -math.inf       # tokens behind the last sequence: nothing to choose from
        s["x"] = _padded(x.to(TYPES[case["logits"]]))
        s["b"] = torch.randn(E, generator=g, device="cuda") * 0.05 if case["bias"] else None
        s["experts"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, k, device="cuda")
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["row_pair"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
        s["row_token"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
        s["position"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    elif op == "route_backward":
        T, E, k = case["T"], case["E"], case["k"]
        s["x"] = _padded((torch.randn(T, E, generator=g, device="cuda") * 1.5).to(TYPES[case["logits"]]))
        s["experts"] = torch.sort(s["x"].float(), dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
        s["dw"] = torch.randn(T, k, generator=g, device="cuda")
        s["dx"] = _empty(T, E, s["x"].dtype)
    elif op in ("combine", "combine_backward"):
        T, k, N = case["T"], case["k"], case["N"]
        E = max(8, k)
        experts = _routing(g, T, k, E)
        if case["drop"]:
            experts[T - int(T * case["drop"]):] = -1
        offsets, row_pair, _, s["position"] = _plan(experts, E)
        rows = int(offsets[E])
        s["row_pair"] = row_pair[:rows].contiguous()
        s["y"] = _padded(torch.randn(rows, N, generator=g, device="cuda").to(TYPES[case["y"]]))
        w = torch.rand(T, k, generator=g, device="cuda") + 0.1
        s["w"] = w / w.sum(1, keepdim=True) if case.get("weighted", True) else None
        if op == "combine":
            s["result"] = _empty(T, N, TYPES[case["out"]])
        else:
            s["dout"] = _padded(torch.randn(T, N, generator=g, device="cuda").to(TYPES[case["out"]]))
            s["dy"] = _empty(rows, N, TYPES[case["y"]])
            s["dw"] = torch.empty(T, k, device="cuda")
    elif op == "quantise_dispatch":
        T, k, K = case["T"], case["k"], case["K"]
        s["x"] = _features(g, T, K, TYPES[case["x"]])
        _, s["row_pair"], s["row_token"], s["position"] = _plan(_routing(g, T, k, max(8, k)), max(8, k))
        s["q_out"] = _empty(T * k, K, TYPES[case["q"]])
        s["scales"] = _empty(_up(K, 128) // 128, T * k, torch.float32)
    elif op == "quantise":
        B, M, K, mode = case["batch"], case["M"], case["K"], case["mode"]
        s["x"] = _features(g, M, K, TYPES[case["x"]], (B,)) * (0.02 if mode.startswith("blocks") else 1.0)
        s["x"] = _padded(s["x"])
        s["q_out"] = _empty(*((M, K) if mode in ("rows", "blocks") else (K, M)), TYPES[case["q"]], (B,))
        mb, kb = _up(M, 128) // 128, _up(K, 128) // 128
        s["scales"] = _empty(*{"rows": (kb, M), "cols": (mb, K), "blocks": (mb, kb), "blocks_t": (kb, mb)}[mode], torch.float32, (B,))
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["a_q"], s["a_s"] = _quantised(_features(g, M, K, torch.bfloat16), "rows", TYPES[case["a"]])
        w = (torch.randn(N, K, generator=g, device="cuda") * 0.02).bfloat16()
        s["b_q"], s["b_s"] = _quantised(w, case["scaling"], TYPES[case["b"]])
        s["result"] = _empty(M, N, TYPES[case["c"]])
    elif op == "grouped":
        G, P, N, K = case["G"], case["P"], case["N"], case["K"]
        s["offsets"], s["most"] = _groups(rng, G, P, case["empty"])
        s["a_q"], s["a_s"] = _quantised(_features(g, P, K, torch.bfloat16), "rows", TYPES[case["a"]])
        w = (torch.randn(G, N, K, generator=g, device="cuda") * 0.02).bfloat16()
        s["b_q"], s["b_s"] = _quantised(w, "blocks", TYPES[case["b"]])
        s["result"] = _empty(P, N, TYPES[case["c"]])
    elif op == "wgrad":
        G, P, N, K = case["G"], case["P"], case["N"], case["K"]
        s["offsets"], s["most"] = _groups(rng, G, P, case["empty"])
        s["dc"] = _padded((torch.randn(P, N, generator=g, device="cuda") * 0.05).bfloat16())
        s["a"] = _padded(torch.randn(P, K, generator=g, device="cuda").bfloat16())
        s["result"] = _empty(N, K, TYPES[case["out"]], (G,))
    if own:  # the library's workspaces, which a program keeps from call to call
        import warp_specialized_tensor_gb300 as wst
        s["ws"] = wst.workspace()
        if op == "route":
            s["ws"] = wst.moe_plan_workspace(case["T"] * case["k"], case["E"])
        elif op in ("product", "grouped"):
            s["ws"] = wst.gemm_fp8_workspace()
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------
def _blocks_of(x, mode):
    """x [B, M, K] in 32 bits as blocks that share a scale, the block's values in the last dimensions."""
    B, M, K = x.shape
    m = 128 if mode != "rows" else 1
    k = 128 if mode != "cols" else 1
    x = torch.nn.functional.pad(x, (0, _up(K, k) - K, 0, _up(M, m) - M))
    return x.view(B, x.shape[1] // m, m, x.shape[2] // k, k)


def _quantised(x, mode, dtype, pow2=False):
    """x [M, K] or [B, M, K] in 8 bits, and the scales: rows [K/128, M], cols [M/128, K] with the values transposed,
    blocks [M/128, K/128], blocks_t the same, both transposed."""
    lead = x.dim() == 3
    x = (x if lead else x[None]).float()
    B, M, K = x.shape
    b = _blocks_of(x, "blocks" if mode == "blocks_t" else mode)
    scale = b.abs().amax(dim=(2, 4)).clamp(min=FLOOR) * torch.tensor(1.0 / LARGEST[dtype], dtype=torch.float32, device=x.device)
    if pow2:  # the smallest power of two that leaves no value above the type's largest (1.75 times a power of two)
        mantissa, e = torch.frexp(b.abs().amax(dim=(2, 4)).clamp(min=FLOOR))
        scale = torch.ldexp(torch.ones_like(mantissa), e - 1 - int(math.log2(LARGEST[dtype] / 1.75)) + (mantissa > 0.875).int())
    q = (b * (1.0 / scale)[:, :, None, :, None]).reshape(B, b.shape[1] * b.shape[2], -1)[:, :M, :K]
    q = q.clamp(-LARGEST[dtype], LARGEST[dtype])
    q = (q.transpose(1, 2) if mode in ("cols", "blocks_t") else q).contiguous().to(dtype)
    scale = scale.transpose(1, 2) if mode in ("rows", "blocks_t") else scale
    q, scale = _padded(q), _padded(scale.contiguous())
    return (q, scale) if lead else (q[0], scale[0])


def _values(q, scale, mode):
    """The numbers that 8-bit values [.., M, K] and their scales stand for, in 32 bits."""
    M, K = q.shape[-2:]
    scale = scale.transpose(-1, -2) if mode == "rows" else scale.repeat_interleave(128, -2)[..., :M, :]
    return q.float() * scale.repeat_interleave(128, -1)[..., :K]


def _scores(x, score, off):
    x = torch.where(off, -math.inf, x)
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _by_group(v, case, off):
    """v with the experts of groups that are not kept at -inf."""
    T, n = v.shape[0], case["groups"]
    g = v.view(T, n, -1)
    best = g.sort(dim=-1, descending=True).values[..., :case["group_best"]]
    score = torch.where(best[..., :1] == -math.inf, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(-1, keepdim=True))[..., 0]
    kept = torch.zeros_like(score, dtype=torch.bool)
    kept.scatter_(1, score.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]], True)
    return torch.where(kept[:, :, None], g, -math.inf).reshape(T, -1)


def _plain_route(s):
    # in 64 bits: two experts' scores may differ by less than 32 bits tell apart
    x = s["x"].double()
    off = x <= OFF
    score = _scores(x, s["score"], off)
    v = torch.where(off, -math.inf, score if s["b"] is None else score + s["b"].double())
    if s["groups"] > 1:
        v = _by_group(v, s, off)
    best = v.sort(dim=1, descending=True, stable=True)
    chosen, live = best.indices[:, :s["k"]], best.values[:, :s["k"]] > -math.inf
    w = torch.where(live, score.gather(1, chosen), 0.0)
    if s["renorm"]:
        w = torch.where(live, w / w.sum(1, keepdim=True), 0.0)
    experts = torch.where(live, chosen, -1).to(torch.int32)
    offsets, row_pair, row_token, position = _plan(experts, s["E"])
    return {"experts": experts, "weights": (s["scale"] * w).float(), "offsets": offsets, "row_pair": row_pair, "row_token": row_token,
            "position": position}


def _plain_route_backward(s):
    x = s["x"].double()
    off = x <= OFF
    score = _scores(x, s["score"], off)
    chosen = s["experts"].long()
    g = s["scale"] * s["dw"].double()
    picked = score.gather(1, chosen)
    if s["renorm"]:
        total = picked.sum(1, keepdim=True)
        g = (g - (g * (picked / total)).sum(1, keepdim=True)) / total
    ds = torch.zeros_like(x).scatter_(1, chosen, g)
    if s["score"] == "sigmoid":
        return ds.mul_(score).mul_(1.0 - score).to(s["x"].dtype)
    return (score * (ds - (ds * score).sum(1, keepdim=True))).to(s["x"].dtype)


def _plain_combine(s):
    at = s["position"].long()
    w = (at >= 0).float() if s["w"] is None else torch.where(at >= 0, s["w"], 0.0)
    y = s["y"].float()[at.clamp(min=0)]
    return (y * w[:, :, None]).sum(1).to(TYPES[s["out"]])


def _plain_combine_backward(s):
    pair = s["row_pair"].long()
    d = s["dout"].float()[pair // s["k"]]
    dy = (d * s["w"].reshape(-1)[pair][:, None]).to(s["y"].dtype)
    dw = torch.zeros(s["w"].numel(), device="cuda").index_copy_(0, pair, (d * s["y"].float()).sum(1))
    return {"dy": dy, "dw": dw.view_as(s["w"])}


def _padded_groups(x, offsets, most):
    """x [P, n] as [G, most, n] in 32 bits, zeros behind each group's rows; and the rows' places."""
    at = offsets[:-1, None].long() + torch.arange(most, device="cuda")
    there = at < offsets[1:, None]
    return x.float()[torch.where(there, at, 0)] * there[:, :, None], at, there


def _plain_grouped(s):
    P, G = s["P"], s["G"]
    a, _, _ = _padded_groups(_values(s["a_q"], s["a_s"], "rows"), s["offsets"], s["most"])
    c = torch.bmm(a, _values(s["b_q"], s["b_s"], "blocks").transpose(1, 2))
    row = torch.arange(P, device="cuda")
    group = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    return c[group, row - s["offsets"][group].long()].to(TYPES[s["c"]])


def _plain_wgrad(s):
    dc, _, _ = _padded_groups(s["dc"], s["offsets"], s["most"])
    a, _, _ = _padded_groups(s["a"], s["offsets"], s["most"])
    return torch.bmm(dc.transpose(1, 2), a).to(TYPES[s["out"]])


def _plain(s):
    op = s["op"]
    if op == "route":
        return _plain_route(s)
    if op == "route_backward":
        return _plain_route_backward(s)
    if op == "combine":
        return _plain_combine(s)
    if op == "combine_backward":
        return _plain_combine_backward(s)
    if op == "quantise_dispatch":
        q, scale = _quantised(s["x"], "rows", TYPES[s["q"]], s["pow2"])
        token = s["row_token"].long()
        return {"q": q.view(torch.uint8)[token].view(q.dtype), "scales": scale[:, token]}
    if op == "quantise":
        q, scale = _quantised(s["x"], s["mode"], TYPES[s["q"]], s["pow2"])
        return {"q": q, "scales": scale}
    if op == "product":
        return (_values(s["a_q"], s["a_s"], "rows") @ _values(s["b_q"], s["b_s"], s["scaling"]).T).to(TYPES[s["c"]])
    if op == "grouped":
        return _plain_grouped(s)
    return _plain_wgrad(s)


# ----------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------
def _own(s):
    import warp_specialized_tensor_gb300 as wst
    op, ws = s["op"], s["ws"]
    if op == "route":
        wst.wst_moe_route(s["x"], s["experts"], s["weights"], score=s["score"], bias=s["b"], groups=s["groups"],
                          top_groups=s["top_groups"], group_best=s["group_best"], renorm=s["renorm"], scale=s["scale"])
        wst.wst_moe_plan(s["experts"], s["E"], s["offsets"], s["row_pair"], s["row_token"], s["position"], workspace=ws)
        return {n: s[n] for n in ("experts", "weights", "offsets", "row_pair", "row_token", "position")}
    if op == "route_backward":
        wst.wst_moe_route_backward(s["x"], s["experts"], s["dw"], s["dx"], score=s["score"], renorm=s["renorm"], scale=s["scale"])
        return s["dx"]
    if op == "combine":
        wst.wst_moe_combine(s["y"], s["position"], s["result"], weights=s["w"], workspace=ws)
        return s["result"]
    if op == "combine_backward":
        wst.wst_moe_combine_backward(s["dout"], s["position"], y=s["y"], weights=s["w"], dy=s["dy"], dweights=s["dw"], workspace=ws)
        return {"dy": s["dy"], "dw": s["dw"]}
    if op == "quantise_dispatch":
        wst.wst_quantize_fp8_dispatch(s["x"], s["position"], s["q_out"], s["scales"], pow2=s["pow2"], workspace=ws)
        return {"q": s["q_out"], "scales": s["scales"]}
    if op == "quantise":
        wst.wst_quantize_fp8(s["x"], s["q_out"], s["scales"], mode=s["mode"], pow2=s["pow2"])
        return {"q": s["q_out"], "scales": s["scales"]}
    if op == "product":
        wst.wst_gemm_fp8(s["a_q"], s["a_s"], s["b_q"], s["b_s"], s["result"], scaling=s["scaling"], workspace=ws)
        return s["result"]
    if op == "grouped":
        wst.wst_grouped_gemm_fp8(s["a_q"], s["a_s"], s["b_q"], s["b_s"], s["offsets"], s["result"], workspace=ws)
        return s["result"]
    wst.wst_grouped_gemm_wgrad_bf16(s["dc"], s["a"], s["offsets"], s["result"], workspace=ws)
    return s["result"]


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2, "e4m3": 1, "e5m2": 1}
    op = case["op"]
    if op == "route":
        T, E, P = case["T"], case["E"], case["T"] * case["k"]
        # logits in; experts, weights, rows' pairs and tokens, pairs' rows and the offsets out
        return {"bytes": T * E * size[case["logits"]] + 20 * P + 4 * (E + 1), "flops": 4 * T * E}
    if op == "route_backward":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 2 * T * E * size[case["logits"]] + 8 * T * k, "flops": 6 * T * E}
    if op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        rows = (T - int(T * case["drop"])) * k
        return {"bytes": rows * N * size[case["y"]] + T * N * size[case["out"]] + T * k * (8 if case["weighted"] else 4), "flops": 2 * rows * N}
    if op == "combine_backward":
        T, k, N = case["T"], case["k"], case["N"]
        rows = (T - int(T * case["drop"])) * k
        return {"bytes": 2 * rows * N * size[case["y"]] + T * N * size[case["out"]] + 12 * T * k, "flops": 3 * rows * N}
    if op == "quantise_dispatch":
        T, k, K = case["T"], case["k"], case["K"]
        return {"bytes": T * K * size[case["x"]] + T * k * (K + 4 * _up(K, 128) // 128 + 4), "flops": 2 * T * K}
    if op == "quantise":
        n = case["batch"] * case["M"] * case["K"]
        return {"bytes": n * (size[case["x"]] + 1) + 4 * n // (128 if case["mode"] in ("rows", "cols") else 16384), "flops": 2 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K + 4 * M * K // 128 + M * N * size[case["c"]], "flops": 2 * M * N * K}
    G, P, N, K = case["G"], case["P"], case["N"], case["K"]
    if op == "grouped":
        used = min(G - case["empty"], P)
        return {"bytes": P * K + 4 * P * K // 128 + used * N * K + P * N * size[case["c"]], "flops": 2 * P * N * K}
    return {"bytes": 2 * P * (N + K) + G * N * K * size[case["out"]], "flops": 2 * P * N * K}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def _exact_scores(x, score):
    if score == "sigmoid":
        return np.where(x <= OFF, 0.0, np.exp(-np.logaddexp(0.0, -np.where(x <= OFF, 0.0, x))))
    e = np.where(x <= OFF, 0.0, np.exp(x - np.maximum(x.max(1, keepdims=True), OFF)))
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def _exact_scale(amax, dtype, pow2):
    amax = np.maximum(amax, FLOOR)
    return np.exp2(np.ceil(np.log2(amax / LARGEST[dtype]))) if pow2 else amax / LARGEST[dtype]


def _exact_quantised(x, mode, dtype, pow2):
    """[B, M, K] in 64 bits on the CPU: the 8-bit values and the scales, laid out as run() returns them."""
    B, M, K = x.shape
    wide = np.zeros((B, _up(M, 128), _up(K, 128)))
    wide[:, :M, :K] = np.abs(x)
    if mode != "rows":
        wide = wide.reshape(B, -1, 128, wide.shape[2]).max(2)
    if mode != "cols":
        wide = wide.reshape(B, wide.shape[1], -1, 128).max(3)
    scale = _exact_scale(wide, dtype, pow2)
    each = scale if mode == "rows" else np.repeat(scale, 128, 1)
    each = each if mode == "cols" else np.repeat(each, 128, 2)
    q = torch.from_numpy(x / each[:, :M, :K]).to(dtype).double().numpy()
    if mode == "rows":
        return q, scale[:, :M].transpose(0, 2, 1)
    if mode == "cols":
        return q.transpose(0, 2, 1), scale[:, :, :K]
    return (q, scale) if mode == "blocks" else (q.transpose(0, 2, 1), scale.transpose(0, 2, 1))


def exact(case, seed):
    op = case["op"]
    if op == "route_backward" and case["T"] * case["k"] * case["E"] > 2 ** 26:
        return None
    s = prepare(case, seed)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    if op == "route":
        x, k, n = host(s["x"]), case["k"], case["groups"]
        score = _exact_scores(x, case["score"])
        v = np.where(x <= OFF, -np.inf, score + (0.0 if s["b"] is None else host(s["b"])))
        g = v.reshape(len(v), n, -1)
        two = -np.sort(-g, axis=2)[:, :, :case["group_best"]]
        total = np.where(two[:, :, 0] > -np.inf, np.where(two > -np.inf, two, 0.0).sum(2), -np.inf)
        rank = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1, kind="stable")
        v = np.where(rank[:, :, None] < case["top_groups"], g, -np.inf).reshape(v.shape)
        chosen = np.argsort(-v, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(np.where(v > -np.inf, score, 0.0), chosen, 1)
        if case["renorm"]:
            w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
        return {"experts": None, "weights": case["scale"] * w, "offsets": None, "row_pair": None, "row_token": None, "position": None}
    if op == "route_backward":
        # by the derivative of each weight, [T, k, E]
        x, at = host(s["x"]), s["experts"].cpu().numpy().astype(np.int64)
        score, T = _exact_scores(x, case["score"]), len(x)
        picked = np.take_along_axis(score, at, 1)
        one = np.zeros((T, case["k"], case["E"]), dtype=bool)
        np.put_along_axis(one, at[:, :, None], True, 2)
        if case["score"] == "sigmoid":
            jac = lambda c: c * one * (picked * (1 - picked))[:, :, None]  # noqa: E731
        else:
            jac = lambda c: c * picked[:, :, None] * (one - score[:, None, :])  # noqa: E731
        d = jac(1.0)
        if case["renorm"]:
            total = picked.sum(1)[:, None, None]
            d = d / total - (picked[:, :, None] / total) * (d.sum(1, keepdims=True) / total)
        return case["scale"] * np.einsum("tk,tke->te", host(s["dw"]), d)
    if op == "combine":
        at, y = s["position"].long(), s["y"].double()
        out = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            w = (at[:, j] >= 0).double() * (1.0 if s["w"] is None else s["w"][:, j].double())
            out += w[:, None] * y[at[:, j].clamp(min=0)]
        return out
    if op == "combine_backward":
        at, d, y = s["position"].long(), s["dout"].double(), s["y"].double()
        dy, dw = torch.zeros_like(y), torch.zeros(*at.shape, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = torch.nonzero(at[:, j] >= 0)[:, 0]
            dy[at[t, j]] = s["w"][t, j].double()[:, None] * d[t]
            dw[t, j] = torch.linalg.vecdot(d[t], y[at[t, j]])
        return {"dy": dy, "dw": dw}
    if op == "quantise_dispatch":
        q, scale = _exact_quantised(host(s["x"])[None], "rows", TYPES[case["q"]], case["pow2"])
        token = s["row_token"].cpu().numpy()
        return {"q": q[0][token], "scales": scale[0][:, token]}
    if op == "quantise":
        q, scale = _exact_quantised(host(s["x"]), case["mode"], TYPES[case["q"]], case["pow2"])
        return {"q": np.ascontiguousarray(q), "scales": np.ascontiguousarray(scale)}
    if op == "product":
        # block by block of K, the scales applied to each block's product
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for i, k in enumerate(range(0, case["K"], 128)):
            b = s["b_s"][i] if case["scaling"] == "rows" else s["b_s"][:, i].repeat_interleave(128)[:case["N"]]
            part = s["a_q"][:, k:k + 128].double() @ s["b_q"][:, k:k + 128].double().T
            out += part * s["a_s"][i].double()[:, None] * b.double()[None]
        return out
    at = s["offsets"].tolist()
    if op == "grouped":
        out = torch.zeros(case["P"], case["N"], dtype=torch.float64, device="cuda")
        ones = torch.ones(128, dtype=torch.float64, device="cuda")
        for j in range(case["G"]):
            a, b = slice(at[j], at[j + 1]), j
            va = s["a_q"][a].double() * torch.kron(s["a_s"][:, a].T.contiguous().double(), ones[None])[:, :case["K"]]
            vb = s["b_q"][b].double() * torch.kron(s["b_s"][b].double(), torch.outer(ones, ones))[:case["N"], :case["K"]]
            out[a] = va @ vb.T
        return out
    return torch.stack([s["dc"][i:j].double().T @ s["a"][i:j].double() for i, j in zip(at[:-1], at[1:])])
