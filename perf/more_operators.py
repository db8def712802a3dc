"""Operators of a decoding step, as measured cases.

Three operators: the append of keys and values to a paged cache with the
position rotation on the way, attention of drafted tokens (a tree, a chain, one
token) over that cache, and products of few rows with 4-bit weights and group
scales, dense and for the experts of a mixture.  `run` with `own` false computes
them by elementary torch operations; with `own` true it calls the library's entry
points.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _append(T, H, Hkv, Dh, rot, style, page, x, drop, far):
    return {"op": "append", "T": T, "H": H, "Hkv": Hkv, "Dh": Dh, "rot": rot, "style": style, "page": page, "x": x, "drop": drop, "far": far}


def _attend(B, n, ctx, H, Hkv, Dh, page, mask, out, ragged=True):
    return {"op": "attend", "B": B, "n": n, "ctx": ctx, "H": H, "Hkv": Hkv, "Dh": Dh, "page": page, "mask": mask, "out": out, "ragged": ragged}


def _product(M, N, K, group, epi, c):
    return {"op": "product", "M": M, "N": N, "K": K, "group": group, "epi": epi, "c": c}


def _experts(G, P, N, K, group, c, empty):
    return {"op": "experts", "G": G, "P": P, "N": N, "K": K, "group": group, "c": c, "empty": empty}


def listed():
    return [
        # the new token of each of 32 sequences, one layer
        dict(_append(32, 32, 8, 128, 128, "halves", 64, "bf16", 0.0, 16384), name="append_step"),
        # the tokens of long prompts, one layer
        dict(_append(16384, 32, 8, 128, 128, "halves", 64, "bf16", 0.0, 16384), name="append_prompt"),
        # narrow heads rotated in part and in pairs, far positions, fp32 projections, tokens behind the last sequence
        dict(_append(5003, 14, 2, 64, 32, "pairs", 16, "f32", 0.05, 1000000), name="append_partial"),
        # plain decoding: one token for each of 32 sequences of about 4096
        dict(_attend(32, 1, 4096, 32, 8, 128, 64, "chain", "bf16"), name="attend_step"),
        # a tree of up to 64 drafted tokens for each of 16 sequences
        dict(_attend(16, 64, 8192, 32, 8, 128, 64, "tree", "bf16"), name="attend_tree"),
        # one token of one very long sequence
        dict(_attend(1, 1, 262143, 32, 8, 128, 128, "chain", "bf16", False), name="attend_long"),
        # a small tree behind a short context, narrow heads, small pages: latency
        dict(_attend(1, 7, 501, 12, 4, 64, 16, "tree", "f32", False), name="attend_short"),
        # chains of some hundred tokens: a prompt that goes in by parts
        dict(_attend(4, 500, 2000, 28, 4, 128, 32, "chain", "bf16"), name="attend_chunk"),
        # one token through a square projection of the benchmark's width
        dict(_product(1, 4096, 4096, 128, "none", "bf16"), name="product_token"),
        # 16 drafted tokens through a large one with an activation
        dict(_product(16, 8192, 8192, 128, "bias_silu", "bf16"), name="product_draft"),
        # more rows, small groups, odd sizes
        dict(_product(61, 1531, 2744, 32, "bias", "f32"), name="product_odd"),
        # the benchmark's experts for a step of 32 tokens, two experts each
        dict(_experts(64, 64, 1536, 4096, 128, "bf16", 20), name="product_experts"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "product", "experts"])
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        Dh = rng.choice([64, 128])
        H = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
        T = _log(rng, 1, min(16384, 16384 * 48 * 128 // ((H + 2 * Hkv) * Dh)))
        return _append(T, H, Hkv, Dh, rng.choice([0, 16, 32, Dh, Dh]), rng.choice(["halves", "pairs"]), rng.choice([16, 32, 64, 128]),
                       rng.choice(["bf16", "bf16", "f32"]), rng.choice([0.0, 0.1]), rng.choice([4096, 131072, 1000000]))
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        n = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 2, 64)])
        B = _log(rng, 1, 64)
        ctx = _log(rng, 1, min(32768, 2 ** 21 // (B * Hkv)))
        return _attend(B, n, ctx, H, Hkv, rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice(["tree", "tree", "chain"]),
                       rng.choice(["bf16", "f32"]))
    group = rng.choice([32, 64, 128])
    if op == "product":
        return _product(_log(rng, 1, 64), _log(rng, 64, 8192), _log(rng, 64, 8192), group, rng.choice(["none", "bias", "bias_silu", "bias_gelu"]),
                        rng.choice(["bf16", "f32"]))
    G = _log(rng, 2, 64)
    return _experts(G, _log(rng, 1, 256), _log(rng, 64, 1536), _log(rng, 64, 4096), group, rng.choice(["bf16", "f32"]), rng.randint(0, G // 2))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _up(n, m):
    return -(-n // m) * m


def _padded(x):
    """The same values in rows that begin on 16 bytes."""
    per = 16 // x.element_size()
    out = torch.zeros(*x.shape[:-1], _up(x.shape[-1], per), dtype=x.dtype, device=x.device)[..., :x.shape[-1]]
    out.copy_(x)
    return out


def _tree(rng, n):
    """Ancestors of each of n nodes, itself among them: each node hangs on the context or on an earlier node."""
    seen = np.zeros((n, n), dtype=bool)
    for i in range(n):
        parent = int(rng.integers(max(-1, i - 12), i)) if i else -1
        if parent >= 0:
            seen[i] = seen[parent]
        seen[i, i] = True
    return seen


def _words(seen, words):
    """Rows of truth values as rows of 32-bit words, bit j % 32 of word j // 32."""
    bits = np.zeros((seen.shape[0], words * 32), dtype=np.uint8)
    bits[:, :seen.shape[1]] = seen
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def _lengths(case):
    """The cached and the new tokens of each sequence: from half of the case's to all of them where the batch is ragged."""
    B, ctx, n = case["B"], case["ctx"], case["n"]
    if not case["ragged"]:
        return np.full(B, ctx), np.full(B, n)
    return np.linspace(ctx // 2, ctx, B).astype(np.int64), np.linspace(max(1, n // 2), n, B).astype(np.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(case)
    if case["op"] == "append":
        T, H, Hkv, Dh, page = case["T"], case["H"], case["Hkv"], case["Dh"], case["page"]
        # the projections of one layer, packed in one row a token
        qkv = torch.randn(T, (H + 2 * Hkv) * Dh, generator=g, device="cuda").to(TYPES[case["x"]])
        q, k, v = qkv.split([H * Dh, Hkv * Dh, Hkv * Dh], dim=1)
        s["q"], s["k"], s["v"] = q.view(T, H, Dh), k.view(T, Hkv, Dh), v.view(T, Hkv, Dh)
        pages = -(-T * 5 // (4 * page)) + 1
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
        live = T - int(T * case["drop"])
        slots[live:] = -1          # tokens behind the last sequence
        s["slots"], s["live"] = slots, live
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda() if half else None
        s["k_cache"] = torch.zeros(pages, page, Hkv, Dh, dtype=torch.bfloat16, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["q_out"] = torch.zeros(T, H, Dh, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "attend":
        B, n, H, Hkv, Dh, page = (case[x] for x in ("B", "n", "H", "Hkv", "Dh", "page"))
        ctx, new = _lengths(case)
        order = rng.permutation(B)       # which sequence is how long
        ctx, new = ctx[order], new[rng.permutation(B)]
        s["lens"] = [(int(c), int(m)) for c, m in zip(ctx, new)]
        offsets = np.concatenate([[0], np.cumsum(new)])
        T = int(offsets[-1])
        need = -(-(ctx + new) // page)
        pages = int(need.sum()) + 3
        order = rng.permutation(pages)
        table, at = np.zeros((B, int(need.max())), dtype=np.int32), 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + need[b]]
            at += int(need[b])
        s["table"] = torch.from_numpy(table).cuda()
        s["offsets"] = torch.from_numpy(offsets.astype(np.int32)).cuda()
        s["context"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
        s["starts"] = [int(o) for o in offsets]
        seen = None
        if case["mask"] == "tree":
            words = -(-n // 32)
            seen = [_tree(rng, int(m)) for m in new]
            s["mask"] = torch.from_numpy(np.concatenate([_words(x, words) for x in seen])).cuda()
        else:
            s["mask"] = None
        # what each sequence's rows see of its own new tokens, for the plain form
        s["seen"] = [torch.from_numpy(seen[b] if seen else np.tri(int(m), dtype=bool)).cuda() for b, m in enumerate(new)]
        s["k_cache"] = torch.randn(pages, page, Hkv, Dh, generator=g, device="cuda", dtype=torch.bfloat16)
        s["v_cache"] = torch.randn(pages, page, Hkv, Dh, generator=g, device="cuda", dtype=torch.bfloat16)
        s["q"] = torch.randn(T, H, Dh, generator=g, device="cuda", dtype=torch.bfloat16)
        s["out_buffer"] = torch.zeros(T, H, Dh, dtype=TYPES[case["out"]], device="cuda")
        s["scale"] = 1.0 / math.sqrt(Dh)
    else:
        N, K, group = case["N"], case["K"], case["group"]
        lead = (case["G"],) if case["op"] == "experts" else ()
        M = case["P"] if lead else case["M"]
        s["a"] = _padded(torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16))
        # two 4-bit numbers a byte, rows that begin on 16 bytes
        s["w"] = torch.randint(0, 256, (*lead, N, _up(-(-K // 2), 16)), generator=g, device="cuda", dtype=torch.uint8)[..., :-(-K // 2)]
        s["scales"] = _padded(((torch.rand(*lead, -(-K // group), N, generator=g, device="cuda") + 0.5) * 0.02).to(torch.bfloat16))
        s["bias"] = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) if case.get("epi", "none") != "none" else None
        per = 16 // torch.empty(0, dtype=TYPES[case["c"]]).element_size()
        s["c_buffer"] = torch.zeros(M, _up(N, per), dtype=TYPES[case["c"]], device="cuda")[:, :N]
        if lead:
            G = case["G"]
            share = rng.uniform(0.5, 1.5, G)
            share[rng.choice(G, case["empty"], replace=False)] = 0.0
            s["starts"] = [0] + [int(x) for x in np.cumsum(rng.multinomial(M, share / share.sum()))]
            s["offsets"] = torch.tensor(s["starts"], dtype=torch.int32, device="cuda")
    if own:
        import warp_specialized_tensor_gb300 as wst
        s["ws"] = {"append": wst.workspace, "attend": wst.tree_attention_workspace}.get(case["op"], wst.gemm_w4_workspace)()
    return s


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _rotated(x, positions, inv_freq, style):
    """x [T, heads, Dh] with its first 2 * len(inv_freq) components rotated."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()      # the angles of far positions need 64 bits
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    r = x.float().clone()
    if style == "halves":
        a, b = r[..., :half].clone(), r[..., half:2 * half].clone()
        r[..., :half], r[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = r[..., :2 * half:2].clone(), r[..., 1:2 * half:2].clone()
        r[..., :2 * half:2], r[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    return r


def _plain_append(s):
    live = s["live"]
    at = s["slots"][:live].long()
    q, k = s["q"][:live].float(), s["k"][:live].float()
    if s["inv_freq"] is not None:
        q = _rotated(q, s["positions"][:live], s["inv_freq"], s["style"])
        k = _rotated(k, s["positions"][:live], s["inv_freq"], s["style"])
    s["q_out"][:live] = q.to(torch.bfloat16)
    s["k_cache"].view(-1, *s["k"].shape[1:])[at] = k.to(torch.bfloat16)
    s["v_cache"].view(-1, *s["v"].shape[1:])[at] = s["v"][:live].to(torch.bfloat16)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attend(s):
    Hkv, Dh, page = s["Hkv"], s["Dh"], s["page"]
    group = s["H"] // Hkv
    for b, (ctx, n) in enumerate(s["lens"]):
        L, t0 = ctx + n, s["starts"][b]
        pages = s["table"][b, :-(-L // page)].long()
        k = s["k_cache"][pages].view(-1, Hkv, Dh)[:L].float().permute(1, 2, 0)        # [Hkv, Dh, L]
        v = s["v_cache"][pages].view(-1, Hkv, Dh)[:L].float().permute(1, 0, 2)        # [Hkv, L, Dh]
        q = s["q"][t0:t0 + n].float().view(n, Hkv, group, Dh).permute(1, 0, 2, 3).reshape(Hkv, n * group, Dh)
        x = torch.matmul(q, k).view(Hkv, n, group, L) * s["scale"]
        x[..., ctx:].masked_fill_(~s["seen"][b][None, :, None, :], -math.inf)
        p = torch.exp(x - x.amax(dim=-1, keepdim=True))
        o = torch.matmul(p.view(Hkv, n * group, L), v) / p.sum(dim=-1).view(Hkv, n * group, 1)
        s["out_buffer"][t0:t0 + n] = o.view(Hkv, n, group, Dh).permute(1, 0, 2, 3).reshape(n, s["H"], Dh).to(s["out_buffer"].dtype)
    return s["out_buffer"]


def _activated(x, bias, epi):
    if epi == "none":
        return x
    x = x + bias.float()
    if epi == "bias_silu":
        return x / (1.0 + torch.exp(-x))
    if epi == "bias_gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return x


def _weights(w, scales, K, group):
    """[N, K] fp32 of 4-bit weights and their scales."""
    q = torch.stack((w & 15, w >> 4), dim=-1).reshape(w.shape[0], -1)[:, :K].float() - 8.0
    return q * scales.float().T.repeat_interleave(group, dim=1)[:, :K]


def _plain_product(s):
    x = torch.matmul(s["a"].float(), _weights(s["w"], s["scales"], s["K"], s["group"]).T)
    s["c_buffer"].copy_(_activated(x, s["bias"], s["epi"]))
    return s["c_buffer"]


def _plain_experts(s):
    for e in range(s["G"]):
        a, b = s["starts"][e], s["starts"][e + 1]
        if b > a:
            s["c_buffer"][a:b] = torch.matmul(s["a"][a:b].float(), _weights(s["w"][e], s["scales"][e], s["K"], s["group"]).T).to(s["c_buffer"].dtype)
    return s["c_buffer"]


# ----------------------------------------------------------------------------
# the library's operators
# ----------------------------------------------------------------------------
def _own(s):
    import warp_specialized_tensor_gb300 as wst
    if s["op"] == "append":
        wst.wst_cache_append_bf16(s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"], inv_freq=s["inv_freq"],
                                  style=s["style"], q=s["q"], q_out=s["q_out"], workspace=s["ws"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if s["op"] == "attend":
        wst.wst_tree_attention_bf16(s["q"], s["offsets"], s["context"], s["k_cache"], s["v_cache"], s["table"], s["out_buffer"],
                                    mask=s["mask"], scale=s["scale"], workspace=s["ws"])
        return s["out_buffer"]
    if s["op"] == "product":
        wst.wst_gemm_w4(s["a"], s["w"], s["scales"], s["c_buffer"], group=s["group"], bias=s["bias"], epi=s["epi"], workspace=s["ws"])
    else:
        wst.wst_grouped_gemm_w4(s["a"], s["w"], s["scales"], s["offsets"], s["c_buffer"], group=s["group"], workspace=s["ws"])
    return s["c_buffer"]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "product": _plain_product, "experts": _plain_experts}[state["op"]](state)


# ----------------------------------------------------------------------------
# work, and the definitions in 64 bits
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] == "append":
        T, H, Hkv, Dh = case["T"], case["H"], case["Hkv"], case["Dh"]
        live = T - int(T * case["drop"])
        size = 4 if case["x"] == "f32" else 2
        return {"bytes": live * (H + 2 * Hkv) * Dh * (size + 2) + 8 * T, "flops": live * (H + Hkv) * case["rot"] * 3}
    if case["op"] == "attend":
        B, n, H, Hkv, Dh = (case[x] for x in ("B", "n", "H", "Hkv", "Dh"))
        lengths = _lengths(case)
        ctx, new = float(lengths[0].mean()), float(lengths[1].mean())
        size = 4 if case["out"] == "f32" else 2
        visible = ctx + (new + 1) / 2
        return {"bytes": int(B * ((ctx + new) * Hkv * Dh * 4 + new * H * Dh * (2 + size) + 4 * (ctx + new) / case["page"])),
                "flops": int(B * new * H * Dh * 4 * visible)}
    N, K = case["N"], case["K"]
    M = case["M"] if case["op"] == "product" else case["P"]
    size = 4 if case["c"] == "f32" else 2
    # every expert that has a row reads its weights
    used = 1
    if case["op"] == "experts":
        full = case["G"] - case["empty"]
        used = full * (1.0 - (1.0 - 1.0 / full) ** M)
    return {"bytes": int(used * (N * -(-K // 2) + 2 * N * -(-K // case["group"])) + 2 * M * K + size * M * N), "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        T, H, Hkv, Dh, live = case["T"], case["H"], case["Hkv"], case["Dh"], s["live"]
        k_cache, v_cache = s["k_cache"].double().reshape(-1, Hkv, Dh), s["v_cache"].double().reshape(-1, Hkv, Dh)
        q_out = s["q_out"].double()
        at = s["slots"][:live].long()

        def turned(x):
            x = x[:live].double()
            if s["inv_freq"] is None:
                return x
            rot = case["rot"]
            z = torch.polar(torch.ones(live, rot // 2, dtype=torch.float64, device="cuda"), torch.outer(s["positions"][:live].double(), s["inv_freq"].double()))
            if case["style"] == "pairs":
                pair = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * z[:, None]
                head = torch.view_as_real(pair).reshape(live, -1, rot)
            else:
                pair = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z[:, None]
                head = torch.cat((pair.real, pair.imag), dim=-1)
            return torch.cat((head, x[..., rot:]), dim=-1)

        q_out[:live] = turned(s["q"])
        k_cache[at], v_cache[at] = turned(s["k"]), s["v"][:live].double()
        shape = s["k_cache"].shape
        return q_out, k_cache.view(shape), v_cache.view(shape)
    if case["op"] == "attend":
        group = case["H"] // case["Hkv"]
        out = torch.zeros(s["out_buffer"].shape, dtype=torch.float64, device="cuda")
        for b, (ctx, n) in enumerate(s["lens"]):
            key = torch.arange(ctx + n, device="cuda")
            page, row = s["table"][b].long()[key // case["page"]], key % case["page"]
            t0 = s["starts"][b]
            open_ = torch.ones(n, ctx + n, dtype=torch.bool, device="cuda")
            open_[:, ctx:] = s["seen"][b]
            for h in range(case["H"]):
                k, v = s["k_cache"][page, row, h // group].double(), s["v_cache"][page, row, h // group].double()
                x = (s["q"][t0:t0 + n, h].double() @ k.T) * s["scale"]
                out[t0:t0 + n, h] = torch.softmax(torch.where(open_, x, -math.inf), dim=1) @ v
        return out
    N, K, group = case["N"], case["K"], case["group"]

    def product(a, w, scales):
        even, odd = (w & 15).double() - 8, (w >> 4).double() - 8
        k = torch.arange(K, device="cuda")
        total = torch.zeros(a.shape[0], N, dtype=torch.float64, device="cuda")
        for parity, q in ((0, even), (1, odd)):
            at = k[k % 2 == parity]
            total += a[:, at].double() @ (q[:, at // 2] * scales.double()[at // group].T).T
        return total

    if case["op"] == "experts":
        out = torch.zeros(s["c_buffer"].shape, dtype=torch.float64, device="cuda")
        for e, (i, j) in enumerate(zip(s["starts"][:-1], s["starts"][1:])):
            if j > i:
                out[i:j] = product(s["a"][i:j], s["w"][e], s["scales"][e])
        return out
    x = product(s["a"], s["w"], s["scales"])
    if case["epi"] != "none":
        x = x + s["bias"].double()
    if case["epi"] == "bias_silu":
        x = x * torch.sigmoid(x)
    elif case["epi"] == "bias_gelu":
        x = x * 0.5 * torch.erfc(-x / math.sqrt(2.0))
    return x
