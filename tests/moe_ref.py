"""Plain 64-bit implementations (numpy, CPU) of the mixture-of-experts operators,
and tolerances derived from the arithmetic the kernels do.  u = 2^-24 is half a
unit of fp32, `half(t)` the rounding of an output type."""
import numpy as np
import torch

U = 2.0 ** -24
OFF = -3.0e38


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def scores(x, score):
    """s [T, E]: 0 where the expert is off."""
    off = x <= OFF
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.where(off, 0.0, 1.0 / (1.0 + np.exp(-x)))
        top = np.where(off, -np.inf, x).max(axis=1, keepdims=True)
        e = np.where(off, 0.0, np.exp(x - np.where(np.isneginf(top), 0.0, top)))
        total = e.sum(axis=1, keepdims=True)
        return np.where(off, 0.0, e / np.where(total == 0, 1.0, total))


def order(v):
    """Indices by descending value, NaN first, ties to the lower index."""
    return np.lexsort((np.arange(v.size), -np.where(np.isnan(v), 0.0, v), ~np.isnan(v)))


def route(x, k, score, bias=None, groups=1, top_groups=1, group_best=1, renorm=True, scale=1.0):
    s = scores(x, score)
    off = x <= OFF
    v = s if bias is None else s + bias
    T, E = x.shape
    experts = np.full((T, k), -1, dtype=np.int64)
    weights = np.zeros((T, k))
    for t in range(T):
        dead = off[t] | np.isneginf(v[t])
        allowed = ~dead
        if groups > 1 and top_groups < groups:
            total = np.full(groups, -np.inf)
            for g in range(groups):
                m = np.arange(g * (E // groups), (g + 1) * (E // groups))
                m = m[~dead[m]]
                if m.size:
                    best = m[order(v[t, m])][:group_best]
                    total[g] = v[t, best].sum()
            kept = order(total)[:top_groups]
            allowed &= np.isin(np.arange(E) // (E // groups), kept)
        # without a bias the logits themselves rank the experts (the same order, by finer values)
        value = x[t] if bias is None and not np.isnan(v[t]).any() else v[t]
        idx = np.nonzero(allowed)[0]
        idx = idx[order(value[idx])][:k]
        experts[t, :idx.size] = idx
        w = s[t, idx]
        weights[t, :idx.size] = scale * (w / w.sum() if renorm and idx.size else w)
    return experts, weights


def route_backward(x, experts, dw, score, renorm, scale):
    """The gradient and the sum of its terms' sizes, from which bounds follow."""
    T, E = x.shape
    s = scores(x, score)
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        slots = [i for i in range(experts.shape[1]) if 0 <= experts[t, i] < E and x[t, experts[t, i]] > OFF]
        e = experts[t, slots]
        g = scale * dw[t, slots]
        if renorm and slots:
            p = s[t, e] / s[t, e].sum()
            mean, amean = (p * g).sum(), (p * abs(g)).sum()
            d = p * (g - mean) * ((1 - s[t, e]) if score == "sigmoid" else 1.0)
            a = p * (abs(g) + amean) * ((1 - s[t, e]) if score == "sigmoid" else 1.0)
            np.add.at(grad[t], e, d)
            np.add.at(size[t], e, a)
        elif score == "sigmoid":
            np.add.at(grad[t], e, g * s[t, e] * (1 - s[t, e]))
            np.add.at(size[t], e, abs(g) * s[t, e] * (1 - s[t, e]))
        else:
            ds, ads = np.zeros(E), np.zeros(E)
            np.add.at(ds, e, g)
            np.add.at(ads, e, abs(g))
            grad[t] = s[t] * (ds - (ds * s[t]).sum())
            size[t] = s[t] * (ads + (ads * s[t]).sum())
    return grad, size


def plan(experts, E):
    flat = experts.reshape(-1)
    k = experts.shape[1]
    live = np.nonzero((flat >= 0) & (flat < E))[0]
    rows = live[np.argsort(flat[live], kind="stable")]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[live], minlength=E))])
    row_pair = np.full(flat.size, -1)
    row_pair[:rows.size] = rows
    row_token = np.where(row_pair >= 0, row_pair // k, -1)
    position = np.full(flat.size, -1)
    position[rows] = np.arange(rows.size)
    return offsets, row_pair, row_token, position.reshape(experts.shape)


def combine(y, position, w):
    """The sum and the sum of its terms' sizes."""
    out, size = np.zeros((position.shape[0], y.shape[1])), np.zeros((position.shape[0], y.shape[1]))
    for t, row in enumerate(position):
        for i, p in enumerate(row):
            if 0 <= p < y.shape[0]:
                out[t] += w[t, i] * y[p]
                size[t] += abs(w[t, i] * y[p])
    return out, size


def quantise(x, mode, dtype, pow2=False):
    """q (the 8-bit tensor) and the scales of x [M, K] (a CPU tensor), each fp32 operation done in fp32."""
    x = x.float().numpy()
    M, K = x.shape
    largest = np.float32(torch.finfo(dtype).max)
    bm, bk = {"rows": (1, 128), "cols": (128, 1)}.get(mode, (128, 128))
    pad = np.zeros((-(-M // bm) * bm, -(-K // bk) * bk), dtype=np.float32)
    pad[:M, :K] = x
    b = pad.reshape(pad.shape[0] // bm, bm, pad.shape[1] // bk, bk)
    amax = np.maximum(np.abs(b).max(axis=(1, 3)), np.float32(2.0 ** -100))  # (maximum keeps NaN)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if pow2:
            e = np.ceil(np.log2(amax.astype(np.float64) / float(largest)))
            scale = np.where(np.isfinite(amax), np.exp2(np.where(np.isfinite(e), e, 0)), amax).astype(np.float32)
        else:
            scale = amax * np.float32(1.0 / float(largest))
        v = b * (np.float32(1.0) / scale)[:, None, :, None]
    v = np.ascontiguousarray(v.reshape(pad.shape)[:M, :K])
    q = torch.from_numpy(np.clip(v, -largest, largest)).to(dtype)
    if mode == "cols":
        return q.t().contiguous(), scale
    if mode == "blocks_t":
        return q.t().contiguous(), np.ascontiguousarray(scale.T)
    return q, (np.ascontiguousarray(scale.T) if mode == "rows" else scale)


def values(q, scale, mode):
    """The numbers that q [M, K] (scales of mode "rows" or "blocks") stands for, in 64 bits."""
    q, scale = f64(q), np.asarray(scale, dtype=np.float64)
    M, K = q.shape
    each = scale.T if mode == "rows" else np.repeat(scale, 128, axis=0)[:M]
    return q * np.repeat(each, 128, axis=1)[:, :K]
