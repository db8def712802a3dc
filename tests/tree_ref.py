"""A paged cache with its sequences, and attention over it in 64 bits, for the tests."""
import numpy as np
import torch


def tree(rng, n, roots=0.1):
    """Which new tokens each of n nodes sees: itself and its ancestors."""
    seen = np.zeros((n, n), dtype=bool)
    for i in range(n):
        if i and rng.random() > roots:
            seen[i] = seen[rng.integers(0, i)]
        seen[i, i] = True
    return seen


def words(seen, count):
    bits = np.zeros((seen.shape[0], count * 32), dtype=np.uint8)
    bits[:, :seen.shape[1]] = seen
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


class Paged:
    """B sequences of (context, new tokens), their keys and values, the cache filled with NaN everywhere else, and
    page tables with rubbish behind each sequence's last page."""

    def __init__(self, lens, H, Hkv, Dh, page, mask="tree", seed=0, layout="plain", size=1.0, behind=0, spare_words=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.Hkv, self.Dh, self.page = lens, H, Hkv, Dh, page
        need = [-(-(c + n) // page) for c, n in lens]
        self.pages = sum(need) + 2
        self.max_pages = max(need + [1]) + 1
        self.T = sum(n for _, n in lens) + behind
        self.q = (torch.randn(self.T, H, Dh, generator=g, device="cuda") * size).bfloat16()
        self.K = [torch.randn(c + n, Hkv, Dh, generator=g, device="cuda").bfloat16() for c, n in lens]
        self.V = [torch.randn(c + n, Hkv, Dh, generator=g, device="cuda").bfloat16() for c, n in lens]
        shape = {"plain": (self.pages, page, Hkv, Dh), "heads": (self.pages, Hkv, page, Dh), "both": (self.pages, 2, page, Hkv, Dh + 8)}[layout]
        caches = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        if layout == "heads":
            caches = [c.transpose(1, 2) for c in caches]
        if layout == "both":
            caches = [caches[0][:, 0, ..., :Dh], caches[0][:, 1, ..., :Dh]]
        self.k_cache, self.v_cache = caches
        order = rng.permutation(self.pages)
        table = rng.integers(-2 ** 31, 2 ** 31 - 1, (len(lens), self.max_pages)).astype(np.int32)
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k
        self.table = torch.from_numpy(table).cuda()
        starts = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
        self.starts = starts.tolist()
        self.offsets = torch.from_numpy(starts).cuda()
        self.context = torch.tensor([c for c, _ in lens], dtype=torch.int32, device="cuda")
        if mask == "tree":
            self.seen = [tree(rng, n) for _, n in lens]
        elif mask == "chain":
            self.seen = [np.tri(n, dtype=bool) for _, n in lens]
        else:  # any set of the new tokens, some empty
            self.seen = [(rng.random((n, n)) < 0.4) & (rng.random((n, 1)) < 0.8) for _, n in lens]
        self.mask = None
        if mask != "chain":
            count = -(-max([n for _, n in lens] + [1]) // 32) + spare_words
            rows = [words(s, count) for s in self.seen] + [np.full((behind, count), -1, dtype=np.int32)]
            # bits behind a sequence's last new token mean nothing
            for (c, n), r in zip(lens, rows):
                extra = words(np.arange(count * 32)[None, :] >= n, count)
                r |= extra
            self.mask = torch.from_numpy(np.concatenate(rows)).cuda()
        self.fill()

    def fill(self):
        for b, (c, n) in enumerate(self.lens):
            key = torch.arange(c + n, device="cuda")
            pg = self.table[b].long()[key // self.page]
            self.k_cache[pg, key % self.page] = self.K[b]
            self.v_cache[pg, key % self.page] = self.V[b]

    def want(self, scale):
        """The result in 64 bits, [tokens, H, Dh], sum p |v| and the largest scale * sum |q k| of a row."""
        out = torch.zeros(self.starts[-1], self.H, self.Dh, dtype=torch.float64, device="cuda")
        size, most = torch.zeros_like(out), torch.zeros(*out.shape[:2], 1, dtype=torch.float64, device="cuda")
        g = self.H // self.Hkv
        for b, (c, n) in enumerate(self.lens):
            if n == 0:
                continue
            seen = torch.ones(n, c + n, dtype=torch.bool, device="cuda")
            seen[:, c:] = torch.from_numpy(self.seen[b]).cuda()
            rows = slice(self.starts[b], self.starts[b] + n)
            for h in range(self.H):
                q, k, v = self.q[rows, h].double(), self.K[b][:, h // g].double(), self.V[b][:, h // g].double()
                x = torch.where(seen, q @ k.T * scale, -float("inf"))
                top = x.amax(dim=1, keepdim=True)
                p = torch.where(seen, torch.exp(x - torch.where(top.isfinite(), top, 0.0)), 0.0)
                total = p.sum(dim=1, keepdim=True)
                p = torch.where(total > 0, p / total, 0.0)
                out[rows, h], size[rows, h] = p @ v, p @ v.abs()
                most[rows, h] = (torch.where(seen, q.abs() @ k.abs().T, 0.0)).amax(dim=1, keepdim=True) * abs(scale)
        return out, size, most

    def tolerance(self, out, size, most, dtype):
        """P is off by half a step of bf16 (for fp32 output by half a step of the last of three bf16, at most 2^-24); a
        score's Dh products are added with an error of at most 2^-22 of their sizes in each of Dh/16 steps, a score's
        error counts twice (P and the sum of P), 2^x and the scaling are good to 2^-21; an output adds 8 steps (three
        times 8 for three parts) of at most 2^-22 for every 128 keys; then the rounding of the result."""
        blocks = max(c + n for c, n in self.lens) / 128 + 2
        parts = 1 if dtype is torch.bfloat16 else 3
        part = 2.0 ** (-8 * parts) + 2 * (self.Dh / 16 * 2.0 ** -22 * most + 2.0 ** -21 * (1 + most)) + 8 * parts * blocks * 2.0 ** -22
        half = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
        return part * size + half * (out.abs() + part * size)
