"""The 8-bit product's hand-over of stages and accumulators, checked on the CPU.

The kernel (csrc/fp8_gemm.cuh) has a ring of stages that one producer fills,
two issuers that take a unit's even and odd K blocks with an accumulator each,
and an epilogue that adds the blocks in order.  A wait names only the parity
of a barrier's phase, so it also passes when the barrier is one phase behind
what the waiting role means: a wait is right only where something else keeps
the two from drifting that far apart.  This test restates the roles and lets
copies complete in any order; an issuer must never multiply a stage whose
copies are not complete, whatever the number of K blocks in a unit.

The split form's epilogue counts in through a barrier of its warps; a warp that
gave up must leave the loop together with the others, or they wait for it."""
import os
import random
import re

import pytest

STAGES = 5
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "warp_specialized_tensor_gb300", "csrc",
                      "fp8_gemm.cuh")


def passes(completed, parity):
    """mbarrier.try_wait.parity on a barrier of which `completed` phases are complete."""
    return (completed & 1) != parity


class Pair:
    """One CTA pair; `order` is what an issuer waits for first."""

    def __init__(self, unit, units, order, rng):
        self.owner = [(b % unit) & 1 for b in range(unit * units)]
        self.order, self.rng = order, rng
        self.full, self.empty, self.accf, self.acce = [0] * STAGES, [0] * STAGES, [0, 0], [0, 0]
        self.loaded = 0                      # blocks the producer has asked for
        self.flying = []                     # blocks whose copies are under way
        self.at = [0, 0]                     # each issuer's next block
        self.waits = [0, 0]                  # how many of its two waits it has passed
        self.used = [0, 0]                   # blocks it has issued
        self.done = 0                        # blocks the epilogue has added
        self.phase = [0, 0]                  # the epilogue's uses of each accumulator
        self.early = 0                       # products on a stage that was not complete

    def producer(self):
        b = self.loaded
        if b == len(self.owner) or not passes(self.empty[b % STAGES], (b // STAGES & 1) ^ 1):
            return False
        self.loaded += 1
        self.flying.append(b)
        return True

    def copy(self, i):
        b = self.flying.pop(i)
        self.full[b % STAGES] += 1

    def issuer(self, me):
        while self.at[me] < len(self.owner) and self.owner[self.at[me]] != me:
            self.at[me] += 1
        b = self.at[me]
        if b == len(self.owner):
            return False
        s = b % STAGES
        full = passes(self.full[s], b // STAGES & 1)
        acc = passes(self.acce[me], (self.used[me] & 1) ^ 1)
        first, second = (full, acc) if self.order == "stage" else (acc, full)
        if not (first if self.waits[me] == 0 else second):
            return False
        self.waits[me] += 1
        if self.waits[me] < 2:
            return True
        if self.full[s] <= b // STAGES:
            self.early += 1
        self.waits[me] = 0
        self.used[me] += 1
        self.at[me] += 1
        self.accf[me] += 1
        self.empty[s] += 1
        return True

    def epilogue(self):
        if self.done == len(self.owner):
            return False
        a = self.owner[self.done]
        if not passes(self.accf[a], self.phase[a] & 1):
            return False
        self.phase[a] += 1
        self.acce[a] += 1
        self.done += 1
        return True

    def run(self):
        rng = self.rng
        for _ in range(400 * len(self.owner)):
            if self.done == len(self.owner) or self.early:
                break
            what = rng.randrange(8)
            if what < 2:
                self.producer()
            elif what == 2 and self.flying:
                self.copy(rng.randrange(len(self.flying)))   # in any order
            elif what < 6:
                self.issuer(what & 1)
            elif what == 6:
                self.epilogue()
        return self


@pytest.mark.parametrize("unit", [1, 2, 3, 4, 5, 6, 7, 11])
def test_no_product_before_its_copies(unit):
    for seed in range(300):
        p = Pair(unit, 40 // unit + 2, "accumulator", random.Random(seed))
        p.run()
        assert p.early == 0
        assert p.done == len(p.owner)


def test_the_other_order_of_the_waits_is_wrong():
    # With three K blocks a unit, an issuer's blocks are up to three apart and the
    # stage between may be a lap behind: the accumulator has to come first.
    assert any(Pair(3, 16, "stage", random.Random(seed)).run().early for seed in range(300))


def test_the_kernel_waits_in_that_order():
    text = open(SOURCE).read()
    issuer = text[text.index("MMA issuers (leader)"):text.index("umma_commit_pair(accf_bar(mine)")]
    waits = re.findall(r"f8_wait<false>\(guard, (\w+)\(", issuer)
    assert waits == ["acce_bar", "full_bar"]


def leave(units, rule, rng, warps=8):
    """The warps of the split epilogue: True if none is left waiting for another.

    A warp's wait for a unit's blocks may run out (or find that another's did); the
    rule says whether it then leaves by itself or by what warp 4 wrote down
    between the two barriers."""
    abort, last = False, None
    state = [dict(unit=0, bar=0, ok=True) for _ in range(warps)]   # bar: barriers passed in this unit
    out = [False] * warps
    waiting = [False] * warps
    for _ in range(5000):
        live = [w for w in range(warps) if not out[w]]
        if not live:
            return True
        ready = [w for w in live if not waiting[w]]
        if not ready:
            if len(live) < warps:
                return False                                       # (a warp that left does not come to the barrier)
            waiting = [False] * warps
            for s in state:
                s["bar"] += 1
            continue
        w = rng.choice(ready)
        s = state[w]
        if s["bar"] == 0:
            if s["unit"] == units:
                out[w] = True
                continue
            if s["ok"] and rng.random() < (0.5 if abort else 0.1):
                s["ok"], abort = False, True
            waiting[w] = True
        elif s["bar"] == 1:
            if w == 0:
                last = "given up" if abort else "store"
            waiting[w] = True
        else:
            if (not s["ok"]) if rule == "alone" else last == "given up":
                out[w] = True
                continue
            s["unit"] += 1
            s["bar"] = 0
    return False


def test_warps_that_give_up_leave_together():
    for seed in range(500):
        assert leave(4, "together", random.Random(seed))
    assert not all(leave(4, "alone", random.Random(seed)) for seed in range(500))


def test_the_kernel_leaves_by_what_was_written_down():
    text = open(SOURCE).read()
    split = text[text.index("if (un.split >= 0) {"):]
    after = split[:split.index("const float* parts")].split("bar.sync 1")[2]
    assert re.findall(r"if \(([^)]*)\) (break|continue);", after) == [("last == 2u", "break"), ("last == 0u", "continue")]


@pytest.fixture(scope="module")
def splits(tmp_path_factory):
    """The kernel's own rule, compiled for the host."""
    import ctypes
    import subprocess
    text = open(SOURCE).read()
    body = re.search(r"__host__ __device__ inline (int f8_splits\(.*?\n}\n)", text, re.S).group(1)
    tile = re.search(r"constexpr int kF8Tile = (\d+);", text).group(1)
    units = int(re.search(r"constexpr int kF8MaxUnits = (\d+);", text).group(1))
    d = tmp_path_factory.mktemp("splits")
    (d / "s.cpp").write_text("constexpr int kF8Tile = %s;\nextern \"C\" %s" % (tile, body))
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(d / "s.so"), str(d / "s.cpp")], check=True)
    fn = ctypes.CDLL(str(d / "s.so")).f8_splits
    fn.argtypes = [ctypes.c_longlong] + [ctypes.c_int] * 4
    return lambda tiles, pairs, M, K: fn(tiles, pairs, -(-K // 128), units, M)


@pytest.mark.parametrize("pairs", [70, 74, 76])
def test_the_sizes_meant_to_split_do(splits, pairs):
    from test_gpu_fp8 import SPLIT_DENSE, SPLIT_GROUPED
    for M, N, K in SPLIT_DENSE:
        tiles = -(-M // 256) * -(-N // 256)
        assert 2 <= splits(tiles, pairs, M, K) <= pairs // tiles
    for sizes, N, K in SPLIT_GROUPED:
        tiles = sum(-(-s // 256) for s in sizes) * -(-N // 256)
        assert 2 <= splits(tiles, pairs, sum(sizes) + 7, K) <= pairs // tiles


def test_the_rule_keeps_every_unit_on_a_pair_of_its_own(splits):
    rng = random.Random(0)
    for _ in range(5000):
        tiles, pairs, M, K = rng.randrange(0, 200), rng.randrange(1, 80), rng.randrange(1, 5000), rng.randrange(1, 20000)
        s = splits(tiles, pairs, M, K)
        assert s >= 1 and (s == 1 or (s * tiles <= min(pairs, 120) and s <= -(-K // 128)))
