"""CPU model of the barriers of the MXFP4 products (k_mx4gemm.cu): the pair kernel's two producers, its MMA issuer and
sixteen epilogue warps, and the split kernel's ring. Roles run in random order, copies and MMAs complete at
random times. Every wait must be for a phase that has really completed, every MMA must read the stage it was issued
for, no accumulator column may be overwritten before it was drained, and every schedule must finish."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_gemm_moe_b200", "csrc", "k_mx4gemm.cu")


class Unsound(Exception):
    pass


class Barrier:
    """An mbarrier: `done` phases completed; a wait for phase p tests the parity of p, as the hardware does."""

    def __init__(self, count):
        self.count, self.pending, self.tx, self.done = count, count, 0, 0

    def _check(self):
        if self.pending == 0 and self.tx == 0:
            self.done += 1
            self.pending = self.count

    def arrive(self, expect=0):
        if self.pending == 0:
            raise Unsound("an arrival too many")
        self.tx += expect
        self.pending -= 1
        self._check()

    def bytes_in(self, n):
        self.tx -= n
        self._check()

    def ready(self, phase):
        if (self.done & 1) == (phase & 1):
            return False  # the phase of this parity is open
        if self.done != phase + 1:
            raise Unsound(f"a wait for phase {phase} passes after {self.done} phases")
        return True


class Engine:
    """Roles (generators that yield a condition to wait for, or None), copies in flight, and tensor operations in order."""

    def __init__(self, rng):
        self.rng, self.roles, self.copies, self.tensor = rng, [], [], []

    def run(self):
        waiting = {r: None for r in self.roles}
        while waiting or self.copies or self.tensor:
            choices = [("role", r) for r, c in waiting.items() if c is None or c()]
            choices += [("copy", i) for i in range(len(self.copies))]
            if self.tensor:
                choices.append(("tensor", 0))
            if not choices:
                raise Unsound("nothing can go on")
            kind, x = self.rng.choice(choices)
            if kind == "role":
                try:
                    waiting[x] = next(x)
                except StopIteration:
                    del waiting[x]
            elif kind == "copy":
                self.copies.pop(x)()
            else:
                self.tensor.pop(0)()


def pair(rng, NS, KS, tiles, warps=16, freed_early=False, freed_count=None):
    """One pair of CTAs over `tiles` tiles of KS stages. freed_early: the drained columns are announced before they are
    read; freed_count: arrivals that complete the announcement."""
    e = Engine(rng)
    full = [Barrier(1) for _ in range(NS)]                                # the even CTA's
    empty = [[Barrier(1) for _ in range(NS)] for _ in range(2)]
    accf = [[Barrier(1) for _ in range(2)] for _ in range(2)]
    freed = Barrier(freed_count or warps)
    ring = [[None] * NS for _ in range(2)]
    # accumulator columns of each CTA: "a" and "s" of the first accumulator, "s" (shared) and "b" of the second
    cols = [{"a": (None, 0), "s": (None, 0), "b": (None, 0)} for _ in range(2)]  # region: (tile, chunks not yet read)
    own = {0: ("s", "a"), 1: ("s", "b")}
    reads = {"s": warps // 2, "a": 3 * warps // 2, "b": 3 * warps // 2}    # chunks of 32 columns, per CTA

    def producer(cta):
        for it in range(tiles * KS):
            s = it % NS
            yield lambda s=s, it=it: empty[cta][s].ready(it // NS - 1)
            if cta == 0:
                full[s].arrive(expect=2)

            def land(s=s, it=it):
                ring[cta][s] = it
                full[s].bytes_in(1)

            e.copies.append(land)
            yield None

    def issuer():
        for it in range(tiles * KS):
            n, ks, s = it // KS, it % KS, it % NS
            if ks == 0 and n > 0:
                yield lambda n=n: freed.ready(n - 1)
            yield lambda s=s, it=it: full[s].ready(it // NS)

            def mma(n=n, ks=ks, s=s, it=it):
                for c in range(2):
                    if ring[c][s] != it:
                        raise Unsound("an MMA reads another stage's data")
                    for r in own[n & 1]:
                        tile, left = cols[c][r]
                        if ks == 0 and left:
                            raise Unsound("an accumulator is overwritten before it was read")
                        if ks and tile != n:
                            raise Unsound("an accumulator changed hands")
                        cols[c][r] = (n, reads[r])

            def commit(bars):
                return lambda: [b.arrive() for b in bars]

            e.tensor.append(mma)
            e.tensor.append(commit([empty[0][s], empty[1][s]]))
            if ks == KS - 1:
                e.tensor.append(commit([accf[0][n & 1], accf[1][n & 1]]))
            yield None

    def epilogue(cta):
        for n in range(tiles):
            yield lambda n=n: accf[cta][n & 1].ready(n >> 1)
            shared, rest = own[n & 1]
            if freed_early:
                freed.arrive()
                yield None
            for j, region in enumerate((shared, rest, rest, rest)):
                tile, left = cols[cta][region]
                if tile != n or left < 1:
                    raise Unsound("an epilogue warp reads another tile's sums")
                cols[cta][region] = (tile, left - 1)
                yield None
                if j == 0 and not freed_early:
                    freed.arrive()
                    yield None

    e.roles = [producer(0), producer(1), issuer()] + [epilogue(w & 1) for w in range(warps)]
    e.run()
    assert all(left == 0 for c in cols for r, (_, left) in c.items())


def split(rng, NS, nk):
    """The split kernel's ring: the first stages' weights and activations are issued before any is consumed."""
    e = Engine(rng)
    full, empty, accf, ring = [Barrier(1) for _ in range(NS)], [Barrier(1) for _ in range(NS)], Barrier(1), [[None, None] for _ in range(NS)]
    sums = []

    def load(it, part):
        s = it % NS

        def land():
            ring[s][part] = it
            full[s].bytes_in(1)

        if part == 0:
            full[s].arrive(expect=2)
        e.copies.append(land)

    def producer():
        ahead = min(nk, NS)
        for part in (0, 1):
            for it in range(ahead):
                load(it, part)
                yield None
        for it in range(ahead, nk):
            yield lambda it=it: empty[it % NS].ready(it // NS - 1)
            load(it, 0)
            load(it, 1)

    def issuer():
        for it in range(nk):
            s = it % NS
            yield lambda s=s, it=it: full[s].ready(it // NS)

            def mma(s=s, it=it):
                if ring[s] != [it, it]:
                    raise Unsound("an MMA reads another stage's data")
                sums.append(it)

            e.tensor += [mma, lambda s=s: empty[s].arrive()]
            if it == nk - 1:
                e.tensor.append(accf.arrive)
            yield None

    def epilogue():
        yield lambda: accf.ready(0)
        assert sums == list(range(nk))

    e.roles = [producer(), issuer(), epilogue()]
    e.run()


def test_model_has_the_kernels_stages():
    with open(SRC) as f:
        src = f.read()
    assert re.search(r"static constexpr int kStages = 6;", src) and re.search(r"kEpiWarps = 8;", src)
    assert re.search(r"mbar_init\(freed, 2 \* C::kEpiWarps\)", src)
    assert re.search(r"split_stages\(int bn\) \{ return 114176 / split_stage_bytes\(bn\); \}", src)


@pytest.mark.parametrize("KS", [1, 2, 5, 6, 7, 13])
@pytest.mark.parametrize("tiles", [1, 2, 3, 6])
def test_pair_protocol(KS, tiles):
    for seed in range(12):
        pair(random.Random(1000 * KS + 10 * tiles + seed), 6, KS, tiles)


@pytest.mark.parametrize("mistake", [dict(freed_early=True), dict(freed_count=8)])
def test_pair_model_catches_an_early_release(mistake):
    """Columns announced before they are read, or by half of the warps, must be found out by some schedule."""
    caught = 0
    for seed in range(60):
        try:
            pair(random.Random(seed), 6, 2, 4, **mistake)
        except Unsound:
            caught += 1
    assert caught > 0


@pytest.mark.parametrize("NS", [3, 4, 5])  # 128, 64 and 16 tokens
@pytest.mark.parametrize("nk", [1, 2, 3, 4, 5, 9, 29])
def test_split_protocol(NS, nk):
    for seed in range(20):
        split(random.Random(100 * nk + seed), NS, nk)
