"""The barriers of the prompt attention kernel (csrc/prompt_attn.cu) as a model on the host, under schedules in which any warp,
copy or MMA may be late.

A wait looks at the parity of a barrier's phase, so a warp that looks only after the phase behind it has ended too takes it
for one that is still to come, and waits for ever.  Each agent (the loading warp, the two that issue MMAs, two softmax warps
of each warpgroup, two that widen codes, every copy in flight, the tensor cores) is slow or fast at random, for a time; what
a tile, the queries, S or O hold is checked where it is read.  The order of waits and arrivals is the kernel's; `without`
takes one of them out, and the schedules then have to find that.
"""
import os
import random
import re

import pytest

STAGES, OUT, WARPS = 5, 3, 2   # bf16: stages, the first one of those that the output passes through; warps of a warpgroup


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, "an arrival too many"
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return self.phase & 1 != parity & 1


class Ring:
    """bf16: the order in which a part's tiles are loaded, and their stages."""

    def __init__(self):
        self.ph = [0] * (STAGES + 1)

    def part(self, one, count):
        self.one, self.count, self.total, self.n = one, count, 2 * count, STAGES + one

    def block(self, t):
        if not self.one:
            return t >> 1, t & 1
        first, w = t >> 2 << 1, t & 3
        if first + 1 < self.count:
            return first + (w & 1), int(w >= 2)
        return first, int(w == 1)

    def at(self, t):
        return t % self.n, (self.ph[t % self.n] ^ t // self.n) & 1

    def k(self, b):
        return self.at(4 * (b >> 1) + (b & 1) if self.one else 2 * b)

    def v(self, b):
        if not self.one:
            return self.at(2 * b + 1)
        return self.at(4 * (b >> 1) + (2 + (b & 1) if b | 1 < self.count else 1))

    def out(self, b):
        st = OUT + (1 if self.one else b)
        return st, self.ph[st] ^ 1

    def done(self):
        for st in range(self.n):
            self.ph[st] ^= (self.total // self.n + (st < self.total % self.n)) & 1


class Ring8:
    """E4M3: four stages of K's codes, two of V's values (4 and 5), taken by the blocks of all parts in turn."""

    def __init__(self):
        self.base = 0

    def part(self, one, count):
        self.one, self.count = one, count

    def k(self, b):
        n = self.base + b
        return n & 3, n >> 2 & 1

    def v(self, b):
        n = self.base + b
        return 4 + (n & 1), n >> 1 & 1

    def out(self, b):
        st = 0 if self.one else b
        return 4 + st, (self.base + 1 - st >> 1) - 1 & 1

    def done(self):
        self.base += self.count


class Kernel:
    def __init__(self, parts, fp8, rng, without=()):
        """parts: (one tile of rows, blocks, whole) each."""
        self.parts, self.fp8, self.rng, self.without = parts, fp8, rng, without
        n = 2 * WARPS
        self.full = [Bar(WARPS if fp8 and st >= 4 else 1) for st in range(STAGES + 1)]
        self.empty = [Bar(2) for _ in range(STAGES + 1)]
        self.code_full, self.code_empty = [Bar(1), Bar(1)], [Bar(WARPS), Bar(WARPS)]
        self.q_full, self.q_empty, self.q_ready = Bar(1), Bar(2), Bar(WARPS)
        self.s_full, self.p_full = [Bar(1), Bar(1)], [Bar(WARPS), Bar(WARPS)]
        self.o_full, self.turn = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
        self.turn[0].arrive()
        self.ml_full, self.o_free, self.out_free = Bar(n), Bar(n), Bar(n)
        self.holds, self.reading = [None] * (STAGES + 1), [0] * (STAGES + 1)   # tiles
        self.codes, self.scales = [None, None], [None] * 8
        self.q, self.q_up = [None, None], [[None] * WARPS, [None] * WARPS]
        self.s, self.o = [[None] * WARPS, [None] * WARPS], [[None] * WARPS, [None] * WARPS]   # by warpgroup and warp
        self.ml = {}
        self.flying, self.pipe = [], []   # what may happen at any time; what the tensor cores do in order
        self.agents = [self.loader(), *(self.mma(b) for b in (0, 1)),
                       *(self.softmax(b, w) for b in (0, 1) for w in range(WARPS))]
        if fp8:
            self.agents += [self.widener(w) for w in range(WARPS)]

    def ring(self):
        return Ring8() if self.fp8 else Ring()

    def names(self):
        out = {}
        for n, x in vars(self).items():
            out |= {n: x} if isinstance(x, Bar) else {f"{n}[{i}]": y for i, y in enumerate(x) if isinstance(y, Bar)} if isinstance(x, list) else {}
        return out

    def run(self):
        rng, wants, slow = self.rng, {}, {}
        alive = list(self.agents)
        steps = 0
        while alive:
            if steps % 200 == 0:   # who is slow, for a time
                slow = {id(a): 10.0 ** -rng.uniform(0, rng.choice([0.5, 4])) for a in self.agents}
                slow["flying"], slow["pipe"] = 10.0 ** -rng.uniform(0, 3), 10.0 ** -rng.uniform(0, 3)
            steps += 1
            ready = [a for a in alive if all(bar.done(par) for bar, par in wants.get(id(a), ()))]
            if not ready and not self.flying and not self.pipe:
                names = {id(x): n for n, x in self.names().items()}
                stuck = [names[id(bar)] for a in alive for bar, par in wants.get(id(a), ()) if not bar.done(par)]
                raise AssertionError(f"a wait without an end among {sorted(set(stuck))}")
            options = ready + (["flying"] if self.flying else []) + (["pipe"] if self.pipe else [])
            pick = rng.choices(options, [slow[x if isinstance(x, str) else id(x)] for x in options])[0]
            if pick == "flying":
                self.flying.pop(rng.randrange(len(self.flying)))()
            elif pick == "pipe":
                self.pipe.pop(0)()
            else:
                try:
                    wants[id(pick)] = next(pick)
                except StopIteration:
                    alive.remove(pick)
        while self.flying or self.pipe:
            (self.flying or self.pipe).pop(0)()

    # ------------------------------------------------------------------------------------------ loads
    def copy(self, where, st, tag, bar):
        where[st] = "loading"

        def land():
            assert where[st] == "loading"
            where[st] = tag
            bar.arrive()
        self.flying.append(land)

    def fill(self, st, tag):
        assert self.reading[st] == 0, "a tile replaced while it is read"
        self.copy(self.holds, st, tag, self.full[st])

    def load_q(self, pi, one, state):
        if pi:
            yield [(self.q_empty, pi - 1)]
        if not one and state["lent"] is not None:
            yield [(self.empty[STAGES], state["lent"])]
            state["lent"] = None
        if not one and not self.fp8:
            assert self.reading[STAGES] == 0
            self.holds[STAGES] = "queries"
        tiles = 1 if one else 2
        for b in range(tiles):
            self.q[b] = "loading"

        def land():
            for b in range(tiles):
                self.q[b] = pi
            self.q_full.arrive()
        self.flying.append(land)

    def loader(self):
        ring, used, blocks, state = self.ring(), set(), 0, {"lent": None}
        for pi, (one, count, _) in enumerate(self.parts):
            ring.part(one, count)
            if pi == 0:
                yield from self.load_q(pi, one, state)
            if self.fp8:
                for i in range(count):
                    st, par = ring.k(i)
                    if blocks >= 4:
                        yield [(self.empty[st], par ^ 1)]
                    self.scales[blocks & 7] = (pi, i)
                    self.fill(st, (pi, "k", i))
                    yield []
                    c = blocks & 1
                    if blocks >= 2:
                        yield [(self.code_empty[c], blocks // 2 - 1)]
                    self.copy(self.codes, c, (pi, i), self.code_full[c])
                    blocks += 1
                    yield []
                    if i == 0 and pi:
                        yield from self.load_q(pi, one, state)
            else:
                read = pi == 0
                for t in range(ring.total):
                    b, v = ring.block(t)
                    st, par = ring.at(t)
                    last = t == ring.total - 1 and "loader looks before the last tile" not in self.without
                    if last and pi and ring.total == 2:
                        yield from self.load_q(pi, one, state)
                    if (st >= OUT or last) and not read:
                        yield [(self.out_free, pi - 1)]
                        read = True
                    if st in used:
                        yield [(self.empty[st], par ^ 1)]
                    self.fill(st, (pi, "v" if v else "k", b))
                    used.add(st)
                    yield []
                    if t == 1 and pi and not (ring.total == 2 and last):
                        yield from self.load_q(pi, one, state)
                if not read:   # (only without the look before the last tile)
                    yield [(self.out_free, pi - 1)]
                if one and ring.total > STAGES:
                    state["lent"] = ring.at(STAGES + (ring.total - ring.n) // ring.n * ring.n)[1]
            ring.done()

    # ------------------------------------------------------------------------------------------ MMAs
    def commit(self, bar):
        self.pipe.append(lambda: self.flying.append(bar.arrive))

    def multiply(self, st, before, after):
        def begin():
            before()
            self.reading[st] += 1

        def end():
            self.reading[st] -= 1
            after()
        self.pipe += [begin, end]

    def mma(self, b):
        ring, p_ph, turn_ph = self.ring(), 0, 0
        for pi, (one, count, _) in enumerate(self.parts):
            ring.part(one, count)
            every, first = (2, b) if one else (1, 0)
            steps, blocks = ((count + 1) // 2, (count + 1 - b) // 2) if one else (count, count)
            yield [(self.q_ready if self.fp8 else self.q_full, pi)]
            for i in range(-1, steps):
                pv, s = 0 <= i < blocks, i + 1 < blocks
                vb, kb = (first + i * every if pv else 0), (first + (i + 1) * every if s else 0)
                (v_st, v_par), (k_st, k_par) = ring.v(vb), ring.k(kb)
                if s:
                    yield [(self.full[k_st], k_par)]
                if pv:
                    yield [(self.full[v_st], v_par)]
                    if i == 0 and pi:
                        yield [(self.o_free, pi - 1)]
                yield [(self.turn[b], turn_ph)] + ([(self.p_full[b], p_ph)] if pv else [])
                p_ph, turn_ph = p_ph ^ pv, turn_ph ^ 1
                times = 2 if one else 1
                if pv:
                    def before(pi=pi, vb=vb, st=v_st, i=i):
                        assert self.holds[st] == (pi, "v", vb) and self.s[b] == [("p", pi, i)] * WARPS
                        assert self.o[b] == ([(pi, i - 1)] * WARPS if i else self.o[b]) and (i or self.o[b] in ([None] * WARPS, ["read"] * WARPS))

                    def after(pi=pi, i=i):
                        self.o[b], self.s[b] = [(pi, i)] * WARPS, [None] * WARPS
                    self.multiply(v_st, before, after)
                if s:
                    def before(pi=pi, kb=kb, st=k_st, one=one):
                        assert self.holds[st] == (pi, "k", kb) and self.s[b] == [None] * WARPS
                        assert self.q[0 if one else b] == (("codes", pi) if self.fp8 else pi)

                    def after(pi=pi, i=i):
                        self.s[b] = [("s", pi, i + 1)] * WARPS
                    self.multiply(k_st, before, after)
                self.turn[b ^ 1].arrive()
                if s:
                    self.commit(self.s_full[b])
                if pv:
                    if not s:
                        self.commit(self.o_full[b])
                    for _ in range(times):
                        self.commit(self.empty[v_st])
                if s:
                    for _ in range(times):
                        self.commit(self.empty[k_st])
                if i + 1 == max(blocks - 1, 0):
                    self.commit(self.q_empty)
                yield []
            ring.done()

    # ------------------------------------------------------------------------------------------ softmax and output
    def softmax(self, b, w):
        ring, steps, outs, merges = self.ring(), 0, 0, 0
        early = "softmax sees the next queries before it is done with a part" not in self.without
        if self.fp8 and early:
            yield [(self.q_ready, 0)]
            if "softmax sees the first queries" not in self.without:
                self.out_free.arrive()
        for pi, (one, count, whole) in enumerate(self.parts):
            ring.part(one, count)
            if self.fp8:
                if not early:
                    yield [(self.q_ready, pi)]
                assert self.q_up[pi & 1] == [pi] * WARPS
                yield []
            had = b if one else 0
            mine = range(had, count, 2 if one else 1)
            for n, blk in enumerate(mine):
                yield [(self.s_full[b], steps)]
                st, par = ring.v(blk)
                if self.fp8 or (blk == count - 1 and (one or b == 0)):   # V's scale; or rows behind the last key
                    yield [(self.full[st], par)]
                    assert self.holds[st] == (pi, "v", blk)
                    assert not self.fp8 or self.scales[ring.base + blk & 7] == (pi, blk)
                assert self.s[b][w] == ("s", pi, n)
                self.s[b][w] = ("p", pi, n)
                self.p_full[b].arrive()
                steps += 1
                yield []
            ring.done()
            if mine:
                yield [(self.o_full[b], outs)]
                outs += 1
            if one:
                if pi:
                    yield [(self.o_free, pi - 1)]
                self.ml[b, w] = pi
                self.ml_full.arrive()
                yield [(self.ml_full, merges)]
                merges += 1
                assert self.ml[b ^ 1, w] == pi
            st, par = ring.out(b)
            if whole:
                yield [(self.empty[st], par)]
                assert self.reading[st] == 0 and self.holds[st] != "loading"
                self.holds[st] = "output"
            if mine:
                assert self.o[b][w] == (pi, len(mine) - 1)
            if one and range(b ^ 1, count, 2):
                assert self.o[b ^ 1][w] in ((pi, len(range(b ^ 1, count, 2)) - 1),)
            yield []
            # (of the last warp that reads it, or O would count as read before the other warpgroup's look)
            self.seen = getattr(self, "seen", {})
            for x in ((0, 1) if one else (b,)):
                key = (pi, x, w)
                self.seen[key] = self.seen.get(key, 0) + 1
                if self.seen[key] == (2 if one else 1) and range(x if one else 0, count, 2 if one else 1):
                    self.o[x][w] = "read"
            self.o_free.arrive()
            yield []
            if whole:
                assert self.holds[st] == "output", "an output's stage was loaded before its rows were stored"
            if self.fp8 and early and pi + 1 < len(self.parts):
                yield [(self.q_ready, pi + 1)]
            self.out_free.arrive()

    # ------------------------------------------------------------------------------------------ E4M3: queries, V's codes
    def widener(self, w):
        ring, n = self.ring(), 0
        for pi, (one, count, _) in enumerate(self.parts):
            ring.part(one, count)
            yield [(self.q_full, pi)]
            for b in range(1 if one else 2):
                assert self.q[b] in (pi, ("half", pi))
                self.q[b] = ("half", pi) if self.q[b] == pi else ("codes", pi)
            self.q_up[pi & 1][w] = pi
            yield []
            self.q_ready.arrive()
            if "softmax sees the next queries before it is done with a part" in self.without or "softmax sees the first queries" in self.without:
                if pi:
                    yield [(self.out_free, pi - 1)]
            else:
                yield [(self.out_free, pi)]
            for i in range(count):
                c, (st, par) = n & 1, ring.v(i)
                yield [(self.code_full[c], n >> 1)]
                if n >= 2:
                    yield [(self.empty[st], par ^ 1)]
                assert self.codes[c] == (pi, i) and self.reading[st] == 0
                self.holds[st] = (pi, "v", i)
                yield []
                assert self.codes[c] == (pi, i)
                self.code_empty[c].arrive()
                self.full[st].arrive()
                n += 1
            ring.done()


SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_05_gb300", "csrc",
                      "prompt_attn.cu")


def test_the_source_has_the_order_of_the_model():
    text = open(SOURCE).read()
    softmax = text[text.index("- softmax and output"):]
    first, last = re.search(r"q_ready, 0, .*?out_free", softmax, re.S), re.search(r"\+\+parts;.*?q_ready, parts & 1.*?out_free\);\s+g = then", softmax, re.S)
    assert first and last and first.start() < softmax.index("while (ok && there)") < last.start()
    assert re.search(r"\(st >= C::kOutStage \|\| last\) && !out_read", text)
    assert re.search(r"mbar_arrive\(&sm.q_ready\);[^;]*out_free, parts & 1", softmax)


def schedules(fp8, n, without=()):
    """How many of n schedules of random parts end badly."""
    bad = []
    for seed in range(n):
        rng = random.Random(seed)
        most = rng.choice([1, 2, 3, 9])
        parts = [(rng.random() < 0.5, rng.randint(1, most), rng.random() < 0.8) for _ in range(rng.randint(1, 8))]
        try:
            Kernel(parts, fp8, rng, without).run()
        except AssertionError as e:
            bad.append((seed, parts, str(e)))
    return bad


@pytest.mark.parametrize("fp8", [False, True])
def test_every_schedule_ends(fp8):
    bad = schedules(fp8, 600)
    assert not bad, bad[:3]


@pytest.mark.parametrize("fp8,without", [(True, "softmax sees the next queries before it is done with a part"),
                                         (True, "softmax sees the first queries"),
                                         (False, "loader looks before the last tile")])
def test_a_look_that_comes_too_late_is_found(fp8, without):
    """Each of these orders is needed: without it some schedules never end."""
    bad = schedules(fp8, 600, (without,))
    assert bad and all("without an end" in e for _, _, e in bad), bad[:3]
