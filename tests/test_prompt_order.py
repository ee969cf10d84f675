"""The order of the prompt kernel's warps, on the host.

A block of the kernel is a copying warp, two warps that issue products and the
softmax warps, which meet at barriers that count phases and are waited for by a
phase's parity.  Such a wait is right only if the barrier cannot complete another
phase before the wait is looked at: then the parity is the old one again, and the
warp sleeps on.  The model below runs the warps' waits and arrivals in the
kernel's order, with delays drawn from a wide range (a warp may stand still
anywhere); what it holds is that every warp comes to its end whatever the delays
are.  Sizes of rings and numbers of barriers are the kernel's.
"""
import heapq
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "serving_router_sigmoid_gb300", "csrc", "k_prompt.cu")


def source():
    with open(SOURCE) as f:
        return f.read()


def constant(name):
    return int(re.search(rf"constexpr int {name} = (\d+);", source()).group(1))


class Barrier:
    def __init__(self, count=1):
        self.count, self.left, self.done, self.asleep = count, count, 0, []


class Block:
    """Warps as generators that yield ("for", cycles) or ("wait", barrier, parity)."""

    def __init__(self, seed):
        self.r, self.now, self.queue, self.n, self.pipe = random.Random(seed), 0.0, [], 0, 0.0

    def at(self, when, what):
        self.n += 1
        heapq.heappush(self.queue, (when, self.n, what))

    def delay(self, base):
        return base * self.r.choice([0.1, 0.5, 1, 1, 1, 2, 6])

    def arrive(self, bar):
        bar.left -= 1
        if bar.left == 0:
            bar.left, bar.done = bar.count, bar.done + 1
            asleep, bar.asleep = bar.asleep, []
            for warp, parity in asleep:  # each looks again, a little later
                self.at(self.now + self.delay(40), lambda w=warp, p=parity: self.look(w, bar, p))

    def look(self, warp, bar, parity):
        if (bar.done & 1) != parity:
            self.step(warp)
        else:
            bar.asleep.append((warp, parity))

    def step(self, warp):
        try:
            kind, *rest = next(warp)
        except StopIteration:
            self.running -= 1
            return
        if kind == "for":
            self.at(self.now + rest[0], lambda: self.step(warp))
        else:
            self.look(warp, rest[0], rest[1])

    def later(self, base, bar):
        self.at(self.now + self.delay(base), lambda: self.arrive(bar))

    def product(self, cycles):
        self.pipe = max(self.pipe, self.now) + cycles
        return self.pipe

    def commit(self, bar, end):  # once what was issued is done
        self.at(max(end, self.now) + 150 + self.delay(100), lambda: self.arrive(bar))

    def run(self, warps):
        """Whether all warps end."""
        self.running = len(warps)
        for w in warps:
            self.at(0.0, lambda w=w: self.step(w))
        while self.queue:
            self.now, _, what = heapq.heappop(self.queue)
            what()
        return self.running == 0


LOOKUP, COPY, SOFTMAX, RESCALE = 900, 900, 350, 500


def two_streams(b, items, nk, nv, slots, tiles_max, fixes_n, start):
    """items: ((tiles of the first stream, of the second), whether the last tile is cleared).  start: what lets
    the second stream begin an item: "count" (of items whose first stream has weights) or "parity"."""
    bars = lambda n, c=1: [Barrier(c) for _ in range(n)]  # noqa: E731
    full, empty, v_fixed = bars(tiles_max), bars(tiles_max, 2), bars(fixes_n)
    q_full, q_empty, s_full, pv_done, o_full, o_empty = (bars(2) for _ in range(6))
    p_ready = [bars(2), bars(2)]
    began = [0]

    def copies():
        room, put, got, sizes, qp, fixes = slots, 0, 0, [], 0, 0

        def take(n):
            nonlocal room, got
            while room < n or put - got == tiles_max:
                yield "wait", empty[got % tiles_max], got // tiles_max & 1
                room += sizes.pop(0)
                got += 1
            sizes.append(n)
            room -= n
        for tiles, cleared in items:
            yield "for", b.delay(LOOKUP)
            for j in range(max(tiles)):
                if j == 0:
                    yield "wait", q_empty[0], qp ^ 1
                    b.later(COPY, q_full[0])
                yield from take(nk)
                b.later(COPY, full[put % tiles_max])
                put += 1
                if j == 0:
                    yield "wait", q_empty[1], qp ^ 1
                    b.later(COPY, q_full[1])
                yield from take(nv)
                b.later(COPY, full[put % tiles_max])
                if cleared and j == max(tiles) - 1:
                    yield "wait", full[put % tiles_max], put // tiles_max & 1
                    yield "for", b.delay(200)
                    b.arrive(v_fixed[fixes % fixes_n])
                    fixes += 1
                put += 1
            qp ^= 1

    def issue(g):
        tile = fixes = qf = oe = theirs = use = 0
        for it, (tiles, cleared) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            mine, other, n = tiles[g], tiles[g ^ 1], max(tiles)
            yield "wait", q_full[g], qf
            qf ^= 1

            def first(j):
                end = b.product(nk * 250)
                t = tile + 2 * j
                b.commit(s_full[g], end)
                for _ in range(1 + (j >= other)):
                    b.commit(empty[t % tiles_max], end)
                if j + 1 == mine:
                    b.commit(q_empty[g], end)
            if g == 1 and mine and other:
                if start == "parity":
                    yield "wait", p_ready[0][0], theirs
                else:
                    while began[0] <= it:
                        yield "for", 50
            theirs ^= other & 1
            if mine:
                yield "wait", full[tile % tiles_max], tile // tiles_max & 1
                first(0)
            else:
                b.commit(q_empty[g], 0)
            for j in range(n):
                fix, t, last = fixes, tile + 2 * j + 1, cleared and j == n - 1
                fixes += last
                if j >= mine:
                    continue
                yield "wait", full[t % tiles_max], t // tiles_max & 1
                if last:
                    yield "wait", v_fixed[fix % fixes_n], fix // fixes_n & 1
                if j == 0:
                    yield "wait", o_empty[g], oe ^ 1
                    oe ^= 1
                yield "wait", p_ready[g][0], use
                b.commit(pv_done[g], b.product(nv * 128))
                yield "wait", p_ready[g][1], use
                use ^= 1
                end = b.product(nv * 128)
                for _ in range(1 + (j >= other)):
                    b.commit(empty[t % tiles_max], end)
                if j + 1 == mine:
                    b.commit(o_full[g], end)
                else:
                    t = tile + 2 * j + 2
                    yield "wait", full[t % tiles_max], t // tiles_max & 1
                    first(j + 1)
            tile += 2 * n

    def softmax(g):
        sf = pd = of = 0
        for it, (tiles, _) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            for j in range(2 * tiles[g]):
                if not j & 1:
                    yield "wait", s_full[g], sf
                    sf ^= 1
                if j and b.r.random() < 0.5:
                    if j & 1:
                        yield "wait", pv_done[g], pd
                    yield "for", b.delay(RESCALE)
                pd ^= j & 1
                yield "for", b.delay(SOFTMAX)
                b.arrive(p_ready[g][j & 1])
                if g == 0 and j == 0:
                    began[0] = it + 1
            if tiles[g]:
                yield "wait", o_full[g], of
                of ^= 1
                yield "for", b.delay(600)
                b.arrive(o_empty[g])
    return b.run([copies(), issue(0), issue(1), softmax(0), softmax(1)])


def one_stream(b, items, nk, nv, slots, fixes_n):
    """items: (tiles, whether the last one is cleared)."""
    bars = lambda n: [Barrier() for _ in range(n)]  # noqa: E731
    full, empty, v_fixed = bars(slots), bars(slots), bars(fixes_n)
    q_full, q_empty, o_full, o_empty = (Barrier() for _ in range(4))
    s_full, p_ready, pv_done = bars(2), bars(2), bars(2)

    def copies():
        here = qp = fixes = 0

        def bring(n):
            nonlocal here
            for _ in range(n):
                yield "wait", empty[here % slots], here // slots & 1 ^ 1
                b.later(COPY, full[here % slots])
                here += 1

        def values(cleared):
            nonlocal fixes
            begin = here
            yield from bring(nv)
            if cleared:
                for at in range(begin, begin + nv):
                    yield "wait", full[at % slots], at // slots & 1
                yield "for", b.delay(200)
                b.arrive(v_fixed[fixes % fixes_n])
                fixes += 1
        for n, cleared in items:
            yield "for", b.delay(LOOKUP)
            yield "wait", q_empty, qp ^ 1
            b.later(COPY, q_full)
            for j in range(n):
                yield from bring(nk)
                if j:
                    yield from values(False)
            yield from values(cleared)
            qp ^= 1

    def products_s():
        at = step = qf = began = 0
        uses = [0, 0]
        for n, _ in items:
            yield "for", b.delay(LOOKUP)
            yield "wait", q_full, qf
            qf ^= 1
            end = 0
            for j in range(n):
                k = step & 1
                step += 1
                if began >> k & 1:
                    yield "wait", pv_done[k], uses[k] ^ 1
                began |= 1 << k
                uses[k] ^= 1
                for c in range(nk):
                    yield "wait", full[at % slots], at // slots & 1
                    end = b.product(250)
                    b.commit(empty[at % slots], end)
                    if c + 1 == nk:
                        b.commit(s_full[k], end)
                    at += 1
                if j:
                    at += nv
            b.commit(q_empty, end)
            at += nv

    def products_o():
        at = step = fixes = oe = 0
        uses = [0, 0]
        for n, cleared in items:
            yield "for", b.delay(LOOKUP)
            at += nk * min(n, 2)
            for j in range(n):
                k = step & 1
                step += 1
                if cleared and j == n - 1:
                    yield "wait", v_fixed[fixes % fixes_n], fixes // fixes_n & 1
                    fixes += 1
                if j == 0:
                    yield "wait", o_empty, oe ^ 1
                    oe ^= 1
                yield "wait", p_ready[k], uses[k]
                uses[k] ^= 1
                for i in range(nv):
                    yield "wait", full[at % slots], at // slots & 1
                    end = b.product(128)
                    b.commit(empty[at % slots], end)
                    if i + 1 == nv:
                        b.commit(pv_done[k], end)
                        if j + 1 == n:
                            b.commit(o_full, end)
                    at += 1
                if j + 2 < n:
                    at += nk

    def softmax():
        sf, pd, of, step = [0, 0], [0, 0], 0, 0
        for n, _ in items:
            yield "for", b.delay(LOOKUP)
            for j in range(n):
                k = step & 1
                step += 1
                yield "wait", s_full[k], sf[k]
                sf[k] ^= 1
                if j and b.r.random() < 0.5:
                    yield "wait", pv_done[k ^ 1], pd[k ^ 1] ^ 1
                    yield "for", b.delay(RESCALE)
                pd[k] ^= 1
                yield "for", b.delay(SOFTMAX)
                b.arrive(p_ready[k])
            yield "wait", o_full, of
            of ^= 1
            yield "for", b.delay(600)
            b.arrive(o_empty)
    return b.run([copies(), products_s(), products_o(), softmax()])


def ring(chunks, streams):
    """Slots of the ring: 13 of 16 KB hold the ring and the queries."""
    return 13 - streams * chunks


# chunks of 64 key dimensions, slots of a tile of values
TWO = [(1, 1), (1, 2), (2, 1), (2, 2), (3, 1), (3, 2)]
ONE = TWO + [(4, 4), (4, 1), (2, 4)]


def draw_two(r):
    items = []
    for _ in range(r.randint(1, 6)):
        n = r.randint(1, 4)
        items.append((r.choice([(n, n), (n, n + 1), (n, n + 2), (n, 0), (0, n), (n + 1, n)]), r.random() < 0.5))
    return items


@pytest.mark.parametrize("nk,nv", TWO)
def test_two_streams_come_to_their_end(nk, nv):
    for seed in range(300):
        items = draw_two(random.Random(seed))
        assert two_streams(Block(seed), items, nk, nv, ring(nk, 2), constant("kTiles"), constant("kFixes"), "count"), (seed, items)


@pytest.mark.parametrize("nk,nv", ONE)
def test_one_stream_comes_to_its_end(nk, nv):
    for seed in range(300):
        r = random.Random(seed)
        items = [(r.choice([1, 1, 1, 2, 3]), r.random() < 0.8) for _ in range(r.randint(1, 8))]
        assert one_stream(Block(seed), items, nk, nv, ring(nk, 1), constant("kFixes")), (seed, items)


def test_the_model_sees_a_phase_that_is_missed():
    """A start by the parity of the first stream's weights, and two barriers of cleared rows, are each overtaken."""
    def two(seed):
        return two_streams(Block(seed), [((2, 3), False)] * 3, 2, 2, ring(2, 2), 8, 4, "parity")

    def one(seed):
        return one_stream(Block(seed), [(1, True)] * 8, 2, 1, ring(2, 1), 2)
    assert not all(two(s) for s in range(300))
    assert not all(one(s) for s in range(300))


def test_the_second_stream_starts_by_a_count():
    text = source()
    assert "wait(&sm.p_ready[0][0]" not in text  # completed once a tile: its parity says nothing of an item
    assert re.search(r"sm\.began", text)


def test_slots_of_the_ring():
    """227 KB less the rest of a block's shared memory are 13 slots."""
    shared = 8 * (2 * constant("kSlots") + constant("kFixes") + 2 * 9) + 4 * (3 + 512)  # barriers; flags and row maxima
    room = 227 * 1024 - 1024 - shared - 64
    assert room // 16384 == 13 and room - 13 * 16384 > 64
