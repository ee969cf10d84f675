"""The order of the prompt kernel's warps, on the host.

A block of the kernel is a copying warp, two warps that issue products and the
softmax warps, which meet at barriers that count phases and are waited for by a
phase's parity.  Such a wait is right only if the barrier can neither complete
another phase before the wait is looked at (the parity is the old one again, and
the warp sleeps on), nor be a phase behind (the parity is that of the phase before
the last, and the warp reads what has not come).  The model below runs the warps'
waits and arrivals in the kernel's order, with delays drawn from a wide range (a
warp or a copy may stand still anywhere); what it holds is that every wait ends, and
with the phase that it is for, whatever the delays are.  Sizes of rings and numbers
of barriers are the kernel's.
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
    """Warps as generators that yield ("for", cycles) or ("wait", barrier, phase): phases count from 0, -1 is
    what came before the first."""

    def __init__(self, seed):
        self.r, self.now, self.queue, self.n, self.pipe = random.Random(seed), 0.0, [], 0, 0.0
        self.wrong, self.last = 0, {}

    def at(self, when, what):
        self.n += 1
        heapq.heappush(self.queue, (when, self.n, what))

    def delay(self, base):
        return base * self.r.choice([0.1, 0.5, 1, 1, 1, 2, 6, 15])

    def arrive(self, bar):
        bar.left -= 1
        if bar.left == 0:
            bar.left, bar.done = bar.count, bar.done + 1
            asleep, bar.asleep = bar.asleep, []
            for warp, phase in asleep:  # each looks again, a little later
                self.at(self.now + self.delay(40), lambda w=warp, p=phase: self.look(w, bar, p))

    def look(self, warp, bar, phase):
        if (bar.done ^ phase) & 1:  # what a wait by parity sees
            self.wrong += bar.done != phase + 1
            self.step(warp)
        else:
            bar.asleep.append((warp, phase))

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

    def commit(self, warp, bar, end):  # once what the warp issued is done; in the order of its commits
        when = max(max(end, self.now) + 150 + self.delay(100), self.last.get(warp, 0.0))
        self.last[warp] = when
        self.at(when, lambda: self.arrive(bar))

    def run(self, warps):
        """Whether all warps end, and every wait was for the phase it saw."""
        self.running = len(warps)
        for w in warps:
            self.at(0.0, lambda w=w: self.step(w))
        while self.queue:
            self.now, _, what = heapq.heappop(self.queue)
            what()
        return self.running == 0 and not self.wrong


LOOKUP, COPY, SOFTMAX, RESCALE = 900, 900, 350, 500


def two_streams(b, items, nk, nv, slots, tiles_max, fixes_n, start="count", skips=False):
    """items: ((tiles of the first stream, of the second), whether the last tile is cleared).  start: what lets
    the second stream begin an item: "count" (of items whose first stream has weights), "parity" (of the
    first stream's weights) or "nothing".  skips: a stream passes by the tiles that only the other one needs,
    which gives them back for both."""
    bars = lambda n, c=1: [Barrier(c) for _ in range(n)]  # noqa: E731
    full, empty, v_fixed = bars(tiles_max), bars(tiles_max, 2), bars(fixes_n)
    q_full, q_empty, s_full, pv_done, o_full, o_empty = (bars(2) for _ in range(6))
    p_ready = [bars(2), bars(2)]
    began = [0]
    turn = lambda ring, n: (ring[n % len(ring)], n // len(ring))  # noqa: E731

    def copies():
        room, put, got, sizes, fixes = slots, 0, 0, [], 0

        def take(n):
            nonlocal room, got
            while room < n or put - got == tiles_max:
                yield "wait", *turn(empty, got)
                room += sizes.pop(0)
                got += 1
            sizes.append(n)
            room -= n
        for it, (tiles, cleared) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            for j in range(max(tiles)):
                if j == 0:
                    yield "wait", q_empty[0], it - 1
                    b.later(COPY, q_full[0])
                yield from take(nk)
                b.later(COPY, full[put % tiles_max])
                put += 1
                if j == 0:
                    yield "wait", q_empty[1], it - 1
                    b.later(COPY, q_full[1])
                yield from take(nv)
                b.later(COPY, full[put % tiles_max])
                if cleared and j == max(tiles) - 1:
                    yield "wait", *turn(full, put)
                    yield "for", b.delay(200)
                    b.arrive(v_fixed[fixes % fixes_n])
                    fixes += 1
                put += 1

    def issue(g):
        tile = fixes = theirs = use = worked = 0
        for it, (tiles, cleared) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            mine, other, n = tiles[g], tiles[g ^ 1], max(tiles)
            yield "wait", q_full[g], it

            def first(j):
                end = b.product(nk * 250)
                b.commit(g, s_full[g], end)
                b.commit(g, empty[(tile + 2 * j) % tiles_max], end)
                if skips and j >= other:
                    b.commit(g, empty[(tile + 2 * j) % tiles_max], end)
                if j + 1 == mine:
                    b.commit(g, q_empty[g], end)
            if g == 1 and mine and other:
                if start == "parity":
                    yield "wait", p_ready[0][0], theirs
                elif start == "count":
                    while began[0] <= it:
                        yield "for", 50
            theirs += other
            if mine:
                yield "wait", *turn(full, tile)
                first(0)
            else:
                b.commit(g, q_empty[g], 0)
            for j in range(n):
                fix, t, last = fixes, tile + 2 * j + 1, cleared and j == n - 1
                fixes += last
                if j >= mine:
                    if not skips:
                        for i in (t - 1, t):
                            yield "wait", *turn(full, i)
                            b.arrive(empty[i % tiles_max])
                    continue
                yield "wait", *turn(full, t)
                if last:
                    yield "wait", *turn(v_fixed, fix)
                if j == 0:
                    yield "wait", o_empty[g], worked - 1
                    worked += 1
                yield "wait", p_ready[g][0], use
                b.commit(g, pv_done[g], b.product(nv * 128))
                yield "wait", p_ready[g][1], use
                use += 1
                end = b.product(nv * 128)
                b.commit(g, empty[t % tiles_max], end)
                if skips and j >= other:
                    b.commit(g, empty[t % tiles_max], end)
                if j + 1 == mine:
                    b.commit(g, o_full[g], end)
                else:
                    yield "wait", *turn(full, t + 1)
                    first(j + 1)
            tile += 2 * n

    def softmax(g):
        done = worked = 0
        for it, (tiles, _) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            for j in range(2 * tiles[g]):
                if not j & 1:
                    yield "wait", s_full[g], done
                if j and b.r.random() < 0.5:
                    if j & 1:
                        yield "wait", pv_done[g], done
                    yield "for", b.delay(RESCALE)
                done += j & 1
                yield "for", b.delay(SOFTMAX)
                b.arrive(p_ready[g][j & 1])
                if g == 0 and j == 0:
                    began[0] = it + 1
            if tiles[g]:
                yield "wait", o_full[g], worked
                worked += 1
                yield "for", b.delay(600)
                b.arrive(o_empty[g])
    return b.run([copies(), issue(0), issue(1), softmax(0), softmax(1)])


def one_stream(b, items, nk, nv, slots, fixes_n, turns):
    """items: (tiles, whether the last one is cleared).  turns: barriers of the copies of keys, and of those of
    values; 0: one barrier for each slot, whatever it holds."""
    bars = lambda n: [Barrier() for _ in range(n)]  # noqa: E731
    full, k_full, v_full, empty, v_fixed = bars(slots), bars(turns), bars(turns), bars(slots), bars(fixes_n)
    q_full, q_empty, o_full, o_empty = (Barrier() for _ in range(4))
    s_full, p_ready, pv_done = bars(2), bars(2), bars(2)
    turn = lambda ring, n: (ring[n % len(ring)], n // len(ring))  # noqa: E731

    def landed(ring, n, at):  # of the n-th copy of keys or values, which is the at-th of all
        return turn(ring, n) if turns else turn(full, at)

    def copies():
        here = keys = vals = fixes = 0

        def bring(ring, n, count):
            nonlocal here
            for i in range(n):
                yield "wait", empty[here % slots], here // slots - 1
                b.later(COPY, landed(ring, count + i, here)[0])
                here += 1

        def values(cleared):
            nonlocal fixes, vals
            begin = here
            yield from bring(v_full, nv, vals)
            if cleared:
                for i in range(nv):
                    yield "wait", *landed(v_full, vals + i, begin + i)
                yield "for", b.delay(200)
                b.arrive(v_fixed[fixes % fixes_n])
                fixes += 1
            vals += nv
        for it, (n, cleared) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            yield "wait", q_empty, it - 1
            b.later(COPY, q_full)
            for j in range(n):
                yield from bring(k_full, nk, keys)
                keys += nk
                if j:
                    yield from values(False)
            yield from values(cleared)

    def products_s():
        at = step = keys = 0
        for it, (n, _) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            yield "wait", q_full, it
            for j in range(n):
                if step >= 2:
                    yield "wait", pv_done[step & 1], step // 2 - 1
                for c in range(nk):
                    yield "wait", *landed(k_full, keys, at)
                    end = b.product(250)
                    b.commit("s", empty[at % slots], end)
                    if c + 1 == nk:
                        b.commit("s", s_full[step & 1], end)
                    at += 1
                    keys += 1
                step += 1
                if j:
                    at += nv
            b.commit("s", q_empty, end)
            at += nv

    def products_o():
        at = step = fixes = vals = 0
        for it, (n, cleared) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            at += nk * min(n, 2)
            for j in range(n):
                if cleared and j == n - 1:
                    yield "wait", *turn(v_fixed, fixes)
                    fixes += 1
                if j == 0:
                    yield "wait", o_empty, it - 1
                yield "wait", p_ready[step & 1], step // 2
                for i in range(nv):
                    yield "wait", *landed(v_full, vals, at)
                    end = b.product(128)
                    b.commit("o", empty[at % slots], end)
                    if i + 1 == nv:
                        b.commit("o", pv_done[step & 1], end)
                        if j + 1 == n:
                            b.commit("o", o_full, end)
                    at += 1
                    vals += 1
                step += 1
                if j + 2 < n:
                    at += nk

    def softmax():
        step = 0
        for it, (n, _) in enumerate(items):
            yield "for", b.delay(LOOKUP)
            for j in range(n):
                yield "wait", s_full[step & 1], step // 2
                if j and b.r.random() < 0.5:
                    yield "wait", pv_done[step & 1 ^ 1], (step - 1) // 2
                    yield "for", b.delay(RESCALE)
                yield "for", b.delay(SOFTMAX)
                b.arrive(p_ready[step & 1])
                step += 1
            yield "wait", o_full, it
            yield "for", b.delay(600)
            b.arrive(o_empty)
    return b.run([copies(), products_s(), products_o(), softmax()])


def ring(chunks, streams):
    """Slots of the ring: 13 of 16 KB hold the ring and the queries."""
    return 13 - streams * chunks


# chunks of 64 key dimensions, slots of a tile of values
TWO = [(1, 1), (1, 2), (2, 1), (2, 2), (3, 1), (3, 2)]
ONE = TWO + [(4, 4), (4, 1), (2, 4), (5, 4), (5, 1), (1, 4)]


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
        for start in ("count", "nothing"):
            block = Block(seed)
            assert two_streams(block, items, nk, nv, ring(nk, 2), constant("kTiles"), constant("kFixes"), start), (seed, items)


@pytest.mark.parametrize("nk,nv", ONE)
def test_one_stream_comes_to_its_end(nk, nv):
    for seed in range(300):
        r = random.Random(seed)
        items = [(r.choice([1, 1, 1, 2, 3]), r.random() < 0.8) for _ in range(r.randint(1, 8))]
        assert one_stream(Block(seed), items, nk, nv, ring(nk, 1), constant("kFixes"), constant("kTurns")), (seed, items)


def test_the_model_sees_a_phase_that_is_missed():
    """A start by the parity of the first stream's weights, tiles that a stream passes by, two barriers of cleared
    rows, and a barrier for each slot of a short ring are each overtaken or behind."""
    def two(seed):
        return two_streams(Block(seed), [((2, 3), False)] * 3, 2, 2, ring(2, 2), 8, 4, "parity")

    def skips(seed):
        return two_streams(Block(seed), [((0, 4), False), ((1, 2), False)] * 4, 1, 1, ring(1, 2), 8, 4, skips=True)

    def fixes(seed):
        return one_stream(Block(seed), [(1, True)] * 8, 2, 1, ring(2, 1), 2, 16)

    def slots(seed):
        return one_stream(Block(seed), [(4, False)] * 3, 5, 4, ring(5, 1), 4, 0)
    for order in (two, skips, fixes, slots):
        assert not all(order(s) for s in range(300)), order


def test_the_second_stream_starts_by_a_count():
    text = source()
    assert "wait(&sm.p_ready[0][0]" not in text  # completed once a tile: its parity says nothing of an item
    assert re.search(r"sm\.began", text)


def test_slots_of_the_ring():
    """227 KB less the rest of a block's shared memory are 13 slots."""
    barriers = constant("kSlots") + 2 * constant("kTurns") + constant("kFixes") + 2 * 9
    shared = 8 * barriers + 4 * (3 + 512)  # and flags, and row maxima
    room = 227 * 1024 - 1024 - shared - 64
    assert room // 16384 == 13 and room - 13 * 16384 > 64


def test_streams_see_every_tile():
    """No stream gives a tile back for the other one."""
    assert not re.search(r"if \(j >= other\)", source())
