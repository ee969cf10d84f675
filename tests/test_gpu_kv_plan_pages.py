"""moe_kv_plan when something runs out: no page is lost.

Whatever the flags say, the pages that left the free list (up to info[1]) are
the ones that table rows received, each once.  A request that needs more pages
than its row holds takes those that fit and no more, so the requests after it
get theirs, and a loop that copies info[1] to the list's head goes on.
"""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

KEEP = -77  # a table entry nobody owns


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def walk(past, new, free, head, table, page, room):
    """The definition, request by request; table: list of rows, updated."""
    flags, taken, start, pos, slot = 0, 0, [0], [], []
    for row, p, n in zip(table, past, new):
        flags |= 8 if p < 0 or n < 0 else 0
        p, n = max(p, 0), max(n, 0)
        have, need = -(-p // page), -(-(p + n) // page)
        flags |= 2 if need > len(row) else 0
        for col in range(have, min(need, len(row))):
            row[col] = free[head + taken] if head + taken < len(free) else -1
            taken += 1
        for i in range(p, p + n):
            at = row[i // page] if i // page < len(row) else -1
            pos.append(i)
            slot.append(at * page + i % page if at >= 0 else -1)
        start.append(start[-1] + n)
    avail = max(len(free) - head, 0)
    flags |= (1 if taken > avail else 0) | (4 if start[-1] > room else 0)
    lens = [max(p, 0) + max(n, 0) for p, n in zip(past, new)]
    pad = max(0, room - len(pos))
    return (start, lens, (pos + [0] * pad)[:room], (slot + [-1] * pad)[:room],
            [start[-1], head + min(taken, avail), flags, max(lens, default=0)])


class Loop:
    """A serving loop's state: lists on the host beside the tensors a call takes."""

    def __init__(self, moe, n, cols, page, n_free, room, seed=0):
        r = random.Random(seed)
        self.page, self.room = page, room
        self.free = r.sample(range(10 * n_free + 10), n_free)
        self.head, self.past = 0, [0] * n
        self.rows = [[KEEP] * cols for _ in range(n)]
        self.table = torch.full((n, cols), KEEP, dtype=torch.int32, device="cuda")
        self.plan = moe.KvPlan(n, room, page)

    def step(self, new):
        start, lens, pos, slot, info = walk(self.past, new, self.free, self.head, self.rows, self.page, self.room)
        p = self.plan.update(i32(self.past), i32(new), i32(self.free), i32([self.head]), self.table)
        assert p.info.tolist() == info
        assert self.table.tolist() == self.rows
        assert p.q_start.tolist() == start and p.seq_len.tolist() == lens
        assert p.positions.tolist() == pos and p.slots.tolist() == slot
        self.head, self.past = info[1], lens
        # the pages in the rows are those that left the list, each once
        held = sorted(v for row in self.rows for v in row if v >= 0)
        assert held == sorted(self.free[:self.head])
        return info[2]


def test_a_full_row_takes_what_fits(moe):
    loop = Loop(moe, 3, 3, 16, 40, 200)
    assert loop.step([30, 60, 50]) == 2  # the second and third need 4 of 3
    assert loop.head == 2 + 3 + 3
    assert loop.step([5, 20, 1]) == 2    # and go on: nothing more for the full rows
    assert loop.head == 9
    assert loop.step([13, 0, 0]) == 2 and loop.head == 9  # the full rows stay flagged


def test_requests_after_a_full_row_get_the_pages(moe):
    loop = Loop(moe, 2, 2, 16, 3, 100)
    assert loop.step([16 * 5, 16]) == 2  # three pages: two for the first, one for the second
    assert loop.head == 3 and loop.rows[1][0] >= 0


@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("n", [1, 40, 600, 1100])
def test_loops_that_overflow_rows_and_list(moe, n, page):
    r = random.Random(100 * n + page)
    loop = Loop(moe, n, 3, page, 2 * n, 8 * n * page, seed=n)
    seen = 0
    for _ in range(6):
        seen |= loop.step([r.choice([0, 1, page, r.randrange(2 * page + 1)]) for _ in range(n)])
    assert n == 1 or seen & 3 == 3


def test_shortages_one_by_one(moe):
    """Each shortage by itself and several at once, from lengths already in the cache."""
    for past, new, page, cols, room, n_free, head in (
            ([10, 20, 0], [30, 40, 50], 16, 8, 200, 4, 0),    # the free list runs out
            ([10, 20, 0], [30, 40, 50], 16, 3, 200, 40, 0),   # rows too short
            ([50, 70, 0], [30, 40, 50], 16, 3, 200, 40, 0),   # lengths already beyond the row
            ([10, 20, 0], [30, 40, 50], 16, 8, 61, 40, 0),    # no room for all tokens
            ([10, -5, 0], [30, 7, -1], 16, 8, 64, 40, 0),     # negative lengths
            ([1, 2], [40, 40], 16, 2, 10, 1, 0),              # several at once
            ([3, 2], [4, 4], 1, 8, 10, 5, 9)):                # a head beyond the list
        held = iter(range(1000, 2000))
        rows = [[next(held) if c < -(-max(p, 0) // page) else KEEP for c in range(cols)] for p in past]
        table, free = i32(rows), list(range(n_free))
        start, lens, pos, slot, info = walk(past, new, free, head, rows, page, room)
        p = moe.KvPlan(len(past), room, page).update(i32(past), i32(new), i32(free), i32([head]), table)
        assert p.info.tolist() == info and table.tolist() == rows
        assert p.q_start.tolist() == start and p.seq_len.tolist() == lens
        assert p.positions.tolist() == pos and p.slots.tolist() == slot
