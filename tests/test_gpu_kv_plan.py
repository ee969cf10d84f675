"""moe_kv_plan against a plain Python walk over the requests: whole numbers,
compared for equality, with the entries that must stay as they were."""
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


def walk(past, new, free, head, table, page, room):
    """The definition, request by request; table: list of rows, updated."""
    flags, taken, start, pos, slot = 0, 0, [0], [], []
    for b, (p, n) in enumerate(zip(past, new)):
        if p < 0 or n < 0:
            flags |= 8
            p, n = max(p, 0), max(n, 0)
        have, need = -(-p // page), -(-(p + n) // page)
        if need > len(table[b]):
            flags |= 2
        for col in range(have, need):
            got = free[head + taken] if head + taken < len(free) else -1
            taken += 1
            if col < len(table[b]):
                table[b][col] = got
        for i in range(p, p + n):
            pos.append(i)
            at = table[b][i // page] if i // page < len(table[b]) else -1
            slot.append(at * page + i % page if at >= 0 else -1)
        start.append(start[-1] + n)
    avail = max(len(free) - head, 0)
    flags |= 1 if taken > avail else 0
    flags |= 4 if start[-1] > room else 0
    lens = [max(p, 0) + max(n, 0) for p, n in zip(past, new)]
    info = [start[-1], head + min(taken, avail), flags, max(lens, default=0)]
    pad = max(0, room - len(pos))
    return start, lens, (pos + [0] * pad)[:room], (slot + [-1] * pad)[:room], info


def check(moe, past, new, page, cols, room, n_free, head=0, wide=0, seed=0, rows=0):
    r = random.Random(seed)
    n = len(past)
    ids = r.sample(range(4 * (n_free + sum(max(p, 0) // page + 1 for p in past)) + 8), n_free + sum(
        max(p, 0) // page + 1 for p in past))
    free, held = ids[:n_free], iter(ids[n_free:])
    table = [[KEEP] * cols for _ in range(n)]
    for row, p in zip(table, past):
        for c in range(min(cols, -(-max(p, 0) // page))):
            row[c] = next(held)
    full = torch.full((n + rows, cols + wide), KEEP, dtype=torch.int32)
    full[:n, :cols] = torch.tensor(table, dtype=torch.int32).view(n, cols)
    dev = full.cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = moe.KvPlan(max(n, 1) + rows, room, page)
    start, lens, pos, slot, info = walk(past, new, free, head, table, page, room)
    full[:n, :cols] = torch.tensor(table, dtype=torch.int32).view(n, cols)
    for _ in range(2):  # a second call on the same inputs gives the same outputs
        plan.update(i32(past), i32(new), i32(free), i32([head]), dev[:, :cols])
        assert plan.info.tolist() == info
        assert plan.q_start.tolist() == start
        assert plan.seq_len.tolist() == lens
        assert plan.positions.tolist() == pos
        assert plan.slots.tolist() == slot
        assert torch.equal(dev.cpu(), full)


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("n", [1, 2, 8, 33, 511, 513, 1500])
def test_ragged_batches(moe, n, page):
    r = random.Random(n * 100 + page)
    past = [r.choice([0, 1, page - 1, page, page + 1, r.randrange(200)]) for _ in range(n)]
    new = [r.choice([0, 1, 1, page, r.randrange(60)]) for _ in range(n)]
    need = sum(-(-(p + q) // page) - -(-p // page) for p, q in zip(past, new))
    cols = max(-(-(p + q) // page) for p, q in zip(past, new)) + 2
    check(moe, past, new, page, cols, sum(new) + r.choice([0, 1, 37]), need + 5, head=3, wide=3, seed=n, rows=2)


def test_one_new_token_each_and_the_largest_batch(moe):
    r = random.Random(5)
    past = [r.randrange(0, 300) for _ in range(8192)]
    check(moe, past, [1] * 8192, 64, 6, 8192, 8192, seed=2)


def test_one_long_request(moe):
    check(moe, [5], [300001], 16, 18752, 300001, 18760)


def test_no_requests_and_no_tokens(moe):
    plan = moe.KvPlan(4, 9, 16)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    plan.update(e, e, e, torch.tensor([0], dtype=torch.int32, device="cuda"),
                torch.empty((0, 3), dtype=torch.int32, device="cuda"))
    assert plan.info.tolist() == [0, 0, 0, 0] and plan.q_start.tolist() == [0]
    assert plan.slots.tolist() == [-1] * 9 and plan.positions.tolist() == [0] * 9
    check(moe, [0, 40, 3], [0, 0, 0], 16, 4, 0, 2)


def test_shortages_are_flagged_and_leave_no_slot(moe):
    check(moe, [10, 20, 0], [30, 40, 50], 16, 8, 200, 4)          # the free list runs out
    check(moe, [10, 20, 0], [30, 40, 50], 16, 3, 200, 40)         # rows too short
    check(moe, [10, 20, 0], [30, 40, 50], 16, 8, 61, 40)          # no room for all tokens
    check(moe, [10, -5, 0], [30, 7, -1], 16, 8, 64, 40)           # negative lengths
    check(moe, [1, 2], [40, 40], 16, 2, 10, 1)                    # several at once
    check(moe, [3, 2], [4, 4], 1, 8, 10, 5, head=9)               # a head beyond the list


def test_side_stream_and_graph(moe):
    past, new = [5, 17, 0], [1, 1, 33]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, free, head = torch.full((3, 8), -1, dtype=torch.int32, device="cuda"), i32(list(range(100, 120))), i32([0])
    table[0, 0], table[1, 0], table[1, 1] = 7, 8, 9
    p, q = i32(past), i32(new)
    plan, s = moe.KvPlan(3, 40, 16), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.update(p, q, free, head, table, stream=s)
    s.synchronize()
    want = plan.slots.tolist()
    plan.slots.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.update(p, q, free, head, table)
    g.replay()
    torch.cuda.synchronize()
    assert plan.slots.tolist() == want
    q += 1  # new lengths, same graph
    g.replay()
    torch.cuda.synchronize()
    assert plan.seq_len.tolist() == [7, 19, 34] and plan.info.tolist()[0] == 38


def test_refusals(moe):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan, t = moe.KvPlan(2, 8, 16), torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    ok = (i32([1, 2]), i32([1, 1]), i32([3, 4]), i32([0]), t)
    plan.update(*ok)
    for bad in ((i32([1, 2, 3]), i32([1, 1, 1])) + ok[2:], (ok[0].cpu(),) + ok[1:], (ok[0].long(),) + ok[1:],
                ok[:1] + (i32([1]),) + ok[2:], ok[:4] + (t[:1],), ok[:4] + (t.t(),), ok[:3] + (i32([0, 1]),) + ok[4:]):
        with pytest.raises(ValueError):
            plan.update(*bad)
    with pytest.raises(moe.MoeError):
        moe.KvPlan(2, 8, 0).update(*ok)
