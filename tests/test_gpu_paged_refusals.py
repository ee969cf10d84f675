"""Arguments that do not fit their field or have another rank are refused as
ValueError, like all other arguments of the paged-cache operators; numbers
beyond fp32 reach the library as infinities and are refused there."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def test_numbers(moe):
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn((2, 4, 64), device="cuda")
    cache = torch.zeros((4, 16, 4, 64), dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros((2, 2), **i32), torch.ones(2, **i32)
    attn, rope = moe.PagedAttention(2, 4, 4, 64), moe.Rope(64)
    attn.decode(q, cache, cache, table, lens)
    for bad in (dict(window=2**31), dict(window=1.5), dict(window=None), dict(scale="1"), dict(v_scale=None)):
        with pytest.raises(ValueError):
            attn.decode(q, cache, cache, table, lens, **bad)
    for bad in (dict(scale=1e39), dict(k_scale=1e300)):
        with pytest.raises(moe.MoeError):
            attn.decode(q, cache, cache, table, lens, **bad)
    slots = torch.arange(2, device="cuda")
    for bad, error in ((dict(k_scale=1e39), moe.MoeError), (dict(v_scale="1"), ValueError)):
        with pytest.raises(error):
            rope.append(q, q, q, lens, slots, cache, cache.clone(), **bad)
    x = torch.randn((2, 64), device="cuda")
    for bad, error in ((dict(alpha=1e39), moe.MoeError), (dict(beta=None), ValueError), (dict(eps="0"), ValueError)):
        with pytest.raises(error):
            moe.block_norm(x, x.clone(), **bad)


def test_plan_ranks(moe):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan, t = moe.KvPlan(2, 8, 16), torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    ok = [i32([1, 2]), i32([1, 1]), i32([3, 4]), i32([0]), t]
    plan.update(*ok)
    for at in range(5):
        for other in (lambda a: a.flatten()[0], lambda a: a[None]):
            bad = list(ok)
            bad[at] = other(bad[at])
            with pytest.raises(ValueError):
                plan.update(*bad)


def test_plan_outputs_as_inputs(moe):
    """The plan's own outputs would be read while they are written; another plan's are fine."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    past, one, free, head = i32([0, 40]), i32([1, 1]), i32([7, 3, 5, 6]), i32([0])
    table = i32([[-1] * 4, [1, 2, 4, -1]])
    plan, other = moe.KvPlan(2, 4, 16), moe.KvPlan(2, 4, 16)
    plan.update(past, one, free, head, table)
    for bad in ((plan.seq_len, one, free, head, table), (past, plan.seq_len, free, head, table),
                (past, one, free, plan.info[1:2], table), (past, one, plan.positions, head, table),
                (table[0, 1:3], one, free, head, table), (past, one, free, table[1, 3:], table)):
        with pytest.raises(moe.MoeError):
            plan.update(*bad)
    other.update(plan.seq_len, one, free, plan.info[1:2], table)
    assert other.seq_len.tolist() == [2, 42] and other.slots.tolist() == [7 * 16 + 1, 4 * 16 + 9, -1, -1]
    assert other.info.tolist() == [2, 1, 0, 42]


def test_tables_near_2_31_tokens(moe):
    """A step that ends at a request's last tokens would end beyond 2^31."""
    q = torch.randn((1, 1, 8), device="cuda")
    cache, lens = torch.zeros((1, 3, 1, 8), dtype=torch.float16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.empty((1, 2**31 // 3), dtype=torch.int32, device="cuda")
    attn = moe.PagedAttention(1, 1, 1, 8)
    with pytest.raises(moe.MoeError):
        attn.decode(q, cache, cache, table, lens)
    attn.decode(q, cache, cache, table[:, :-22], lens)
