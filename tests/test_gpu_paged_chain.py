"""The paged-cache operators one after another in a CUDA graph, where each call's
kernel is resident before the one it takes its inputs from has ended, against
the same calls with a synchronisation after each: the same bits."""
import os
import sys

import pytest
import torch

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu

STEPS, N, HEADS, KV, DIM, PAGE = 10, 7, 8, 2, 128, 16


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


class Chain:
    """Decode steps of plan -> rope -> attention -> norm, and nothing between them."""

    def __init__(self, moe, act, cache):
        g = torch.Generator(device="cuda").manual_seed(5)
        new = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        i32 = dict(dtype=torch.int32, device="cuda")
        self.moe, width = moe, HEADS * DIM
        self.plans = [moe.KvPlan(N, N, PAGE) for _ in range(STEPS)]
        self.rope, self.attn = moe.Rope(DIM, interleaved=True), moe.PagedAttention(N, HEADS, KV, DIM)
        self.one, self.free = torch.ones(N, **i32), torch.randperm(400, generator=g, device="cuda").to(torch.int32)
        self.start = torch.tensor([0, 15, 16, 40, 700, 3, 100], **i32)
        self.table0 = torch.full((N, 60), -1, **i32)
        ids = iter(range(400, 600))
        for b, n in enumerate(self.start.tolist()):
            for c in range(-(-n // PAGE)):
                self.table0[b, c] = next(ids)
        self.x0, self.w_post, self.w_pre = new(N, width).to(act), 1 + 0.1 * new(width), 1 + 0.1 * new(width)
        self.kv = [new(N, KV, DIM).to(act) for _ in range(2 * STEPS)]
        self.cache0 = [new(600, PAGE, KV, DIM).to(cache).view(torch.uint8) for _ in range(2)]
        self.cache = [torch.empty_like(c).view(cache) for c in self.cache0]
        self.table, self.q = torch.empty_like(self.table0), torch.empty_like(self.x0)
        self.out = [(torch.empty((N, width), dtype=act, device="cuda"), torch.empty((N, HEADS), device="cuda"),
                     torch.empty((N, width), dtype=act, device="cuda"), torch.empty((N, width), dtype=act, device="cuda"))
                    for _ in range(STEPS)]

    def reset(self):
        self.table.copy_(self.table0)
        for c, z in zip(self.cache, self.cache0):
            c.view(torch.uint8).copy_(z)
        for step in self.out:
            for t in step:
                t.fill_(7.0)

    def run(self, between):
        past, head, x = self.start, torch.zeros(1, dtype=torch.int32, device="cuda"), self.x0
        for i, plan in enumerate(self.plans):
            att, lse, res, nrm = self.out[i]
            plan.update(past, self.one, self.free, head, self.table)
            between()
            q = x.unflatten(1, (HEADS, DIM))
            self.rope.append(q, self.kv[2 * i], self.kv[2 * i + 1], plan.positions, plan.slots, *self.cache,
                             q_out=self.q.unflatten(1, (HEADS, DIM)))
            between()
            self.attn.decode(self.q.unflatten(1, (HEADS, DIM)), *self.cache, self.table, plan.seq_len,
                             out=att.unflatten(1, (HEADS, DIM)), lse=lse)
            between()
            self.moe.block_norm(x, att, w_post=self.w_post, w_pre=self.w_pre, out=res, normed=nrm)
            between()
            past, head, x = plan.seq_len, plan.info[1:2], nrm

    def results(self):
        got = [t.clone() for step in self.out for t in step] + [self.table.clone()]
        got += [c.view(torch.uint8).clone() for c in self.cache]
        return got + [t.clone() for p in self.plans for t in (p.seq_len, p.positions, p.slots, p.info, p.q_start)]


@pytest.mark.parametrize("act,cache", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16),
                                       (torch.float16, torch.float8_e4m3fn)])
def test_overlapped_launches_see_the_outputs_before_them(moe, act, cache):
    chain = Chain(moe, act, cache)
    chain.reset()
    chain.run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = chain.results()
    assert all(int(p.info[2]) == 0 for p in chain.plans)
    assert all(torch.isfinite(t.float()).all() for step in chain.out for t in step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain.run(lambda: None)
    for _ in range(10):
        chain.reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(chain.results(), want))


def test_the_example_block_in_a_graph(moe):
    """Norms and the MoE layer's kernel, which overlaps them, in the example's decode step."""
    import decode_block as ex
    block = ex.Block(3, pages=64)
    g = torch.Generator(device="cuda").manual_seed(2)
    lengths = torch.tensor([9, 30, 2], dtype=torch.int32, device="cuda")
    block.prompt(torch.randn((41, block.cfg.D), generator=g, device="cuda"), lengths)
    x0 = torch.randn((3, block.cfg.D), generator=g, device="cuda")
    state = [t.clone() for t in (block.head, block.past, block.table)]
    # the layer's part of a step by itself: norm -> experts -> join, kernel after kernel
    y = torch.randn((3, block.cfg.D), generator=g, device="cuda")

    def joined(between):
        x, outs = x0, []
        for _ in range(6):
            r, h = moe.block_norm(x, y, w_post=block.w.post, gate=block.w.gate, w_pre=block.w.moe, eps=ex.EPS)
            between()
            m = block.layer.forward(h)
            between()
            x, _ = moe.block_norm(r, m)
            between()
            outs += [r, h, m, x]
        return outs

    want = joined(torch.cuda.synchronize)
    steps, x = [], x0
    for _ in range(4):
        x = block.step(x).out
        torch.cuda.synchronize()
        steps.append(x)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        got = joined(lambda: None)
    with torch.cuda.graph(g2):
        out, x = [], x0
        for _ in range(4):
            x = block.step(x).out
            out.append(x)
    for _ in range(10):
        for t in got + out:
            t.fill_(3.0)
        g1.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for t, z in zip((block.head, block.past, block.table), state):
            t.copy_(z)
        g2.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, steps))
    assert block.layer.device_status() == 0
    block.layer.close()
