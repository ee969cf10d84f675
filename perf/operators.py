"""The attention half of a decode step on a paged key-value cache, as cases to measure.

Four operators, each in a plain form (elementary torch operations in 32 bits, rounded once at the end) and, where
`own` is true, as calls of this package:

  plan   page allocation, positions and cache slots of the tokens a batch of requests brings
  rope   rotary positions on queries and keys; the rotated keys and the values written into the paged cache
  attn   attention of one new token per request over the paged cache
  norm   gated residual update of a block's output with the norms after and before it

`listed` gives the cases, `draw` another one of the same ranges, `prepare` what a program holds before the call, `run`
one pass, `work` what a pass cannot do without, `exact` the result in 64 bits from the definition.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode step of a small batch: one new token a request; latency is all there is
        dict(name="plan decode 8", op="plan", requests=8, new=1, past=3000, page=64, spare=0, lens=1),
        # a prefill wave of 512 ragged requests, some of them with a cached prefix; the token buffers have room to spare
        dict(name="plan prefill 512", op="plan", requests=512, new=700, past=400, page=16, spare=1000, lens=2),
        # one decoded token, 32 query and 8 key heads, interleaved pairs
        dict(name="rope decode 1", op="rope", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, rot_at=0, interleaved=True,
             scaling="none", kind="bf16", cache="bf16", page=64, start=2900),
        # a 2048-token prefill in the activations' fp32, rotating only the last 64 of 128 dimensions
        dict(name="rope prefill 2048 part", op="rope", tokens=2048, heads=32, kv_heads=8, dim=128, rot=64, rot_at=64,
             interleaved=True, scaling="linear", kind="f32", cache="bf16", page=64, start=0),
        # a long prefill chunk far into a long context, halves layout, frequencies scaled by parts, 8-bit cache
        dict(name="rope prefill 16384 e4m3", op="rope", tokens=16384, heads=64, kv_heads=8, dim=128, rot=128, rot_at=0,
             interleaved=False, scaling="parts", kind="bf16", cache="e4m3", page=64, start=114000),
        # one request early in its life
        dict(name="attn 1 x 777", op="attn", requests=1, longest=777, lens=0, heads=32, kv_heads=8, dim=128, kind="bf16",
             cache="bf16", page=16, window=0, by_head=False),
        # the verify batch's size: eight ragged requests of a few thousand tokens
        dict(name="attn 8 x 4100", op="attn", requests=8, longest=4100, lens=3, heads=64, kv_heads=8, dim=128, kind="bf16",
             cache="bf16", page=64, window=0, by_head=False),
        # a full serving batch, lengths spread over two orders of magnitude
        dict(name="attn 64 x 32768", op="attn", requests=64, longest=32768, lens=4, heads=64, kv_heads=8, dim=128,
             kind="bf16", cache="bf16", page=64, window=0, by_head=True),
        # two very long contexts in an 8-bit cache
        dict(name="attn 2 x 131072 e4m3", op="attn", requests=2, longest=131072, lens=0, heads=32, kv_heads=8, dim=128,
             kind="f16", cache="e4m3", page=64, window=0, by_head=False),
        # fp32 activations, a key head for each query head of 64 dimensions, a sliding window
        dict(name="attn 32 x 5000 f32 window", op="attn", requests=32, longest=5000, lens=5, heads=16, kv_heads=16, dim=64,
             kind="f32", cache="f16", page=32, window=1024, by_head=False),
        # one decoded token of the hidden size that the layer's configurations use, fp32 residual stream
        dict(name="norm 1 x 6144", op="norm", tokens=1, dim=6144, kind="f32", post=True, pre=True, gate="none"),
        # a prefill of 2048 tokens, a gate value for each channel of each token
        dict(name="norm 2048 x 6144 gated", op="norm", tokens=2048, dim=6144, kind="f32", post=True, pre=True, gate="full"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "attn", "attn", "norm"])
    if op == "plan":
        n = _log(rng, 1, 2048)
        new = rng.choice([1, _log(rng, 1, max(1, 262144 // n))])
        return dict(op=op, requests=n, new=new, past=_log(rng, 1, 20000), page=rng.choice([16, 32, 48, 64, 128]),
                    spare=rng.choice([0, rng.randrange(1, 2000)]), lens=rng.randrange(1, 1 << 20))
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([dim, dim // 2, 32])
        kv = rng.choice([1, 2, 4, 8, 16])
        kind = rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=kv * rng.choice([1, 2, 4, 5, 8]) if kv < 16 else 16, kv_heads=kv,
                    dim=dim, rot=rot, rot_at=rng.choice([0, dim - rot]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "parts"]), kind=kind,
                    cache=rng.choice(["f16" if kind == "f16" else "bf16", "e4m3"]), page=rng.choice([16, 32, 48, 64]),
                    start=_log(rng, 1, 120000))
    if op == "attn":
        kv, group, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 5, 8, 12, 16]), rng.choice([64, 80, 96, 128, 256])
        n = _log(rng, 1, 128)
        kind = rng.choice(["bf16", "bf16", "f16", "f32"])
        cache = rng.choice(["f16" if kind == "f16" else "bf16", "e4m3"])
        # the cache of a drawn case holds 0.5 GB of keys and values at most
        most = 5e8 / (n * kv * dim * 2 * SIZE[cache])
        longest = _log(rng, 1, int(max(1, min(131072, most))))
        return dict(op=op, requests=n, longest=longest, lens=rng.choice([0, rng.randrange(1, 1 << 20)]), heads=kv * group,
                    kv_heads=kv, dim=dim, kind=kind, cache=cache, page=rng.choice([16, 32, 48, 64, 128]),
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), by_head=rng.random() < 0.5)
    return dict(op=op, tokens=_log(rng, 1, 4096), dim=rng.choice([64, 256, 1000, 1536, 2049, 4096, 5120, 6144, 8192]),
                kind=rng.choice(["f32", "f32", "bf16", "f16"]), post=rng.random() < 0.7, pre=rng.random() < 0.8,
                gate=rng.choice(["none", "token", "channel", "full"]))


# ------------------------------------------------------------------ inputs

def _ragged(seed, n, longest):
    """n lengths of 1..longest, spread over their logarithm; seed 0: all the longest."""
    if seed == 0:
        return [longest] * n
    r = random.Random(seed)
    got = [_log(r, max(1, longest // 100), longest) for _ in range(n)]
    got[r.randrange(n)] = longest
    return got


def _plan_lens(c):
    r = random.Random(c["lens"])
    new = [1] * c["requests"] if c["new"] == 1 else [r.randrange(1, 2 * c["new"]) for _ in range(c["requests"])]
    past = [r.randrange(0, 2 * c["past"]) for _ in range(c["requests"])]
    if c["new"] > 1:  # a cached prefix is the exception in a prefill
        past = [p if r.random() < 0.3 else 0 for p in past]
    return past, new


def _pages(n, page):
    return -(-n // page)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, kind, std=1.0):
    if kind == "e4m3":
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * std).to(DT[kind])
    return torch.randn(shape, generator=g, device="cuda", dtype=DT[kind]) * std


def _turns(c):
    """Radians a position turns each pair by, in 64 bits, and the factor on cos and sin."""
    half, base, s = c["rot"] // 2, 10000.0, 8.0
    i = torch.arange(half, dtype=torch.float64)
    if c["scaling"] == "ntk":
        base = base * s ** (c["rot"] / (c["rot"] - 2))
    theta = base ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        theta = theta / s
    if c["scaling"] == "parts":
        keep = ((16384 * theta / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        theta = theta * (keep + (1 - keep) / s)
        return theta, 0.1 * math.log(s) + 1.0
    return theta, 1.0


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(c=c)
    if c["op"] == "plan":
        past, new = _plan_lens(c)
        n, page = c["requests"], c["page"]
        have, need = [_pages(p, page) for p in past], [_pages(p + q, page) for p, q in zip(past, new)]
        pool = sum(need) + 64
        ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table = torch.full((n, max(need) + 3), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(table.shape[1], device="cuda")
        held = torch.tensor(have, device="cuda")
        first = held.cumsum(0) - held
        table = torch.where(col < held[:, None], ids[(first[:, None] + col).clamp(max=pool - 1)], table).contiguous()
        st.update(past=torch.tensor(past, dtype=torch.int32, device="cuda"),
                  new=torch.tensor(new, dtype=torch.int32, device="cuda"), table=table, free=ids[sum(have):].contiguous(),
                  head=torch.zeros(1, dtype=torch.int32, device="cuda"), room=sum(new) + c["spare"])
        if own:
            import serving_router_sigmoid_gb300 as moe
            st["plan"] = moe.KvPlan(n, st["room"], page, device="cuda")
        return st
    if c["op"] == "rope":
        t, d, page = c["tokens"], c["dim"], c["page"]
        width = (c["heads"] + 2 * c["kv_heads"]) * d
        qkv = _normal(g, (t, width), c["kind"])  # as one projection gives them
        q, k, v = qkv.split([c["heads"] * d, c["kv_heads"] * d, c["kv_heads"] * d], dim=1)
        pages = _pages(t, page) + 3
        ids = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(t, device="cuda")
        shape = (pages, page, c["kv_heads"], d)
        st.update(q=q.unflatten(1, (c["heads"], d)), k=k.unflatten(1, (c["kv_heads"], d)),
                  v=v.unflatten(1, (c["kv_heads"], d)), slots=ids[at // page] * page + at % page,
                  positions=(at + c["start"]).to(torch.int32), k_cache=_normal(g, shape, c["cache"]),
                  v_cache=_normal(g, shape, c["cache"]), scales=(0.0225, 0.0175) if c["cache"] == "e4m3" else (1.0, 1.0))
        theta, amp = _turns(c)
        if own:
            import serving_router_sigmoid_gb300 as moe
            st["rope"] = moe.Rope(c["rot"], base=10000.0, interleaved=c["interleaved"], rot_offset=c["rot_at"],
                                  scaling=c["scaling"], factor=8.0, original_len=16384, device="cuda")
        else:  # the table of cos and sin that such a program keeps
            turn = torch.arange(c["start"] + t, dtype=torch.float64, device="cuda")[:, None] * theta.cuda()
            st["cos"], st["sin"] = (turn.cos() * amp).float(), (turn.sin() * amp).float()
        return st
    if c["op"] == "attn":
        n, d, page = c["requests"], c["dim"], c["page"]
        lens = _ragged(c["lens"], n, c["longest"])
        held = torch.tensor([_pages(x, page) for x in lens], device="cuda")
        pages = int(sum(_pages(x, page) for x in lens)) + 2
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        first = held.cumsum(0) - held
        col = torch.arange(_pages(c["longest"], page) + 1, device="cuda")
        table = torch.where(col < held[:, None], ids[(first[:, None] + col).clamp(max=pages - 1)], -1)
        shape = (pages, c["kv_heads"], page, d) if c["by_head"] else (pages, page, c["kv_heads"], d)
        k, v = _normal(g, shape, c["cache"]), _normal(g, shape, c["cache"])
        if c["by_head"]:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        st.update(q=_normal(g, (n, c["heads"], d), c["kind"], 2.0), k_cache=k, v_cache=v,
                  table=table.to(torch.int32).contiguous(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  scales=(0.9, 1.1) if c["cache"] == "e4m3" else (1.0, 1.0), scale=1 / math.sqrt(d))
        if own:
            import serving_router_sigmoid_gb300 as moe
            st["attn"] = moe.PagedAttention(n, c["heads"], c["kv_heads"], d, device="cuda")
        return st
    t, d = c["tokens"], c["dim"]
    gate = {"none": None, "token": (t, 1), "channel": (1, d), "full": (t, d)}[c["gate"]]
    st.update(x=_normal(g, (t, d), c["kind"], 3.0), y=_normal(g, (t, d), c["kind"]),
              post=1 + _normal(g, (d,), "f32", 0.1) if c["post"] else None,
              pre=1 + _normal(g, (d,), "f32", 0.1) if c["pre"] else None,
              gate=None if gate is None else _normal(g, gate, c["kind"]), alpha=1.0, beta=0.5)
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["c"]["op"]](state)


def _plain_plan(s):
    page, past, new, free, table = s["c"]["page"], s["past"], s["new"], s["free"], s["table"]
    have, need = (past + page - 1) // page, (past + new + page - 1) // page
    take = need - have
    first = s["head"] + take.cumsum(0) - take
    col = torch.arange(table.shape[1], device=table.device, dtype=torch.int32)
    taken = (col >= have[:, None]) & (col < need[:, None])
    table.copy_(torch.where(taken, free[(first[:, None] + col - have[:, None]).clamp(0, free.numel() - 1)], table))
    end = new.cumsum(0)
    tok = torch.arange(s["room"], device=table.device)
    req = torch.searchsorted(end, tok, right=True).clamp(max=new.numel() - 1)
    pos = past[req] + tok - (end - new)[req]
    slot = table[req, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    live = tok < end[-1]
    start = torch.cat([torch.zeros_like(end[:1]), end]).int()
    lens = past + new
    info = torch.stack([end[-1].int(), (s["head"][0] + take.sum()).int(), torch.zeros_like(past[0]), lens.max()]).int()
    return dict(table=table, start=start, lens=lens, positions=torch.where(live, pos, 0).int(),
                slots=torch.where(live, slot, -1), info=info)


def _own_plan(s):
    p = s["plan"]
    p.update(s["past"], s["new"], s["free"], s["head"], s["table"])
    return dict(table=s["table"], start=p.q_start, lens=p.seq_len, positions=p.positions, slots=p.slots, info=p.info)


def _rotate(x, cos, sin, c):
    x = x.float()
    part = x[..., c["rot_at"]:c["rot_at"] + c["rot"]]
    a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else part.chunk(2, dim=-1)
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], dim=-1).flatten(-2) if c["interleaved"] else torch.cat([a, b], dim=-1)
    return torch.cat([x[..., :c["rot_at"]], turned, x[..., c["rot_at"] + c["rot"]:]], dim=-1)


def _stored(x, scale, kind):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(DT[kind]) if kind == "e4m3" else x.to(DT[kind])


def _put(cache, slots, rows):
    """cache.flatten(0, 1)[slots] = rows, on the bytes where the type is an 8-bit one."""
    if rows.element_size() == 1:
        cache, rows = cache.view(torch.uint8), rows.view(torch.uint8)
    cache.view(-1, *cache.shape[2:])[slots] = rows


def _plain_rope(s):
    c = s["c"]
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    _put(s["k_cache"], s["slots"], _stored(_rotate(s["k"], cos, sin, c), s["scales"][0], c["cache"]))
    _put(s["v_cache"], s["slots"], _stored(s["v"].float(), s["scales"][1], c["cache"]))
    return dict(q=_rotate(s["q"], cos, sin, c).to(s["q"].dtype), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_rope(s):
    q = s["rope"].append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                         k_scale=s["scales"][0], v_scale=s["scales"][1])
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _gathered(cache, table):
    """Every request's rows of the cache, [requests, longest, heads, dim] in 32 bits."""
    at = table.clamp(min=0).long()
    rows = cache.view(torch.uint8)[at].view(cache.dtype) if cache.element_size() == 1 else cache[at]
    return rows.flatten(1, 2).float()


def _plain_attn(s):
    c, lens = s["c"], s["lens"]
    k, v = _gathered(s["k_cache"], s["table"]), _gathered(s["v_cache"], s["table"])
    at = torch.arange(k.shape[1], device=k.device)
    seen = at < lens[:, None]
    if c["window"]:
        seen = seen & (at >= lens[:, None] - c["window"])
    v = torch.where(seen[:, :, None, None], v, 0)
    q = s["q"].float().unflatten(1, (c["kv_heads"], -1)) * (s["scale"] * s["scales"][0])
    score = q @ k.permute(0, 2, 3, 1)  # [requests, kv head, group, longest]
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v.transpose(1, 2)) / total * s["scales"][1]
    return dict(out=out.flatten(1, 2).to(s["q"].dtype), lse=(top + total.log()).flatten(1))


def _own_attn(s):
    out, lse = s["attn"].decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["scale"],
                                window=s["c"]["window"], k_scale=s["scales"][0], v_scale=s["scales"][1])
    return dict(out=out, lse=lse)


def _unit(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_norm(s):
    u = s["y"].float()
    if s["post"] is not None:
        u = _unit(u, s["post"])
    if s["gate"] is not None:
        u = u / (1 + (-s["gate"].float()).exp())
    r = s["alpha"] * s["x"].float() + s["beta"] * u
    got = dict(out=r.to(s["x"].dtype))
    if s["pre"] is not None:
        got["normed"] = _unit(r, s["pre"]).to(s["x"].dtype)
    return got


def _own_norm(s):
    import serving_router_sigmoid_gb300 as moe
    out, normed = moe.block_norm(s["x"], s["y"], w_post=s["post"], gate=s["gate"], gate_act="sigmoid", w_pre=s["pre"],
                                 alpha=s["alpha"], beta=s["beta"], eps=EPS)
    return dict(out=out) if normed is None else dict(out=out, normed=normed)


_plain = dict(plan=_plain_plan, rope=_plain_rope, attn=_plain_attn, norm=_plain_norm)
_own = dict(plan=_own_plan, rope=_own_rope, attn=_own_attn, norm=_own_norm)


# ------------------------------------------------------------------ what a pass needs

def work(case):
    c = case
    if c["op"] == "plan":
        past, new = _plan_lens(c)
        pages = sum(_pages(p + n, c["page"]) - _pages(p, c["page"]) for p, n in zip(past, new))
        # both lengths in, both tables out; a position and a slot a token; each page id read and written
        return dict(bytes=16 * c["requests"] + 12 * (sum(new) + c["spare"]) + 8 * pages, flops=0)
    if c["op"] == "rope":
        one, cached = SIZE[c["kind"]], SIZE[c["cache"]]
        turned = (c["heads"] + c["kv_heads"]) * c["rot"]
        return dict(bytes=c["tokens"] * c["dim"] * (2 * one * c["heads"] + 2 * c["kv_heads"] * (one + cached)) + 12 * c["tokens"],
                    flops=3 * c["tokens"] * turned)
    if c["op"] == "attn":
        lens = [min(x, c["window"] or x) for x in _ragged(c["lens"], c["requests"], c["longest"])]
        rows = sum(lens)
        return dict(bytes=2 * rows * c["kv_heads"] * c["dim"] * SIZE[c["cache"]]
                    + c["requests"] * c["heads"] * (2 * c["dim"] * SIZE[c["kind"]] + 4) + 4 * sum(_pages(x, c["page"]) for x in lens),
                    flops=4 * rows * c["heads"] * c["dim"])
    t, d, one = c["tokens"], c["dim"], SIZE[c["kind"]]
    gate = {"none": 0, "token": t, "channel": d, "full": t * d}[c["gate"]]
    return dict(bytes=one * (t * d * (3 + c["pre"]) + gate) + 4 * d * (c["post"] + c["pre"]), flops=t * d * 12)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "plan":
        return None  # whole numbers only
    if c["op"] == "rope":
        theta, amp = _turns(c)
        angle = s["positions"].double()[:, None] * theta.to("cuda")
        w = torch.polar(torch.full_like(angle, amp), angle)[:, None]

        def turn(x):
            x = x.double().clone()
            lo, half = c["rot_at"], c["rot"] // 2
            at = torch.arange(half, device="cuda")
            i, j = (lo + 2 * at, lo + 2 * at + 1) if c["interleaved"] else (lo + at, lo + half + at)
            z = torch.complex(x[..., i], x[..., j]) * w
            x[..., i], x[..., j] = z.real, z.imag
            return x

        def filled(cache, rows, scale):
            got = cache.double().flatten(0, 1)
            got[s["slots"]] = rows / scale
            return got.view(cache.shape)

        return dict(q=turn(s["q"]), k_cache=filled(s["k_cache"], turn(s["k"]), s["scales"][0]),
                    v_cache=filled(s["v_cache"], s["v"].double(), s["scales"][1]))
    if c["op"] == "attn":
        out, lse = [], []
        for b, n in enumerate(_ragged(c["lens"], c["requests"], c["longest"])):
            at = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device="cuda")
            rows = s["table"][b].long()[at // c["page"]], at % c["page"]
            k, v = ((x.view(torch.uint8)[rows].view(x.dtype) if x.element_size() == 1 else x[rows]).double() * f
                    for x, f in ((s["k_cache"], s["scales"][0]), (s["v_cache"], s["scales"][1])))
            q = s["q"][b].double().unflatten(0, (c["kv_heads"], -1))
            score = torch.einsum("hgd,lhd->hgl", q, k) * s["scale"]
            lse.append(torch.logsumexp(score, -1).flatten())
            out.append(torch.einsum("hgl,lhd->hgd", torch.softmax(score, -1), v).flatten(0, 1))
        return dict(out=torch.stack(out), lse=torch.stack(lse))
    x, u = s["x"].double(), s["y"].double()
    if s["post"] is not None:
        u = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * s["post"].double()
    if s["gate"] is not None:
        u = u * torch.sigmoid(s["gate"].double())
    r = s["alpha"] * x + s["beta"] * u
    if s["pre"] is None:
        return dict(out=r)
    return dict(out=r, normed=r / (r.square().mean(-1, keepdim=True) + EPS).sqrt() * s["pre"].double())
