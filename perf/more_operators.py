"""FP8 block-scaled products and latent attention, as cases to measure.

What the dense half of a block with a compressed key-value cache computes around the MoE layer, for checkpoints whose
matrices are E4M3 codes with one scale a 128 x 128 block.  Four operators, each in a plain form (elementary torch
operations in 32 bits, rounded once at the end) and, where `own` is true, as calls of this package:

  quant   activations as E4M3 codes with one scale for each 128 of a row
  linear  the product of such activations with an E4M3 matrix
  decode  one new token a request over a paged cache of latent rows that all heads share (absorbed form): a row is the
          key, and its first part is the value
  prompt  ragged prompts, keys and values expanded a head, the rotary part of the keys shared by all heads

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
BLOCK = 128


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token of the layer's hidden size, in the fp32 that the block's norms give
        dict(name="quant 1 x 6144", op="quant", tokens=1, dim=6144, kind="f32"),
        # a 2048-token prefill of it, from 16-bit activations
        dict(name="quant 2048 x 6144", op="quant", tokens=2048, dim=6144, kind="bf16"),
        # one decoded token through a down projection to a 2048-wide query latent; the matrix has to be read, no more
        dict(name="linear 1: 6144 -> 2048", op="linear", tokens=1, inner=6144, outer=2048, kind="bf16"),
        # the verify batch's 8 tokens through the query projection of 64 heads of 192
        dict(name="linear 8: 2048 -> 12288", op="linear", tokens=8, inner=2048, outer=12288, kind="bf16"),
        # a ragged batch to the shared latent and rotary row (512 + 64), fp32 as the MoE layer's stream
        dict(name="linear 300: 6144 -> 576", op="linear", tokens=300, inner=6144, outer=576, kind="f32"),
        # the output projection of 64 heads of 128 in a 2048-token prefill
        dict(name="linear 2048: 8192 -> 6144", op="linear", tokens=2048, inner=8192, outer=6144, kind="bf16"),
        # one request early in its life
        dict(name="decode 1 x 777", op="decode", requests=1, longest=777, lens=0, heads=64, latent=512, rope=64, kind="bf16",
             cache="bf16", page=16),
        # a full serving batch, lengths spread over two orders of magnitude, 128 heads
        dict(name="decode 64 x 16384", op="decode", requests=64, longest=16384, lens=4, heads=128, latent=512, rope=64,
             kind="bf16", cache="bf16", page=64),
        # two very long contexts in an 8-bit cache
        dict(name="decode 2 x 131072 e4m3", op="decode", requests=2, longest=131072, lens=0, heads=64, latent=512, rope=64,
             kind="f16", cache="e4m3", page=64),
        # a few short ragged prompts, each behind a cached prefix
        dict(name="prompt 5 x 250", op="prompt", requests=5, longest=250, prefix=130, lens=7, heads=16, nope=128, rope=64,
             v=128, kind="f16", causal=True),
        # a 2048-token prompt of 64 heads of 128 + 64
        dict(name="prompt 2048", op="prompt", requests=1, longest=2048, prefix=0, lens=0, heads=64, nope=128, rope=64,
             v=128, kind="bf16", causal=True),
        # a chunk of a long prompt over everything before it, wide heads
        dict(name="prompt 1000 of 5000 wide", op="prompt", requests=1, longest=1000, prefix=4000, lens=0, heads=32,
             nope=192, rope=64, v=256, kind="bf16", causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "decode", "decode", "prompt", "prompt"])
    if op == "quant":
        return dict(op=op, tokens=_log(rng, 1, 4096), dim=rng.choice([64, 128, 512, 576, 1040, 2048, 5120, 6144]),
                    kind=rng.choice(["f32", "bf16", "f16"]))
    if op == "linear":
        inner, outer = rng.choice([64, 512, 576, 1040, 2048, 5120, 6144, 8192]), _log(rng, 24, 16384)
        most = 2048 * 8192 * 6144 // (inner * outer)
        return dict(op=op, tokens=_log(rng, 1, max(1, min(4096, most))), inner=inner, outer=outer,
                    kind=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "decode":
        heads = rng.choice([4, 8, 16, 20, 32, 48, 64, 96, 128])
        latent, rope = rng.choice([(512, 64), (512, 64), (256, 64), (512, 32), (384, 64), (128, 16)])
        kind = rng.choice(["bf16", "bf16", "f16"])
        n = _log(rng, 1, 128)
        # a drawn case's cache holds 300k tokens at most, and its plain form 3 GB of logits
        longest = _log(rng, 1, int(max(1, min(131072, 300000 // n, 7e8 // (n * heads)))))
        return dict(op=op, requests=n, longest=longest, lens=rng.choice([0, rng.randrange(1, 1 << 20)]), heads=heads,
                    latent=latent, rope=rope, kind=kind, cache=rng.choice([kind, kind, "e4m3"]),
                    page=rng.choice([1, 16, 32, 48, 64, 128]))
    heads, n = rng.choice([1, 4, 16, 24, 32, 64]), rng.choice([1, 1, 2, 3, 5, 8, 20])
    nope, rope, v = rng.choice([(128, 64, 128), (128, 64, 128), (192, 64, 256), (64, 32, 64), (96, 64, 80), (64, 64, 192)])
    room = 2e8 / (n * heads)  # of logits, padded
    longest = _log(rng, 1, int(min(2048, math.sqrt(room))))
    prefix = rng.choice([0, _log(rng, 1, int(max(1, min(8192, room / longest - longest))))])
    return dict(op=op, requests=n, longest=longest, prefix=prefix, lens=rng.choice([0, rng.randrange(1, 1 << 20)]),
                heads=heads, nope=nope, rope=rope, v=v, kind=rng.choice(["bf16", "bf16", "f16"]),
                causal=rng.random() < 0.8)


# ------------------------------------------------------------------ inputs

def _ragged(seed, n, longest):
    """n lengths of 1..longest, spread over their logarithm; seed 0: all the longest."""
    if seed == 0:
        return [longest] * n
    r = random.Random(seed)
    got = [_log(r, max(1, longest // 100), longest) for _ in range(n)]
    got[r.randrange(n)] = longest
    return got


def _prompts(c):
    """New tokens and tokens before them, a request."""
    new = _ragged(c["lens"], c["requests"], c["longest"])
    if not c["prefix"] or not c["lens"]:
        return new, [c["prefix"]] * len(new)
    r = random.Random(c["lens"] + 1)
    return new, [r.randrange(0, c["prefix"] + 1) for _ in new]


def _pages(n, page):
    return -(-n // page)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, kind, std=1.0):
    if kind == "e4m3":
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * std).to(DT[kind])
    return torch.randn(shape, generator=g, device="cuda", dtype=DT[kind]) * std


def _groups(x, block=BLOCK):
    """x [n, dim] as [n, groups, block], zeros behind its end."""
    n, dim = x.shape
    return torch.nn.functional.pad(x, (0, -dim % block)).view(n, -1, block)


def _spread(s, rows, cols):
    """The scales of 128 x 128 blocks, one an element."""
    return s.repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def _quantised(x):
    """Codes and scales of the rows of x, in 32 bits."""
    g = _groups(x.float())
    s = (g.abs().amax(-1) / E4M3_MAX).clamp(min=1e-12)
    q = (g / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :x.shape[1]]
    return q.to(DT["e4m3"]), s


def _activations(g, tokens, dim, kind):
    """Rows as a norm leaves them: channels of unequal size, a few of them large."""
    size = torch.randn(dim, generator=g, device="cuda").mul(0.7).exp()
    return (_normal(g, (tokens, dim), "f32") * size).to(DT[kind])


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = dict(c=c)
    if c["op"] == "quant":
        st.update(x=_activations(g, c["tokens"], c["dim"], c["kind"]))
        return st
    if c["op"] == "linear":
        x8, xs = _quantised(_activations(g, c["tokens"], c["inner"], "f32"))
        w = _normal(g, (c["outer"], c["inner"]), "f32", 0.02)
        rows, cols = _pages(c["outer"], BLOCK), _pages(c["inner"], BLOCK)
        pad = torch.nn.functional.pad(w, (0, cols * BLOCK - c["inner"], 0, rows * BLOCK - c["outer"]))
        ws = pad.view(rows, BLOCK, cols, BLOCK).abs().amax((1, 3)) / E4M3_MAX
        w8 = (w / _spread(ws, c["outer"], c["inner"])).clamp(-E4M3_MAX, E4M3_MAX).to(DT["e4m3"])
        st.update(x8=x8, xs=xs, w8=w8, ws=ws)
        return st
    if c["op"] == "decode":
        n, d, page = c["requests"], c["latent"] + c["rope"], c["page"]
        lens = _ragged(c["lens"], n, c["longest"])
        held = torch.tensor([_pages(x, page) for x in lens], device="cuda")
        pages = int(sum(_pages(x, page) for x in lens)) + 2
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        first = held.cumsum(0) - held
        col = torch.arange(_pages(c["longest"], page) + 1, device="cuda")
        table = torch.where(col < held[:, None], ids[(first[:, None] + col).clamp(max=pages - 1)], -1)
        st.update(q=_normal(g, (n, c["heads"], d), c["kind"]), cache=_normal(g, (pages, page, 1, d), c["cache"]),
                  table=table.to(torch.int32).contiguous(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  k_scale=0.9 if c["cache"] == "e4m3" else 1.0, scale=1 / math.sqrt(128 + c["rope"]))
        if own:
            import serving_router_sigmoid_gb300 as moe
            st["attn"] = moe.LatentAttention(n, c["heads"], c["latent"], c["rope"], device="cuda")
        return st
    new, past = _prompts(c)
    keys, h = [a + b for a, b in zip(new, past)], c["heads"]
    start = lambda v: torch.tensor([0] + v, device="cuda").cumsum(0).int()  # noqa: E731
    kv = _normal(g, (sum(keys), h, c["nope"] + c["v"]), c["kind"])  # as one projection gives them
    row = _normal(g, (sum(keys), 512 + c["rope"]), c["kind"])       # the latent row and its rotary part
    st.update(q=_normal(g, (sum(new), h, c["nope"] + c["rope"]), c["kind"]), k=kv[..., :c["nope"]], v=kv[..., c["nope"]:],
              k_rope=row[:, 512:], q_start=start(new), kv_start=start(keys), most=(max(new), max(keys)),
              scale=1 / math.sqrt(c["nope"] + c["rope"]))
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["c"]["op"]](state)


def _plain_quant(s):
    q, scale = _quantised(s["x"])
    return dict(x8=q, scale=scale)


def _own_quant(s):
    import serving_router_sigmoid_gb300 as moe
    x8, scale = moe.quant_act_fp8(s["x"])
    return dict(x8=x8, scale=scale)


def _plain_linear(s):
    c = s["c"]
    x = s["x8"].float() * s["xs"].repeat_interleave(BLOCK, 1)[:, :c["inner"]]
    w = s["w8"].float() * _spread(s["ws"], c["outer"], c["inner"])
    return dict(out=(x @ w.T).to(DT[c["kind"]]))


def _own_linear(s):
    import serving_router_sigmoid_gb300 as moe
    return dict(out=moe.fp8_linear(s["x8"], s["xs"], s["w8"], s["ws"], dtype=DT[s["c"]["kind"]]))


def _plain_decode(s):
    c, lens = s["c"], s["lens"]
    at = s["table"].clamp(min=0).long()
    cache = s["cache"][:, :, 0]
    rows = cache.view(torch.uint8)[at].view(cache.dtype) if cache.element_size() == 1 else cache[at]
    k = rows.flatten(1, 2).float() * s["k_scale"]  # [requests, longest, latent + rope]
    seen = torch.arange(k.shape[1], device=k.device) < lens[:, None]
    k = torch.where(seen[..., None], k, 0)
    score = (s["q"].float() * s["scale"]) @ k.transpose(1, 2)  # [requests, heads, longest]
    score = torch.where(seen[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ k[..., :c["latent"]]) / total
    return dict(out=out.to(s["q"].dtype), lse=(top + total.log())[..., 0])


def _own_decode(s):
    out, lse = s["attn"].decode(s["q"], s["cache"], s["table"], s["lens"], s["scale"], k_scale=s["k_scale"])
    return dict(out=out, lse=lse)


def _plain_prompt(s):
    c, q0, k0 = s["c"], s["q_start"].long(), s["kv_start"].long()
    nq, nk = q0.diff()[:, None], k0.diff()[:, None]
    i, j = (torch.arange(m, device=q0.device) for m in s["most"])
    qi, kj = (q0[:-1, None] + i).clamp(max=s["q"].shape[0] - 1), (k0[:-1, None] + j).clamp(max=s["v"].shape[0] - 1)
    q = s["q"][qi].float().transpose(1, 2) * s["scale"]  # [requests, heads, longest, nope + rope]
    key = s["k"][kj].float().permute(0, 2, 3, 1)
    score = q[..., :c["nope"]] @ key + q[..., c["nope"]:] @ s["k_rope"][kj].float().transpose(1, 2)[:, None]
    seen = (j < nk)[:, None, :] & (i < nq)[..., None]
    if c["causal"]:
        seen = seen & (j <= (nk - nq)[..., None] + i[:, None])
    score = torch.where(seen[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ s["v"][kj].float().transpose(1, 2)) / total
    live = i < nq
    return dict(out=out.transpose(1, 2)[live].to(s["q"].dtype), lse=(top + total.log())[..., 0].transpose(1, 2)[live])


def _own_prompt(s):
    import serving_router_sigmoid_gb300 as moe
    out, lse = moe.latent_prompt(s["q"], s["k"], s["k_rope"], s["v"], s["q_start"], s["kv_start"], s["scale"],
                                 causal=s["c"]["causal"])
    return dict(out=out, lse=lse)


_plain = dict(quant=_plain_quant, linear=_plain_linear, decode=_plain_decode, prompt=_plain_prompt)
_own = dict(quant=_own_quant, linear=_own_linear, decode=_own_decode, prompt=_own_prompt)


# ------------------------------------------------------------------ what a pass needs

def work(case):
    c = case
    if c["op"] == "quant":
        n = c["tokens"] * c["dim"]
        return dict(bytes=n * (SIZE[c["kind"]] + 1) + 4 * c["tokens"] * _pages(c["dim"], BLOCK), flops=3 * n)
    if c["op"] == "linear":
        t, i, o = c["tokens"], c["inner"], c["outer"]
        scales = 4 * _pages(i, BLOCK) * (t + _pages(o, BLOCK))
        return dict(bytes=t * i + o * i + scales + t * o * SIZE[c["kind"]], flops=2 * t * i * o)
    if c["op"] == "decode":
        lens, d = _ragged(c["lens"], c["requests"], c["longest"]), c["latent"] + c["rope"]
        rows = sum(lens)
        return dict(bytes=rows * d * SIZE[c["cache"]] + c["requests"] * c["heads"] * ((d + c["latent"]) * SIZE[c["kind"]] + 4)
                    + 4 * sum(_pages(x, c["page"]) for x in lens), flops=2 * rows * c["heads"] * (d + c["latent"]))
    new, past = _prompts(c)
    keys, queries, h, one = sum(new) + sum(past), sum(new), c["heads"], SIZE[c["kind"]]
    pairs = sum(n * p + (n * (n + 1) // 2 if c["causal"] else n * n) for n, p in zip(new, past))
    return dict(bytes=one * (queries * h * (c["nope"] + c["rope"] + c["v"]) + keys * (h * (c["nope"] + c["v"]) + c["rope"]))
                + 4 * queries * h, flops=2 * pairs * h * (c["nope"] + c["rope"] + c["v"]))


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "quant":
        parts = [p.double() for p in s["x"].split(BLOCK, dim=1)]
        scale = [p.abs().max(dim=1).values.div(448).clamp(min=1e-12) for p in parts]
        return dict(x8=torch.cat([p / m[:, None] for p, m in zip(parts, scale)], 1), scale=torch.stack(scale, 1))
    if c["op"] == "linear":
        got = torch.zeros((c["tokens"], c["outer"]), dtype=torch.float64, device="cuda")
        row = torch.arange(c["outer"], device="cuda") // BLOCK
        for b in range(s["xs"].shape[1]):  # a block of the contraction after another
            at = slice(b * BLOCK, min(c["inner"], (b + 1) * BLOCK))
            got += (s["x8"][:, at].double() @ s["w8"][:, at].double().T) * s["xs"][:, b, None].double() * s["ws"][row, b].double()
        return dict(out=got)
    if c["op"] == "decode":
        out, lse = [], []
        for b, n in enumerate(_ragged(c["lens"], c["requests"], c["longest"])):
            at = torch.arange(n, device="cuda")
            rows, cache = s["table"][b].long()[at // c["page"]] * c["page"] + at % c["page"], s["cache"].flatten(0, 2)
            k = (cache.view(torch.uint8)[rows].view(cache.dtype) if cache.element_size() == 1 else cache[rows]).double()
            k = k * s["k_scale"]
            score = s["q"][b].double() @ k.T * s["scale"]
            lse.append(torch.logsumexp(score, -1))
            out.append(torch.softmax(score, -1) @ k[:, :c["latent"]])
        return dict(out=torch.stack(out), lse=torch.stack(lse))
    out, lse, q0, k0 = [], [], 0, 0
    for nq, past in zip(*_prompts(c)):
        nk = nq + past
        shared = s["k_rope"][k0:k0 + nk].double()
        hidden = torch.ones((nq, nk), dtype=torch.bool, device="cuda").triu(past + 1) if c["causal"] else None
        heads = []
        for h in range(c["heads"]):
            key = torch.cat([s["k"][k0:k0 + nk, h].double(), shared], 1)
            score = s["q"][q0:q0 + nq, h].double() @ key.T * s["scale"]
            if hidden is not None:
                score = score.masked_fill(hidden, -math.inf)
            heads.append((torch.softmax(score, -1) @ s["v"][k0:k0 + nk, h].double(), torch.logsumexp(score, -1)))
        out.append(torch.stack([a for a, _ in heads], 1))
        lse.append(torch.stack([b for _, b in heads], 1))
        q0, k0 = q0 + nq, k0 + nk
    return dict(out=torch.cat(out), lse=torch.cat(lse))
