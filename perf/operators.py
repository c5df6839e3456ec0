"""The cases that measure the cache's positional, scoring, eviction and cross-attention operators.

Each case is one pass of one operator:
  rope     rotary positions with several axes, applied to queries and keys on the way into the cache
  step     decode attention of one new token per sequence that adds its weights to the tokens' scores
  prompt   causal attention of whole prompts or chunks that adds its weights to the tokens' scores
  evict    per-head eviction of the tokens with the lowest scores, the rest moved together
  cross    attention of ragged query chunks over an encoder's cached states of another length
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3_MAX = 448.0


# ---- the cases ------------------------------------------------------------------------------------
def listed():
    return [
        # One decode step's new tokens of a 7B-shape batch: 64 tokens, all heads of their own. Latency.
        dict(name="rope_step", op="rope", dtype="bf16", cache="16", tokens=64, heads=32, kv_heads=32, head_size=128,
             rotary=128, axes=3, interleaved=False, block_size=16),
        # A long video prompt of a 70B-shape model: time, height and width positions. Bandwidth.
        dict(name="rope_prompt", op="rope", dtype="bf16", cache="16", tokens=16384, heads=64, kv_heads=8, head_size=128,
             rotary=128, axes=3, interleaved=False, block_size=8),
        # An odd number of image tokens into an FP8 cache: two axes, pairs side by side, half of each head rotated.
        dict(name="rope_fp8", op="rope", dtype="f16", cache="fp8", tokens=5003, heads=32, kv_heads=8, head_size=128,
             rotary=64, axes=2, interleaved=True, block_size=32),
        # One sequence's next token over a short context: the smallest call of a serving loop.
        dict(name="step_one", op="step", dtype="f16", cache="16", seqs=1, heads=32, kv_heads=8, head_size=128,
             block_size=16, min_len=701, max_len=701),
        # A 7B-shape decode batch (every query head has its own keys), ragged contexts.
        dict(name="step_mha", op="step", dtype="bf16", cache="16", seqs=64, heads=32, kv_heads=32, head_size=128,
             block_size=16, min_len=512, max_len=1996),
        # A 70B-shape decode batch with grouped heads, contexts from short to long.
        dict(name="step_gqa", op="step", dtype="bf16", cache="16", seqs=128, heads=64, kv_heads=8, head_size=128,
             block_size=8, min_len=131, max_len=4092),
        # Whole prompts, every row of which scores the prompt's tokens.
        dict(name="prompt_all", op="prompt", dtype="bf16", cache="16", seqs=8, heads=32, kv_heads=8, head_size=128,
             block_size=16, min_len=300, max_len=2048, chunk=0, window=0),
        # 512-token chunks over longer contexts in an FP8 cache; only the last 64 rows of each chunk score.
        dict(name="prompt_chunk", op="prompt", dtype="bf16", cache="fp8", seqs=16, heads=32, kv_heads=8, head_size=128,
             block_size=16, min_len=1024, max_len=4096, chunk=512, window=64),
        # Long contexts cut to 2048 tokens a head.
        dict(name="evict_long", op="evict", dtype="bf16", cache="16", seqs=16, kv_heads=8, head_size=128, block_size=16,
             min_len=4096, max_len=16384, budget=2048, sink=4, recent=512),
        # A few short ragged sequences, one of them already below the budget; FP8 codes move as they are.
        dict(name="evict_short", op="evict", dtype="f16", cache="fp8", seqs=5, kv_heads=4, head_size=128, block_size=8,
             min_len=97, max_len=901, budget=129, sink=1, recent=31),
        # Text prompts over image states: ragged queries, ragged encoder lengths.
        dict(name="cross_prompt", op="cross", dtype="bf16", cache="16", seqs=16, heads=32, kv_heads=32, head_size=128,
             block_size=16, min_q=33, max_q=512, min_len=577, max_len=1601),
        # One new token per sequence over the encoder's states.
        dict(name="cross_step", op="cross", dtype="bf16", cache="16", seqs=32, heads=32, kv_heads=8, head_size=128,
             block_size=32, min_q=1, max_q=1, min_len=577, max_len=6404),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "step", "prompt", "evict", "cross"])
    cache = rng.choice(["16", "16", "fp8"])
    d = 128 if cache == "fp8" else rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), cache=cache, kv_heads=kv_heads, head_size=d,
             block_size=rng.choice([8, 16, 32, 64]))
    if op != "evict":
        group = rng.choice([g for g in (1, 2, 4, 8) if g * kv_heads <= 64])
        c["heads"] = group * kv_heads
    if op == "rope":
        c["tokens"] = _log(rng, 1, 12000)
        c["rotary"] = rng.choice([d, d, d // 2, 32])
        c["axes"] = rng.choice([1, 2, 3])
        c["interleaved"] = rng.choice([False, True])
        return c
    if op == "prompt":
        c["max_len"] = _log(rng, 3, 2300)
        rows = 2 ** 27 // (c["heads"] * c["max_len"])  # query rows whose scores a plain pass can hold
        c["chunk"] = rng.choice([0, 0, min(c["max_len"], _log(rng, 1, 512))])
        c["seqs"] = max(1, min(_log(rng, 1, 24), rows // (c["chunk"] or c["max_len"])))
        c["window"] = rng.choice([0, 0, _log(rng, 1, 100)])
    elif op == "cross":
        c["max_len"] = _log(rng, 1, 6000)
        c["max_q"] = rng.choice([1, _log(rng, 1, 600)])
        c["seqs"] = max(1, min(_log(rng, 1, 48), 2 ** 28 // (c["heads"] * c["max_len"] * c["max_q"])))
        c["seqs"] = max(1, min(c["seqs"], 2 ** 29 // (kv_heads * d * c["max_len"])))
        c["min_q"] = max(1, c["max_q"] // rng.randint(1, 9))
    else:
        c["max_len"] = _log(rng, 3, 16000)
        c["seqs"] = max(1, min(_log(rng, 1, 120), (2 ** 27 if op == "evict" else 2 ** 28) // (kv_heads * d * c["max_len"])))
    c["min_len"] = max(1, c["max_len"] // rng.randint(1, 12))
    if op == "prompt" and c["chunk"]:
        c["min_len"] = max(c["min_len"], c["chunk"])
    if op == "evict":
        c["budget"] = max(2, c["max_len"] // rng.randint(2, 9))
        c["sink"] = rng.randint(0, min(8, c["budget"] // 2))
        c["recent"] = rng.randint(0, c["budget"] // 2)
    return c


# ---- sizes that a case fixes ----------------------------------------------------------------------
def _spread(lo, hi, n, salt):
    """n lengths from lo to hi, both among them, in an order that only the case fixes."""
    v = [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]
    random.Random(salt).shuffle(v)
    return v


def _lens(case):
    return _spread(case["min_len"], case["max_len"], case["seqs"], 1)


def _q_lens(case):
    if case["op"] == "cross":
        return _spread(case["min_q"], case["max_q"], case["seqs"], 2)
    return [min(n, case["chunk"] or n) for n in _lens(case)]


def work(case):
    d, hk, e = case["head_size"], case["kv_heads"], 2
    ec = 1 if case["cache"] == "fp8" else 2
    if case["op"] == "rope":
        t, h, r = case["tokens"], case["heads"], case["rotary"]
        return {"bytes": t * (2 * h * d * e + 2 * hk * d * (e + ec) + 4 * case["axes"] + 8), "flops": t * (h + hk) * r * 3}
    lens = _lens(case)
    blocks = sum(-(-n // case["block_size"]) for n in lens)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens) * hk
        rows = case["seqs"] * hk
        return {"bytes": 4 * sum(lens) * hk + kept * (4 * d * ec + 4) + rows * 4 * case["max_len"] + 4 * blocks,
                "flops": sum(lens) * hk}
    h = case["heads"]
    q = [1] * len(lens) if case["op"] == "step" else _q_lens(case)
    n_bytes = 2 * sum(q) * h * d * e + 2 * sum(lens) * hk * d * ec + 4 * blocks
    if case["op"] == "cross":
        return {"bytes": n_bytes, "flops": 4 * d * h * sum(a * b for a, b in zip(q, lens))}
    n_bytes += 8 * sum(lens) * hk  # scores read and written
    if case["op"] == "step":
        return {"bytes": n_bytes, "flops": 4 * d * h * sum(lens)}
    pairs = lambda n, l: n * l - n * (n - 1) // 2  # noqa: E731  keys that the last n rows of l see together
    rows = [min(n, case["window"] or n) for n in q]
    return {"bytes": n_bytes, "flops": 4 * d * h * sum(map(pairs, q, lens)) + 2 * d * h * sum(map(pairs, rows, lens))}


# ---- inputs ---------------------------------------------------------------------------------------
def _encode(x, scale):
    """E4M3 codes of x / scale, rounded to nearest even, saturating."""
    return (x.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _pool(case, gen, blocks, st):
    shape = (blocks, case["block_size"], case["kv_heads"], case["head_size"])
    dt = DTYPES[case["dtype"]]
    for name in ("key_cache", "value_cache"):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=dt)
        if case["cache"] == "fp8":
            s = torch.rand(case["kv_heads"], generator=gen, device="cuda") * 0.01 + 0.01
            st["k_scale" if name == "key_cache" else "v_scale"] = s
            x = _encode(x, s[:, None])
        st[name] = x


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(case, gen, lens, first_of=None):
    """A block table over scattered blocks; columns past a sequence's blocks hold block 0."""
    bs = case["block_size"]
    counts = _ints([-(-n // bs) for n in lens])
    width = -(-max(lens) // bs)
    order = torch.randperm(int(sum(-(-n // bs) for n in lens)), generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    start = torch.cumsum(counts, 0) - counts
    table = order[(start[:, None] + col).clamp(max=order.numel() - 1)]
    return torch.where(col < counts[:, None], table, 0).to(torch.int32).contiguous(), order.numel()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case, k_scale=None, v_scale=None, ws=None)
    dt, d = DTYPES[case["dtype"]], case["head_size"]
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    if case["op"] == "rope":
        t, bs, half = case["tokens"], case["block_size"], case["rotary"] // 2
        st["query"] = randn(t, case["heads"], d)
        st["query_out"] = torch.empty_like(st["query"])
        st["key"], st["value"] = randn(t, case["kv_heads"], d), randn(t, case["kv_heads"], d)
        blocks = -(-t // bs) + 2
        _pool(case, gen, blocks, st)
        st["slots"] = torch.randperm(blocks * bs, generator=gen, device="cuda")[:t].contiguous()
        # Far positions on the first axis (a long conversation or video), small grids on the others.
        far = torch.randint(0, 900000, (1,), generator=gen, device="cuda")
        grid = torch.randint(0, 4096, (case["axes"], t), generator=gen, device="cuda")
        grid[0] += far
        st["positions"] = grid.to(torch.int32).contiguous()
        st["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        st["freq_axis"] = (torch.arange(half, device="cuda") * case["axes"] // half).to(torch.int32)
        return st
    lens = _lens(case)
    st["scale"] = 1.0 / math.sqrt(d)
    st["table"], blocks = _tables(case, gen, lens)
    st["lens"] = _ints(lens)
    rows = (case["seqs"], case["kv_heads"], case["max_len"])
    if case["op"] in ("step", "prompt", "evict"):
        # Accumulated weights: a few heavy tokens, many light ones, some that nothing has looked at yet.
        x = torch.rand(rows, generator=gen, device="cuda")
        st["scores"] = torch.where(x < 0.05, torch.zeros_like(x), x.pow(8) * 3)
        st["scores"].masked_fill_(torch.arange(rows[2], device="cuda") >= st["lens"][:, None, None], 0.0)
    if case["op"] == "evict":
        to, more = _tables(case, gen, [min(n, case["budget"]) for n in lens])
        st["dst_table"] = (to + blocks).to(torch.int32).contiguous()
        st["scores_out"] = torch.zeros(rows, device="cuda")
        st["kept"] = torch.zeros((case["seqs"], case["kv_heads"], case["budget"]), dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.zeros(case["seqs"], dtype=torch.int32, device="cuda")
        _pool(case, gen, blocks + more, st)
    else:
        q = [1] * len(lens) if case["op"] == "step" else _q_lens(case)
        st["query"] = randn(sum(q), case["heads"], d)
        st["out"] = torch.empty_like(st["query"])
        st["q_start"] = _ints([sum(q[:i]) for i in range(len(q) + 1)])
        st["max_q"] = max(q)
        _pool(case, gen, blocks, st)
    if own:  # the scratch memory that a serving program allocates once
        from pagedattention_paged_kv_attention_b200 import pagedattn as P
        s, h = case["seqs"], case.get("heads", 0)
        if case["op"] == "step":
            st["ws"] = P.make_accumulate_workspace(s, h, case["kv_heads"], d, case["max_len"])
        elif case["op"] == "prompt":
            st["ws"] = P.make_prefill_accumulate_workspace(st["query"].shape[0], h)
        elif case["op"] == "cross":
            st["ws"] = P.make_cross_workspace(s, st["query"].shape[0], h, case["kv_heads"], d, st["max_q"], case["max_len"])
        else:
            st["ws"] = P.make_evict_workspace()
    return st


# ---- one pass -------------------------------------------------------------------------------------
def _values(case, cache):
    """A cache as the values it stands for: E4M3 codes are returned as such."""
    return cache.view(torch.float8_e4m3fn) if case["cache"] == "fp8" else cache


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        from pagedattention_paged_kv_attention_b200 import pagedattn as P
        fp8 = dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
        if op == "rope":
            P.rope_reshape_and_cache(st["query_out"], st["query"], st["key"], st["value"], st["key_cache"], st["value_cache"],
                                     st["slots"], st["positions"], st["inv_freq"], st["freq_axis"],
                                     interleaved=case["interleaved"], **fp8)
        elif op == "step":
            P.paged_attention_accumulate(st["out"], st["scores"], st["query"], st["key_cache"], st["value_cache"],
                                         st["table"], st["lens"], st["scale"], case["max_len"], st["ws"], **fp8)
        elif op == "prompt":
            P.paged_prefill_accumulate(st["out"], st["scores"], st["query"], st["key_cache"], st["value_cache"],
                                       st["table"], st["lens"], st["q_start"], st["scale"], st["max_q"],
                                       case["max_len"], st["ws"], window=case["window"], **fp8)
        elif op == "evict":
            P.evict_tokens(st["kept"], st["new_lens"], st["scores_out"], st["scores"], st["key_cache"],
                           st["value_cache"], st["table"], st["dst_table"], st["lens"], case["budget"], case["sink"],
                           case["recent"], case["max_len"], st["ws"])
        else:
            P.paged_cross_attention(st["out"], st["query"], st["key_cache"], st["value_cache"], st["table"], st["lens"],
                                    st["q_start"], st["scale"], st["max_q"], case["max_len"], st["ws"], **fp8)
    else:
        {"rope": _rope, "step": _attend, "prompt": _attend, "evict": _evict, "cross": _attend}[op](st)
    if op == "rope":
        return {"query": st["query_out"], "key_cache": _values(case, st["key_cache"]), "value_cache": _values(case, st["value_cache"])}
    if op == "evict":
        return {"kept": st["kept"], "new_lens": st["new_lens"], "scores": st["scores_out"],
                "key_cache": _values(case, st["key_cache"]), "value_cache": _values(case, st["value_cache"])}
    if op == "cross":
        return {"out": st["out"]}
    return {"out": st["out"], "scores": st["scores"]}


# ---- the plain forms ------------------------------------------------------------------------------
def _rotate(st, x):
    case = st["case"]
    r = case["rotary"]
    # Far positions: the angle needs more than 32 bits before its cosine is taken.
    angle = st["positions"].double()[st["freq_axis"].long()].t() * st["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    x = x.float()
    y = x.clone()
    lo = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
    hi = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
    y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
    y[..., hi] = x[..., hi] * cos + x[..., lo] * sin
    return y


def _rope(st):
    case = st["case"]
    st["query_out"].copy_(_rotate(st, st["query"]))
    blk, off = st["slots"] // case["block_size"], st["slots"] % case["block_size"]
    k, v = _rotate(st, st["key"]), st["value"].float()
    if case["cache"] == "fp8":
        st["key_cache"][blk, off] = _encode(k, st["k_scale"][:, None])
        st["value_cache"][blk, off] = _encode(v, st["v_scale"][:, None])
    else:
        st["key_cache"][blk, off] = k.to(st["key_cache"].dtype)
        st["value_cache"][blk, off] = v.to(st["value_cache"].dtype)


def _gathered(st, which):
    """[S][kv head][max_len][d] in 32 bits, through the block table."""
    case = st["case"]
    t = torch.arange(case["max_len"], device="cuda")
    blk = st["table"].long()[:, t // case["block_size"]]
    x = _values(case, st[which + "_cache"]).permute(2, 0, 1, 3)[:, blk, t % case["block_size"]].float()
    if case["cache"] == "fp8":
        x = x * st["k_scale" if which == "key" else "v_scale"][:, None, None, None]
    return x.transpose(0, 1)


def _attend(st):
    case = st["case"]
    s, hk, d = case["seqs"], case["kv_heads"], case["head_size"]
    g = case["heads"] // hk
    # The packed rows, a sequence's rows side by side: row j of sequence s at [s][j].
    j = torch.arange(st["max_q"], device="cuda")
    first, n = st["q_start"][:-1].long(), (st["q_start"][1:] - st["q_start"][:-1]).long()
    real = j < n[:, None]
    q = st["query"].float()[torch.where(real, first[:, None] + j, 0)]
    q = q.view(s, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(s, hk, -1, d)
    k = _gathered(st, "key")
    z = (q @ k.transpose(2, 3) * st["scale"]).view(s, hk, g, -1, case["max_len"])
    del k
    t = torch.arange(case["max_len"], device="cuda")
    if case["op"] == "prompt":
        last = st["lens"].long()[:, None] - n[:, None] + j
    else:
        last = (st["lens"].long()[:, None] - 1).expand(s, st["max_q"])
    z.masked_fill_((t > last[:, :, None])[:, None, None], float("-inf"))
    z -= z.amax(-1, keepdim=True)
    z.exp_()
    z /= z.sum(-1, keepdim=True)
    o = (z.view(s, hk, -1, case["max_len"]) @ _gathered(st, "value")).view(s, hk, g, -1, d)
    o = o.permute(0, 3, 1, 2, 4).reshape(s, -1, hk * g, d)
    at = torch.arange(st["query"].shape[0], device="cuda")
    seq = (at[:, None] >= st["q_start"][1:]).sum(1)
    st["out"].copy_(o[seq, at - first[seq]])
    if case["op"] != "cross":
        counted = real & (j >= n[:, None] - case.get("window", 0)) if case.get("window", 0) else real
        z *= counted[:, None, None, :, None]
        st["scores"] += z.sum((2, 3))


def _evict(st):
    case = st["case"]
    bs, budget, n = case["block_size"], case["budget"], st["lens"].long()[:, None, None]
    t = torch.arange(case["max_len"], device="cuda")
    rank = st["scores"].masked_fill((t < case["sink"]) | ((t >= n - case["recent"]) & (t < n)), float("inf"))
    rank = rank.masked_fill(t >= n, float("-inf"))
    best = rank.sort(dim=-1, descending=True, stable=True)[1][..., :budget]
    new = n.clamp(max=budget)
    place = torch.arange(budget, device="cuda")
    best = torch.where(place < new, best, case["max_len"]).sort(-1)[0]
    real = (place < new).expand_as(best)
    st["kept"].copy_(torch.where(real, best, -1))
    st["new_lens"].copy_(new[:, 0, 0])
    best = torch.where(real, best, 0)
    st["scores_out"].zero_()
    st["scores_out"][..., :budget] = st["scores"].gather(2, best) * real
    head = torch.arange(case["kv_heads"], device="cuda")[None, :, None]
    seq = torch.arange(case["seqs"], device="cuda")[:, None, None]
    src_blk, src_off = st["table"].long()[seq, best // bs], best % bs
    dst_blk = st["dst_table"].long()[seq, (place // bs)[None, None]].expand_as(best)
    dst_off, head = (place % bs).expand_as(best), head.expand_as(best)
    for cache in (st["key_cache"], st["value_cache"]):
        cache[dst_blk[real], dst_off[real], head[real]] = cache[src_blk[real], src_off[real], head[real]]


# ---- the definitions in 64 bits -------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "evict": _exact_evict}.get(case["op"], _exact_attention)(case, st)


def _exact_rope(case, st):
    r, t = case["rotary"], case["tokens"]
    turn = torch.empty(t, r // 2, dtype=torch.complex128, device="cuda")
    for i in range(r // 2):
        a = st["positions"][int(st["freq_axis"][i])].double() * float(st["inv_freq"][i])
        turn[:, i] = torch.complex(a.cos(), a.sin())

    def rotated(x):
        x = x.double()
        pair = x[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
        y = y.flatten(-2) if case["interleaved"] else y.transpose(-1, -2).flatten(-2)
        return torch.cat([y, x[..., r:]], -1)

    out = {"query": rotated(st["query"])}
    for name, x in (("key", rotated(st["key"])), ("value", st["value"].double())):
        pool = _values(case, st[name + "_cache"]).double().flatten(0, 1)
        if case["cache"] == "fp8":
            # The code's value: the nearest E4M3 number (8 steps an octave, the least octave from 2^-6).
            x = (x / st["k_scale" if name == "key" else "v_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(x / step) * step
        pool[st["slots"]] = x
        out[name + "_cache"] = pool.view(st[name + "_cache"].shape)
    return out


def _exact_attention(case, st):
    hk, bs, d = case["kv_heads"], case["block_size"], case["head_size"]
    g, lens, start = case["heads"] // hk, st["lens"].tolist(), st["q_start"].tolist()
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device="cuda")
    scores = st["scores"].double() if case["op"] != "cross" else None
    for s, length in enumerate(lens):
        rows, n = slice(start[s], start[s + 1]), start[s + 1] - start[s]
        blocks = st["table"][s, : -(-length // bs)].long()
        k, v = (_values(case, st[w])[blocks].double().flatten(0, 1)[:length] for w in ("key_cache", "value_cache"))
        keys = torch.arange(length, device="cuda")
        seen = torch.ones(n, length, dtype=torch.bool, device="cuda")
        if case["op"] == "prompt":
            seen = keys <= torch.arange(length - n, length, device="cuda")[:, None]
        for h in range(hk):
            ks, vs = (1.0, 1.0) if case["cache"] != "fp8" else (st["k_scale"][h].double(), st["v_scale"][h].double())
            for a in range(h * g, h * g + g):
                z = st["query"][rows, a].double() @ k[:, h].t() * (ks * st["scale"])
                p = torch.softmax(torch.where(seen, z, -math.inf), -1)
                out[rows, a] = p @ v[:, h] * vs
                if scores is not None:
                    scores[s, h, :length] += p[-(case.get("window", 0) or n):].sum(0)
    return {"out": out} if scores is None else {"out": out, "scores": scores}


def _exact_evict(case, st):
    # Moves and comparisons only: the values are those of the inputs.
    bs, lens = case["block_size"], st["lens"].tolist()
    scores, table, to = st["scores"].cpu(), st["table"].cpu(), st["dst_table"].cpu()
    moved = torch.zeros_like(scores, dtype=torch.float64)
    kept = torch.full(st["kept"].shape, -1, dtype=torch.int64)
    pools = [_values(case, st[w]).double() for w in ("key_cache", "value_cache")]
    for s, length in enumerate(lens):
        new = min(length, case["budget"])
        for h in range(case["kv_heads"]):
            guarded = set(range(min(case["sink"], length))) | set(range(max(0, length - case["recent"]), length))
            row = scores[s, h, :length].tolist()
            order = sorted(range(length), key=lambda t: (t not in guarded, -row[t], t))
            keep = torch.tensor(sorted(order[:new]))
            kept[s, h, :new] = keep
            moved[s, h, :new] = scores[s, h][keep].double()
            place = torch.arange(new)
            for pool in pools:
                pool[to[s, place // bs].long(), place % bs, h] = pool[table[s, keep // bs].long(), keep % bs, h]
    return {"kept": kept, "new_lens": torch.tensor([min(n, case["budget"]) for n in lens]), "scores": moved,
            "key_cache": pools[0], "value_cache": pools[1]}
