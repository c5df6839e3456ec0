"""Eviction by accumulated attention weight: the attention calls that add their weights to the tokens'
scores (bounds of operator_refs, outputs equal to the plain calls bit for bit), the eviction itself
(exact), and a run of them as a serving loop makes it."""
import pytest
import torch

from operator_refs import (DTYPES, U, attention, evict, gather, half_step, make_pool, poison_unused, rotate,
                           scatter_tables)

pytestmark = pytest.mark.gpu
SENTINEL = -12345.0


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


def make(lens, chunks, H, Hkv, d, bs, dtype="bf16", cache="16", seed=0, tail=0, junk=None, stride=None):
    """chunks None: one new token per sequence (decode)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(lens=list(lens), bs=bs, info=(DTYPES[dtype], cache), scale=d ** -0.5)
    st["chunks"] = list(chunks) if chunks is not None else [1] * len(lens)
    st["table"], nb = scatter_tables(gen, lens, bs, junk=junk)
    st["kc"], st["vc"], st["ks"], st["vs"], st["k64"], st["v64"] = make_pool(gen, nb, bs, Hkv, d, DTYPES[dtype], cache)
    poison_unused((st["kc"], st["vc"]), st["table"], lens, bs)
    T = sum(st["chunks"]) + tail
    st["q"] = torch.randn(T, H, d, generator=gen, device="cuda").to(DTYPES[dtype])
    if tail:
        st["q"][-tail:] = float("nan")
    st["q_start"] = torch.tensor([sum(st["chunks"][:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    st["cl"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["max_len"] = max(lens)
    st["scores"] = torch.rand(len(lens), Hkv, stride or max(1, max(lens)), generator=gen, device="cuda")
    for s, n in enumerate(lens):
        st["scores"][s, :, n:] = SENTINEL
    return st


def step(P, st, out, ws=None, part=0, scores=None):
    S, H, d = st["q"].shape
    Hkv = st["kc"].shape[2]
    if ws is None:
        ws = P.make_accumulate_workspace(S, H, Hkv, d, st["max_len"], part)
    P.paged_attention_accumulate(out, st["scores"] if scores is None else scores, st["q"], st["kc"], st["vc"],
                                 st["table"], st["cl"], st["scale"], st["max_len"], ws, k_scale=st["ks"],
                                 v_scale=st["vs"], partition_size=part)
    return ws


def prompt(P, st, out, window=0, ws=None):
    T, H, d = st["q"].shape
    if ws is None:
        ws = P.make_prefill_accumulate_workspace(T, H)
    P.paged_prefill_accumulate(out, st["scores"], st["q"], st["kc"], st["vc"], st["table"], st["cl"], st["q_start"],
                               st["scale"], max(st["chunks"]), st["max_len"], ws, window=window, k_scale=st["ks"],
                               v_scale=st["vs"])
    return ws


def check(st, before, out, window=0, seqs=None):
    for s, (L, n) in enumerate(zip(st["lens"], st["chunks"])):
        if seqs is not None and s not in seqs:
            continue
        got = st["scores"][s].double()
        assert torch.equal(st["scores"][s, :, L:], before[s, :, L:])
        if n == 0 or L == 0:
            assert torch.equal(st["scores"][s], before[s])
            assert out is None or bool((out[int(st["q_start"][s]):int(st["q_start"][s]) + n] == 0).all())
            continue
        rows = slice(int(st["q_start"][s]), int(st["q_start"][s]) + n)
        k, v = gather(st["k64"], st["table"], s, L, st["bs"]), gather(st["v64"], st["table"], s, L, st["bs"])
        counted = min(window or n, n)
        ref, bound, add, rel = attention(st["q"][rows], k, v, rows, st["scale"], True, counted, st["info"])
        if out is not None:
            o = out[rows].double()
            assert bool((o - ref).abs().le(bound).all()), (s, float(((o - ref).abs() - bound).max()))
        was = before[s, :, :L].double()
        err = (got[:, :L] - was - add).abs()
        # weights below 2^-126 flush to zero
        ok = err <= rel * add + 2 * U * (was.abs() + add) + counted * st["q"].shape[1] * 2.0 ** -126
        assert bool(ok.all()), (s, float((err / (rel * add + 2 * U * (was.abs() + add))).max()))


STEP = [
    # lens, H, Hkv, d, bs, partition, options
    ([1], 1, 1, 64, 8, 0, {}),
    ([1, 0, 7, 8, 9, 63, 64, 65], 8, 8, 128, 16, 0, {}),
    ([127, 128, 129, 1000, 3], 8, 2, 128, 16, 64, {}),
    ([700, 31], 32, 4, 128, 8, 128, dict(dtype="f16", stride=811)),
    ([513, 1, 2500], 16, 1, 64, 32, 0, dict(dtype="f16")),
    ([300, 290], 12, 4, 64, 64, 64, {}),                             # 3 heads a group
    ([400, 65], 10, 10, 64, 16, 64, {}),
    ([260, 1025], 72, 1, 128, 16, 192, dict(stride=1100)),           # 72 heads: more than one batch of statistics
    ([900, 33, 0, 17], 8, 8, 128, 16, 0, dict(cache="fp8")),
    ([901, 1700, 8], 16, 2, 128, 32, 320, dict(cache="fp8", dtype="f16")),
    ([640, 111], 8, 4, 128, 8, 64, dict(cache="fp8_block")),
    ([640, 111], 4, 4, 128, 16, 64, dict(cache="fp8_block", dtype="f16")),
    ([3000, 10, 0], 24, 8, 128, 16, 0, dict(junk=-7)),
]


@pytest.mark.parametrize("case", STEP, ids=lambda c: "L%s_H%d_%d_d%d_bs%d_p%d_%s" % (
    "-".join(map(str, c[0])), *c[1:6], "-".join(map(str, c[6].values()))))
def test_step_against_the_formula(P, case):
    lens, H, Hkv, d, bs, part, opt = case
    st = make(lens, None, H, Hkv, d, bs, seed=sum(lens) + H, **opt)
    before = st["scores"].clone()
    out, plain = torch.full_like(st["q"], float("nan")), torch.empty_like(st["q"])
    ws = step(P, st, out, part=part)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    if part:  # left open, the two calls may choose different partitions
        ws2 = P.make_workspace(*st["q"].shape[:2], Hkv, d, st["max_len"], part)
        P.paged_attention(plain, st["q"], st["kc"], st["vc"], st["table"], st["cl"], st["scale"], st["max_len"], ws2,
                          k_scale=st["ks"], v_scale=st["vs"], partition_size=part)
        assert torch.equal(out.view(torch.int16), plain.view(torch.int16))
    check(st, before, out)
    again = before.clone()
    step(P, st, out, ws=ws, part=part, scores=again)
    assert torch.equal(again, st["scores"])


def test_step_weights_of_extreme_scores(P):
    """One key far above the rest takes the whole weight; equal keys share it."""
    st = make([200, 200], None, 4, 2, 64, 16, seed=1)
    st["k64"][:] = 0
    st["k64"][st["table"][0, 3], 5] = 60 * st["q"][0, ::2].double()
    st["kc"].copy_(st["k64"])
    st["vc"].nan_to_num_()
    st["k64"] = st["kc"].double()
    before = st["scores"].clone()
    out = torch.empty_like(st["q"])
    step(P, st, out, part=64)
    check(st, before, None)
    add = (st["scores"] - before)[1, :, :200]
    assert bool((add - 2 / 200).abs().max() < 1e-6)


PROMPT = [
    # lens, chunks, H, Hkv, d, bs, window, options
    ([1], [1], 1, 1, 64, 8, 0, {}),
    ([5, 129, 64], [5, 129, 64], 8, 2, 128, 16, 0, {}),
    ([128, 127, 300], [128, 1, 0], 4, 4, 64, 32, 0, dict(dtype="f16")),
    ([700, 1300], [333, 513], 8, 8, 128, 8, 0, {}),
    ([600, 300], [257, 300], 16, 1, 128, 16, 0, dict(dtype="f16", stride=640)),
    ([1025, 40], [700, 40], 8, 2, 128, 16, 31, {}),
    ([1025, 40], [700, 40], 32, 2, 64, 64, 1, {}),
    ([500, 513], [500, 130], 8, 8, 128, 16, 200, dict(dtype="f16")),
    ([900, 33], [70, 33], 8, 8, 128, 16, 0, dict(cache="fp8")),
    ([640, 1111], [640, 100], 8, 4, 128, 8, 64, dict(cache="fp8_block")),
    ([300, 555], [300, 1], 8, 2, 128, 128, 0, dict(cache="fp8", dtype="f16", junk=-9)),
    ([260, 130], [260, 100], 128, 1, 64, 128, 0, dict(dtype="f16")),
    ([390], [390], 8, 1, 128, 16, 5, dict(cache="fp8_block", dtype="f16")),
]


@pytest.mark.parametrize("case", PROMPT, ids=lambda c: "L%s_n%s_H%d_%d_d%d_bs%d_w%d_%s" % (
    "-".join(map(str, c[0])), "-".join(map(str, c[1])), *c[2:7], "-".join(map(str, c[7].values()))))
def test_prompt_against_the_formula(P, case):
    lens, chunks, H, Hkv, d, bs, window, opt = case
    st = make(lens, chunks, H, Hkv, d, bs, seed=sum(lens) + H, **opt)
    before = st["scores"].clone()
    out, plain = torch.full_like(st["q"], float("nan")), torch.empty_like(st["q"])
    ws = prompt(P, st, out, window)
    P.paged_prefill(plain, st["q"], st["kc"], st["vc"], st["table"], st["cl"], st["q_start"], st["scale"],
                    max(chunks), torch.zeros(64, dtype=torch.int32, device="cuda"), k_scale=st["ks"], v_scale=st["vs"])
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    assert torch.equal(out.view(torch.int16), plain.view(torch.int16))
    check(st, before, out, window)
    first = st["scores"].clone()
    st["scores"].copy_(before)
    prompt(P, st, out, window, ws=ws)
    assert torch.equal(first, st["scores"])


def test_rows_behind_the_last_sequence_stay(P):
    st = make([200, 90], [64, 90], 8, 2, 128, 16, tail=5, seed=4)
    before = st["scores"].clone()
    out = torch.full_like(st["q"], 7.0)
    prompt(P, st, out)
    check(st, before, out)
    assert bool((out[-5:] == 7).all())


def test_invalid_lengths_leave_the_scores(P):
    st = make([200, 90, 300], [64, 90, 10], 8, 2, 128, 16, seed=5)
    before = st["scores"].clone()
    st["cl"][0] = 63                               # shorter than its chunk
    st["cl"][1] = 5000                             # past its table
    out = torch.zeros_like(st["q"])
    ws = prompt(P, st, out)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_CONTEXT_LEN
    assert torch.equal(st["scores"][:2], before[:2])
    check(st, before, out, seqs={2})
    st = make([200, 90, 300], None, 8, 2, 128, 16, seed=5)
    before = st["scores"].clone()
    st["cl"][0], st["cl"][1] = -1, 5000
    ws = step(P, st, torch.zeros_like(st["q"]))
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_CONTEXT_LEN
    assert torch.equal(st["scores"][:2], before[:2])
    check(st, before, None, seqs={2})


def test_empty_contexts_and_chunks(P):
    """A padded decode batch whose sequences are all empty, and a prompt call without any new token."""
    st = make([0, 0], None, 8, 2, 128, 16, seed=1)
    before = st["scores"].clone()
    out = torch.full_like(st["q"], 7.0)
    ws = step(P, st, out)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0 and bool((out == 0).all()) and torch.equal(st["scores"], before)
    st = make([90, 40], [0, 0], 8, 2, 128, 16, tail=3, seed=2)
    before = st["scores"].clone()
    out = torch.full_like(st["q"], 7.0)
    st["chunks"] = [1]                               # max_q_len 1
    ws = prompt(P, st, out)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0 and bool((out == 7).all()) and torch.equal(st["scores"], before)


def test_a_chunk_longer_than_announced_leaves_the_scores(P):
    st = make([300, 90], [300, 40], 8, 8, 128, 16, seed=7)
    before = st["scores"].clone()
    out = torch.zeros_like(st["q"])
    ws = P.make_prefill_accumulate_workspace(340, 8)
    P.paged_prefill_accumulate(out, st["scores"], st["q"], st["kc"], st["vc"], st["table"], st["cl"], st["q_start"],
                               st["scale"], 40, 300, ws)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_CONTEXT_LEN
    assert torch.equal(st["scores"][0], before[0])
    check(st, before, out, seqs={1})


def test_blocks_outside_the_pool_make_the_scores_nan(P):
    st = make([200, 90], [200, 90], 8, 2, 128, 16, seed=6)
    before = st["scores"].clone()
    st["table"][0, 12] = st["kc"].shape[0]          # tokens 192..199
    ws = prompt(P, st, torch.zeros_like(st["q"]))
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_BLOCK_ID
    assert bool(st["scores"][0, :, :200].isnan().all())
    check(st, before, None, seqs={1})
    st = make([200, 90], None, 8, 2, 128, 16, seed=6)
    before = st["scores"].clone()
    st["table"][0, 12] = -1
    ws = step(P, st, torch.zeros_like(st["q"]), part=64)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_BLOCK_ID
    assert bool(st["scores"][0, :, :200].isnan().all())
    check(st, before, None, seqs={1})


# ---- eviction ---------------------------------------------------------------------------------------
def evict_call(P, st, budget, sink, recent, dst, scores_out=None, ws=None):
    S, Hkv = len(st["lens"]), st["kc"].shape[2]
    kept = torch.full((S, Hkv, budget), -99, dtype=torch.int32, device="cuda")
    new = torch.full((S,), -99, dtype=torch.int32, device="cuda")
    so = torch.full_like(st["scores"], SENTINEL) if scores_out is None else scores_out
    ws = P.make_evict_workspace() if ws is None else ws
    P.evict_tokens(kept, new, so, st["scores"], st["kc"], st["vc"], st["table"], dst, st["cl"], budget, sink, recent,
                   st["max_len"], ws)
    return kept, new, so, ws


def rows_of(cache, table, s, idx, bs):
    return cache[table[s].long()[idx // bs], idx % bs]


def check_evict(st, before, dst, budget, sink, recent, kept, new, so, seqs=None):
    scores0, kc0, vc0 = before
    bs, Hkv = st["bs"], kc0.shape[2]
    want_k, want_v = kc0.clone(), vc0.clone()
    for s, L in enumerate(st["lens"]):
        if seqs is not None and s not in seqs:
            continue
        n = min(L, budget)
        assert int(new[s]) == n
        for h in range(Hkv):
            ids = evict(scores0[s, h], L, budget, sink, recent)
            assert kept[s, h].tolist() == ids + [-1] * (budget - n), (s, h)
            idx = torch.tensor(ids, device="cuda", dtype=torch.long)
            exp = torch.zeros_like(so[s, h])
            exp[:n] = scores0[s, h][idx]
            assert torch.equal(so[s, h].view(torch.int32), exp.view(torch.int32))
            j = torch.arange(n, device="cuda")
            for want, was in ((want_k, kc0), (want_v, vc0)):
                want[dst[s].long()[j // bs], j % bs, h] = rows_of(was, st["table"], s, idx, bs)[torch.arange(n), h]
    for got, want in ((st["kc"], want_k), (st["vc"], want_v)):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


def fresh_destinations(st, gen, lens, budget):
    """Blocks that no sequence reads, appended to the pool."""
    S, bs = len(lens), st["bs"]
    width = max(1, -(-min(budget, max(lens)) // bs))
    nb = st["kc"].shape[0]
    dst = nb + torch.randperm(S * width, generator=gen, device="cuda").view(S, width)
    for name in ("kc", "vc"):
        more = torch.zeros((S * width, *st[name].shape[1:]), dtype=st[name].dtype, device="cuda")
        st[name] = torch.cat([st[name], more])
    return dst.to(torch.int32).contiguous()


EVICT = [
    # lens, Hkv, d, bs, budget, sink, recent, options
    ([1], 1, 64, 8, 1, 0, 0, {}),
    ([2, 0, 9, 8, 7], 2, 64, 8, 8, 1, 2, {}),
    ([100, 33, 64, 65], 4, 128, 16, 64, 4, 16, {}),
    ([700, 31, 32], 3, 128, 32, 32, 0, 32, dict(dtype="f16")),       # only the recent ones
    ([700, 129], 2, 128, 16, 7, 7, 0, {}),                           # only the first ones
    ([1500, 4000, 77], 2, 128, 16, 1000, 3, 200, dict(cache="fp8")),
    ([2049, 1025], 1, 64, 64, 1024, 0, 0, dict(stride=3001)),
    ([5000], 2, 8, 4, 2500, 1, 1, {}),                               # rows of 16 bytes
    ([260, 300], 2, 24, 16, 130, 2, 9, {}),                          # rows of 48 bytes: a ragged strip
    ([120, 20], 2, 512, 16, 33, 0, 4, dict(junk=-5)),                # rows of 1024 bytes
]


@pytest.mark.parametrize("place", ["apart", "in_place", "own_table"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "L%s_H%d_d%d_bs%d_b%d_s%d_r%d_%s" % (
    "-".join(map(str, c[0])), *c[1:7], "-".join(map(str, c[7].values()))))
def test_evict_is_exact(P, case, place):
    lens, Hkv, d, bs, budget, sink, recent, opt = case
    st = make(lens, None, Hkv, Hkv, d, bs, seed=sum(lens), **opt)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = st["scores"]
    x.copy_(torch.where(x > 0.5, x, (x * 16).floor() / 8))           # many equal scores, zeros among them
    if place == "apart":
        dst = fresh_destinations(st, gen, lens, budget)
    else:
        dst = st["table"] if place == "in_place" else st["table"].clone()
    before = st["scores"].clone(), st["kc"].clone(), st["vc"].clone()
    out = st["scores"] if place == "in_place" else None
    kept, new, so, ws = evict_call(P, st, budget, sink, recent, dst, scores_out=out)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    check_evict(st, before, dst, budget, sink, recent, kept, new, so)


def test_evict_scores_out_of_the_ordinary(P):
    """Infinities, NaN, both zeros, subnormals and negative scores keep their order; NaN ranks with -inf."""
    st = make([64, 64, 64], None, 1, 1, 64, 8, seed=3)
    inf, nan = float("inf"), float("nan")
    odd = [0.0, -0.0, inf, -inf, nan, 1e-42, -1e-42, 3.0, -3.0, 1e38, -1e38, nan, -0.0, 0.0, inf, 5.0]
    st["scores"][:] = torch.tensor(odd * 4, device="cuda")
    st["scores"][1] = nan
    st["scores"][2, 0] = 1.0
    for budget in (1, 2, 5, 9, 17, 30, 45, 52, 63):
        st2 = dict(st, kc=st["kc"].clone(), vc=st["vc"].clone())
        before = st["scores"].clone(), st["kc"].clone(), st["vc"].clone()
        kept, new, so, _ = evict_call(P, st2, budget, 0, 0, st["table"])
        check_evict(st2, before, st["table"], budget, 0, 0, kept, new, so)


def test_evict_flags_bad_lengths_and_blocks(P):
    st = make([50, 60, 70, 80], None, 2, 2, 64, 8, seed=8)
    st["cl"][0] = -1
    st["cl"][1] = 8 * st["table"].shape[1] + 1
    st["cl"][2] = 81                               # past max_context_len
    before = st["scores"].clone(), st["kc"].clone(), st["vc"].clone()
    kept, new, so, ws = evict_call(P, st, 20, 1, 3, st["table"])
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_CONTEXT_LEN
    assert new[:3].tolist() == [0, 0, 0] and bool((kept[:3] == -1).all())
    assert bool((so[:3] == SENTINEL).all())
    check_evict(st, before, st["table"], 20, 1, 3, kept, new, so, seqs={3})
    st = make([50, 60], None, 2, 2, 64, 8, seed=9)
    st["table"][0, 0] = st["kc"].shape[0]
    before = st["scores"].clone(), st["kc"].clone(), st["vc"].clone()
    kept, new, so, ws = evict_call(P, st, 20, 0, 0, st["table"].clone())
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_BLOCK_ID
    assert new.tolist() == [20, 20]


def test_evict_twice_changes_nothing_more(P):
    st = make([900, 64], None, 2, 2, 128, 16, seed=10)
    kept, new, so, ws = evict_call(P, st, 100, 4, 20, st["table"], scores_out=st["scores"])
    st["cl"].copy_(new)
    was = st["kc"].clone(), st["vc"].clone(), st["scores"].clone()
    kept, new2, so, ws = evict_call(P, st, 100, 4, 20, st["table"], scores_out=st["scores"], ws=ws)
    assert new2.tolist() == [100, 64]
    assert kept[0, 0].tolist() == list(range(100))
    for a, b in zip((st["kc"], st["vc"], st["scores"]), was):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---- together ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(P, graph):
    """A prompt with time, height and width positions is cached, scored and cut; then every new token is
    cached and scored, and the cache is cut again whenever it has grown past its budget. The reference keeps
    each head's tokens as lists in 64 bits; which tokens stay is checked against the definition on the
    kernels' own scores, whose values are checked on their own."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    S, H, Hkv, d, bs, budget, sink, recent, steps = 3, 8, 2, 128, 16, 96, 4, 24, 9
    dt, scale, room = torch.bfloat16, 128 ** -0.5, 4
    lens = [150, 70, 301]
    width = -(-(max(lens) + steps) // bs)
    NB = S * width
    table = torch.randperm(NB, generator=gen, device="cuda").view(S, width).to(torch.int32)
    kc, vc = (torch.zeros(NB, bs, Hkv, d, dtype=dt, device="cuda") for _ in range(2))
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)).float()
    axis = (torch.arange(64, device="cuda") * 3 // 64).to(torch.int32)
    scores = torch.zeros(S, Hkv, max(lens) + steps, device="cuda")
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q_start = torch.tensor([0, 150, 220, 521], dtype=torch.int32, device="cuda")
    T = sum(lens)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731

    def slots_of(s, t):
        return table[s].long()[t // bs] * bs + t % bs

    # prompt
    q, k, v = randn(T, H, d), randn(T, Hkv, d), randn(T, Hkv, d)
    pos = torch.randint(0, 50, (3, T), generator=gen, device="cuda").to(torch.int32)
    slots = torch.cat([slots_of(s, torch.arange(n, device="cuda")) for s, n in enumerate(lens)])
    qr, out = torch.empty_like(q), torch.empty_like(q)
    P.rope_reshape_and_cache(qr, q, k, v, kc, vc, slots, pos, inv, axis)
    pws = P.make_prefill_accumulate_workspace(T, H)
    P.paged_prefill_accumulate(out, scores, qr, kc, vc, table, cl, q_start, scale, max(lens), max(lens), pws, window=32)
    info = (dt, "16")

    def turned(x, p, got):  # got, the kernel's rotation of x, is the formula's to its rounding
        ref, size = rotate(x, p, inv, axis, False)
        assert bool((got.double() - ref).abs().le(half_step(dt) * ref.abs() + 2.0 ** -20 * size + 2.0 ** -25).all())
        return got.double()

    turned(q, pos, qr)
    keys, values = [], []
    for s, n in enumerate(lens):
        rows = slice(int(q_start[s]), int(q_start[s]) + n)
        keys.append(turned(k[rows], pos[:, rows], gather(kc, table, s, n, bs)))
        values.append(v[rows].double())
        ref, bound, add, rel = attention(qr[rows], keys[s], values[s], rows, scale, True, 32, info)
        assert bool((out[rows].double() - ref).abs().le(bound).all())
        assert bool((scores[s, :, :n].double() - add).abs().le(rel * add + 2 * U * add).all())
    cap = max(lens) + steps
    kept = torch.zeros(S, Hkv, budget, dtype=torch.int32, device="cuda")
    new = torch.zeros(S, dtype=torch.int32, device="cuda")
    ews = P.make_evict_workspace()

    def cut():
        P.evict_tokens(kept, new, scores, scores, kc, vc, table, table, cl, budget, sink, recent, cap, ews)
        cl.copy_(new)

    def cut_reference(was_scores, was_lens):
        for s in range(S):
            per = []
            for h in range(Hkv):
                ids = evict(was_scores[s, h], was_lens[s], budget, sink, recent)
                assert kept[s, h, :len(ids)].tolist() == ids
                per.append(torch.tensor(ids, device="cuda"))
            keys[s] = torch.stack([keys[s][per[h], h] for h in range(Hkv)], 1)
            values[s] = torch.stack([values[s][per[h], h] for h in range(Hkv)], 1)

    was, was_lens = scores.clone(), cl.tolist()
    cut()
    cut_reference(was, was_lens)
    assert cl.tolist() == [min(n, budget) for n in lens]

    # steps
    q, k, v = randn(S, H, d), randn(S, Hkv, d), randn(S, Hkv, d)
    pos = torch.zeros(3, S, dtype=torch.int32, device="cuda")
    slot = torch.zeros(S, dtype=torch.int64, device="cuda")
    qr, out = torch.empty_like(q), torch.empty_like(q)
    ws = P.make_accumulate_workspace(S, H, Hkv, d, budget + room)

    def one():
        P.rope_reshape_and_cache(qr, q, k, v, kc, vc, slot, pos, inv, axis)
        P.paged_attention_accumulate(out, scores, qr, kc, vc, table, cl, scale, budget + room, ws)

    g = None
    for i in range(steps):
        q.copy_(randn(S, H, d)), k.copy_(randn(S, Hkv, d)), v.copy_(randn(S, Hkv, d))
        pos.fill_(400 + i)
        at = cl.clone()
        slot.copy_(torch.stack([slots_of(s, at[s].long()) for s in range(S)]))
        cl.add_(1)
        before = scores.clone()
        if graph and i == 1:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                one()
        if g is not None:
            g.replay()
        else:
            one()
        for s in range(S):
            nk = turned(k[s:s + 1], pos[:, s:s + 1], gather(kc, table, s, int(cl[s]), bs)[-1:])
            keys[s] = torch.cat([keys[s], nk])
            values[s] = torch.cat([values[s], v[s:s + 1].double()])
            n = keys[s].shape[0]
            assert n == int(cl[s])
            ref, bound, add, rel = attention(qr[s:s + 1], keys[s], values[s], None, scale, True, 1, info)
            assert bool((out[s:s + 1].double() - ref).abs().le(bound).all())
            err = (scores[s, :, :n] - before[s, :, :n]).double() - add
            assert bool(err.abs().le(rel * add + 2 * U * (before[s, :, :n].double() + add)).all())
        if int(cl.max()) >= budget + room:
            was, was_lens = scores.clone(), cl.tolist()
            cut()
            cut_reference(was, was_lens)
    assert P.get_device_error(ws) == 0 and P.get_device_error(pws) == 0 and P.get_device_error(ews) == 0


def test_prefill_step_evict_with_the_block_manager(P):
    """Sequences that share a prompt's blocks are cut by the manager's plan: shared blocks are replaced, the prompt's
    owner keeps its tokens, freed blocks come back, and decoding goes on over what was kept."""
    from pagedattention_paged_kv_attention_b200.block_manager import BlockManager
    gen = torch.Generator(device="cuda").manual_seed(33)
    H, Hkv, d, bs, NB, budget, dt = 4, 2, 64, 8, 64, 20, torch.float16
    bm = BlockManager(NB, bs)
    kc, vc = (torch.full((NB, bs, Hkv, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    slots = torch.from_numpy(bm.add_sequence(0, 50).copy()).cuda()
    k, v = randn(50, Hkv, d), randn(50, Hkv, d)
    P.reshape_and_cache(k, v, kc, vc, slots)
    bm.fork(0, 1)
    s2 = torch.from_numpy(bm.add_sequence(2, 30, 0, 24).copy()).cuda()  # shares 3 blocks
    k2, v2 = randn(30, Hkv, d), randn(30, Hkv, d)
    k2[:24], v2[:24] = k[:24], v[:24]
    P.reshape_and_cache(k2[24:].contiguous(), v2[24:].contiguous(), kc, vc, s2)
    logical = {0: (k, v), 1: (k, v), 2: (k2, v2)}
    free = bm.num_free_blocks()[0]
    tables, dst, lens = bm.plan_evict([1, 2], budget, 8, 3)
    assert lens.tolist() == [50, 30]
    assert bm.sequence_info(1) == (20, 3, False) and bm.sequence_info(2) == (20, 3, False)
    # 6 shared blocks are replaced; sequence 0 owns all its blocks alone now; one block of sequence 2 is free again
    assert bm.num_free_blocks()[0] == free - 6 + 1
    scores = torch.rand(2, Hkv, 56, generator=gen, device="cuda")
    kept = torch.zeros(2, Hkv, budget, dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    cuda = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    was = scores.clone()
    P.evict_tokens(kept, new, scores, scores, kc, vc, cuda(tables), cuda(dst), cuda(lens), budget, 2, 5, 56,
                   P.make_evict_workspace())
    assert new.tolist() == [20, 20]
    t0, l0 = bm.block_tables([0], 8)
    assert l0.tolist() == [50]
    assert torch.equal(gather(kc, cuda(t0), 0, 50, bs), k)             # the prompt's owner reads what it wrote
    slots, cow, tables, lens = bm.plan_decode([1, 2], 8)
    assert len(cow) == 0 and lens.tolist() == [21, 21]
    nk, nv, q = randn(2, Hkv, d), randn(2, Hkv, d), randn(2, H, d)
    P.reshape_and_cache(nk, nv, kc, vc, cuda(slots))
    out = torch.empty_like(q)
    before = scores.clone()
    P.paged_attention_accumulate(out, scores, q, kc, vc, cuda(tables), cuda(lens), 0.125, 21,
                                 P.make_accumulate_workspace(2, H, Hkv, d, 21))
    for i, s in enumerate((1, 2)):
        per = []
        for h in range(Hkv):
            ids = evict(was[i, h], len(logical[s][0]), budget, 2, 5)
            assert kept[i, h].tolist() == ids
            per.append(torch.tensor(ids, device="cuda"))
        keys, values = (torch.cat([torch.stack([logical[s][w][per[h], h] for h in range(Hkv)], 1), x[i:i + 1]]).double()
                        for w, x in ((0, nk), (1, nv)))
        ref, bound, add, rel = attention(q[i:i + 1], keys, values, None, 0.125, True, 1, (dt, "16"))
        assert bool((out[i:i + 1].double() - ref).abs().le(bound).all())
        err = (scores[i, :, :21] - before[i, :, :21]).double() - add
        assert bool(err.abs().le(rel * add + 2 * U * (before[i, :, :21].double() + add)).all())
