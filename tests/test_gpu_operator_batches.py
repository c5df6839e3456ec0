"""Calls with more work items than the GPU has SMs, so that CTAs take several items one after another: scoring decode
and single-token cross attention (tickets, in order of size or, for large batches, as they come), scoring prefill
(items dealt and drawn, several rings of them a CTA) and eviction (more tokens a CTA than its registers hold)."""
import pytest
import torch

import test_gpu_cross as X
import test_gpu_eviction as E

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


def ragged(n, lo, hi, seed):
    g = torch.Generator().manual_seed(seed)
    return [hi, lo] + torch.randint(lo, hi + 1, (n - 2,), generator=g).tolist()


STEP = [
    # sequences, shortest, longest, H, Hkv, d, bs, partition, options: at least 300 items, in several head blocks
    (40, 0, 700, 8, 8, 128, 16, 64, {}),
    (40, 0, 700, 16, 8, 64, 16, 64, dict(dtype="f16")),
    (33, 1, 900, 32, 8, 128, 8, 64, dict(stride=901)),
    (60, 1, 400, 24, 8, 128, 16, 64, {}),                            # 3 heads a group
    (24, 100, 1000, 40, 2, 128, 16, 64, dict(dtype="f16")),          # 20 heads a group: three subgroups
    (20, 0, 600, 12, 12, 128, 32, 64, {}),                           # a second block of heads, half empty
    (40, 0, 700, 8, 8, 128, 16, 64, dict(cache="fp8")),
    (40, 0, 700, 32, 8, 128, 16, 64, dict(cache="fp8", dtype="f16")),
    (40, 0, 700, 16, 8, 128, 8, 64, dict(cache="fp8_block")),
    (40, 1, 700, 8, 8, 128, 16, 128, dict(cache="fp8_block", dtype="f16")),
    (200, 0, 300, 16, 8, 64, 16, 0, {}),                             # the library's partitions
    (1100, 0, 40, 8, 8, 64, 8, 0, {}),                               # too many sequences for an order by size
]


@pytest.mark.parametrize("case", STEP, ids=lambda c: "S%d_L%d-%d_H%d_%d_d%d_bs%d_p%d_%s" % (
    *c[:8], "-".join(map(str, c[8].values()))))
def test_scoring_steps_of_many_items(P, case):
    S, lo, hi, H, Hkv, d, bs, part, opt = case
    st = E.make(ragged(S, lo, hi, S + hi), None, H, Hkv, d, bs, seed=S + H, **opt)
    before = st["scores"].clone()
    out = torch.full_like(st["q"], float("nan"))
    ws = E.step(P, st, out, part=part)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    E.check(st, before, out)
    again, second = before.clone(), torch.full_like(st["q"], float("nan"))
    E.step(P, st, second, ws=ws, part=part, scores=again)            # the work counters are back at zero
    assert torch.equal(again, st["scores"]) and torch.equal(out, second)


CROSS = [
    # sequences, shortest, longest, H, Hkv, d, bs, options
    (100, 0, 2000, 8, 8, 128, 16, {}),
    (64, 1, 3000, 32, 8, 128, 32, dict(dtype="f16")),
    (300, 0, 700, 16, 4, 64, 16, {}),
    (90, 0, 1500, 8, 8, 128, 16, dict(cache="fp8")),
    (70, 5, 2500, 16, 8, 128, 8, dict(cache="fp8_block", dtype="f16")),
    (1100, 0, 60, 8, 8, 64, 8, {}),
]


@pytest.mark.parametrize("case", CROSS, ids=lambda c: "S%d_L%d-%d_H%d_%d_d%d_bs%d_%s" % (
    *c[:7], "-".join(map(str, c[7].values()))))
def test_single_token_cross_attention_of_many_items(P, case):
    S, lo, hi, H, Hkv, d, bs, opt = case
    lens = ragged(S, lo, hi, S)
    chunks = [0 if i % 5 == 3 else 1 for i in range(S)]              # some sequences have no query row
    st = X.make(lens, chunks, H, Hkv, d, bs, seed=S + H, tail=2, **opt)
    out = torch.full_like(st["q"], 7.0)
    ws = X.call(P, st, out)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    X.check(st, out)
    assert bool((out[-2:] == 7).all())
    again = torch.full_like(st["q"], 7.0)
    X.call(P, st, again, ws=ws)
    assert torch.equal(out, again)


PROMPT = [
    # sequences, shortest, longest, longest chunk, H, Hkv, d, bs, window, options: 5 items a CTA and more
    (8, 700, 1500, 1500, 16, 16, 128, 16, 0, {}),                    # drawn
    (6, 900, 1300, 1000, 32, 16, 64, 16, 0, dict(dtype="f16")),
    (10, 300, 1700, 640, 16, 16, 128, 8, 0, dict(cache="fp8")),      # no more than 6 tiles: dealt
    (16, 1, 1500, 70, 16, 16, 128, 16, 0, {}),
    (12, 200, 1400, 1400, 16, 16, 64, 32, 40, {}),
    (9, 400, 1500, 300, 32, 16, 128, 16, 300, dict(cache="fp8_block", dtype="f16")),
]


@pytest.mark.parametrize("case", PROMPT, ids=lambda c: "S%d_L%d-%d_n%d_H%d_%d_d%d_bs%d_w%d_%s" % (
    *c[:9], "-".join(map(str, c[9].values()))))
def test_scoring_prompts_of_many_items(P, case):
    S, lo, hi, most, H, Hkv, d, bs, window, opt = case
    lens = ragged(S, lo, hi, S)
    chunks = [min(n, most) for n in lens]
    chunks[2] = 0
    assert sum(-(-n // 128) for n in lens) * Hkv > 5 * 148
    st = E.make(lens, chunks, H, Hkv, d, bs, seed=S + H, **opt)
    before = st["scores"].clone()
    out = torch.full_like(st["q"], float("nan"))
    ws = E.prompt(P, st, out, window)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    E.check(st, before, out, window)
    first, second = st["scores"].clone(), torch.full_like(st["q"], float("nan"))
    st["scores"].copy_(before)
    E.prompt(P, st, second, window, ws=ws)
    assert torch.equal(first, st["scores"]) and torch.equal(out, second)


EVICT = [
    # lens, Hkv, d, bs, budget, sink, recent, options: more than 4096 tokens a CTA
    ([40001, 33000], 1, 8, 16, 2048, 4, 100, {}),                    # 8 CTAs a row, two tiles each
    ([70000], 2, 16, 64, 30011, 0, 0, dict(cache="fp8")),
    ([33000, 17], 1, 8, 16, 32990, 3, 9, {}),
    ([9000, 4097, 8193] + [50] * 97, 3, 8, 16, 3000, 1, 7, {}),      # one CTA a row
    ([4500, 12289] + [1] * 297, 1, 8, 8, 4400, 0, 4400, {}),         # only the recent ones
]


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("place", ["apart", "in_place"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "S%d_L%d_H%d_d%d_bs%d_b%d" % (len(c[0]), *c[0][:1], *c[1:5]))
def test_eviction_of_more_tokens_than_a_tile(P, case, place, ties):
    lens, Hkv, d, bs, budget, sink, recent, opt = case
    st = E.make(lens, None, Hkv, Hkv, d, bs, seed=lens[0], **opt)
    if ties:
        st["scores"].copy_((st["scores"] * 16).floor() / 8)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dst = E.fresh_destinations(st, gen, lens, budget) if place == "apart" else st["table"]
    before = st["scores"].clone(), st["kc"].clone(), st["vc"].clone()
    kept, new, so, ws = E.evict_call(P, st, budget, sink, recent, dst,
                                     scores_out=st["scores"] if place == "in_place" else None)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    E.check_evict(st, before, dst, budget, sink, recent, kept, new, so)
