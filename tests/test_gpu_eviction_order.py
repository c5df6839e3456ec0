"""Eviction whose rows move into blocks that are read: a slot may be written only after every CTA of its cluster has
read the rows that come from it. A cut of a few tokens keeps sources and destinations within a round of each other
along the whole row. Results are exact."""
import pytest
import torch

from test_gpu_eviction import check_evict, evict_call, fresh_destinations, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


def cut(P, lens, Hkv, d, bs, budget, sink, recent, place, seed, **opt):
    st = make(lens, None, Hkv, Hkv, d, bs, seed=seed, **opt)
    for c in ("kc", "vc"):  # no code or value repeats by chance along a row
        st[c].view(torch.uint8).random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(seed + 1))
    dst = st["table"]
    if place == "mixed":  # as after a fork: some of a sequence's blocks are replaced, the others are its own
        fresh = fresh_destinations(st, torch.Generator(device="cuda").manual_seed(2), lens, budget)
        dst = st["table"][:, :fresh.shape[1]].clone()
        dst[:, 1::3] = fresh[:, 1::3]
    before = st["scores"].clone(), st["kc"].clone(), st["vc"].clone()
    kept, new, so, ws = evict_call(P, st, budget, sink, recent, dst, scores_out=st["scores"])
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    check_evict(st, before, dst, budget, sink, recent, kept, new, so)


CASES = [
    # lens, Hkv, d, bs, budget, sink, recent, options: 2 to 8 CTAs a row
    ([2052], 2, 128, 16, 2048, 4, 64, {}),
    ([4100, 4097, 300], 8, 128, 16, 4096, 0, 0, {}),
    ([16384], 4, 128, 16, 16380, 4, 512, {}),
    ([9000, 8200], 4, 128, 32, 8192, 1, 31, dict(cache="fp8", dtype="f16")),
    ([3000, 3010], 3, 512, 8, 2990, 0, 100, {}),                     # four strips a row
    ([3000, 3010], 3, 24, 8, 2995, 3, 0, dict(dtype="f16")),         # rows of 48 bytes
    ([4100] * 40, 4, 64, 16, 4090, 2, 20, {}),                       # 3 CTAs a row, every SM busy
]


@pytest.mark.parametrize("place", ["in_place", "mixed"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "S%d_L%d_H%d_d%d_bs%d_b%d_%s" % (
    len(c[0]), c[0][0], *c[1:5], "-".join(map(str, c[7].values()))))
def test_a_cut_of_a_few_tokens_is_exact(P, case, place):
    lens, Hkv, d, bs, budget, sink, recent, opt = case
    for seed in range(2 if len(lens) > 9 else 5):
        cut(P, lens, Hkv, d, bs, budget, sink, recent, place, 10 * seed + budget, **opt)


def test_rows_of_one_cta_and_several_stages(P):
    """More rows than clusters of two fit: one CTA moves a row in several stages, over slots that it reads."""
    cut(P, [4990] + [17] * 39, 8, 8, 16, 4980, 1, 9, "in_place", 3)
