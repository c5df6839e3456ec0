"""The scales that evict_tokens is given: per-head ones of the cache are accepted, others refused before it runs."""
import pytest
import torch

import test_gpu_eviction as E

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


def call(P, st, k_scale):
    kept = torch.full((2, 2, 30), -99, dtype=torch.int32, device="cuda")
    new = torch.full((2,), -99, dtype=torch.int32, device="cuda")
    P.evict_tokens(kept, new, st["scores"], st["scores"], st["kc"], st["vc"], st["table"], st["table"], st["cl"], 30, 2,
                   5, st["max_len"], P.make_evict_workspace(), k_scale=k_scale)
    return kept, new


def test_scales_of_another_cache_are_refused(P):
    st = E.make([100, 31], None, 2, 2, 128, 16, cache="fp8", seed=4)
    before = st["scores"].clone(), st["kc"].clone(), st["vc"].clone()
    NB = st["kc"].shape[0]
    for bad in (torch.ones(3, device="cuda"), torch.ones(NB + 1, 2, device="cuda"), torch.ones(2, 1, 1, device="cuda"),
                torch.ones(2), torch.ones(2, device="cuda").double(), torch.ones(2, 4, device="cuda")[:, 0]):
        with pytest.raises(ValueError):
            call(P, st, bad)
    with pytest.raises(TypeError):
        call(P, st, [1.0, 1.0])
    with pytest.raises(P.PagedAttnError):
        call(P, st, torch.ones(NB, 2, device="cuda"))
    torch.cuda.synchronize()
    for now, was in zip((st["scores"], st["kc"], st["vc"]), before):
        assert torch.equal(now, was)
    kept, new = call(P, st, st["ks"])
    E.check_evict(st, before, st["table"], 30, 2, 5, kept, new, st["scores"])
