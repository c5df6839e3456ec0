"""Contexts longer than the call's max_context_len, inside its block table and its last partition all the same: they
are flagged, their rows are NaN, their scores stay, and nothing behind the workspace's rows of scores is written."""
import pytest
import torch

import test_gpu_cross as X
import test_gpu_eviction as E

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


@pytest.mark.parametrize("max_len,part", [(2040, 704), (2040, 0), (70, 128), (0, 64)])
@pytest.mark.parametrize("H", [8, 32, 2])
@pytest.mark.parametrize("cache", ["16", "fp8"])
def test_a_scoring_step_past_the_announced_length(P, max_len, part, H, cache):
    covered = max(1, -(-max_len // (part or 64))) * (part or 64)
    lens = [max_len, covered, max(max_len - 5, 0), max_len + 1]    # the last rows end the workspace
    Hkv, d = min(H, 8), 128
    st = E.make(lens, None, H, Hkv, d, 16, cache=cache, seed=max_len + H, stride=covered + 3)
    st["max_len"] = max_len
    before = st["scores"].clone()
    n = P.accumulate_workspace_size(4, H, Hkv, d, max_len, part)
    memory = torch.zeros(n + (4 << 20), dtype=torch.uint8, device="cuda")
    memory[n:] = 0xA5
    out = torch.full_like(st["q"], 7.0)
    E.step(P, st, out, ws=memory[:n], part=part)
    torch.cuda.synchronize()
    assert P.get_device_error(memory[:n]) == P.PA_DEVERR_CONTEXT_LEN
    assert bool((memory[n:] == 0xA5).all())
    E.check(st, before, out, seqs={0, 2})
    for s in (1, 3):
        assert lens[s] > max_len and torch.equal(st["scores"][s], before[s]) and bool(out[s].isnan().all())


@pytest.mark.parametrize("H", [8, 16])
def test_single_token_cross_attention_past_the_announced_length(P, H):
    st = X.make([40, 700, 699, 703, 650], [1, 1, 1, 1, 1], H, 8, 128, 16, seed=H)
    out = torch.full_like(st["q"], 7.0)
    ws = X.call(P, st, out, max_len=699)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_CONTEXT_LEN
    assert bool(out[1].isnan().all()) and bool(out[3].isnan().all())
    X.check(st, out, seqs={0, 2, 4})
