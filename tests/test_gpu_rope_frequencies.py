"""Frequencies that the rotary write does not use may hold anything."""
import pytest
import torch

import test_gpu_rope as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


@pytest.mark.parametrize("cache", ["16", "fp8"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
def test_a_pair_without_an_axis_reads_no_frequency(P, cache, il, junk):
    st = R.make(dict(T=9, H=4, Hkv=2, d=128, r=128, axes=2, bs=8, cache=cache), seed=6)
    st["axis"][5], st["axis"][60] = -1, 2
    known = st["inv"].clone()
    st["inv"][5] = st["inv"][60] = junk
    before = st["kc"].clone(), st["vc"].clone()
    out = torch.empty_like(st["q"])
    R.call(P, st, out, il)
    R.check(dict(st, inv=known), before, out, il)
