"""The workspaces of scoring decode and cross attention without a GPU: a size holds for the arguments it was asked for.
A smaller call may need more, its own query says how much, and a buffer below that is refused before any CUDA call."""
import pytest

import test_abi_operators as A

TOO_SMALL = 3
P = A.P  # the module's fixture


def cross_size(P, S, T, max_q, max_len, H=32, Hkv=32):
    return P.lib.pa_paged_cross_attention_workspace_size(S, T, H, Hkv, 128, max_q, max_len)


@pytest.mark.parametrize("S,T,max_q", [(4, 2048, 512), (1, 512, 512), (32, 32, 1), (1, 1, 1)])
def test_cross_attention_of_a_smaller_batch_needs_its_own_size(P, S, T, max_q):
    prompts, need = cross_size(P, 32, 32 * 512, 512, 1601), cross_size(P, S, T, max_q, 1601)
    assert prompts == 256 < need
    sizes = dict(num_seqs=S, num_q_tokens=T, num_heads=32, num_kv_heads=32, max_q_len=max_q, max_context_len=1601)
    for n in (prompts, need - 1):
        over = dict(sizes, workspace_bytes=n)
        assert A.refuse(P.lib.pa_paged_cross_attention, A.cross_args(P), over) == TOO_SMALL


@pytest.mark.parametrize("larger,smaller", [((95, 100), (94, 100)), ((4, 2369), (4, 2368)), ((14, 701), (13, 701))])
def test_a_scoring_step_of_a_smaller_batch_needs_its_own_size(P, larger, smaller):
    size = lambda S, L: P.lib.pa_paged_attention_accumulate_workspace_size(S, 32, 8, 128, L, 0)  # noqa: E731
    have, need = size(*larger), size(*smaller)
    assert have < need
    S, L = smaller
    sizes = dict(num_seqs=S, num_heads=32, num_kv_heads=8, max_context_len=L, score_stride=L)
    for n in (have, need - 1):
        over = dict(sizes, workspace_bytes=n)
        assert A.refuse(P.lib.pa_paged_attention_accumulate, A.step_args(P), over) == TOO_SMALL
