"""The positional, scoring, eviction and cross-attention entry points without a GPU: workspace sizes as
documented, and bad arguments refused with a status before any CUDA call."""
import pytest


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import build
    build.build()
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


def refuse(fn, base, over):
    unknown = set(over) - set(base)
    assert not unknown, unknown
    return fn(*dict(base, **over).values())


def rope_args(P):
    return dict(query_out=16, query_out_stride=1024, query=32, query_stride=1024, key=16, key_stride=256, value=16,
                value_stride=256, in_dtype=P.PA_BF16, key_cache=16, value_cache=16, kv_dtype=P.PA_BF16, k_scale=None,
                v_scale=None, slot_mapping=16, positions=16, num_axes=3, inv_freq=16, freq_axis=16, rotary_size=128,
                interleaved=0, num_tokens=4, num_heads=8, num_kv_heads=2, head_size=128, block_size=16, num_blocks=10,
                stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(query_out=None), 1), (dict(query=None), 1), (dict(key=None), 1), (dict(value=None), 1),
    (dict(positions=None), 1), (dict(inv_freq=None), 1), (dict(freq_axis=None), 1), (dict(slot_mapping=None), 1),
    (dict(query=24), 1), (dict(key_cache=8), 1), (dict(slot_mapping=4), 1), (dict(positions=2), 1),
    (dict(num_tokens=-1), 1), (dict(num_heads=0), 1), (dict(num_axes=0), 1), (dict(rotary_size=0), 1),
    (dict(rotary_size=130), 1), (dict(rotary_size=63), 1), (dict(interleaved=2), 1), (dict(num_blocks=0), 1),
    (dict(query_stride=1016), 1), (dict(key_stride=128), 1), (dict(query_out=32, query_out_stride=2048), 1),
    (dict(in_dtype=2), 1), (dict(in_dtype=9), 1), (dict(kv_dtype=2), 1), (dict(kv_dtype=4, k_scale=16, v_scale=16), 1),
    (dict(kv_dtype=0), 2), (dict(rotary_size=24), 2), (dict(head_size=516, query_stride=8256, query_out_stride=8256,
                                                            key_stride=2048, value_stride=2048), 2),
    (dict(query_stride=1028), 2), (dict(value_stride=260), 2),
    (dict(rotary_size=528, head_size=528, query_stride=8448, query_out_stride=8448, key_stride=2112,
          value_stride=2112), 2),
    (dict(num_tokens=0, query=None, positions=None), 0),
])
def test_rope_refuses(P, over, status):
    assert refuse(P.lib.pa_rope_reshape_and_cache, rope_args(P), over) == status


def step_args(P):
    return dict(out=16, scores=16, score_stride=64, query=16, q_dtype=P.PA_BF16, key_cache=16, value_cache=16,
                kv_dtype=P.PA_BF16, k_scale=None, v_scale=None, block_tables=16, max_blocks_per_seq=4, context_lens=16,
                num_seqs=2, num_heads=8, num_kv_heads=2, head_size=128, block_size=16, num_blocks=10,
                max_context_len=64, scale=0.1, partition_size=0, workspace=16, workspace_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(out=None), 1), (dict(scores=None), 1), (dict(scores=6), 1), (dict(score_stride=63), 1),
    (dict(score_stride=0, max_context_len=0), 1), (dict(workspace=None), 1), (dict(kv_dtype=2), 1),
    (dict(partition_size=100), 1), (dict(head_size=96), 2), (dict(block_size=4), 2), (dict(kv_dtype=0), 2),
    (dict(workspace_bytes=256), 3), (dict(num_seqs=0, scores=None), 0),
])
def test_step_refuses(P, over, status):
    assert refuse(P.lib.pa_paged_attention_accumulate, step_args(P), over) == status


def prompt_args(P):
    return dict(out=16, scores=16, score_stride=64, query=16, q_dtype=P.PA_BF16, key_cache=16, value_cache=16,
                kv_dtype=P.PA_BF16, k_scale=None, v_scale=None, block_tables=16, max_blocks_per_seq=4, context_lens=16,
                q_start=16, num_seqs=2, num_q_tokens=20, num_heads=8, num_kv_heads=2, head_size=128, block_size=16,
                num_blocks=10, max_q_len=16, max_context_len=64, window=0, scale=0.1, workspace=16,
                workspace_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(out=None), 1), (dict(scores=None), 1), (dict(scores=6), 1), (dict(score_stride=63), 1),
    (dict(max_context_len=-1), 1), (dict(window=-1), 1), (dict(q_start=None), 1), (dict(workspace=8), 1),
    (dict(scale=0.0), 1), (dict(num_heads=6, num_kv_heads=4), 1), (dict(kv_dtype=3), 1), (dict(head_size=96), 2),
    (dict(block_size=4), 2), (dict(num_heads=12, num_kv_heads=4), 2), (dict(workspace_bytes=256 + 639), 3),
    (dict(num_seqs=0, scores=None), 0), (dict(num_q_tokens=0), 0), (dict(max_q_len=0), 0),
])
def test_prompt_refuses(P, over, status):
    assert refuse(P.lib.pa_paged_prefill_accumulate, prompt_args(P), over) == status


def cross_args(P):
    a = prompt_args(P)
    for k in ("scores", "score_stride", "window"):
        del a[k]
    return a


@pytest.mark.parametrize("over,status", [
    (dict(out=None), 1), (dict(query=8), 1), (dict(max_context_len=-1), 1), (dict(q_start=None), 1),
    (dict(scale=float("nan")), 1), (dict(num_heads=6, num_kv_heads=4), 1), (dict(num_heads=0), 1), (dict(kv_dtype=2), 1),
    (dict(head_size=96), 2), (dict(block_size=4), 2), (dict(num_heads=12, num_kv_heads=4), 2), (dict(kv_dtype=0), 2),
    (dict(workspace_bytes=255), 3), (dict(max_q_len=1, max_context_len=100000, workspace_bytes=4096), 3),
    (dict(num_seqs=0, query=None), 0), (dict(num_q_tokens=0), 0),
])
def test_cross_refuses(P, over, status):
    assert refuse(P.lib.pa_paged_cross_attention, cross_args(P), over) == status


def evict_args(P):
    return dict(kept=16, new_lens=16, scores_out=16, scores=16, score_stride=64, key_cache=16, value_cache=16,
                kv_dtype=P.PA_BF16, block_tables=16, max_blocks_per_seq=4, dst_block_tables=16,
                max_dst_blocks_per_seq=2, context_lens=32, num_seqs=2, num_kv_heads=2, head_size=128, block_size=16,
                num_blocks=10, max_context_len=64, budget=32, num_sink=4, num_recent=8, workspace=16,
                workspace_bytes=256, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(kept=None), 1), (dict(new_lens=None), 1), (dict(scores=None), 1), (dict(scores_out=None), 1),
    (dict(key_cache=8), 1), (dict(workspace=None), 1), (dict(new_lens=32), 1), (dict(score_stride=63), 1),
    (dict(budget=0), 1), (dict(num_sink=-1), 1), (dict(num_recent=-1), 1), (dict(num_sink=20, num_recent=13), 1),
    (dict(num_sink=2 ** 31 - 1, num_recent=2 ** 31 - 1), 1), (dict(budget=33, max_dst_blocks_per_seq=2), 1),
    (dict(kv_dtype=9), 1), (dict(num_seqs=-1), 1), (dict(kv_dtype=3), 2), (dict(head_size=12), 2),
    (dict(head_size=520), 2), (dict(num_seqs=65536), 2), (dict(workspace_bytes=255), 3),
    (dict(num_seqs=0, kept=None), 0),
])
def test_evict_refuses(P, over, status):
    assert refuse(P.lib.pa_evict_tokens, evict_args(P), over) == status


def test_workspace_sizes(P):
    lib = P.lib
    S, H, Hkv, d, L = 8, 32, 8, 128, 4000
    parts = -(-L // P.partition_size(S, H, Hkv, L))
    n = lib.pa_paged_attention_accumulate_workspace_size(S, H, Hkv, d, L, 0)
    assert n >= P.workspace_size(S, H, Hkv, d, L) + S * H * (4 * 4032 + 8 * parts)
    assert lib.pa_paged_attention_accumulate_workspace_size(S, H, 3, d, L, 0) == 0
    assert lib.pa_paged_attention_accumulate_workspace_size(S, H, Hkv, d, -1, 0) == 0
    assert lib.pa_paged_attention_accumulate_workspace_size(S, H, Hkv, d, L, 100) == 0
    assert lib.pa_paged_prefill_accumulate_workspace_size(100, 8) == 256 + 3328
    assert lib.pa_paged_prefill_accumulate_workspace_size(0, 8) == 256
    assert lib.pa_paged_prefill_accumulate_workspace_size(-1, 8) == 0
    assert lib.pa_paged_prefill_accumulate_workspace_size(5, 0) == 0
    size = lib.pa_paged_cross_attention_workspace_size
    assert size(64, 64 * 500, 32, 32, 128, 500, 1600) == 256            # enough query tiles: no split
    assert size(1, 300, 8, 8, 128, 300, 20000) > 256 + 300 * 8 * 128 * 4  # few query tiles: keys split
    assert size(1, 1, 8, 3, 128, 1, 100) == 0 and size(1, 1, 0, 1, 128, 1, 100) == 0
    assert size(1, 1, 8, 8, 128, -1, 100) == 0 and size(1, 1, 8, 8, 128, 1, -1) == 0
    for make, args in ((P.make_cross_workspace, (1, 1, 8, 3, 128, 1, 100)),
                       (P.make_accumulate_workspace, (8, 32, 3, 128, 100)),
                       (P.make_prefill_accumulate_workspace, (-1, 8))):
        with pytest.raises(ValueError):
            make(*args, device="cpu")


def test_binding_checks_shapes_before_the_library(P):
    """Mismatched shapes, types, strides and CPU tensors raise before any pointer is passed on."""
    import torch
    bf = torch.bfloat16
    q, kv = torch.zeros(4, 8, 128, dtype=bf), torch.zeros(4, 2, 128, dtype=bf)
    cache = torch.zeros(10, 16, 2, 128, dtype=bf)
    slots, pos = torch.zeros(4, dtype=torch.int64), torch.zeros(3, 4, dtype=torch.int32)
    inv, axis = torch.zeros(64), torch.zeros(64, dtype=torch.int32)
    good = [q, q, kv, kv, cache, cache, slots, pos, inv, axis]
    for i, bad in ((0, q[:3]), (2, kv[:3]), (4, cache[:9]), (6, slots[:3]), (7, pos[:, :3]), (8, inv[:5]),
                   (1, q.transpose(0, 1)), (2, kv.float())):
        with pytest.raises(ValueError):
            P.rope_reshape_and_cache(*good[:i], bad, *good[i + 1:])
    with pytest.raises(ValueError):
        P.rope_reshape_and_cache(*good)                                  # CPU tensors
    table, lens = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    scores, ws = torch.zeros(4, 2, 64), torch.zeros(4096, dtype=torch.uint8)
    for sc, tb, ln in ((scores[:3], table, lens), (scores[:, :1], table, lens), (scores, table[:3], lens),
                       (scores, table, lens[:3]), (scores, table, lens)):
        with pytest.raises(ValueError):
            P.paged_attention_accumulate(q, sc, q, cache, cache, tb, ln, 0.1, 32, ws)
    start = torch.zeros(5, dtype=torch.int32)
    for st in (start[:4], start):
        with pytest.raises(ValueError):
            P.paged_cross_attention(q, q, cache, cache, table, lens, st, 0.1, 4, 32, ws)
        with pytest.raises(ValueError):
            P.paged_prefill_accumulate(q, scores, q, cache, cache, table, lens, st, 0.1, 4, 32, ws)
    kept, new = torch.zeros(4, 2, 16, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for k, n, so in ((kept[..., :15], new, scores), (kept, new[:3], scores), (kept, new, scores[..., :63]),
                     (kept, new, scores)):
        with pytest.raises(ValueError):
            P.evict_tokens(k, n, so, scores, cache, cache, table, table, lens, 16, 1, 2, 32, ws)
