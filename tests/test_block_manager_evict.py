"""The block manager's eviction plan (CPU): destinations are a sequence's own blocks, or fresh ones where it shares
them; no destination is read by another sequence of the call; failures change nothing."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def BM():
    from pagedattention_paged_kv_attention_b200 import build
    build.build()
    from pagedattention_paged_kv_attention_b200 import block_manager
    return block_manager


def state(bm, ids):
    return [bm.ref_count(b) for b in range(bm.num_blocks)], bm.num_free_blocks(), [bm.sequence_info(s) for s in ids]


@pytest.mark.parametrize("seed", range(12))
def test_random_pools(BM, seed):
    rng = np.random.default_rng(seed)
    bs, nb = int(rng.choice([1, 2, 4, 16])), int(rng.integers(20, 90))
    bm = BM.BlockManager(nb, bs)
    ids = []
    for i in range(int(rng.integers(1, 9))):
        try:
            kind = rng.integers(3)
            if kind == 0 or not ids:
                bm.add_sequence(i, int(rng.integers(0, 6 * bs + 2)))
            elif kind == 1:
                bm.fork(int(rng.choice(ids)), i)
            else:
                p = int(rng.choice(ids))
                k = min(bm.sequence_info(p)[0], int(rng.integers(0, 4 * bs)))
                bm.add_sequence(i, k + int(rng.integers(0, 2 * bs)), p, k)
            ids.append(i)
        except BM.OutOfBlocks:
            pass
    budget = int(rng.integers(1, 4 * bs + 1))
    sel = [int(s) for s in rng.permutation(ids)[:int(rng.integers(1, len(ids) + 1))]]
    old = {s: (bm.sequence_info(s)[0], bm.block_tables([s], 99, pad=-1)[0][0].tolist()) for s in ids}
    refs = [bm.ref_count(b) for b in range(nb)]
    free = {b for b in range(nb) if refs[b] == 0}
    keep = {s: -(-min(old[s][0], budget) // bs) for s in sel}
    need = sum(refs[b] > 1 for s in sel if old[s][0] > budget for b in old[s][1][:keep[s]])
    if need > len(free):
        before = state(bm, ids)
        with pytest.raises(BM.OutOfBlocks):
            bm.plan_evict(sel, budget, 99, 99)
        assert state(bm, ids) == before
        return
    tables, dst, lens = bm.plan_evict(sel, budget, 99, 99, pad=-1)
    seen = {}
    for i, s in enumerate(sel):
        tokens, blocks = old[s]
        assert lens[i] == tokens and tables[i].tolist() == blocks
        d = dst[i].tolist()
        assert all(b == -1 for b in d[keep[s]:]) and bm.sequence_info(s)[0] == min(tokens, budget)
        assert bm.block_tables([s], 99, pad=-1)[0][0].tolist() == d
        for j, b in enumerate(d[:keep[s]]):
            if tokens <= budget or refs[blocks[j]] == 1:
                assert b == blocks[j]
            else:
                assert b in free and b not in seen
                seen[b] = s
    owners = [0] * nb
    for s in ids:
        for b in bm.block_tables([s], 99, pad=-1)[0][0].tolist():
            if b >= 0:
                owners[b] += 1
    assert owners == [bm.ref_count(b) for b in range(nb)]
    assert bm.num_free_blocks()[0] == owners.count(0)
    bm.append_slots(ids[:1]) if bm.num_free_blocks()[0] else None


def test_refusals_change_nothing(BM):
    bm = BM.BlockManager(16, 4, 8)
    bm.add_sequence(0, 18)
    bm.add_sequence(1, 3)
    bm.add_sequence(2, 5)
    bm.swap_out(2)
    before = state(bm, [0, 1, 2])
    for args in (([0], 0, 9, 9), ([0], -1, 9, 9), ([0, 0], 4, 9, 9), ([2], 4, 9, 9), ([7], 4, 9, 9), ([0], 12, 4, 9),
                 ([0], 12, 9, 2), ([0, 1], 12, 9, 0)):
        with pytest.raises(Exception) as e:
            bm.plan_evict(*args)
        assert "INVALID_ARGUMENT" in str(e.value)
        assert state(bm, [0, 1, 2]) == before
    tables, dst, lens = bm.plan_evict([], 4, 2, 2)
    assert len(lens) == 0 and state(bm, [0, 1, 2]) == before
    tables, dst, lens = bm.plan_evict([0, 1], 12, 5, 3, pad=9)
    assert tables.tolist() == [[0, 1, 2, 3, 4], [5, 9, 9, 9, 9]] and dst.tolist() == [[0, 1, 2], [5, 9, 9]]
    assert lens.tolist() == [18, 3] and bm.sequence_info(0) == (12, 3, False)
