"""Cross attention over an encoder's cached states against the formula in 64 bits (operator_refs' bounds)."""
import pytest
import torch

from operator_refs import DTYPES, attention, gather, make_pool, poison_unused, scatter_tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


def make(lens, chunks, H, Hkv, d, bs, dtype="bf16", cache="16", seed=0, tail=0, junk=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(lens=lens, chunks=chunks, bs=bs, info=(DTYPES[dtype], cache), scale=d ** -0.5)
    st["table"], nb = scatter_tables(gen, lens, bs, junk=junk)
    st["kc"], st["vc"], st["ks"], st["vs"], st["k64"], st["v64"] = make_pool(gen, nb, bs, Hkv, d, DTYPES[dtype], cache)
    poison_unused((st["kc"], st["vc"]), st["table"], lens, bs)
    T = sum(chunks) + tail
    st["q"] = torch.randn(T, H, d, generator=gen, device="cuda").to(DTYPES[dtype])
    if tail:
        st["q"][-tail:] = float("nan")
    st["q_start"] = torch.tensor([sum(chunks[:i]) for i in range(len(chunks) + 1)], dtype=torch.int32, device="cuda")
    st["cl"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return st


def call(P, st, out, ws=None, max_q=None, max_len=None):
    S, (T, H, d) = len(st["lens"]), st["q"].shape
    max_q = max(st["chunks"]) if max_q is None else max_q
    max_len = max(st["lens"]) if max_len is None else max_len
    if ws is None:
        ws = P.make_cross_workspace(S, T, H, st["kc"].shape[2], d, max_q, max_len)
    P.paged_cross_attention(out, st["q"], st["kc"], st["vc"], st["table"], st["cl"], st["q_start"], st["scale"], max_q,
                            max_len, ws, k_scale=st["ks"], v_scale=st["vs"])
    return ws


def check(st, out, seqs=None):
    for s, (L, n) in enumerate(zip(st["lens"], st["chunks"])):
        if n == 0 or (seqs is not None and s not in seqs):
            continue
        rows = slice(int(st["q_start"][s]), int(st["q_start"][s]) + n)
        got = out[rows].double()
        if L == 0:
            assert bool((got == 0).all())
            continue
        k, v = gather(st["k64"], st["table"], s, L, st["bs"]), gather(st["v64"], st["table"], s, L, st["bs"])
        ref, bound, _, _ = attention(st["q"][rows], k, v, rows, st["scale"], False, 1, st["info"])
        assert bool((got - ref).abs().le(bound).all()), (s, float(((got - ref).abs() - bound).max()))


CASES = [
    # lens, chunks, H, Hkv, d, bs, options
    ([1], [1], 1, 1, 64, 8, {}),
    ([5, 0, 129, 64], [3, 2, 1, 130], 8, 2, 128, 16, {}),
    ([127, 128, 1, 300], [257, 1, 0, 40], 4, 4, 64, 32, dict(dtype="f16")),
    ([700, 1300], [1, 1], 32, 4, 128, 8, {}),                        # decode rows, keys split
    ([2049, 77, 513], [1, 1, 1], 8, 8, 128, 64, dict(dtype="f16")),
    ([1500, 1025, 0, 40], [5, 33, 4, 9], 16, 1, 128, 16, {}),        # 16 heads share a kv head, split
    ([900, 33], [70, 300], 8, 8, 128, 16, dict(cache="fp8")),
    ([901, 1700, 8], [1, 1, 1], 16, 2, 128, 32, dict(cache="fp8", dtype="f16")),
    ([640, 1111], [20, 1], 8, 4, 128, 8, dict(cache="fp8_block")),
    ([640, 1111], [1, 1], 8, 1, 128, 16, dict(cache="fp8_block", dtype="f16")),
    ([300, 555], [1, 1], 8, 2, 64, 128, {}),
    ([300, 2000], [64, 33], 128, 1, 64, 128, dict(dtype="f16")),
    ([3000, 10, 0], [1, 1, 1], 24, 8, 128, 16, dict(junk=-7)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "L%s_n%s_H%d_%d_d%d_bs%d_%s" % (
    "-".join(map(str, c[0])), "-".join(map(str, c[1])), *c[2:6], "-".join(map(str, c[6].values()))))
def test_cross_against_the_formula(P, case):
    lens, chunks, H, Hkv, d, bs, opt = case
    if 128 % (H // Hkv):
        st = make(lens, chunks, H, Hkv, d, bs, **opt)
        with pytest.raises(P.PagedAttnError):
            call(P, st, torch.empty_like(st["q"]))
        return
    st = make(lens, chunks, H, Hkv, d, bs, seed=sum(lens), **opt)
    out = torch.full_like(st["q"], float("nan"))
    ws = call(P, st, out)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    check(st, out)


@pytest.mark.parametrize("chunks", [[1, 0, 1], [1, 1, 1], [9, 0, 2]])
def test_rows_behind_the_last_sequence_and_empty_chunks_stay(P, chunks):
    st = make([900, 50, 1024], chunks, 8, 2, 128, 16, tail=3, seed=2)
    out = torch.full_like(st["q"], 7.0)
    call(P, st, out, max_q=max(chunks) + 5, max_len=1500)
    check(st, out)
    assert bool((out[-3:] == 7).all())


@pytest.mark.parametrize("chunks", [[1, 1, 1, 1], [4, 2, 3, 1]])
def test_invalid_lengths_are_flagged_and_their_rows_are_nan(P, chunks):
    st = make([40, 300, 700, 650], chunks, 8, 2, 128, 16, seed=3)
    st["cl"][0] = -3
    st["cl"][1] = 16 * st["table"].shape[1] + 1    # past its table
    out = torch.zeros_like(st["q"])
    ws = call(P, st, out, max_len=699 if chunks[0] == 4 else 10000)  # 700 is past 699
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_CONTEXT_LEN
    bad = [0, 1, 2] if chunks[0] == 4 else [0, 1]
    for s in bad:
        assert bool(out[st["q_start"][s]:st["q_start"][s + 1]].isnan().all())
    check(st, out, seqs={3})


def test_a_chunk_longer_than_announced_is_flagged(P):
    st = make([300, 700], [3, 1], 8, 2, 128, 16, seed=4)           # three rows where one is announced
    out = torch.zeros_like(st["q"])
    ws = call(P, st, out, max_q=1)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_CONTEXT_LEN
    check(st, out, seqs={1})
    assert bool((out[:3] == 0).all())
    st = make([300, 2000], [300, 40], 8, 8, 128, 16, seed=4)       # 256 rows are covered
    out = torch.zeros_like(st["q"])
    ws = call(P, st, out, max_q=40)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == P.PA_DEVERR_CONTEXT_LEN
    assert bool(out[:256].isnan().all()) and bool((out[256:300] == 0).all())
    check(st, out, seqs={1})
    st = make([3000, 300], [60, 40], 8, 8, 128, 16, seed=4)        # more than announced, but covered: computed
    out = torch.zeros_like(st["q"])
    ws = call(P, st, out, ws=P.make_cross_workspace(2, 100, 8, 8, 128, 40, 3000), max_q=40)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    check(st, out)


@pytest.mark.parametrize("n", [1, 5])
def test_results_repeat_and_do_not_depend_on_the_other_sequences(P, n):
    st = make([1900, 33, 800], [n, n, n], 16, 4, 128, 16, seed=6)
    a, b = torch.empty_like(st["q"]), torch.empty_like(st["q"])
    ws = call(P, st, a)
    for _ in range(3):
        call(P, st, b, ws=ws)
        assert torch.equal(a, b)


def test_graph_replay_follows_lengths_and_queries(P):
    st = make([1900, 33, 800], [1, 1, 1], 16, 4, 128, 16, seed=7)
    out = torch.empty_like(st["q"])
    ws = call(P, st, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(P, st, out, ws=ws)
    st["q"].normal_()
    st["lens"] = [1024, 0, 799]
    st["cl"].copy_(torch.tensor(st["lens"]))
    g.replay()
    check(st, out)
