"""Ways of calling the rotary write, scoring, eviction and cross attention that their formulas do not show: every 16-bit
value under far scales, another stream, and two graphs over one workspace. Results are compared bit for bit, with
the plain cache write and with an eager run on the default stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_every_value_gets_the_code_of_the_plain_write(P, dt, interleaved):
    T, Hkv, d, bs = 64 * 8, 8, 128, 16
    scales = [2e-38, 1e-30, 0.0078125, 0.01, 0.3, 3.0, 448.0, 1e30]
    every = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(dt)
    every = torch.where(every.isfinite(), every, torch.ones_like(every))
    v = every.view(64, Hkv, d)                   # heads in turn, so that each value meets each scale
    v = torch.cat([v.roll(i, 1) for i in range(Hkv)]).contiguous()
    ks = torch.tensor(scales, device="cuda")
    vs = ks.flip(0).contiguous()
    slots = torch.randperm(T, generator=torch.Generator().manual_seed(1)).cuda()
    caches = [torch.zeros(T // bs, bs, Hkv, d, dtype=torch.uint8, device="cuda") for _ in range(4)]
    q = torch.zeros(T, 2, d, dtype=dt, device="cuda")
    P.rope_reshape_and_cache(q, q, v, v, caches[0], caches[1], slots, torch.zeros(2, T, dtype=torch.int32, device="cuda"),
                             torch.ones(d // 2, device="cuda"), torch.zeros(d // 2, dtype=torch.int32, device="cuda"),
                             interleaved=interleaved, k_scale=ks, v_scale=vs)
    P.reshape_and_cache(v, v, caches[2], caches[3], slots, k_scale=ks, v_scale=vs)
    assert torch.equal(caches[1], caches[3])
    # At position 0 a key is x - 0 y: x itself, but for the sign of a zero.
    a, b = (torch.where(c & 0x7f == 0, torch.zeros_like(c), c) for c in (caches[0], caches[2]))
    assert torch.equal(a, b)


def state(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    S, H, Hkv, d, bs = 3, 8, 2, 128, 16
    lens, width = [700, 33, 1300], 82
    NB = S * width
    st = dict(S=S, H=H, Hkv=Hkv, d=d, lens=lens, max_len=width * bs)
    st["table"] = torch.randperm(NB, generator=gen, device="cuda").view(S, width).to(torch.int32)
    st["kc"], st["vc"] = (torch.randn(NB, bs, Hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    st["cl"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["q"] = torch.randn(40, H, d, generator=gen, device="cuda").bfloat16()
    st["scores"] = torch.zeros(S, Hkv, st["max_len"], device="cuda")
    st["outs"] = [torch.zeros_like(st["q"]) for _ in range(4)]
    st["kept"] = torch.zeros(S, Hkv, 256, dtype=torch.int32, device="cuda")
    st["new"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    starts = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st["chunks"], st["ones"] = starts(0, 20, 21, 40), starts(0, 1, 2, 3)
    return st


def workspaces(P, st):
    S, H, Hkv, d, m = st["S"], st["H"], st["Hkv"], st["d"], st["max_len"]
    return [P.make_prefill_accumulate_workspace(40, H), P.make_accumulate_workspace(S, H, Hkv, d, m),
            P.make_cross_workspace(S, 40, H, Hkv, d, 20, m), P.make_cross_workspace(S, S, H, Hkv, d, 1, m),
            P.make_evict_workspace()]


def steps(P, st, ws):
    scale, m, kv = st["d"] ** -0.5, st["max_len"], (st["kc"], st["vc"], st["table"])
    o = st["outs"]
    P.paged_prefill_accumulate(o[0], st["scores"], st["q"], *kv, st["cl"], st["chunks"], scale, 20, m, ws[0], window=7)
    P.paged_attention_accumulate(o[1][:3], st["scores"], st["q"][:3], *kv, st["cl"], scale, m, ws[1])
    P.paged_cross_attention(o[2], st["q"], *kv, st["cl"], st["chunks"], scale, 20, m, ws[2])
    P.paged_cross_attention(o[3][:3], st["q"][:3], *kv, st["cl"], st["ones"], scale, 1, m, ws[3])
    P.evict_tokens(st["kept"], st["new"], st["scores"], st["scores"], st["kc"], st["vc"], st["table"], st["table"],
                   st["cl"], 256, 4, 64, m, ws[4])
    st["cl"].copy_(st["new"])


def results(st):
    return [*st["outs"], st["scores"], st["kept"], st["new"], st["kc"], st["vc"]]


def same(a, b):
    for x, y in zip(results(a), results(b)):
        assert torch.equal(x, y)


def test_another_stream(P):
    a, b = state(1), state(1)
    steps(P, a, workspaces(P, a))
    ws = workspaces(P, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps(P, b, ws)
    torch.cuda.current_stream().wait_stream(side)
    same(a, b)
    assert all(P.get_device_error(w) == 0 for w in ws)


def test_two_graphs_share_workspaces(P):
    """Two states, each with a graph of its own over the same workspaces, replayed in turn."""
    eager, graphed = [state(2), state(3)], [state(2), state(3)]
    warm = state(2)
    ws = workspaces(P, warm)
    steps(P, warm, ws)
    graphs = []
    for st in graphed:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            steps(P, st, ws)
        graphs.append(g)
    for _ in range(2):                           # the second pass starts from the evicted caches
        for st in eager:
            steps(P, st, workspaces(P, st))
        for g in graphs:
            g.replay()
        for a, b in zip(eager, graphed):
            same(a, b)
    assert all(P.get_device_error(w) == 0 for w in ws)


LONE = [  # context lengths, chunk, query heads, kv heads, head size, cache
    ([129, 256, 257, 384, 385, 128, 1], 5, 4, 4, 128, "16"),       # 2, 2, 3, 3, 4 key tiles; 1 and 1: one warpgroup
    ([1000, 1, 640, 511, 1153, 2048, 2049], 128, 4, 4, 128, "16"),
    ([1000, 130, 640, 511, 0, 2048, 700], 33, 8, 2, 64, "16"),
    ([900, 129, 640, 255, 1153], 9, 16, 2, 128, "fp8"),
    ([900, 129, 640, 257, 1153], 17, 4, 4, 128, "fp8_block"),
    ([1500, 3, 5000], 7, 2, 1, 128, "16"),                         # keys shared by several CTAs as well
]


@pytest.mark.parametrize("case", LONE, ids=lambda c: "L%s_n%d_H%d_%d_d%d_%s" % ("-".join(map(str, c[0])), *c[1:]))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_cross_attention_of_lone_query_tiles(P, case, dtype):
    import test_gpu_cross as X
    lens, n, H, Hkv, d, cache = case
    chunks = [n] * len(lens)
    st = X.make(lens, chunks, H, Hkv, d, 16, seed=sum(lens), cache=cache, dtype=dtype)
    out = torch.full_like(st["q"], float("nan"))
    ws = X.call(P, st, out)
    torch.cuda.synchronize()
    assert P.get_device_error(ws) == 0
    X.check(st, out)
    again = torch.empty_like(out)
    X.call(P, st, again, ws=ws)
    assert torch.equal(out, again)
