"""Rotary positions with several axes on the way into the cache, against the formula in 64 bits.

Tolerance of a turned element: its angle is off by at most 2^-21 rad (the turns' fraction rounded to fp32, pi 2^-24;
sine and cosine within 2^-22), and two products and a sum add 3 roundings of 2^-24, together less than 2^-20 of
the pair's size |a| + |b|; then one rounding to the output type, half a step of the value.
"""
import pytest
import torch

from operator_refs import DTYPES, half_step, rotate

pytestmark = pytest.mark.gpu
SLACK = 2.0 ** -20


@pytest.fixture(scope="module")
def P():
    from pagedattention_paged_kv_attention_b200 import pagedattn
    return pagedattn


def make(case, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, H, Hkv, d, r, axes, bs = (case[k] for k in ("T", "H", "Hkv", "d", "r", "axes", "bs"))
    dt = DTYPES[case.get("dtype", "bf16")]
    st = dict(dt=dt)
    if case.get("fused"):  # slices of one projection, rows (H + 2 Hkv) d apart
        qkv = torch.randn(T, H + 2 * Hkv, d, generator=gen, device="cuda").to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        st["q"], st["k"], st["v"] = (torch.randn(T, n, d, generator=gen, device="cuda").to(dt) for n in (H, Hkv, Hkv))
    NB = -(-T // bs) + 3
    st["cache"] = cache = case.get("cache", "16")
    st["ks"] = st["vs"] = None
    if cache == "16":
        st["kc"], st["vc"] = (torch.randn(NB, bs, Hkv, d, generator=gen, device="cuda").to(dt) for _ in range(2))
    else:
        st["kc"], st["vc"] = (torch.randint(0, 120, (NB, bs, Hkv, d), generator=gen, device="cuda").to(torch.uint8)
                              for _ in range(2))
        shape = (Hkv,) if cache == "fp8" else (NB, Hkv)
        st["ks"], st["vs"] = (torch.rand(shape, generator=gen, device="cuda") * 0.02 + 0.005 for _ in range(2))
    st["slots"] = torch.randperm(NB * bs, generator=gen, device="cuda")[:T].contiguous()
    st["pos"] = torch.randint(0, case.get("far", 1000), (axes, T), generator=gen, device="cuda").to(torch.int32)
    st["inv"] = 10000.0 ** (-torch.arange(r // 2, dtype=torch.float64, device="cuda") / (r // 2))
    st["inv"] = st["inv"].float()
    st["axis"] = torch.randint(0, axes, (r // 2,), generator=gen, device="cuda").to(torch.int32)
    return st


def call(P, st, out, interleaved, **over):
    a = dict(st, **over)
    return P.rope_reshape_and_cache(out, a["q"], a["k"], a["v"], a["kc"], a["vc"], a["slots"], a["pos"], a["inv"],
                                    a["axis"], interleaved=interleaved, k_scale=a["ks"], v_scale=a["vs"])


def check(st, before, out, interleaved):
    kc0, vc0 = before
    ref, size = rotate(st["q"], st["pos"], st["inv"], st["axis"], interleaved)
    err = (out.double() - ref).abs()
    assert bool((err <= half_step(st["dt"]) * ref.abs() + SLACK * size + 2.0 ** -25).all()), float(err.max())
    bs = st["kc"].shape[1]
    ok = (st["slots"] >= 0) & (st["slots"] < st["kc"].shape[0] * bs)
    slots = st["slots"][ok]
    blk, off = slots // bs, slots % bs
    kref, ksize = rotate(st["k"][ok], st["pos"][:, ok], st["inv"], st["axis"], interleaved)
    touched = torch.zeros(st["kc"].shape[:2], dtype=torch.bool, device="cuda")
    touched[blk, off] = True
    for now, was in ((st["kc"], kc0), (st["vc"], vc0)):
        assert torch.equal(now[~touched].view(torch.uint8), was[~touched].view(torch.uint8))
    if st["cache"] == "16":
        assert torch.equal(st["vc"][blk, off], st["v"][ok])
        kerr = (st["kc"][blk, off].double() - kref).abs()
        assert bool((kerr <= half_step(st["dt"]) * kref.abs() + SLACK * ksize + 2.0 ** -25).all()), float(kerr.max())
        return
    ks, vs = (x[None, :, None] if x.dim() == 1 else x[blk][:, :, None] for x in (st["ks"], st["vs"]))
    codes = (st["v"][ok].float() / vs).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(st["vc"][blk, off], codes.view(torch.uint8))
    got = st["kc"][blk, off].view(torch.float8_e4m3fn).double()
    want = (kref / ks.double()).clamp(-448, 448)
    slack = half_step(torch.float8_e4m3fn) * want.abs() + 2.0 ** -10 + SLACK * ksize / ks.double()
    # below the normal range (2^-6) a step is 2^-9, half of it 2^-10
    slack = torch.where(want.abs() > 2.0 ** -5, slack - 2.0 ** -10, slack)
    assert bool(((got - want).abs() <= slack).all()), float((got - want).abs().max())


CASES = [
    dict(T=1, H=1, Hkv=1, d=64, r=64, axes=1, bs=8),
    dict(T=7, H=8, Hkv=2, d=128, r=128, axes=3, bs=16, dtype="f16"),
    dict(T=33, H=12, Hkv=4, d=128, r=32, axes=2, bs=8, il=True),
    dict(T=130, H=32, Hkv=32, d=64, r=16, axes=1, bs=64, far=1000000),
    dict(T=65, H=64, Hkv=1, d=128, r=64, axes=5, bs=32, dtype="f16", il=True, fused=True, far=2 ** 31 - 1),
    dict(T=19, H=5, Hkv=5, d=80, r=48, axes=3, bs=4, fused=True),
    dict(T=40, H=8, Hkv=8, d=128, r=128, axes=3, bs=16, cache="fp8", far=900000),
    dict(T=41, H=16, Hkv=2, d=128, r=64, axes=2, bs=8, cache="fp8_block", il=True, dtype="f16"),
    dict(T=9, H=2, Hkv=2, d=520, r=512, axes=3, bs=16, cache="fp8", dtype="f16", fused=True),
    dict(T=5, H=3, Hkv=3, d=16, r=16, axes=1, bs=8),
    dict(T=5, H=70, Hkv=1, d=16, r=16, axes=2, bs=8, il=True),
    dict(T=3, H=2, Hkv=1, d=8192, r=512, axes=2, bs=2),
    dict(T=3000, H=4, Hkv=2, d=128, r=128, axes=3, bs=16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "_".join(f"{k}{v}" for k, v in c.items()))
def test_rope_against_the_formula(P, case):
    st = make(case, seed=len(str(case)))
    before = st["kc"].clone(), st["vc"].clone()
    out = torch.full(st["q"].shape, float("nan"), dtype=st["dt"], device="cuda")
    call(P, st, out, case.get("il", False))
    check(st, before, out, case.get("il", False))


@pytest.mark.parametrize("il", [False, True])
def test_in_place_padding_negative_positions_and_foreign_axes(P, il):
    st = make(dict(T=23, H=4, Hkv=2, d=64, r=64, axes=2, bs=8, fused=True), seed=5)
    st["slots"][::4] = -1                        # padding
    st["slots"][5] = st["kc"].shape[0] * 8       # past the pool
    st["slots"][6] = 2 ** 40
    st["pos"] -= 500
    st["axis"][3] = 2                            # no such axis: not turned
    st["axis"][4] = -1
    before = st["kc"].clone(), st["vc"].clone()
    q0 = st["q"].clone()
    call(P, st, st["q"], il)                     # turned in place
    out = st["q"].clone()
    check(dict(st, q=q0), before, out, il)


def test_one_axis_equals_the_ordinary_embedding_and_zero_position_is_the_identity(P):
    st = make(dict(T=12, H=4, Hkv=4, d=128, r=128, axes=1, bs=16), seed=9)
    st["pos"].zero_()
    out = torch.empty_like(st["q"])
    call(P, st, out, False)
    assert torch.equal(out, st["q"])
    bs = 16
    assert torch.equal(st["kc"][st["slots"] // bs, st["slots"] % bs], st["k"])


def test_empty_batch_and_another_stream(P):
    st = make(dict(T=6, H=2, Hkv=2, d=64, r=64, axes=1, bs=8), seed=3)
    empty = {k: st[k][:0] for k in ("q", "k", "v", "slots")}
    call(P, st, torch.empty_like(empty["q"]), False, pos=st["pos"][:, :0].contiguous(), **empty)
    before = st["kc"].clone(), st["vc"].clone()
    out = torch.empty_like(st["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(P, st, out, False)
    torch.cuda.current_stream().wait_stream(side)
    check(st, before, out, False)


def test_graph_replay_follows_new_inputs(P):
    st = make(dict(T=10, H=4, Hkv=2, d=128, r=128, axes=3, bs=16), seed=4)
    out = torch.empty_like(st["q"])
    call(P, st, out, False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(P, st, out, False)
    st["q"].normal_()
    st["pos"].add_(77)
    before = st["kc"].clone(), st["vc"].clone()
    g.replay()
    check(st, before, out, False)
