"""Plain 64-bit forms of the positional, scoring, eviction and cross-attention operators, and the error
bounds their tests hold the kernels to.

Bounds are derived, not fitted. u = 2^-24 is half a step of fp32 relative to the value, h(T) = eps(T) / 2
that of a type T.
  score z = log2(e) scale q.k in fp32:  |dz| <= (d + 4) 2u A + rounding of the operands, A = max sum_i |q_i k_i|
      log2(e) scale (each of d products' additions may truncate, 2u; FP8 caches on the tensor cores take a
      bf16 query as f16, off by 2^-25 below f16's normal range; per-block scales may multiply the keys in f16,
      h(f16) A).
  weight p = 2^(z - lse):  rel(p) <= ln2 (2 |dz| + 4u (max|z| + log2 L)) + 8u (two exp2, 2u each, and the
      sum's) + L u (the sum's additions).
  output:  h(T_P) (sum p|v| + |out|) for the weights' rounding (the sum may take rounded or unrounded
      weights), + (rel(p) + 2 L u) sum p|v|, + h(out) |out|; f16 weights below the normal range: 2^-24 L max|v|;
      per-block value scales: 2 h(f16) sum p|v|.
  score sums:  rel(p) per term, u per addition.
"""
import math

import torch

U = 2.0 ** -24
LOG2E = math.log2(math.e)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def half_step(t):
    return torch.finfo(t).eps / 2


def make_pool(gen, num_blocks, block_size, kv_heads, d, dtype, cache, device="cuda"):
    """(key_cache, value_cache, k_scale, v_scale, keys and values in 64 bits as the codes stand for them).
    cache: "16", "fp8" (per-kv-head scales) or "fp8_block"."""
    out, scales, values = [], [], []
    for _ in range(2):
        x = torch.randn(num_blocks, block_size, kv_heads, d, generator=gen, device=device)
        if cache == "16":
            c = x.to(dtype)
            out.append(c)
            scales.append(None)
            values.append(c.double())
            continue
        shape = (kv_heads,) if cache == "fp8" else (num_blocks, kv_heads)
        s = torch.rand(shape, generator=gen, device=device) * 0.01 + 0.01
        sb = s[None, None, :, None] if cache == "fp8" else s[:, None, :, None]
        c = (x / sb).clamp(-448, 448).to(torch.float8_e4m3fn)
        out.append(c.view(torch.uint8))
        scales.append(s)
        values.append(c.double() * sb.double())
    return out[0], out[1], scales[0], scales[1], values[0], values[1]


def scatter_tables(gen, lens, block_size, extra=3, junk=None, device="cuda"):
    """Block tables over shuffled blocks; entries past a sequence's blocks hold `junk` (or block ids)."""
    counts = [-(-n // block_size) for n in lens]
    total = sum(counts)
    order = torch.randperm(total + extra, generator=gen, device=device).to(torch.int32)
    width = max(1, max(counts)) + 1
    table = torch.full((len(lens), width), int(order[-1]) if junk is None else junk, dtype=torch.int32, device=device)
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = order[at:at + c]
        at += c
    return table, total + extra


def gather(values, table, s, length, block_size):
    """[length, kv_heads, d] of sequence s."""
    t = torch.arange(length, device=values.device)
    return values[table[s].long()[t // block_size], t % block_size]


def poison_unused(caches, table, lens, block_size):
    """Every cache slot that no sequence uses becomes NaN (16-bit NaN, or the E4M3 NaN code)."""
    nb, bs = caches[0].shape[:2]
    used = torch.zeros(nb, bs, dtype=torch.bool, device=caches[0].device)
    for s, n in enumerate(lens):
        t = torch.arange(n, device=used.device)
        used[table[s].long()[t // block_size], t % block_size] = True
    for c in caches:
        c[~used] = 0x7F if c.dtype == torch.uint8 else float("nan")


def attention(query, keys, values, rows, scale, causal, counted, info):
    """One sequence. query [n, H, d], keys/values [L, Hkv, d] (64 bits). Returns out, its bound, the weights
    summed over the last `counted` rows and each kv head's query heads [Hkv, L], and their relative bound."""
    n, H, d = query.shape
    L, Hkv, _ = keys.shape
    dtype, cache = info
    g = H // Hkv
    q = query.double().view(n, Hkv, g, d)
    z = torch.einsum("nkgd,lkd->nkgl", q, keys) * (scale * LOG2E)
    a = float(torch.einsum("nkgd,lkd->nkgl", q.abs(), keys.abs()).max()) * scale * LOG2E if L else 0.0
    if causal:
        pos = torch.arange(L - n, L, device=z.device)
        z = z.masked_fill((torch.arange(L, device=z.device) > pos[:, None])[:, None, None], -math.inf)
    zmax = float(z[z.isfinite()].abs().max()) if L else 0.0
    p = torch.softmax(z * math.log(2.0), -1)
    out = torch.einsum("nkgl,lkd->nkgd", p, values).reshape(n, H, d)
    mass = torch.einsum("nkgl,lkd->nkgd", p, values.abs()).reshape(n, H, d)
    dz = (d + 4) * 2 * U * a
    mma = torch.float16 if cache != "16" else dtype
    vmax = float(values.abs().max()) if L else 0.0
    kmax = float(keys.abs().max()) if L else 0.0
    if cache != "16":
        dz += d * 2.0 ** -25 * kmax * scale * LOG2E
    if cache == "fp8_block":
        dz += half_step(torch.float16) * a
    rel = math.log(2) * (2 * dz + 4 * U * (zmax + math.log2(max(L, 2)))) + 8 * U + L * U
    bound = half_step(mma) * (mass + out.abs()) + (rel + 2 * L * U) * mass + half_step(dtype) * out.abs()
    if mma == torch.float16:
        bound = bound + 2.0 ** -24 * L * vmax
    if cache == "fp8_block":
        bound = bound + 2 * half_step(torch.float16) * mass
    bound = bound + 2.0 ** -24  # the least step of an f16 output
    return out, bound, p[n - counted:].sum((0, 2)), rel + counted * g * U


def rotate(x, positions, inv_freq, freq_axis, interleaved):
    """x [T, heads, d] by multi-axis rotary positions; 64 bits. Also |a| + |b| of each element's pair."""
    x = x.double()
    half = inv_freq.numel()
    r = 2 * half
    ok = (freq_axis >= 0) & (freq_axis < positions.shape[0])
    pos = positions.double()[torch.where(ok, freq_axis, 0).long()] * ok[:, None]
    ang = (pos * inv_freq.double()[:, None]).t()[:, None]
    c, s = ang.cos(), ang.sin()
    lo = slice(0, r, 2) if interleaved else slice(0, half)
    hi = slice(1, r, 2) if interleaved else slice(half, r)
    y, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    size[..., lo] = size[..., hi] = a.abs() + b.abs()
    return y, size


def evict(scores, length, budget, sink, recent):
    """Kept token indices (rising) of one row of scores, per the definition."""
    if length <= budget:
        return list(range(length))
    w = [-math.inf if x != x else x for x in scores.tolist()]
    ends = set(range(sink)) | set(range(length - recent, length))
    order = sorted((t for t in range(length) if t not in ends), key=lambda t: (-w[t], t))
    return sorted(ends | set(order[:budget - len(ends)]))
