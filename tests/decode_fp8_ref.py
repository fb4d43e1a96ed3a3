"""The operators on an 8-bit cache and on 4-bit weights from their definitions, in 64 bits on the CPU,
and the bounds the GPU tests hold the kernels to (decode_ref.py has the symbols: U, TINY, E)."""
from __future__ import annotations

import math

import torch

from decode_ref import E, TINY, U, assert_close  # noqa: F401

E4M3 = torch.float8_e4m3fn


def nearest_e4m3(y):
    """The nearest number of E4M3 (ties to even, no overflow in these tests); NaN for a non-finite."""
    exponent = torch.frexp(y.abs())[1] - 1                    # floor(log2 |y|)
    step = torch.ldexp(torch.ones_like(y), exponent.clamp(min=-6) - 3)
    r = torch.round(y / step) * step
    assert not (r.abs()[y.isfinite()] > 448).any()
    return torch.where(y.isfinite(), r, torch.full_like(y, math.nan))


def need_of(x):
    """The least e >= 0 with max |x| <= 448 * 2^(e - 127), over the finite elements of x."""
    top = float(x[x.isfinite()].abs().max()) if x.isfinite().any() else 0.0
    e = 0
    while top > 448 * 2.0 ** (e - 127):
        e += 1
    return e


def quantize_cache(x, codes, scale, slots):
    """(codes as values, scale) after tokens' x [tokens, h, d] go to the cache codes [pages, page, h,
    d] with scale [pages, blocks, h]: block by block, head by head."""
    x = x.double().cpu()
    pages, page, h, d = codes.shape
    block = page // scale.shape[1]
    c = codes.float().double().cpu().reshape(-1, block, h, d).clone()
    s = scale.cpu().long().reshape(-1, h).clone()
    by_block = {}
    for t, slot in enumerate(slots.tolist()):
        if 0 <= slot < pages * page:
            by_block.setdefault(slot // block, []).append((slot % block, t))
    for b, tokens in by_block.items():
        first, last = tokens[0][0], tokens[-1][0]
        assert [o for o, _ in tokens] == list(range(first, last + 1))
        for j in range(h):
            new = x[[t for _, t in tokens], j]
            e = need_of(new)
            if first:
                e = max(e, int(s[b, j]))
                c[b, :, j] = nearest_e4m3(c[b, :, j] * 2.0 ** (int(s[b, j]) - e))
            c[b, first:last + 1, j] = nearest_e4m3(new * 2.0 ** (127 - e))
            s[b, j] = e
    return c.view(codes.shape), s.to(torch.uint8).view(scale.shape)


def values(codes, scale):
    """What a cache holds, in 64 bits."""
    block = codes.shape[1] // scale.shape[1]
    e = scale.cpu().long().repeat_interleave(block, 1)[..., None]
    by = torch.where(e == 255, math.nan, torch.ldexp(torch.ones_like(e, dtype=torch.float64), e - 127))
    return codes.view(E4M3).float().double().cpu() * by


def paged_attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale, window, sinks):
    """(o, lse, o's bound, lse's bound).  A score's error is at most es: (d + 4) 4 e sum |q K| scale of
    the tensor core's fp32 sums, 2^-38 of the largest element of q for each of d products (bfloat16
    queries that become float16), and 8 e of the score itself.  A weight's relative error is that, and
    2^-18 for the exponentials (2^-22 each, one more where the running maximum grows), its two pieces
    (2^-22) and the sums' fp32 roundings, of which there is one more for every slice of 16 tokens at
    least; what its pieces leave out may also be 2^-40 of the largest scale's weight."""
    dt = q.dtype
    q = q.double().cpu()
    k, v = values(k_cache, k_scale), values(v_cache, v_scale)
    n, h_q, d = q.shape
    page, h_kv = k.shape[1], k.shape[2]
    o = torch.zeros(n, h_q, d, dtype=torch.float64)
    lse = torch.full((n, h_q), -math.inf, dtype=torch.float64)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    for i, length in enumerate(lens.tolist()):
        if not 0 < length <= table.shape[1] * page:
            continue
        start = max(0, length - window) if window else 0
        at = torch.cat([torch.arange(min(sinks, start)), torch.arange(start, length)])
        rows = table[i].cpu().long()[at // page]
        for m in range(h_q):
            kv = m // (h_q // h_kv)
            K, V = k[rows, at % page, kv], v[rows, at % page, kv]
            x = scale * (K @ q[i, m])
            es = float((abs(scale) * (K.abs() @ q[i, m].abs())).max()) * (d + 4) * 4 * E + \
                8 * E * float(x.abs().max())
            if dt == torch.bfloat16:
                es += abs(scale) * 2.0 ** -38 * float(q[i, m].abs().max()) * float(K.abs().sum(1).max())
            lse[i, m] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[i, m])
            o[i, m] = p @ V
            rel = 2 * es + 2.0 ** -18 + len(at) / 16 * E
            ob[i, m] = rel * (p @ V.abs()) + 2.0 ** -40 * 448 * len(at) * \
                2.0 ** (float(v_scale.cpu()[rows, at % page // (page // v_scale.shape[1]), kv].max()) - 127)
            lb[i, m] = es + 2.0 ** -18 + len(at) / 16 * E + 4 * E * abs(float(lse[i, m]))
    return o, lse, ob, lb


def linear_w4(x, codes, scales, group, zeros=None, bias=None, activation="none"):
    """(y, y's bound before its rounding): products are exact, and of the fp32 sums of a group's
    columns and of the groups each term may take a unit roundoff of the tensor core (2 e) a time, some
    16 more for the scaling, the parts and the bias; GELU's slope is below 1.13 and its error 2^-20."""
    x = x.double().cpu()
    pairs = codes.cpu().long()
    n, k = codes.shape[0], 2 * codes.shape[1]
    code = torch.stack([pairs % 16, pairs // 16], -1).view(n, k).double()
    at = torch.arange(k) // group
    z = 8.0 if zeros is None else zeros.cpu().double()[:, at]
    w = (code - z) * scales.cpu().double()[:, at]
    y = x @ w.T
    bound = (min(group, k) + scales.shape[1] + 16) * 2 * E * (x.abs() @ w.abs().T)
    if bias is not None:
        y = y + bias.double().cpu()
        bound = bound + 2 * E * bias.double().cpu().abs()
    if activation == "relu":
        y = torch.where(y < 0, torch.zeros_like(y), y)
    elif activation == "gelu":
        y = y * torch.special.ndtr(y)
        bound = 1.13 * bound + 2.0 ** -20 * y.abs()
    return y, bound


def paged_attention_by_weight(q, c, table, lens, scale):
    """(o, lse, o's bound, lse's bound) as paged_attention gives them for all of a sequence's tokens, but that
    what the pieces of a weight leave out is held to the weights: they keep 2^-25 where the slice's largest
    product of weight and scale stands for 2^7 at least (2^15, but that scales up to 2^8 apart are left as they
    are), so a token's part is off by 2^-32 of the largest such product, times its code.  (c: the four tensors of
    a cache.)"""
    dt = q.dtype
    q = q.double().cpu()
    k, v = values(c["k_cache"], c["k_scale"]), values(c["v_cache"], c["v_scale"])
    page, h_kv = k.shape[1], k.shape[2]
    block = page // c["v_scale"].shape[1]
    o = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    for i, length in enumerate(lens.tolist()):
        at = torch.arange(length)
        rows = table[i].cpu().long()[at // page]
        for m in range(q.shape[1]):
            kv = m // (q.shape[1] // h_kv)
            K, V = k[rows, at % page, kv], v[rows, at % page, kv]
            by = torch.ldexp(torch.ones(length, dtype=torch.float64),
                             c["v_scale"].cpu().long()[rows, at % page // block, kv] - 127)
            x = scale * (K @ q[i, m])
            es = float((abs(scale) * (K.abs() @ q[i, m].abs())).max()) * (q.shape[2] + 4) * 4 * E + \
                8 * E * float(x.abs().max())
            if dt == torch.bfloat16:
                es += abs(scale) * 2.0 ** -38 * float(q[i, m].abs().max()) * float(K.abs().sum(1).max())
            lse[i, m] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[i, m])
            o[i, m] = p @ V
            rel = 2 * es + 2.0 ** -18 + length / 16 * E
            ob[i, m] = rel * (p @ V.abs()) + 2.0 ** -32 * 448 * length * float((p * by).max())
            lb[i, m] = es + 2.0 ** -18 + length / 16 * E + 4 * E * abs(float(lse[i, m]))
    return o, lse, ob, lb
