"""The decode-step operators from their definitions, in 64 bits on the CPU, and the bounds the GPU
tests hold the kernels to.

Each bound is derived from the kernels' arithmetic: U is the 16-bit type's unit roundoff (half an
ulp: 2^-8 bfloat16, 2^-11 float16), TINY the 16-bit type's rounding error where it is subnormal, and
E = 2^-24 the roundoff of fp32, of which a sum of m terms takes at most m per unit of the sum of
magnitudes."""
from __future__ import annotations

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
E = 2.0 ** -24


def gdn_step(q, k, v, alpha, beta, state, scale, slots=None):
    """(o, state, o's bound, state's bound).  With A the largest row norm of a state or value on
    the way, keys of norm at most 1 and |beta| <= 1, a token adds at most 160 e A to a row (two sums
    of 128 terms and a handful of roundings)."""
    q, k, v, alpha, beta = (x.double().cpu() for x in (q, k, v, alpha, beta))
    state = state.double().cpu().clone()
    n, tokens, h_q, d = q.shape
    h_k, h_v = k.shape[2], v.shape[2]
    h_o = max(h_q, h_v)
    o = torch.zeros(n, tokens, h_o, d, dtype=torch.float64)
    ob, sb = torch.zeros_like(o), torch.zeros_like(state)
    slots = range(n) if slots is None else slots.tolist()
    for i, slot in enumerate(slots):
        if not 0 <= slot < state.shape[0]:
            continue
        for j in range(h_v):
            S = state[slot, j]
            kj = j // (h_v // h_k)
            if h_q == h_k:
                heads = [(kj, j)]
            else:
                heads = [(m, m) for m in range(h_q) if m // (h_q // h_v) == j]
            A = max(float(S.norm(dim=1).max()), 1e-30)
            for t in range(tokens):
                S = alpha[i, t, j] * S
                u = beta[i, t, j] * (v[i, t, j] - S @ k[i, t, kj])
                S = S + torch.outer(u, k[i, t, kj])
                A = max(A, float(S.norm(dim=1).max()), float(v[i, t, j].abs().max()))
                for m, to in heads:
                    o[i, t, to] = scale * (S @ q[i, t, m])
                    ob[i, t, to] = abs(scale) * float(q[i, t, m].norm()) * (t + 2) * 160 * E * A
            state[slot, j] = S
            sb[slot, j] = (tokens + 1) * 160 * E * A
    return o, state, ob, sb


def qk_norm_rope(x, w, norm, eps, positions, table, sections, interleaved):
    """(y, y's bound before the rounding to 16 bits): relative d / 2 + 16 roundings on each of the
    two elements that a rotation mixes."""
    x = x.double().cpu()
    d = x.shape[-1]
    if norm == "rms":
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    elif norm == "l2":
        x = x / (x.pow(2).sum(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        x = x * w.double().cpu()
    big = x.abs().clone()
    if table is not None:
        half = table.shape[1] // 2
        pos = positions.cpu().long().reshape(-1, x.shape[0])
        axis = [a for a, s in enumerate(sections or [half]) for _ in range(s)]
        y = x.clone()
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, half + j)
            c, s = (table[pos[axis[j]], half * f + j].double().cpu()[:, None] for f in (0, 1))
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., b] * c + x[..., a] * s
            big[..., a] = big[..., b] = x[..., a].abs() + x[..., b].abs()
        x = y
    return x, (d / 2 + 16) * E * big


def paged_attention(q, k_cache, v_cache, table, lens, scale, window):
    """(o, lse, o's bound, lse's bound).  A score's error is at most es = (d + 4) 4 e sum |q K|
    scale (the tensor core's fp32 sums) plus 8 e of the score itself; a weight's relative error is
    that, 2^-20 for the exponentials, and at most U / 2 for the 16-bit pieces that carry it (float16's,
    scaled by 2^15, lose at most 2^-40 of the largest weight); o mixes them with |V|."""
    dt = q.dtype
    q, kc, vc = (x.double().cpu() for x in (q, k_cache, v_cache))
    n, h_q, d = q.shape
    page, h_kv = kc.shape[1], kc.shape[2]
    o = torch.zeros(n, h_q, d, dtype=torch.float64)
    lse = torch.full((n, h_q), float("-inf"), dtype=torch.float64)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    for i, length in enumerate(lens.tolist()):
        if not 0 < length <= table.shape[1] * page:
            continue
        at = torch.arange(max(0, length - window) if window else 0, length)
        rows = table[i].cpu().long()[at // page]
        for m in range(h_q):
            kv = m // (h_q // h_kv)
            K, V = kc[rows, at % page, kv], vc[rows, at % page, kv]
            x = scale * (K @ q[i, m])
            es = float((abs(scale) * (K.abs() @ q[i, m].abs())).max()) * (d + 4) * 4 * E + \
                8 * E * float(x.abs().max())
            lse[i, m] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[i, m])
            o[i, m] = p @ V
            small = 2.0 ** -40 * float(p.max()) if dt == torch.float16 else 0.0
            ob[i, m] = (2 * es + 2.0 ** -20 + U[dt] / 2) * (p @ V.abs()) + small * V.abs().sum(0)
            lb[i, m] = es + 2.0 ** -20 + 4 * E * abs(float(lse[i, m]))
    return o, lse, ob, lb


def assert_close(got, ref, bound, where):
    """got (16 or 32 bits) within its own rounding of the reference, plus ``bound``."""
    u, tiny = U.get(got.dtype, 2 * E), TINY.get(got.dtype, 0.0)
    x = got.double().cpu()
    assert x.shape == ref.shape, where
    inf = ref == float("-inf")
    assert torch.equal(x == float("-inf"), inf), f"{where}: infinities differ"
    ref, x, bound = ref.masked_fill(inf, 0), x.masked_fill(inf, 0), bound.masked_fill(inf, 0)
    err, tol = (x - ref).abs(), u * ref.abs() + tiny + bound
    bad = ~(err <= tol)
    assert not bad.any(), (f"{where}: {int(bad.sum())} of {bad.numel()} out of bound, worst err/tol "
                           f"{float((err / tol.clamp_min(1e-300)).nan_to_num(1e9).max()):.3f}, "
                           f"first at {bad.nonzero()[0].tolist()}")
