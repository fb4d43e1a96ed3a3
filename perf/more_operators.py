"""Cases of the decode-step operators on few bits: the write to a paged cache of E4M3 codes with one
E8M0 scale for each block of tokens and head, the reading back, the attention of one new token over
that cache (with a sliding window and first tokens that stay visible), and the linear layer with
4-bit weights and a scale for each group of them.

``run`` computes each operator in elementary torch operations in 32 bits (``own`` false) or through
the package's entry points (``own`` true); ``exact`` computes the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # -- the write to the cache
        # one new token of each of 20 conversations: most go on in a block that older tokens began
        dict(name="write_20x1", op="write", dtype="bf16", n=20, each=1, h=8, d=128, page=16,
             block=16),
        # a prompt of 32768 tokens
        dict(name="write_1x32768", op="write", dtype="bf16", n=1, each=32768, h=8, d=128, page=64,
             block=16),
        # short ragged prompts, wide heads, blocks of an odd size
        dict(name="write_9x200_d256", op="write", dtype="fp16", n=9, each=200, h=2, d=256, page=60,
             block=20),
        # -- the reading back
        # a short conversation's keys and values, narrow heads, blocks of an odd size
        dict(name="read_500_d64", op="read", dtype="fp16", tokens=500, h=12, d=64, page=20, block=10),
        # a long document's
        dict(name="read_200001_d256", op="read", dtype="bf16", tokens=200001, h=2, d=256, page=64,
             block=64),
        # -- attention over the cache
        # one short conversation
        dict(name="attn_1x500", op="attn", dtype="bf16", n=1, longest=500, h_q=32, h_kv=8, d=128,
             page=16, block=16, window=0, sinks=0),
        # a full server: lengths from nothing to 8192
        dict(name="attn_64x8192_ragged", op="attn", dtype="bf16", n=64, longest=8192, h_q=32,
             h_kv=8, d=128, page=16, block=16, window=0, sinks=0),
        # one very long document, wide heads
        dict(name="attn_1x200001_d256", op="attn", dtype="bf16", n=1, longest=200001, h_q=16,
             h_kv=2, d=256, page=64, block=64, window=0, sinks=0),
        # a sliding window and four first tokens, one key head per query head, odd pages and blocks
        dict(name="attn_37x5000_sinks", op="attn", dtype="fp16", n=37, longest=5000, h_q=12,
             h_kv=12, d=64, page=20, block=10, window=1000, sinks=4),
        # -- the linear layer
        # one user's token through an attention projection
        dict(name="w4_1x4096x4096", op="w4", dtype="bf16", m=1, n=4096, k=4096, group=128,
             zeros=False, bias=False, act="none"),
        # a few tokens, an odd number of outputs, small groups
        dict(name="w4_7x5000x1024", op="w4", dtype="fp16", m=7, n=5000, k=1024, group=32,
             zeros=True, bias=True, act="gelu"),
        # a server's batch through the layer that widens
        dict(name="w4_48x14336x4096", op="w4", dtype="bf16", m=48, n=14336, k=4096, group=128,
             zeros=True, bias=False, act="none"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _paging(rng):
    block = rng.choice([1, 8, 10, 16, 16, 16, 20, 32, 64])
    return dict(page=block * rng.choice([1, 1, 2, 4]), block=block)


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "w4", "w4"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "w4":
        k = 32 * _log(rng, 8, 448)
        n = _log(rng, 256, 16384)
        m = _log(rng, 1, max(1, min(64, 48 * 14336 * 4096 // (n * k))))
        return dict(op=op, dtype=dtype, m=m, n=n, k=k, group=rng.choice([32, 64, 128, 128, 160]),
                    zeros=rng.random() < 0.5, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "none", "relu", "gelu"]))
    d = rng.choice([64, 128, 128, 256])
    if op in ("write", "read"):
        h = rng.choice([1, 2, 4, 8, 12])
        most = max(64, 32768 * 8 * 128 // (h * d))
        if op == "read":
            return dict(op=op, dtype=dtype, tokens=_log(rng, 1, min(200000, 2 * most)), h=h, d=d,
                        **_paging(rng))
        n = _log(rng, 1, 256)
        each = rng.choice([1, _log(rng, 2, max(2, most // n))])
        return dict(op=op, dtype=dtype, n=n, each=each, h=h, d=d, **_paging(rng))
    h_kv = rng.choice([1, 2, 4, 8])
    h_q = h_kv * rng.choice([1, 3, 4, 8, 16])
    n = _log(rng, 1, 200)
    most = max(64, min(200000, 64 * 8192 * 8 * 128 // (2 * n * h_kv * d)))
    longest = _log(rng, 40, most)
    window = rng.choice([0, 0, 0, max(1, longest // 3)])
    return dict(op=op, dtype=dtype, n=n, longest=longest, h_q=h_q, h_kv=h_kv, d=d, window=window,
                sinks=rng.choice([0, 1, 4, 21]) if window else 0, **_paging(rng))


# ---- inputs ------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _package():
    import blackwell_tensor_core_fp16_gb300 as package
    return package


def prepare(case, seed):
    g = _generator(seed)
    return {"case": case, **{"write": _prepare_write, "read": _prepare_read, "attn": _prepare_attn,
                             "w4": _prepare_w4}[case["op"]](case, g)}


def _power(e):
    """2^(e - 127) in float32, for whole e in 0 .. 254."""
    e = e.to(torch.int32)
    return torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _need(top):
    """The least e >= 0 with top <= 448 * 2^(e - 127), for finite top >= 0."""
    m, x = torch.frexp(top)                     # top = m * 2^x, 0.5 <= m < 1
    e = 127 + x - 9 + (m > 0.875).to(x.dtype)   # 448 = 0.875 * 2^9
    return torch.where(top > 0, e, torch.zeros_like(e)).clamp(min=0)


def _pool(g, pages, page, block, h, d):
    """A pool of pages whose blocks hold normal values of a size of their own, quantised: codes
    [pages, page, h, d] and scales [pages, page // block, h]."""
    codes = torch.empty(pages, page, h, d, dtype=E4M3, device="cuda")
    scale = torch.empty(pages, page // block, h, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (page * h * d))
    for p in range(0, pages, step):             # in parts: the pool may be large
        x = _normal(g, min(step, pages - p), page // block, block, h, d)
        x *= torch.exp2(_normal(g, *x.shape[:2], 1, h, 1))
        e = _need(x.abs().amax((2, 4)))
        codes[p:p + step] = (x * _power(254 - e)[:, :, None, :, None]).to(E4M3).flatten(1, 2)
        scale[p:p + step] = e.to(torch.uint8)
    return codes, scale


def _pages(g, used, width, total=None):
    """A page table in which each sequence has `used` pages of a pool of `total`, in no order, and
    the pool's size (None: two pages more than are used)."""
    total = int(used.sum()) + 2 if total is None else total
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = (used.cumsum(0) - used)[:, None] + torch.arange(width, device="cuda")
    table = torch.where(torch.arange(width, device="cuda") < used[:, None],
                        order[at.clamp(max=total - 1)], torch.zeros_like(order[:1]))
    return table.contiguous(), total


def _prepare_write(c, g):
    """New tokens of n sequences, one after the other, as the norm leaves keys and the projection
    values, and the cache with what older tokens left in it.  One sequence starts anew, and so does
    one with a long prompt; some tokens are larger than those before them."""
    n, page, h, d, dt = c["n"], c["page"], c["h"], c["d"], DTYPES[c["dtype"]]
    if c["each"] > 1 and n > 1:
        new = torch.randint(1, c["each"] + 1, (n,), generator=g, device="cuda")
        new[0] = c["each"]
    else:
        new = torch.full((n,), c["each"], device="cuda")
    before = torch.randint(0, 3 * page, (n,), generator=g, device="cuda")
    before[0] = 0 if c["each"] > 1 else before[0]
    width = (3 * page + c["each"] + page - 1) // page
    table, total = _pages(g, (before + new + page - 1) // page, width, n * width + 2)
    t = int(new.sum())
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), new)
    pos = before[seq] + torch.arange(t, device="cuda") - (new.cumsum(0) - new)[seq]
    slots = (table[seq, pos // page] * page + pos % page).to(torch.int32)
    packed = _normal(g, t, 2 * h, d) * torch.exp2(1.5 * _normal(g, t, 1, 1))
    packed = packed.to(dt)
    kc, ks = _pool(g, total, page, c["block"], h, d)
    vc, vs = _pool(g, total, page, c["block"], h, d)
    return {"k": packed[:, :h], "v": packed[:, h:], "k_cache": kc, "v_cache": vc, "k_scale": ks,
            "v_scale": vs, "slots": slots}


def _prepare_read(c, g):
    """One sequence's places in the pool."""
    t, page = c["tokens"], c["page"]
    used = torch.full((1,), -(-t // page), device="cuda")
    table, total = _pages(g, used, int(used))
    pos = torch.arange(t, device="cuda")
    kc, ks = _pool(g, total, page, c["block"], c["h"], c["d"])
    vc, vs = _pool(g, total, page, c["block"], c["h"], c["d"])
    return {"k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs,
            "slots": (table[0, pos // page] * page + pos % page).to(torch.int32)}


def _prepare_attn(c, g):
    """One query per sequence, the pool, and lengths between nothing and the longest; one sequence
    alone has the longest."""
    n, d, page = c["n"], c["d"], c["page"]
    if n > 1:
        lens = torch.randint(0, c["longest"] + 1, (n,), generator=g, device="cuda")
        lens[0], lens[n // 2] = c["longest"], 0
    else:
        lens = torch.full((1,), c["longest"], device="cuda")
    table, total = _pages(g, (lens + page - 1) // page, -(-c["longest"] // page))
    kc, ks = _pool(g, total, page, c["block"], c["h_kv"], d)
    vc, vs = _pool(g, total, page, c["block"], c["h_kv"], d)
    s = {"q": _normal(g, n, c["h_q"], d).to(DTYPES[c["dtype"]]), "k_cache": kc, "v_cache": vc,
         "k_scale": ks, "v_scale": vs, "table": table, "lens": lens.to(torch.int32),
         "scale": d ** -0.5, "window": c["window"] or None, "sinks": c["sinks"]}
    if own:
        s["workspace"] = _package().paged_attention_fp8_workspace(c["h_q"], c["h_kv"], d, "cuda")
    return s


def _prepare_w4(c, g):
    """Activations, the weights' codes (two a byte, the even column's in the lower half), a scale
    for each group of a row's columns, and the code that stands for zero (8 where none is kept)."""
    m, n, k, dt = c["m"], c["n"], c["k"], DTYPES[c["dtype"]]
    groups = -(-k // c["group"])
    s = {"x": _normal(g, m, k).to(dt),
         "codes": torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8),
         "scales": (0.25 * k ** -0.5 * (0.5 + torch.rand(n, groups, generator=g, device="cuda"))).to(dt),
         "zeros": None, "bias": None}
    if c["zeros"]:
        s["zeros"] = torch.randint(5, 11, (n, groups), generator=g, device="cuda", dtype=torch.uint8)
    if c["bias"]:
        s["bias"] = (0.5 * _normal(g, n)).to(dt)
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "write":
        return _own_write(s) if own else _plain_write(s)
    if op == "read":
        return _own_read(s) if own else _plain_read(s)
    if op == "attn":
        return _own_attn(s) if own else _plain_attn(s)
    return _own_w4(s) if own else _plain_w4(s)


_CACHE = ("k_cache", "v_cache", "k_scale", "v_scale")


def _own_write(s):
    _package().quantize_cache(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"],
                              s["v_scale"], s["slots"])
    return {x: s[x] for x in _CACHE}


def _plain_write(s):
    block = s["case"]["block"]
    where = s["slots"].long()
    b = where // block
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x.float()
        h = x.shape[1]
        codes, e = cache.view(-1, block, h, x.shape[2]), scale.view(-1, h)
        need = torch.zeros(e.shape, dtype=torch.int32, device=e.device)
        need.scatter_reduce_(0, b[:, None].expand(-1, h), _need(x.abs().amax(-1)).to(torch.int32),
                             "amax")
        first = torch.full_like(e[:, 0], block, dtype=torch.int64)     # offset of the first new token
        first.scatter_reduce_(0, b, where % block, "amin")
        old = torch.where((first > 0)[:, None], e.to(torch.int32), torch.zeros_like(need))
        grown = torch.maximum(old, need)
        grown = torch.where((first < block)[:, None], grown, e.to(torch.int32))
        # older codes go down by as much as their scale grows
        down = _power(127 + e.to(torch.int32) - grown)
        down = torch.where(((first > 0) & (first < block))[:, None], down, torch.ones_like(down))
        codes.copy_((codes.float() * down[:, None, :, None]).to(E4M3))
        codes.flatten(0, 1)[where] = (x * _power(254 - grown)[b][..., None]).to(E4M3)
        e.copy_(grown)
    return {x: s[x] for x in _CACHE}


def _own_read(s):
    k, v = _package().dequantize_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                       s["slots"], dtype=DTYPES[s["case"]["dtype"]])
    return {"k": k, "v": v}


def _rows(cache, scale, where):
    """The values that the cache holds at `where`, in float32."""
    block = cache.shape[1] // scale.shape[1]
    return cache.flatten(0, 1)[where].float() * _power(scale.flatten(0, 1)[where // block])[..., None]


def _plain_read(s):
    where, dt = s["slots"].long(), DTYPES[s["case"]["dtype"]]
    return {"k": _rows(s["k_cache"], s["k_scale"], where).to(dt),
            "v": _rows(s["v_cache"], s["v_scale"], where).to(dt)}


def _own_attn(s):
    o, lse = _package().paged_attention_fp8(
        s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
        scale=s["scale"], window=s["window"], sinks=s["sinks"], return_lse=True,
        workspace=s["workspace"])
    return {"o": o, "lse": lse}


def _plain_attn(s):
    page, h_kv, dt = s["k_cache"].shape[1], s["k_cache"].shape[2], s["q"].dtype
    at = torch.arange(int(s["case"]["longest"]), device="cuda")
    where = s["table"][:, at // page].long() * page + at % page
    k = _rows(s["k_cache"], s["k_scale"], where).transpose(1, 2)     # [n, h_kv, tokens, d]
    v = _rows(s["v_cache"], s["v_scale"], where).transpose(1, 2)
    lens = s["lens"][:, None]
    seen = at < lens
    if s["window"]:
        seen = seen & ((at >= lens - s["window"]) | (at < s["sinks"]))
    q = s["q"].float().unflatten(1, (h_kv, -1))
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))
    return {"o": o.flatten(1, 2).to(dt), "lse": lse.flatten(1)}


def _own_w4(s):
    c = s["case"]
    return {"y": _package().linear_w4(s["x"], s["codes"], s["scales"], c["group"], zeros=s["zeros"],
                                      bias=s["bias"], activation=c["act"])}


def _plain_w4(s):
    c = s["case"]
    w = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=-1).flatten(1).float()
    z = s["zeros"].float() if s["zeros"] is not None else torch.full_like(s["scales"], 8).float()
    group = torch.arange(c["k"], device="cuda") // c["group"]
    w = (w - z[:, group]) * s["scales"].float()[:, group]
    y = s["x"].float() @ w.T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["act"] == "relu":
        y = y.clamp(min=0)
    elif c["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    return {"y": y.to(s["x"].dtype)}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(c):
    if c["op"] == "write":
        t = c["n"] * (c["each"] + 1) / 2 if c["n"] > 1 else c["each"]
        items = 2 * t * c["h"] * c["d"]
        return {"bytes": items * 3 + 4 * t + 2 * max(t / c["block"], c["n"]) * c["h"],
                "flops": 2 * items}
    if c["op"] == "read":
        items = 2 * c["tokens"] * c["h"] * c["d"]
        return {"bytes": items * 3 + 4 * c["tokens"] + 2 * c["tokens"] / c["block"] * c["h"],
                "flops": items}
    if c["op"] == "w4":
        m, n, k = c["m"], c["n"], c["k"]
        groups = -(-k // c["group"])
        return {"bytes": n * k / 2 + n * groups * (3 if c["zeros"] else 2) + 2 * m * (n + k) +
                (2 * n if c["bias"] else 0), "flops": 2 * m * n * k}
    tokens = _expected_tokens(c)
    return {"bytes": 2 * tokens * c["h_kv"] * (c["d"] + 1 / c["block"]) + 4 * tokens / c["page"] +
            c["n"] * c["h_q"] * (4 * c["d"] + 4), "flops": 4 * tokens * c["h_q"] * c["d"]}


def _expected_tokens(c):
    """Cached tokens that a pass attends to, over all sequences: lengths are uniform on
    0 .. longest but for the two that are set."""
    w = c["window"] + c["sinks"] if c["window"] else c["longest"]
    if c["n"] == 1:
        return min(c["longest"], w)
    L = c["longest"]
    w = min(w, L)
    mean = (w * (w + 1) / 2 + (L - w) * w) / (L + 1)
    return w + (c["n"] - 2) * mean


# ---- the definition in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attn": _exact_attn,
            "w4": _exact_w4}[case["op"]](case, s)


def _power64(e):
    """2^e in float64, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest_e4m3(y):
    """The nearest number of three fraction bits and exponents from -6 on, ties to even."""
    step = _power64(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_write(c, s):
    """Token by token over the blocks' offsets: one new token of every block at a time tells where
    its block's new ones begin and how large they are."""
    block, where = c["block"], s["slots"].long()
    out = {}
    for kind in "kv":
        cache, scale = s[kind + "_cache"], s[kind + "_scale"]
        x = s[kind].double()
        values = torch.full((cache.shape[0] * cache.shape[1], *cache.shape[2:]), math.nan,
                            dtype=torch.float64, device="cuda")
        values[where] = x
        new = torch.zeros(len(values), dtype=torch.bool, device="cuda")
        new[where] = True
        values, new = values.unflatten(0, (-1, block)), new.unflatten(0, (-1, block))
        codes = cache.double().reshape(values.shape)
        before = scale.long().flatten(0, 1)
        top = values.abs().nan_to_num(nan=0.0).amax((1, 3))                  # [blocks, h]
        need = torch.round(torch.log2(top.clamp(min=2.0 ** -150) / 448))     # or one more or less
        need = need - (448 * _power64(need - 1) >= top).double()
        need = (need + (448 * _power64(need) < top)).clamp(min=-127) + 127
        touched, begun = new.any(1), ~new[:, 0]
        after = torch.where((touched & begun)[:, None], torch.maximum(before.double(), need), need)
        after = torch.where(touched[:, None], after, before.double())
        older = torch.where(touched & begun, 1.0, 0.0)[:, None] * (before - after)
        kept = _nearest_e4m3(codes * _power64(older)[:, None, :, None])
        written = _nearest_e4m3(values * _power64(127 - after)[:, None, :, None])
        out[kind + "_cache"] = torch.where(new[..., None, None], written, kept).view(cache.shape)
        out[kind + "_scale"] = after.to(torch.uint8).view(scale.shape)
    return out


def _exact_rows(cache, scale, page, offset):
    block = cache.shape[1] // scale.shape[1]
    return cache[page, offset].double() * \
        _power64(scale[page, offset // block].long() - 127)[..., None]


def _exact_read(c, s):
    page, offset = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    return {"k": _exact_rows(s["k_cache"], s["k_scale"], page, offset),
            "v": _exact_rows(s["v_cache"], s["v_scale"], page, offset)}


def _exact_attn(c, s):
    n, d, group = c["n"], c["d"], c["h_q"] // c["h_kv"]
    o = torch.zeros(n, c["h_q"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, c["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        start = max(0, length - (c["window"] or length))
        at = torch.cat([torch.arange(min(c["sinks"], start), device="cuda"),
                        torch.arange(start, length, device="cuda")])
        page = s["table"][i, at // c["page"]].long()
        k, v = (_exact_rows(s[x + "_cache"], s[x + "_scale"], page, at % c["page"])
                .repeat_interleave(group, dim=1) for x in "kv")
        x = torch.einsum("hd,thd->ht", s["q"][i].double(), k) * s["scale"]
        lse[i] = torch.logsumexp(x, dim=1)
        o[i] = torch.einsum("ht,thd->hd", torch.exp(x - lse[i][:, None]), v)
    return {"o": o, "lse": lse}


def _exact_w4(c, s):
    y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
    for g, k0 in enumerate(range(0, c["k"], c["group"])):
        k1 = min(c["k"], k0 + c["group"])
        pairs = s["codes"][:, k0 // 2:k1 // 2].int()
        x = s["x"][:, k0:k1].double()
        z = s["zeros"][:, g].double()[:, None] if c["zeros"] else 8.0
        even, odd = (pairs % 16).double() - z, (pairs // 16).double() - z
        part = x[:, 0::2] @ even.T + x[:, 1::2] @ odd.T
        y += part * s["scales"][:, g].double()
    if c["bias"]:
        y += s["bias"].double()
    if c["act"] == "relu":
        y = torch.relu(y)
    elif c["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    return {"y": y}
