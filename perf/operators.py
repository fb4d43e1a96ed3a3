"""Cases of the decode-step operators: the gated delta rule's recurrent step, the per-head norm and
rotation of queries and keys with the write to the paged cache, and the attention of one new token
over that cache.

``run`` computes each operator in elementary torch operations in 32 bits (``own`` false) or through
the package's entry points (``own`` true); ``exact`` computes the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # -- gated delta rule, recurrent: states of 128 x 128 per value head
        # one user at a prompt: the latency of one layer's step
        dict(name="step_1x1_h8_hv16", op="step", dtype="bf16", n=1, tokens=1, h_q=8, h_k=8, h_v=16),
        # the packed prefill's 20 sequences, carried on
        dict(name="step_20x1_h8_hv16", op="step", dtype="bf16", n=20, tokens=1, h_q=8, h_k=8,
             h_v=16),
        # a full server
        dict(name="step_256x1_h16_hv32", op="step", dtype="bf16", n=256, tokens=1, h_q=16, h_k=16,
             h_v=32),
        # drafted tokens checked in one call, grouped queries, fp16
        dict(name="step_77x4_hq16_h4_hv8", op="step", dtype="fp16", n=77, tokens=4, h_q=16, h_k=4,
             h_v=8),
        # -- norm and rotation
        # three sequences' new tokens on their way to the cache
        dict(name="norm_3_cache", op="norm", dtype="bf16", tokens=3, h_q=32, h_k=8, d=128,
             norm="rms", rot=128, axes=1, interleaved=False, page=16),
        # q and k of a delta-rule prefill (8192 packed tokens): unit length, no rotation
        dict(name="norm_8192_l2", op="norm", dtype="bf16", tokens=8192, h_q=8, h_k=8, d=128,
             norm="l2", rot=0, axes=1, interleaved=False, page=0),
        # a prompt of image patches: positions in time, height and width
        dict(name="norm_32768_axes3_cache", op="norm", dtype="bf16", tokens=32768, h_q=32, h_k=8,
             d=128, norm="rms", rot=128, axes=3, interleaved=False, page=64),
        # wide heads, a quarter of each rotated in neighbouring pairs, an odd token count
        dict(name="norm_1021_d256_rot64", op="norm", dtype="fp16", tokens=1021, h_q=16, h_k=2,
             d=256, norm="rms", rot=64, axes=1, interleaved=True, page=0),
        # -- attention over the paged cache
        # one short conversation
        dict(name="attn_1x500", op="attn", dtype="bf16", n=1, longest=500, h_q=32, h_kv=8, d=128,
             page=16, window=0),
        # a full server: lengths from nothing to 8192
        dict(name="attn_64x8192_ragged", op="attn", dtype="bf16", n=64, longest=8192, h_q=32,
             h_kv=8, d=128, page=16, window=0),
        # one very long document, wide heads
        dict(name="attn_1x200001_d256", op="attn", dtype="bf16", n=1, longest=200001, h_q=16,
             h_kv=2, d=256, page=64, window=0),
        # a sliding window, one key head per query head, pages of an odd size
        dict(name="attn_37x5000_window", op="attn", dtype="fp16", n=37, longest=5000, h_q=12,
             h_kv=12, d=64, page=20, window=1000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "norm", "attn"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "step":
        h_k = rng.choice([1, 2, 4, 8, 16])
        layout = rng.choice(["same", "values", "values", "queries"])
        h_v = h_k * (rng.choice([2, 4]) if layout == "values" and h_k < 16 else 1)
        h_q = h_v * rng.choice([2, 4]) if layout == "queries" else h_k
        most = max(1, 256 * 32 // h_v)
        tokens = rng.choice([1, 1, 1, 2, 3, 5, 8])
        n = _log(rng, 1, min(1500, most) if tokens == 1 else max(1, min(1500, most) // 2))
        return dict(op=op, dtype=dtype, n=n, tokens=tokens, h_q=h_q, h_k=h_k, h_v=h_v)
    if op == "norm":
        d = rng.choice([64, 128, 128, 256])
        h_k = rng.choice([1, 2, 4, 8])
        h_q = h_k * rng.choice([1, 3, 4, 8])
        norm = rng.choice(["rms", "rms", "l2"])
        rot = 0 if norm == "l2" else rng.choice([d, d, d // 2, d // 4])
        axes = rng.choice([1, 1, 3]) if rot >= 64 else 1
        most = max(16, min(65536, 32768 * 48 * 128 // ((h_q + 2 * h_k) * d)))
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, most), h_q=h_q, h_k=h_k, d=d,
                    norm=norm, rot=rot, axes=axes, interleaved=bool(rot and rng.random() < 0.3),
                    page=0 if norm == "l2" else rng.choice([0, 16, 16, 20, 64]))
    d = rng.choice([64, 128, 128, 256])
    h_kv = rng.choice([1, 2, 4, 8])
    h_q = h_kv * rng.choice([1, 3, 4, 8, 16])
    n = _log(rng, 1, 200)
    # at most the bytes of the largest listed case, whose lengths are half its longest on average
    most = max(64, min(200000, 64 * 8192 * 8 * 128 // (2 * n * h_kv * d)))
    longest = _log(rng, 40, most)
    return dict(op=op, dtype=dtype, n=n, longest=longest, h_q=h_q, h_kv=h_kv, d=d,
                page=rng.choice([16, 16, 20, 32, 64, 128]),
                window=rng.choice([0, 0, 0, max(1, longest // 3)]))


# ---- inputs ------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _package():
    import blackwell_tensor_core_fp16_gb300 as package
    return package


def prepare(case, seed):
    g = _generator(seed)
    return {"case": case, **{"step": _prepare_step, "norm": _prepare_norm,
                             "attn": _prepare_attn}[case["op"]](case, g)}


def _prepare_step(c, g):
    """q, k, v as one projection leaves them (side by side), gates, and a pool of states with more
    slots than sequences, in which every sequence has a slot of its own."""
    n, t, dt = c["n"], c["tokens"], DTYPES[c["dtype"]]
    h_q, h_k, h_v = c["h_q"], c["h_k"], c["h_v"]
    packed = torch.cat([_unit(_normal(g, n, t, h_q + h_k, 128)), _normal(g, n, t, h_v, 128)],
                       dim=2).to(dt)
    slots = n + 1 + n // 8
    state = 0.1 * _normal(g, slots, h_v, 128, 128)
    alpha = torch.exp(-0.1 * torch.rand(n, t, h_v, generator=g, device="cuda"))
    beta = torch.sigmoid(_normal(g, n, t, h_v))
    where = torch.randperm(slots, generator=g, device="cuda")[:n].to(torch.int32)
    return {"q": packed[:, :, :h_q], "k": packed[:, :, h_q:h_q + h_k], "v": packed[:, :, h_q + h_k:],
            "alpha": alpha, "beta": beta, "state": state, "slots": where, "scale": 128 ** -0.5}


def _prepare_norm(c, g):
    """The projection's output (queries, keys and values of a token side by side), the norms'
    weights, the table of the angles and the tokens' positions, and the cache with their slots."""
    t, d, dt = c["tokens"], c["d"], DTYPES[c["dtype"]]
    h_q, h_k, rot, axes, page = c["h_q"], c["h_k"], c["rot"], c["axes"], c["page"]
    packed = (1.5 * _normal(g, t, h_q + 2 * h_k, d)).to(dt)
    s = {"q": packed[:, :h_q], "k": packed[:, h_q:h_q + h_k], "v": packed[:, h_q + h_k:],
         "q_weight": None, "k_weight": None, "rotary": None, "positions": None, "sections": None,
         "k_cache": None, "v_cache": None, "slots": None}
    if c["norm"] == "rms":
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * _normal(g, d)).to(dt) for _ in range(2))
    if rot:
        longest = 40000
        rate = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(longest, dtype=torch.float64, device="cuda")[:, None] * rate
        s["rotary"] = torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)
        shape = (t,) if axes == 1 else (axes, t)
        s["positions"] = torch.randint(0, longest, shape, generator=g, device="cuda",
                                       dtype=torch.int32)
        if axes == 3:
            half = rot // 2
            s["sections"] = (half - 2 * (3 * half // 8), 3 * half // 8, 3 * half // 8)
    if page:
        pages = -(-t // page) + 3
        s["k_cache"], s["v_cache"] = (_normal(g, pages, page, h_k, d).to(dt) for _ in range(2))
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:t].to(torch.int32)
    return s


def _prepare_attn(c, g):
    """One query per sequence, the pool of pages in the order in which a server hands them out
    (none), and lengths between nothing and the longest; one sequence alone has the longest."""
    n, d, dt, page = c["n"], c["d"], DTYPES[c["dtype"]], c["page"]
    if n > 1:
        lens = torch.randint(0, c["longest"] + 1, (n,), generator=g, device="cuda")
        lens[0], lens[n // 2] = c["longest"], 0
    else:
        lens = torch.full((1,), c["longest"], device="cuda")
    width = -(-c["longest"] // page)
    used = (lens + page - 1) // page
    total = int(used.sum()) + 2
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = (used.cumsum(0) - used)[:, None] + torch.arange(width, device="cuda")
    table = torch.where(torch.arange(width, device="cuda") < used[:, None],
                        order[at.clamp(max=total - 1)], torch.zeros_like(order[:1]))
    # one draw of pages in 32 bits would be large: they are drawn in 16
    pool = [torch.empty(total, page, c["h_kv"], d, dtype=dt, device="cuda").normal_(generator=g)
            for _ in range(2)]
    s = {"q": (2.0 * _normal(g, n, c["h_q"], d)).to(dt), "k_cache": pool[0], "v_cache": pool[1],
         "table": table.contiguous(), "lens": lens.to(torch.int32), "scale": d ** -0.5,
         "window": c["window"] or None}
    if own:
        s["workspace"] = _package().paged_attention_workspace(c["h_q"], c["h_kv"], d, "cuda")
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "step":
        return _own_step(s) if own else _plain_step(s)
    if op == "norm":
        return _own_norm(s) if own else _plain_norm(s)
    return _own_attn(s) if own else _plain_attn(s)


def _own_step(s):
    o = _package().gated_delta_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["state"],
                                    s["scale"], slots=s["slots"])
    return {"o": o, "state": s["state"]}


def _plain_step(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    h_q, h_k, h_v = q.shape[2], k.shape[2], v.shape[2]
    k = k.repeat_interleave(h_v // h_k, dim=2)
    if h_q == h_k:
        q = q.repeat_interleave(h_v // h_k, dim=2)
    q = q.unflatten(2, (h_v, -1))               # [n, tokens, h_v, queries of the state, 128]
    where = s["slots"].long()
    S = s["state"][where]
    outs = []
    for t in range(q.shape[1]):                 # the recurrence goes token by token
        S = S * s["alpha"][:, t, :, None, None]
        u = s["beta"][:, t, :, None] * (v[:, t] - (S @ k[:, t, :, :, None])[..., 0])
        S = S + u[..., None] * k[:, t, :, None, :]
        outs.append((q[:, t] @ S.transpose(-1, -2)).flatten(1, 2) * s["scale"])
    s["state"][where] = S
    return {"o": torch.stack(outs, dim=1).to(s["q"].dtype), "state": s["state"]}


def _own_norm(s):
    c = s["case"]
    q, k = _package().qk_norm_rope(
        s["q"], s["k"], s["q_weight"], s["k_weight"], norm=c["norm"], eps=1e-6,
        positions=s["positions"], rotary=s["rotary"], sections=s["sections"],
        interleaved=c["interleaved"], v=s["v"] if c["page"] else None, k_cache=s["k_cache"],
        v_cache=s["v_cache"], slots=s["slots"])
    if c["page"]:
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"q": q, "k": k}


def _plain_norm(s):
    c = s["case"]
    cos = sin = None
    if c["rot"]:
        half, pos = c["rot"] // 2, s["positions"].long()
        if s["sections"]:
            rows = s["rotary"][pos]                                  # [axes, t, rot]
            axis = torch.repeat_interleave(torch.arange(3, device="cuda"),
                                           torch.tensor(s["sections"], device="cuda"),
                                           output_size=half)
            pair = torch.arange(half, device="cuda")
            cos, sin = rows[axis, :, pair].T, rows[axis, :, half + pair].T
        else:
            rows = s["rotary"][pos]
            cos, sin = rows[:, :half], rows[:, half:]
        cos, sin = cos[:, None], sin[:, None]

    def one(x, w):
        x = x.float()
        m = (x * x).sum(-1, keepdim=True)
        x = x * torch.rsqrt((m / x.shape[-1] if c["norm"] == "rms" else m) + 1e-6)
        if w is not None:
            x = x * w.float()
        if not c["rot"]:
            return x
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([r, rest], dim=-1)

    dt = s["q"].dtype
    q, k = one(s["q"], s["q_weight"]).to(dt), one(s["k"], s["k_weight"]).to(dt)
    if not c["page"]:
        return {"q": q, "k": k}
    where = s["slots"].long()
    s["k_cache"].flatten(0, 1)[where] = k
    s["v_cache"].flatten(0, 1)[where] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attn(s):
    o, lse = _package().paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                        scale=s["scale"], window=s["window"], return_lse=True,
                                        workspace=s["workspace"])
    return {"o": o, "lse": lse}


def _plain_attn(s):
    h_kv, dt = s["k_cache"].shape[2], s["q"].dtype
    table = s["table"].long()
    k = s["k_cache"][table].flatten(1, 2).transpose(1, 2).float()    # [n, h_kv, tokens, d]
    v = s["v_cache"][table].flatten(1, 2).transpose(1, 2).float()
    at = torch.arange(k.shape[2], device="cuda")
    lens = s["lens"][:, None]
    seen = at < lens
    if s["window"]:
        seen = seen & (at >= lens - s["window"])
    q = s["q"].float().unflatten(1, (h_kv, -1))
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))
    return {"o": o.flatten(1, 2).to(dt), "lse": lse.flatten(1)}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(c):
    if c["op"] == "step":
        n, t = c["n"], c["tokens"]
        h_o = max(c["h_q"], c["h_v"])
        io = 2 * 128 * (c["h_q"] + c["h_k"] + c["h_v"] + h_o) + 8 * c["h_v"]
        return {"bytes": n * (2 * 4 * c["h_v"] * 128 * 128 + t * io + 4),
                "flops": n * t * 2 * 128 * 128 * (2 * c["h_v"] + h_o)}
    if c["op"] == "norm":
        t, d = c["tokens"], c["d"]
        moved = 2 * 2 * (c["h_q"] + c["h_k"] * (2 if c["page"] else 1)) * d
        per = moved + (4 if c["page"] else 0) + (4 * c["axes"] + 4 * c["rot"] if c["rot"] else 0)
        return {"bytes": t * per, "flops": t * (c["h_q"] + c["h_k"]) * (4 * d + 3 * c["rot"])}
    tokens = _expected_tokens(c)
    kv = 2 * 2 * tokens * c["h_kv"] * c["d"]
    return {"bytes": kv + 4 * tokens / c["page"] + c["n"] * c["h_q"] * (4 * c["d"] + 4),
            "flops": 4 * tokens * c["h_q"] * c["d"]}


def _expected_tokens(c):
    """Cached tokens that a pass attends to, over all sequences: lengths are uniform on
    0 .. longest but for the two that are set."""
    if c["n"] == 1:
        return min(c["longest"], c["window"] or c["longest"])
    L, w = c["longest"], c["window"] or c["longest"]
    w = min(w, L)
    mean = (w * (w + 1) / 2 + (L - w) * w) / (L + 1)
    return w + (c["n"] - 2) * mean


# ---- the definition in 64 bits -------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "norm": _exact_norm, "attn": _exact_attn}[case["op"]](case, s)


def _exact_step(c, s):
    q, k, v = (s[x].double() for x in "qkv")
    alpha, beta = s["alpha"].double(), s["beta"].double()
    state = s["state"].double()
    h_v = c["h_v"]
    h_o = max(c["h_q"], h_v)
    o = torch.empty(c["n"], c["tokens"], h_o, 128, dtype=torch.float64, device="cuda")
    where = s["slots"].long()
    for j in range(h_v):
        S = state[where, j]                                          # [n, 128, 128]
        kj = j // (h_v // c["h_k"])
        heads = [(kj, j)] if c["h_q"] == c["h_k"] else [(m, m) for m in range(h_o)
                                                        if m // (h_o // h_v) == j]
        for t in range(c["tokens"]):
            S = alpha[:, t, j, None, None] * S
            update = beta[:, t, j, None] * (v[:, t, j] - torch.einsum("nvk,nk->nv", S, k[:, t, kj]))
            S = S + torch.einsum("nv,nk->nvk", update, k[:, t, kj])
            for m, to in heads:
                o[:, t, to] = s["scale"] * torch.einsum("nvk,nk->nv", S, q[:, t, m])
        state[where, j] = S
    return {"o": o, "state": state}


def _exact_norm(c, s):
    def one(x, w):
        x = x.double()
        square = x.pow(2)
        x = x / ((square.mean(-1, keepdim=True) if c["norm"] == "rms"
                  else square.sum(-1, keepdim=True)) + 1e-6).sqrt()
        x = x if w is None else x * w.double()
        half = c["rot"] // 2
        first = 0
        for axis, size in enumerate(s["sections"] or ([half] if half else [])):
            pos = (s["positions"][axis] if c["axes"] > 1 else s["positions"]).long()
            table = s["rotary"].double()[pos]
            for j in range(first, first + size):
                a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, half + j)
                z = torch.complex(x[..., a], x[..., b]) * \
                    torch.complex(table[:, j], table[:, half + j])[:, None]
                x[..., a], x[..., b] = z.real, z.imag
            first += size
        return x

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if not c["page"]:
        return {"q": q, "k": k}
    caches = []
    for cache, rows in ((s["k_cache"], k), (s["v_cache"], s["v"].double())):
        cache = cache.double()
        at = s["slots"].long()
        cache[at // c["page"], at % c["page"]] = rows
        caches.append(cache)
    return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attn(c, s):
    n, d, group = c["n"], c["d"], c["h_q"] // c["h_kv"]
    o = torch.zeros(n, c["h_q"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, c["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        at = torch.arange(max(0, length - (c["window"] or length)), length, device="cuda")
        page = s["table"][i, at // c["page"]].long()
        k, v = (s[x][page, at % c["page"]].double().repeat_interleave(group, dim=1)
                for x in ("k_cache", "v_cache"))
        x = torch.einsum("hd,thd->ht", s["q"][i].double(), k) * s["scale"]
        lse[i] = torch.logsumexp(x, dim=1)
        o[i] = torch.einsum("ht,thd->hd", torch.exp(x - lse[i][:, None]), v)
    return {"o": o, "lse": lse}
