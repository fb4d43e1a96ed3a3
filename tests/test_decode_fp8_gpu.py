"""The operators on an 8-bit cache and on 4-bit weights on the GPU against their definitions in 64 bits
(tests/decode_fp8_ref.py has the definitions and the derivation of the bounds)."""
from __future__ import annotations

import math

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
import decode_fp8_ref as ref
from decode_fp8_ref import E4M3
from test_decode_gpu import cuda_library, generator, no_refusals_left, normal  # noqa: F401

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])


def pool(gen, pages, page, block, h, d, spread=4.0):
    """A cache of normal values in blocks of sizes of their own (on the CPU)."""
    x = normal(gen, pages, page // block, block, h, d)
    x = x * torch.exp2(spread * normal(gen, pages, page // block, 1, h, 1))
    top = x.abs().amax((2, 4))
    e = torch.ceil(torch.log2(top / 448)).long() + 127
    codes = (x * torch.exp2(127.0 - e)[:, :, None, :, None]).to(E4M3).flatten(1, 2)
    return codes, e.to(torch.uint8)


def caches(gen, pages, page, block, h, d, **kw):
    (kc, ks), (vc, vs) = (pool(gen, pages, page, block, h, d, **kw) for _ in range(2))
    return {"k_cache": kc.cuda(), "v_cache": vc.cuda(), "k_scale": ks.cuda(), "v_scale": vs.cuda()}


def check_cache(got, before, x, slots, where):
    """The cache after x [kind: k, v] went to slots, every byte of it."""
    for kind in "kv":
        codes, scale = ref.quantize_cache(x[kind], before[kind + "_cache"], before[kind + "_scale"], slots)
        assert torch.equal(got[kind + "_scale"].cpu(), scale), f"{where}: {kind} scales"
        c = got[kind + "_cache"].float().double().cpu()
        assert torch.equal(c.isnan(), codes.isnan()), f"{where}: {kind} NaN"
        bad = (c != codes) & ~codes.isnan()
        assert not bad.any(), f"{where}: {kind} codes differ at {bad.nonzero()[0].tolist()}"


def write(c, x, slots, **kw):
    g.quantize_cache(x["k"], x["v"], c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], slots, **kw)


def places(gen, n, most, page, before=None, pages=None):
    """Slots of n sequences' new tokens, 1 .. most each, on pages of their own in no order."""
    new = torch.randint(1, most + 1, (n,), generator=gen)
    old = torch.randint(0, 2 * page, (n,), generator=gen) if before is None else torch.tensor(before)
    width = int((old + new + page - 1).max()) // page
    order = torch.randperm(n * width, generator=gen)
    out = []
    for i in range(n):
        pos = torch.arange(int(old[i]), int(old[i] + new[i]))
        out.append(order[i * width + pos // page] * page + pos % page)
    return torch.cat(out).to(torch.int32), n * width


# ---- the write ---------------------------------------------------------------------------------------

@DTYPES
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h,page,block", [(1, 16, 16), (2, 32, 8), (3, 20, 10), (8, 16, 1), (2, 192, 96),
                                          (1, 48, 48), (12, 6, 3)])
@pytest.mark.parametrize("n,most", [(1, 1), (5, 1), (3, 40), (2, 230)])
def test_write(n, most, h, page, block, d, dtype):
    gen = generator(n * 1000 + most + d + block)
    slots, pages = places(gen, n, most, page)
    c = caches(gen, pages, page, block, h, d)
    before = {x: y.clone() for x, y in c.items()}
    x = {kind: (normal(gen, len(slots), h, d) * torch.exp2(4 * normal(gen, len(slots), 1, 1))).to(dtype).cuda()
         for kind in "kv"}
    write(c, x, slots.cuda())
    check_cache(c, before, x, slots, f"{n} x {most}")
    # once more: the scales have grown already, so older codes stay
    again = {a: b.clone() for a, b in c.items()}
    write(c, x, slots.cuda())
    check_cache(c, again, x, slots, "again")


def test_write_many_tokens():
    """More tokens than any launch keeps resident, with windows whose tokens begin many blocks."""
    gen = generator(3)
    h, d, page, block = 4, 128, 16, 16
    slots, pages = places(gen, 900, 20, page)
    c = caches(gen, pages, page, block, h, d)
    before = {x: y.clone() for x, y in c.items()}
    x = {kind: normal(gen, len(slots), h, d).bfloat16().cuda() for kind in "kv"}
    write(c, x, slots.cuda())
    check_cache(c, before, x, slots, "many")


@pytest.mark.parametrize("tokens,h,page,block,d,dtype", [
    (700, 8, 16, 16, 128, torch.bfloat16), (1900, 8, 8, 8, 128, torch.float16), (4000, 8, 16, 16, 128, torch.bfloat16),
    (2600, 12, 6, 3, 64, torch.float16), (1900, 8, 4, 1, 256, torch.bfloat16), (15500, 2, 16, 16, 64, torch.bfloat16),
    (31000, 1, 8, 4, 128, torch.float16), (8000, 2, 32, 16, 256, torch.float16)])
def test_write_of_many_sequences_tokens(tokens, h, page, block, d, dtype):
    """A token each of many sequences, at any place of its block, between some longer runs, inactive and
    refused tokens; scales that grow and that do not, infinities and NaN."""
    gen = generator(tokens + d + block)
    per = page // block
    where = torch.randperm(tokens + 64, generator=gen)[:tokens]          # blocks
    slots = where * block + torch.randint(0, block, (tokens,), generator=gen)
    slots[torch.rand(tokens, generator=gen) < 0.1] = -1
    slots[::97] = -1                              # (so that the next one, of the same block, begins a run)
    if block > 1:
        for at in range(1, tokens - 1, 97):       # runs of two
            slots[at] = where[at] * block
            slots[at + 1] = where[at] * block + 1
    wrong = torch.zeros(tokens, dtype=torch.bool)
    again = torch.arange(50, tokens, 331)         # the place of a token a little before
    for at in again.tolist():
        if slots[at - 20] >= 0 and slots[at] >= 0 and (at - 20) % 97 > 2 and at % 97 > 2:
            slots[at] = slots[at - 20]
            wrong[at] = True
    slots = slots.to(torch.int32)
    pages = -(-(tokens + 64) // per)
    c = caches(gen, pages, page, block, h, d)
    before = {a: b.clone() for a, b in c.items()}
    x = {kind: (normal(gen, tokens, h, d) * torch.exp2(4 * normal(gen, tokens, 1, 1))).to(dtype) for kind in "kv"}
    x["k"][5::41, 0, 3] = math.inf
    x["v"][7::53, -1, :] = math.nan
    x["v"][9::59] = 0
    x = {kind: y.cuda() for kind, y in x.items()}
    write(c, x, slots.cuda())
    kept = ((slots >= 0) & ~wrong).nonzero().flatten()
    check_cache(c, before, {kind: y[kept.cuda()] for kind, y in x.items()}, slots[kept], "tokens")
    if wrong.any():
        with pytest.raises(g.GemmError, match="cache slot"):
            g.check_decode_status()


def test_write_token_by_token():
    """A block filled one token a call, each larger than the last: every growth of the scale."""
    gen = generator(4)
    c = caches(gen, 2, 16, 16, 2, 64)
    for t in range(32):
        before = {x: y.clone() for x, y in c.items()}
        slots = torch.tensor([16 + t if t < 16 else t - 16], dtype=torch.int32)
        x = {kind: (normal(gen, 1, 2, 64) * 1.7 ** (t % 16)).half().cuda() for kind in "kv"}
        write(c, x, slots.cuda())
        check_cache(c, before, x, slots, f"token {t}")


@DTYPES
def test_write_of_odd_values(dtype):
    """Zeros, subnormal numbers, the type's largest, infinities and NaN, whose neighbours stay exact; an
    old scale that stands for NaN, and one so small that older codes vanish."""
    gen = generator(5)
    h, d = 2, 128
    big = torch.finfo(dtype).max
    tiny = 2.0 ** (-133 if dtype == torch.bfloat16 else -24)
    x = normal(gen, 9, h, d)
    x[0], x[1], x[2] = 0, tiny, -big
    x[3, 0, 5], x[3, 1, 7] = math.inf, -math.inf
    x[4, 0, :] = math.nan
    x[5, 1, 0:128:3] = math.inf
    x[6] = 448 * 0.25
    x[7] = 450 * 0.25
    x = {"k": x.to(dtype).cuda(), "v": x.flip(-1).to(dtype).cuda()}
    slots = torch.arange(0, 9 * 8, 8, dtype=torch.int32)
    slots[8] += 3
    for scale in (0, 1, 120, 200, 255):
        c = caches(gen, 9, 8, 8, h, d)
        for kind in "kv":
            c[kind + "_scale"][8] = scale
        before = {a: b.clone() for a, b in c.items()}
        write(c, x, slots.cuda())
        if scale == 255:                         # a block of NaN stays one, whatever its codes
            for kind in "kv":
                assert bool((c[kind + "_scale"][8] == 255).all())
            continue
        check_cache(c, before, x, slots, f"scale {scale}")


def test_write_to_strided_caches():
    """Keys and values side by side in one projection, heads outside the tokens in the cache, scales
    between others: what lies between stays."""
    gen = generator(6)
    h, d, page, block, pages = 3, 64, 12, 4, 4
    packed = normal(gen, 20, 3 * h, d).bfloat16().cuda()
    store = torch.full((pages, 2, h, page + 1, 2 * d), 9.0).to(E4M3).cuda()
    scales = torch.full((pages, page // block, h, 3), 77, dtype=torch.uint8).cuda()
    c = {"k_cache": store[:, 0, :, :page, :d].transpose(1, 2), "v_cache": store[:, 1, :, :page, :d].transpose(1, 2),
         "k_scale": scales[..., 0], "v_scale": scales[..., 2]}
    before = {a: b.clone() for a, b in c.items()}
    x = {"k": packed[:, h:2 * h], "v": packed[:, 2 * h:]}
    slots = torch.cat([torch.arange(30, 46), torch.arange(2, 6)]).to(torch.int32)
    write(c, x, slots.cuda())
    check_cache(c, before, x, slots, "strided")
    assert bool((store[..., page, :].float() == 9).all() and (store[..., d:].float() == 9).all())
    assert bool((scales[..., 1] == 77).all())
    # keys of one head for all
    one = {kind: y[:, :1].expand(-1, h, -1) for kind, y in x.items()}
    before = {a: b.clone() for a, b in c.items()}
    write(c, one, slots.cuda())
    check_cache(c, before, one, slots, "broadcast")


@pytest.mark.parametrize("bad,kept", [
    ([0, 1, -1, -1, 16, 17], [0, 1, 4, 5]), ([-1] * 6, []),
    ([0, 2, 3, 16, 17, 18], [0, 3, 4, 5]),                   # a gap: refused with what continues it
    ([5, 4, 16, 17, 18, 19], [0, 2, 3, 4, 5]),               # backwards
    ([5, 5, 16, 17, 18, 19], [0, 2, 3, 4, 5]),               # the same place twice
    ([64, 0, 1, 2, -2, 2 ** 31 - 1], [1, 2, 3]), ([-2 ** 31, 63, 0, 1, 2, 3], [1, 2, 3, 4, 5]),
])
@pytest.mark.parametrize("many", [False, True])
def test_write_refusals(bad, kept, many):
    """Refused and inactive tokens are not written and the rest is, with few tokens and with many
    (which go by windows: 3000 inactive ones follow)."""
    gen = generator(7)
    slots = torch.tensor(bad + [-1] * (3000 if many else 0), dtype=torch.int32)
    c = caches(gen, 4, 16, 8, 2, 64)
    before = {a: b.clone() for a, b in c.items()}
    x = {kind: normal(gen, len(slots), 2, 64).half().cuda() for kind in "kv"}
    write(c, x, slots.cuda())
    check_cache(c, before, {kind: y[kept] for kind, y in x.items()}, slots[kept], "kept")
    if len(kept) < sum(s != -1 for s in bad):
        with pytest.raises(g.GemmError, match="cache slot"):
            g.check_decode_status()


@pytest.mark.parametrize("apart", [2, 3, 15, 16, 17, 31, 32, 33, 64, 100, 127, 128])
@pytest.mark.parametrize("again", [[0, 1], [1, 2], [3], [-1, 1]])
@pytest.mark.parametrize("lead,many", [(0, False), (0, True), (11, True)])
def test_write_of_a_block_in_two_runs(apart, again, lead, many):
    """A block's tokens that are `apart` tokens behind its first ones and do not continue them, the same
    place among them: refused, as are those that continue them.  What lies between and behind is written."""
    gen = generator(apart)
    others = iter(range(8, 8 * 400, 8))
    slots = [next(others) for _ in range(lead)] + [0]
    slots += [next(others) for _ in range(apart - 1)]
    first = len(slots)
    slots += again + [next(others) + 5]
    last = len(slots) - 1
    slots = torch.tensor(slots + [-1] * (3000 if many else 0), dtype=torch.int32)
    kept = list(range(first)) + [last]
    c = caches(gen, 200, 16, 8, 2, 64)
    before = {a: b.clone() for a, b in c.items()}
    x = {kind: normal(gen, len(slots), 2, 64).half().cuda() for kind in "kv"}
    write(c, x, slots.cuda())
    check_cache(c, before, {kind: y[kept] for kind, y in x.items()}, slots[kept], "kept")
    with pytest.raises(g.GemmError, match="cache slot"):
        g.check_decode_status()


def test_write_and_read_on_another_stream_and_in_a_graph():
    gen = generator(8)
    slots, pages = places(gen, 4, 30, 16)
    slots = slots.cuda()
    c = caches(gen, pages, 16, 16, 2, 128)
    x = {kind: normal(gen, len(slots), 2, 128).bfloat16().cuda() for kind in "kv"}
    before = {a: b.clone() for a, b in c.items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    write(c, x, slots, stream=stream)
    k, v = g.dequantize_cache(*(c[a] for a in ("k_cache", "v_cache", "k_scale", "v_scale")), slots,
                              stream=stream)
    stream.synchronize()
    check_cache(c, before, x, slots.cpu(), "stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        write(c, x, slots)
        out = g.dequantize_cache(*(c[a] for a in ("k_cache", "v_cache", "k_scale", "v_scale")), slots)
    for a, b in before.items():
        c[a].copy_(b)
    x["k"].mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    check_cache(c, before, x, slots.cpu(), "graph")
    assert torch.equal(out[1], v) and not torch.equal(out[0], k)


# ---- the reading back --------------------------------------------------------------------------------

def rounded(x, dtype):
    """x in 64 bits rounded once to dtype (what holds: a 32-bit number with a power of two's factor)."""
    return x.to(dtype)


@DTYPES
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,h,page,block", [(1, 1, 16, 16), (7, 3, 20, 10), (333, 12, 6, 3),
                                                 (1000, 8, 64, 64), (50, 40, 16, 16)])
def test_read(tokens, h, page, block, d, dtype):
    gen = generator(tokens + d)
    pages = -(-tokens // page) + 2
    c = caches(gen, pages, page, block, h, d, spread=20.0 if dtype == torch.bfloat16 else 5.0)
    slots = torch.randperm(pages * page, generator=gen)[:tokens].to(torch.int32)
    slots[tokens // 2] = -1 if tokens > 1 else slots[0]
    got = g.dequantize_cache(*(c[a] for a in ("k_cache", "v_cache", "k_scale", "v_scale")), slots.cuda(),
                             dtype=dtype)
    for kind, y in zip("kv", got):
        want = rounded(ref.values(c[kind + "_cache"], c[kind + "_scale"]).flatten(0, 1)[slots.long()], dtype)
        want[slots == -1] = 0
        assert y.dtype == dtype and torch.equal(y.cpu(), want), kind


def test_read_into_strided_tensors_and_refusals():
    gen = generator(9)
    c = caches(gen, 4, 16, 8, 2, 64)
    c["k_scale"][0, 0, 0], c["k_scale"][0, 0, 1], c["k_scale"][0, 1, 0] = 255, 254, 0
    c["v_cache"].view(torch.uint8)[0, 3, 1, 5] = 0x7f
    slots = torch.tensor([0, 64, 3, -5, -1, 17, 9], dtype=torch.int32, device="cuda")
    packed = torch.full((7, 6, 64), 5.0, dtype=torch.float16, device="cuda")
    g.dequantize_cache(c["k_cache"].view(torch.uint8), c["v_cache"], c["k_scale"], c["v_scale"], slots,
                       torch.float16, k_out=packed[:, 1:3], v_out=packed[:, 4:])
    with pytest.raises(g.GemmError, match="cache slot"):
        g.check_decode_status()
    at = slots.cpu().long()
    for kind, y in (("k", packed[:, 1:3]), ("v", packed[:, 4:])):
        want = rounded(ref.values(c[kind + "_cache"], c[kind + "_scale"]).flatten(0, 1)[at.clamp(0, 63)],
                       torch.float16)
        want[(at < 0) | (at > 63)] = 0
        assert torch.equal(y.cpu().isnan(), want.isnan())
        assert torch.equal(y.cpu().nan_to_num(nan=0.0), want.nan_to_num(nan=0.0)), kind
    assert bool((packed[:, 0] == 5).all() and (packed[:, 3] == 5).all())


# ---- attention ---------------------------------------------------------------------------------------

def attention_inputs(gen, lens, h_q, h_kv, d, page, block, dtype, width=None, spread=1.0, extra=2):
    lens = torch.tensor(lens, dtype=torch.int32)
    used = (lens.clamp(min=0) + page - 1) // page
    width = max(1, int(used.max())) if width is None else width
    total = int(used.sum()) + extra
    order = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.full((len(lens), width), 2 ** 30, dtype=torch.int32)     # past the length: not read
    at = 0
    for i, u in enumerate(used.tolist()):
        table[i, :u] = order[at:at + u]
        at += u
    c = caches(gen, total, page, block, h_kv, d, spread=spread)
    q = normal(gen, len(lens), h_q, d).to(dtype).cuda()
    return q, c, table.cuda(), lens.cuda()


def attend(q, c, table, lens, **kw):
    return g.paged_attention_fp8(q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], table, lens, **kw)


def check_attention(q, c, table, lens, where, scale=None, window=None, sinks=0, **kw):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    o, lse = attend(q, c, table, lens, scale=scale, window=window, sinks=sinks, return_lse=True, **kw)
    o_ref, lse_ref, ob, lb = ref.paged_attention(q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
                                                 table, lens, scale, window, sinks)
    ref.assert_close(o, o_ref, ob, f"{where}: o")
    ref.assert_close(lse, lse_ref, lb, f"{where}: lse")
    return o, lse


@DTYPES
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (4, 4), (6, 2), (8, 1), (9, 1), (16, 1), (24, 1), (40, 2)])
@pytest.mark.parametrize("page,block", [(16, 16), (20, 10), (64, 32), (5, 1)])
def test_attention(page, block, h_q, h_kv, d, dtype):
    gen = generator(d + h_q + page)
    args = attention_inputs(gen, [1, 0, 17, 130, 64, 301], h_q, h_kv, d, page, block, dtype)
    check_attention(*args, "ragged")


@DTYPES
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page,block", [(16, 8), (12, 12)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (16, 16), (33, 17), (100, 4), (100, 40),
                                          (250, 130), (1000, 4)])
def test_window_and_first_tokens(window, sinks, page, block, d, dtype):
    gen = generator(window + sinks + d)
    lens = [1, 0, window, window + 1, min(window + sinks, 400), min(window + sinks + 1, 400), 300, 131]
    args = attention_inputs(gen, lens, 6, 2, d, page, block, dtype)
    check_attention(*args, "window", window=window, sinks=sinks)


@DTYPES
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 1, 128), (16, 1, 256), (3, 1, 64), (16, 1, 64)])
def test_long_sequences(h_q, h_kv, d, dtype):
    """Ranges that are cut into parts and joined: one long sequence, and it beside short ones."""
    gen = generator(11)
    args = attention_inputs(gen, [40007], h_q, h_kv, d, 64, 16, dtype)
    check_attention(*args, "one")
    args = attention_inputs(gen, [5, 20011, 0, 333, 1, 9000], h_q, h_kv, d, 20, 20, dtype)
    check_attention(*args, "beside short ones")
    check_attention(*args, "windows", window=3001, sinks=70)


def test_many_sequences():
    """More items than the join lists one by one; checked against single calls."""
    gen = generator(12)
    lens = torch.randint(0, 90, (300,), generator=gen).tolist()
    q, c, table, lens = attention_inputs(gen, lens, 8, 4, 128, 16, 16, torch.bfloat16)
    o, lse = attend(q, c, table, lens, return_lse=True)
    pick = [0, 1, 77, 150, 298, 299]
    few = (q[pick], c, table[pick], lens[pick])
    o_ref, lse_ref, ob, lb = ref.paged_attention(few[0], *(c[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")),
                                                 few[2], few[3], 128 ** -0.5, None, 0)
    ref.assert_close(o[pick], o_ref, ob, "o")
    ref.assert_close(lse[pick], lse_ref, lb, "lse")
    assert bool(o.isfinite().all())


def test_wide_table_and_workspace():
    """A table much wider than the lengths need takes the other launch; both give the same within their
    bounds, with one workspace after another's use of it."""
    gen = generator(13)
    q, c, table, lens = attention_inputs(gen, [500, 33], 32, 8, 128, 16, 16, torch.bfloat16)
    ws = g.paged_attention_fp8_workspace(32, 8, 128)
    ws.fill_(255)
    check_attention(q, c, table, lens, "narrow", workspace=ws)
    wide = torch.cat([table, torch.full((2, 2000), -1, dtype=torch.int32, device="cuda")], 1)
    check_attention(q, c, wide, lens, "wide", workspace=ws)
    check_attention(q, c, wide, lens, "wide again", workspace=ws, out=torch.empty_like(q))
    copy = q.clone()
    want = attend(copy, c, wide, lens)
    assert torch.equal(attend(copy, c, wide, lens, out=copy), want)


@DTYPES
@pytest.mark.parametrize("page", [16, 20])
def test_unseen_contents_reach_no_result(page, dtype):
    """NaN in codes and scales wherever no token is seen: past the length in its last page and block,
    between first tokens and window, in pages of others."""
    gen = generator(14)
    lens = [page * 3 + 3, page * 12 + 5, 2]
    q, c, table, lens = attention_inputs(gen, lens, 4, 2, 128, page, page // 4, dtype)
    window, sinks = page * 4, 5
    seen = torch.zeros(c["k_cache"].shape[:2], dtype=torch.bool)
    for i, length in enumerate(lens.tolist()):
        start = max(0, length - window)
        for t in list(range(min(sinks, start))) + list(range(start, length)):
            seen[table[i, t // page].item(), t % page] = True
    blocks = seen.unflatten(1, (4, -1)).any(-1)
    clean = {x: y.clone() for x, y in c.items()}
    for kind in "kv":
        c[kind + "_cache"].view(torch.uint8)[~seen.cuda()] = 0x7f
        c[kind + "_scale"][~blocks.cuda()] = 255
    o, lse = attend(q, c, table, lens, window=window, sinks=sinks, return_lse=True)
    want = attend(q, clean, table, lens, window=window, sinks=sinks, return_lse=True)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_seen_nan_reaches_its_heads_alone():
    gen = generator(15)
    q, c, table, lens = attention_inputs(gen, [100, 100], 4, 2, 128, 16, 16, torch.bfloat16)
    clean = attend(q, c, table, lens)
    c["v_cache"].view(torch.uint8)[table[0, 2], 3, 1, 7] = 0xff            # one element: of heads 2 and 3
    c["k_scale"][table[1, 1], 0, 0] = 255                    # a block of keys: of heads 0 and 1
    o, lse = attend(q, c, table, lens, return_lse=True)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[0, 2:, 7] = True
    bad[1, :2] = True
    assert torch.equal(o.isnan(), bad)
    assert torch.equal(o[~bad], clean[~bad])
    assert torch.equal(lse.isnan().cpu(), torch.tensor([[False] * 4, [True, True, False, False]]))


@DTYPES
def test_scales_far_apart(dtype):
    """Blocks of sizes 2^-20 .. 2^20 of each other (values), queries of sizes far from 1."""
    gen = generator(16)
    q, c, table, lens = attention_inputs(gen, [200, 77], 4, 2, 128, 16, 8, dtype)
    c["v_scale"] = (c["v_scale"].int() + torch.randint(-20, 21, c["v_scale"].shape, generator=gen).cuda()
                    ).to(torch.uint8)
    check_attention(q, c, table, lens, "values")
    small = 2.0 ** -100 if dtype == torch.bfloat16 else 2.0 ** -12
    for by in (small, 1 / small / 2 if dtype == torch.bfloat16 else 2.0 ** 10):
        check_attention((q.double() * by).to(dtype), c, table, lens, f"queries by {by}", scale=128 ** -0.5 / by)
    c["v_scale"][:] = 0
    check_attention(q, c, table, lens, "the smallest scale")
    big = 240 if dtype == torch.bfloat16 else 127
    c["v_scale"][:] = big
    check_attention(q, c, table, lens, "a large scale")


def test_queries_that_are_no_numbers():
    gen = generator(17)
    q, c, table, lens = attention_inputs(gen, [60, 40], 4, 2, 64, 16, 16, torch.bfloat16)
    clean = attend(q, c, table, lens)
    q[0, 1, 5] = math.nan
    q[1, 2] = 0
    o, lse = attend(q, c, table, lens, return_lse=True)
    assert bool(o[0, 1].isnan().all()) and bool(lse[0, 1].isnan())
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[0, 1] = keep[1, 2] = False
    assert torch.equal(o[keep], clean[keep])
    check_attention(q[1:], c, table[1:], lens[1:], "a query of zeros")


def test_attention_refusals():
    gen = generator(18)
    q, c, table, lens = attention_inputs(gen, [30, 40, 50], 4, 2, 128, 16, 16, torch.bfloat16)
    clean = attend(q, c, table, lens)
    for bad in (-1, 16 * table.shape[1] + 1, 2 ** 31 - 1, -2 ** 31):
        at = lens.clone()
        at[1] = bad
        o, lse = attend(q, c, table, at, return_lse=True)
        assert torch.equal(o[[0, 2]], clean[[0, 2]])
        assert bool((o[1] == 0).all()) and bool((lse[1] == -math.inf).all())
        with pytest.raises(g.GemmError, match="sequence length"):
            g.check_decode_status()
    for bad in (-1, c["k_cache"].shape[0], 2 ** 31 - 1):
        other = table.clone()
        other[1, 1] = bad
        o = attend(q, c, other, lens)
        assert torch.equal(o[[0, 2]], clean[[0, 2]])
        with pytest.raises(g.GemmError, match="page number"):
            g.check_decode_status()
    with pytest.raises(ValueError, match="sinks come with a window"):
        attend(q, c, table, lens, sinks=2)
    with pytest.raises(ValueError, match="sinks"):
        attend(q, c, table, lens, window=4, sinks=-1)
    with pytest.raises(ValueError, match="window"):
        attend(q, c, table, lens, window=0)
    with pytest.raises(ValueError, match="scales do not share"):
        attend(q, {**c, "k_scale": c["k_scale"].repeat(1, 3, 1)}, table, lens)
    with pytest.raises(ValueError, match="v_scale must be"):
        attend(q, {**c, "v_scale": c["v_scale"].repeat(1, 2, 1)}, table, lens)
    with pytest.raises(ValueError, match="k_cache must be torch.float8"):
        attend(q, {**c, "k_cache": c["k_cache"].half()}, table, lens)
    with pytest.raises(g.GemmError, match="workspace of"):
        attend(q, c, table, lens, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(g.GemmError, match="workspace shares memory"):
        ws = g.paged_attention_fp8_workspace(4, 2, 128)
        attend(q, c, table, lens, workspace=ws, out=ws[:q.numel() * 2].view(torch.bfloat16).view(q.shape))


def test_attention_without_tokens_or_pages():
    gen = generator(19)
    q, c, table, lens = attention_inputs(gen, [0, 0], 4, 2, 64, 16, 16, torch.float16)
    o, lse = attend(q, c, table, lens, return_lse=True)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    none = {x: y[:0] for x, y in c.items()}
    o = attend(q, none, table[:, :0], lens)
    assert bool((o == 0).all())
    assert attend(q[:0], c, table[:0], lens[:0]).shape == (0, 4, 64)


def test_recorded_attention_follows_lengths_and_tables():
    gen = generator(20)
    q, c, table, lens = attention_inputs(gen, [300, 40, 1000], 8, 2, 128, 16, 16, torch.bfloat16)
    attend(q, c, table, lens, window=500, sinks=4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = attend(q, c, table, lens, window=500, sinks=4, return_lse=True)
    for now in ([300, 40, 1000], [17, 0, 999], [304, 48, 1]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        o_ref, lse_ref, ob, lb = ref.paged_attention(q, *(c[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")),
                                                     table, lens, 128 ** -0.5, 500, 4)
        ref.assert_close(o, o_ref, ob, f"{now}: o")
        ref.assert_close(lse, lse_ref, lb, f"{now}: lse")


def test_graphs_that_share_a_workspace():
    """Two recorded calls with one workspace between them, replayed in turn, and a third on its own on
    another stream at the same time."""
    gen = generator(22)
    first = attention_inputs(gen, [900, 0, 77], 8, 2, 128, 16, 16, torch.bfloat16)
    second = attention_inputs(gen, [5, 4000], 8, 2, 128, 20, 10, torch.bfloat16)
    want = [attend(*x) for x in (first, second)]
    ws = g.paged_attention_fp8_workspace(8, 2, 128)
    graphs, outs = [], []
    for x in (first, second):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(attend(*x, workspace=ws))
        graphs.append(graph)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for o in outs:
            o.zero_()
        for graph in graphs:
            graph.replay()
        with torch.cuda.stream(stream):
            other = attend(*second)
        torch.cuda.synchronize()
        for o, w in zip(outs + [other], want + want[1:]):
            assert torch.equal(o, w)


def test_cache_past_32_bits():
    """Pages whose bytes lie past 2^32 of the cache's first."""
    gen = generator(21)
    h, d, page = 8, 128, 64
    pages = (1 << 32) // (page * h * d) + 70
    big = [torch.empty(pages, page, h, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages, 4, h, dtype=torch.uint8, device="cuda") for _ in range(2)]
    q = normal(gen, 2, 16, d).bfloat16().cuda()
    lens = torch.tensor([150, 64], dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, 1, pages - 60], [pages - 2, 0, 0]], dtype=torch.int32, device="cuda")
    at = torch.cat([torch.arange(150), torch.arange(64)])
    seq = torch.tensor([0] * 150 + [1] * 64)
    slots = (table.cpu()[seq, at // page].long() * page + at % page).to(torch.int32).cuda()
    x = {kind: normal(gen, 214, h, d).bfloat16().cuda() for kind in "kv"}
    c = {"k_cache": big[0].view(E4M3), "v_cache": big[1].view(E4M3), "k_scale": scales[0], "v_scale": scales[1]}
    write(c, x, slots)
    k, v = g.dequantize_cache(*big, *scales, slots)
    used = table.flatten().unique().long()
    few = {a: b[used] for a, b in c.items()}
    for kind, y in (("k", k), ("v", v)):
        scale = x[kind].double().abs().cpu()
        err = (y.double().cpu() - x[kind].double().cpu()).abs()
        assert bool((err <= 2.0 ** -4 * scale + 2.0 ** -10 * 6 * 2.0 ** -6).all()), kind
    o = attend(q, c, table, lens)
    small = torch.searchsorted(used, table.long()).to(torch.int32)
    check_attention(q, few, small, lens, "the same in a small cache")
    assert torch.equal(o, attend(q, few, small, lens))


# ---- the linear layer --------------------------------------------------------------------------------

def weights(gen, n, k, group, dtype, zeros, bias):
    groups = -(-k // group) if k else 0
    s = {"codes": torch.randint(0, 256, (n, k // 2), generator=gen, dtype=torch.uint8).cuda(),
         "scales": (torch.rand(n, groups, generator=gen) + 0.1).to(dtype).cuda(), "group": group}
    if zeros:
        s["zeros"] = torch.randint(0, 16, (n, groups), generator=gen, dtype=torch.uint8).cuda()
    if bias:
        s["bias"] = (3 * normal(gen, n)).to(dtype).cuda()
    return s


def check_linear(x, s, where, **kw):
    y = g.linear_w4(x, **s, **kw)
    kw.pop("out", None), kw.pop("stream", None)
    y_ref, bound = ref.linear_w4(x, **s, **kw)
    ref.assert_close(y, y_ref, bound, where)
    return y


@DTYPES
@pytest.mark.parametrize("k,group", [(32, 32), (64, 128), (256, 32), (288, 64), (1024, 96), (4128, 128),
                                     (2048, 160), (512, 512), (1056, 1056)])
@pytest.mark.parametrize("n", [1, 129, 700])
@pytest.mark.parametrize("m", [1, 8, 9, 33])
def test_linear(m, n, k, group, dtype):
    gen = generator(m + n + k)
    x = (0.2 * normal(gen, m, k)).to(dtype).cuda()
    check_linear(x, weights(gen, n, k, group, dtype, m % 2 == 0, n % 2 == 1), f"{m} x {n} x {k}",
                 activation=("none", "relu", "gelu")[(m + n) % 3])


@DTYPES
@pytest.mark.parametrize("m", [2, 5, 7, 16, 17, 24, 32, 64, 70, 200])
@pytest.mark.parametrize("activation", ["none", "relu", "gelu"])
def test_linear_tokens(m, activation, dtype):
    gen = generator(m)
    x = (0.3 * normal(gen, m, 640)).to(dtype).cuda()
    check_linear(x, weights(gen, 300, 640, 64, dtype, True, True), f"{m} tokens", activation=activation)


@pytest.mark.parametrize("n,k", [(5000, 1024), (20000, 512), (128, 8192), (1000, 14336)])
def test_linear_shapes(n, k):
    """Outputs for more blocks than the GPU holds, and so few that their columns are shared out."""
    gen = generator(n)
    x = (0.1 * normal(gen, 3, k)).bfloat16().cuda()
    check_linear(x, weights(gen, n, k, 128, torch.bfloat16, True, False), f"{n} x {k}")


@DTYPES
@pytest.mark.parametrize("n,k,group", [(128, 8192, 128), (1000, 14336, 64), (20000, 512, 32), (130, 4128, 96),
                                       (2500, 2080, 128)])
@pytest.mark.parametrize("m", [7, 16, 31, 64, 129])
def test_linear_shapes_of_more_tokens(m, n, k, group, dtype):
    """Columns shared out by two, four and eight, more blocks than the GPU holds, and last chunks of 32 and
    64 columns."""
    gen = generator(n + m)
    x = (0.1 * normal(gen, m, k)).to(dtype).cuda()
    check_linear(x, weights(gen, n, k, group, dtype, True, False), f"{m} x {n} x {k}")


@pytest.mark.parametrize("m", [9, 40, 100])
def test_linear_of_strided_tokens(m):
    """Tokens between others, and the same one for all; what other calls left on the chip (NaN) reaches
    no result."""
    gen = generator(m)
    n, k = 200, 352
    s = weights(gen, n, k, 96, torch.float16, True, True)
    nothing = torch.full((128, k), math.nan, dtype=torch.float16, device="cuda")
    packed = (0.3 * normal(gen, m, 3, k)).half().cuda()
    out = torch.full((m, 2, n + 3), 7.0, dtype=torch.float16, device="cuda")
    g.linear_w4(nothing, **s)
    check_linear(packed[:, 1], s, "strided", out=out[:, 1, :n])
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 1, n:] == 7).all())
    g.linear_w4(nothing, **s)
    check_linear(packed[:1, 2].expand(m, k), s, "broadcast")


def test_linear_beside_other_work():
    """The same results from calls on two streams at once, beside a matrix product on a third."""
    gen = generator(36)
    cases = [((0.2 * normal(gen, m, k)).half().cuda(), weights(gen, n, k, 128, torch.float16, True, False))
             for m, n, k in ((3, 1024, 4096), (16, 4096, 4096), (64, 1024, 4096), (48, 5000, 1024))]
    want = [g.linear_w4(x, **s) for x, s in cases]
    A, B = (torch.randn(1024, 2048, dtype=torch.float16, device="cuda") for _ in range(2))
    product = g.linear(A, B)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(24):
        got += [(j, g.linear_w4(cases[j][0], **cases[j][1], stream=streams[i % 2]))
                for j in ((i + 1) % 4, (i // 2) % 4)]
        if i % 3 == 0:
            got.append((-1, g.linear(A, B, stream=streams[2])))
    torch.cuda.synchronize()
    for j, y in got:
        assert torch.equal(y, want[j] if j >= 0 else product), j
    g.check_decode_status()


def test_linear_of_strided_operands():
    gen = generator(31)
    n, k = 200, 320
    store = torch.randint(0, 256, (n, 192), generator=gen, dtype=torch.uint8).cuda()
    scales = (torch.rand(n, 13, generator=gen) + 0.1).half().cuda()
    zeros = torch.randint(0, 256, (n, 17), generator=gen, dtype=torch.uint8).cuda()
    packed = (0.3 * normal(gen, 6, 2 * k)).half().cuda()
    out = torch.full((6, 2, n + 3), 7.0, dtype=torch.float16, device="cuda")
    s = dict(codes=store[:, 16:16 + k // 2], scales=scales[:, 2:7], zeros=zeros[:, 5:10], group=64)
    want, bound = ref.linear_w4(packed[:, k:], **{**s, "zeros": s["zeros"] & 15})
    y = g.linear_w4(packed[:, k:], **s, out=out[:, 1, :n])
    assert y.data_ptr() == out[:, 1].data_ptr()
    ref.assert_close(y, want, bound, "strided")
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 1, n:] == 7).all())
    one = packed[:1, :k].expand(6, k)                         # the same token for all
    check_linear(one, {**s, "zeros": s["zeros"] & 15}, "broadcast")


def test_linear_of_what_is_no_number():
    """An infinity or NaN of a token reaches its own outputs alone; one of a scale its row's."""
    gen = generator(32)
    x = normal(gen, 10, 256).bfloat16().cuda()
    s = weights(gen, 40, 256, 64, torch.bfloat16, True, False)
    clean = g.linear_w4(x, **s)
    x[3, 100], x[9, 5] = math.inf, math.nan
    s["scales"][7, 2] = math.nan
    y = g.linear_w4(x, **s)
    y_ref, _ = ref.linear_w4(x, **s)
    assert torch.equal(y.isfinite().cpu(), y_ref.isfinite())
    keep = y.isfinite()
    assert bool(keep[:3, :7].all()) and not keep[3].any() and not keep[:, 7].any()
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("m", [3, 20])
@pytest.mark.parametrize("exponent", [-118, -100, 100, 112])
def test_linear_of_small_and_large_tokens(m, exponent):
    """Elements near the ends of bfloat16's range: nothing is flushed to zero or overflows on the way."""
    gen = generator(m)
    x = (normal(gen, m, 256).double() * 2.0 ** exponent).bfloat16().cuda()
    check_linear(x, weights(gen, 200, 256, 128, torch.bfloat16, True, False), f"2^{exponent}")


def test_linear_without_columns_and_refusals():
    gen = generator(33)
    s = weights(gen, 5, 0, 32, torch.float16, False, True)
    y = g.linear_w4(torch.empty(3, 0, dtype=torch.float16, device="cuda"), **s)
    assert torch.equal(y, s["bias"].expand(3, 5))
    s = weights(gen, 8, 64, 32, torch.float16, True, True)
    x = normal(gen, 4, 64).half().cuda()
    assert g.linear_w4(x[:0], **s).shape == (0, 8)
    with pytest.raises(ValueError, match="codes must be"):
        g.linear_w4(x[:, :32], **s)
    with pytest.raises(ValueError, match="scales must be"):
        g.linear_w4(x, **{**s, "group": 64})
    with pytest.raises(ValueError, match="scales must be torch.bfloat16"):
        g.linear_w4(x.bfloat16(), **s)
    with pytest.raises(ValueError, match="group"):
        g.linear_w4(x, **{**s, "group": 0})
    with pytest.raises(ValueError, match="zeros must be"):
        g.linear_w4(x, **{**s, "zeros": s["zeros"][:, :1]})
    with pytest.raises(g.GemmError, match="y shares memory with x"):
        g.linear_w4(x, **s, out=x[:, :8])
    with pytest.raises(g.GemmError, match="multiples of 32"):
        g.linear_w4(x[:, :48], s["codes"][:, :24], s["scales"][:, :2], 32)
    with pytest.raises(ValueError, match="overlap"):
        g.linear_w4(x, **s, out=torch.empty(8, dtype=torch.float16, device="cuda").expand(4, 8))


def test_linear_on_another_stream_and_in_a_graph():
    gen = generator(34)
    x = normal(gen, 4, 1024).bfloat16().cuda()
    s = weights(gen, 384, 1024, 128, torch.bfloat16, True, False)
    want = g.linear_w4(x, **s)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    y = g.linear_w4(x, **s, stream=stream)
    stream.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = g.linear_w4(g.linear_w4(x, **s, activation="relu")[:, :384].repeat(1, 3)[:, :1024], **s)
    graph.replay()
    first = y.clone()
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(first, y)
    step = g.linear_w4(g.linear_w4(x, **s, activation="relu").repeat(1, 3)[:, :1024], **s)
    assert torch.equal(step, y)


@DTYPES
def test_quantised_weights_through_the_layer(dtype):
    """quantize_weight_w4's operands give what the weights that they stand for give."""
    gen = generator(35)
    W = (0.05 * normal(gen, 200, 512)).to(dtype).cuda()
    x = normal(gen, 6, 512).to(dtype).cuda()
    for zeros in (True, False):
        codes, scales, z = g.quantize_weight_w4(W, 64, zeros)
        check_linear(x, dict(codes=codes, scales=scales, zeros=z, group=64), f"zeros {zeros}")


def test_pages_without_tokens_are_refused():
    """(their blocks of no token divide by 0)"""
    x = torch.zeros(2, 1, 64, dtype=torch.float16, device="cuda")
    codes = torch.zeros(3, 0, 1, 64, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(3, 1, 1, dtype=torch.uint8, device="cuda")
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="hold a token"):
        g.quantize_cache(x, x, codes, codes, scale, scale, at)
    with pytest.raises(ValueError, match="hold a token"):
        g.dequantize_cache(codes, codes, scale, scale, at)
    with pytest.raises(ValueError, match="hold a token"):
        g.paged_attention_fp8(x, codes, codes, scale, scale, at[:, None], at)


@DTYPES
@pytest.mark.parametrize("h_q,h_kv,d", [(4, 2, 64), (9, 1, 64), (4, 2, 128), (12, 1, 128), (4, 2, 256), (16, 1, 256)])
@pytest.mark.parametrize("whole", [False, True], ids=["blocks", "stretch"])
@pytest.mark.parametrize("apart,weight", [(5, 0), (12, -40), (30, 0), (60, 0), (60, -40), (100, 0), (100, -60),
                                          (110, -100)])
def test_large_values_of_little_weight(apart, weight, whole, h_q, h_kv, d, dtype):
    """Blocks whose values are 2^apart larger, with weights 2^(weight - apart) of the others', so that they
    matter as much or not at all: among the others' blocks, and as the first 1000 tokens of 1500.  (2^110 times
    codes to 448, over 1000 tokens, stays a number of fp32, in which a part of a sequence is summed by itself.)"""
    gen = generator(apart + d + h_q)
    q, c, table, lens = attention_inputs(gen, [40, 1500, 9], h_q, h_kv, d, 16, 8, dtype)
    c = {x: y.cpu() for x, y in c.items()}
    q = (torch.rand(3, h_q, d, generator=gen) + 0.5).to(dtype).cuda()
    k = 0.1 * normal(gen, *c["k_cache"].shape)
    large = torch.rand(c["k_cache"].shape[0], 2, generator=gen) < 0.3                  # pages, blocks
    if whole:
        large[:] = False
        large[table[1, :1000 // 16].cpu().long()] = True
    score = (apart - weight) * math.log(2)                                             # of which e^-score is left
    k[large.repeat_interleave(8, 1)] = -score / d ** 0.5                               # (queries are 1 on average)
    e = torch.where(large, 127 - 4, 127 - 8)[..., None].expand(-1, -1, h_kv)
    c["k_scale"] = e.to(torch.uint8).contiguous()
    c["k_cache"] = (k * torch.exp2(127.0 - e)[:, :, None, :, None].expand(-1, -1, 8, -1, -1).flatten(1, 2)).to(E4M3)
    c["v_scale"] = (c["v_scale"].int() + apart * large[..., None].int()).to(torch.uint8)
    c = {x: y.cuda() for x, y in c.items()}
    o, lse = attend(q, c, table, lens, return_lse=True)
    o_ref, lse_ref, ob, lb = ref.paged_attention_by_weight(q, c, table, lens, d ** -0.5)
    # (a short sequence may have large values alone: from half a step past the type's largest number on, what a
    # value within the bound is rounded to is infinity)
    most = torch.finfo(dtype).max
    most += ref.U[dtype] * 2.0 ** math.floor(math.log2(most))
    past = o.cpu().double() == o_ref.sign() * math.inf
    assert bool((o_ref.abs() + ob >= most)[past].all()) and bool(past[o_ref.abs() - ob >= most].all())
    ref.assert_close(o.cpu().masked_fill(past, 0), o_ref.masked_fill(past, 0), ob.masked_fill(past, 0), "o")
    ref.assert_close(lse, lse_ref, lb, "lse")


@pytest.mark.parametrize("m", [1, 6, 12, 40])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("scale,token", [(122, -122), (126, -126), (127, -133), (-110, 110), (-126, 118), (-66, -60),
                                         (0, -133), (0, -126), (0, 118)])
def test_linear_of_small_and_large_scales(scale, token, group, m):
    """Scales and elements at either end of bfloat16's range, subnormal elements among them: a sum of 128
    products of elements below 2^121 stays below 2^134."""
    gen = generator(m + scale)
    x = (normal(gen, m, 384).double() * 2.0 ** token).bfloat16().cuda()
    s = weights(gen, 150, 384, group, torch.bfloat16, True, False)
    s["scales"] = (0.9 * s["scales"].double() * 2.0 ** scale).bfloat16()
    check_linear(x, s, f"2^{scale} x 2^{token}")


@pytest.mark.parametrize("apart", [129, 143, 144, 145, 159, 160])
@pytest.mark.parametrize("again", [[0, 1], [3], [-1, 1]])
@pytest.mark.parametrize("many", [0, 3000, 9000, 17000])
@pytest.mark.parametrize("last_of_window", [False, True])
def test_write_of_a_block_in_two_runs_far_apart(last_of_window, many, again, apart):
    """The farthest second runs that are refused, at the first and at the last token of a window, with windows of
    1, 2, 8 and 16 tokens."""
    gen = generator(apart + many)
    lead = ((15 if last_of_window else 0) - apart) % 16
    others = iter(range(8, 8 * 400, 8))
    between = apart - 1 - (again[0] == -1)       # (inactive, and the run behind it is `apart` behind)
    slots = [next(others) for _ in range(lead)] + [0] + [next(others) for _ in range(between)]
    kept = list(range(len(slots)))
    slots += again
    slots = torch.tensor(slots + [-1] * many, dtype=torch.int32)
    c = caches(gen, 200, 16, 8, 2, 64)
    before = {a: b.clone() for a, b in c.items()}
    x = {kind: normal(gen, len(slots), 2, 64).half().cuda() for kind in "kv"}
    write(c, x, slots.cuda())
    check_cache(c, before, {kind: y[kept] for kind, y in x.items()}, slots[kept], "kept")
    with pytest.raises(g.GemmError, match="cache slot"):
        g.check_decode_status()
