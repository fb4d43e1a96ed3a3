"""The decode-step operators on the GPU where they can go wrong: results that cancel, infinities,
sequences whose every score is masked, operands that share memory, and the kernels' less travelled
paths."""
from __future__ import annotations

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
import decode_ref as ref
from test_decode_gpu import (attn_inputs, cache_pair, cuda_library, generator,  # noqa: F401
                             no_refusals_left, norm_call, norm_inputs, norm_refs, normal,
                             step_inputs)

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])


# ---- attention: the weights' bits -------------------------------------------------------------------

def cancelling(lens, h_q, h_kv, d, dtype, seed):
    """Token 0 of each sequence outweighs the others (by up to e) and has a zero value; the others
    come in pairs of nearly the same weight and the values 3 and -3.  Queries and keys have two
    elements each, chosen so that every score before its scale is exact in fp32."""
    s = attn_inputs(lens, h_q, h_kv, d, 16, dtype, seed=seed)
    gen = generator(seed + 90)
    n = len(lens)
    s["q"].zero_()
    s["q"][..., 0] = (2 + torch.randint(0, 64, (n, h_q), generator=gen) / 32.0).to(dtype).cuda()
    s["q"][..., 1] = (0.5 + torch.randint(0, 64, (n, h_q), generator=gen) / 128.0).to(dtype).cuda()
    for i, length in enumerate(lens):
        tok = torch.arange(length)
        pair, second = (tok + 1) // 2, (tok + 1) % 2
        key, value = torch.zeros(length, h_kv, d), torch.zeros(length, h_kv, d)
        base = -torch.randint(1, 64, (length // 2 + 1, h_kv), generator=gen) / 64.0
        base[0] = 0.0
        key[..., 0] = base[pair]
        key[..., 1] = 2.0 ** -10 * second[:, None]
        value[:] = (3.0 - 6.0 * second)[:, None, None]
        value[0] = 0.0
        if length % 2 == 0:
            value[-1] = 0.0
        pg, of = s["table"][i].long()[tok.cuda() // 16], tok.cuda() % 16
        s["k_cache"][pg, of], s["v_cache"][pg, of] = key.to(dtype).cuda(), value.to(dtype).cuda()
    return s


@DTYPES
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (16, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[3] * 40 + [5, 18, 300], [700, 9000]], ids=["short", "long"])
def test_attention_weights_keep_their_bits(lens, d, h_q, h_kv, dtype):
    """Results that are small differences of large terms, whose rounding to 16 bits hides nothing.
    The scale and its product with log2 e (3 e of scores up to 1.5), the reference's subtraction (e) and
    the exponential (4 e) bend a weight, its pieces by 2 e at most, and the sums of a matrix
    product, of a warp's and of the blocks' by a few e more: 24 e of p |V| in all, where a weight
    rounded twice to 8 bits is off by up to 128 e."""
    s = cancelling(lens, h_q, h_kv, d, dtype, seed=d + h_q)
    o_ref, l_ref, _, _ = ref.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                             s["lens"], 0.25, None)
    o, lse = g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], scale=0.25,
                               return_lse=True)
    ref.assert_close(o, o_ref, torch.full_like(o_ref, 24 * ref.E * 3.0), "o")
    ref.assert_close(lse, l_ref, 24 * ref.E * (1 + l_ref.abs()), "lse")


@DTYPES
def test_attention_long_sums_lose_nothing(dtype):
    """A sequence a block, so that each warp adds up hundreds of slices, of values whose second half
    undoes the first: the result is 0, and what is left of it is what the running sums lost.  With
    P the sum of p |V| each of 512 additions rounds a sum of P / 4 on average by e at most, and a
    slice's matrix products lose 12 e of their own sum: 144 e P in all.  (A running sum in the
    matrix products, six of them a slice, loses about 0.75 e of P / 4 with each: 576 e P.)"""
    n = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    page, d, length = 64, 64, 65536
    gen = generator(101)
    half = torch.zeros(length // 2, d)
    half[:, 0] = torch.where(torch.arange(length // 2) % 16 == 0, 0.0,
                             -torch.randint(1, 64, (length // 2,), generator=gen) / 64.0)
    size = torch.randint(64, 128, (d,), generator=gen) / 32.0
    value = torch.where(half[:, :1] == 0, 0.0, size)
    cache = [torch.cat(x).view(-1, page, 1, d).to(dtype).cuda()
             for x in ((half, half), (value, -value))]
    q = torch.zeros(n, 1, d)
    q[..., 0] = 2 + torch.randint(0, 64, (n, 1), generator=gen) / 32.0
    table = torch.arange(length // page, dtype=torch.int32, device="cuda").expand(n, -1)
    lens = torch.full((n,), length, dtype=torch.int32, device="cuda")
    o = g.paged_attention(q.to(dtype).cuda(), *cache, table, lens, scale=0.25)
    ref.assert_close(o, torch.zeros(n, 1, d, dtype=torch.float64),
                     (144 * ref.E * size.double()).expand(n, 1, d), "o")


# ---- attention: infinities --------------------------------------------------------------------------

def on_split_path(s, to=4096):
    """The same call with a page table so wide that no cluster takes it (entries past a sequence's
    pages are not read)."""
    n, width = s["table"].shape
    wide = torch.full((n, width + to // int(s["k_cache"].shape[1])), 2 ** 31 - 1, dtype=torch.int32,
                      device="cuda")
    wide[:, :width] = s["table"]
    return dict(s, table=wide)


def assert_as_defined(o, o_ref, bound, where):
    """Infinities and NaN where the definition has them, the rest within its bound."""
    x = o.double().cpu()
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(kind(x), kind(o_ref)), f"{where}: {kind.__name__}"
    rest = o_ref.isfinite()
    ref.assert_close(o.cpu()[rest], o_ref[rest], bound[rest], where)


@DTYPES
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (16, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_infinite_values(d, h_q, h_kv, dtype):
    """An infinite cached value makes its element of the results infinite, whatever its weight and
    its sign, two of opposite signs NaN, and nothing else changes; short sequences and long ones, on clusters
    and on the split path, joined and not."""
    s = attn_inputs([1, 40, 300, 3000, 9], h_q, h_kv, d, 16, dtype, seed=d + h_q)
    place = lambda i, t: (s["table"][i, t // 16].long(), t % 16, 0)     # noqa: E731
    inf = float("inf")
    s["v_cache"][place(0, 0)][3], s["v_cache"][place(0, 0)][4] = inf, -inf
    for i, t in ((1, 39), (2, 150), (3, 2999)):
        s["v_cache"][place(i, t)][0] = inf
        s["v_cache"][place(i, t)][1] = -inf
        s["v_cache"][place(i, t)][2] = inf
        s["v_cache"][place(i, t - 20)][2] = -inf
    for case in (s, on_split_path(s)):
        o_ref, l_ref, ob, lb = ref.paged_attention(case["q"], case["k_cache"], case["v_cache"],
                                                   case["table"], case["lens"], d ** -0.5, None)
        o, lse = g.paged_attention(case["q"], case["k_cache"], case["v_cache"], case["table"],
                                   case["lens"], return_lse=True)
        assert int(o_ref.isinf().sum()) == 8 * h_q // h_kv and int(o_ref.isnan().sum()) == 3 * h_q // h_kv
        assert_as_defined(o, o_ref, ob, "o")
        ref.assert_close(lse, l_ref, lb, "lse")


@DTYPES
def test_attention_infinite_values_of_small_weight(dtype):
    """Weights of 2^-60 and 2^-100 of the largest still carry an infinite value."""
    s = attn_inputs([1000, 33], 8, 2, 64, 16, dtype, seed=7)
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    s["k_cache"][~s["k_cache"].isnan()] = 0.0
    for i, t, score in ((0, 5, -41.5), (0, 700, -69.5), (1, 20, -69.5)):
        at = (s["table"][i, t // 16].long(), t % 16)
        s["k_cache"][at][:, 0] = score
        s["v_cache"][at][:, 9 + t % 2] = float("-inf")
    for case in (s, on_split_path(s)):
        o_ref, _, ob, _ = ref.paged_attention(case["q"], case["k_cache"], case["v_cache"],
                                              case["table"], case["lens"], 1.0, None)
        o = g.paged_attention(case["q"], case["k_cache"], case["v_cache"], case["table"],
                              case["lens"], scale=1.0)
        assert int(o_ref.isneginf().sum()) == 3 * 8
        assert_as_defined(o, o_ref, ob, "o")


@DTYPES
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (16, 1)])
def test_attention_every_score_minus_infinity(h_q, h_kv, d, dtype):
    """A sequence whose every score is -infinity has the result of an empty one, whatever its values
    hold, beside sequences that go on as ever: in clusters, in blocks of their own, and joined."""
    s = attn_inputs([1, 40, 40, 300, 3000, 3000, 17], h_q, h_kv, d, 16, dtype, seed=d + h_q)
    s["q"].abs_().clamp_(min=0.01)
    for i in (0, 2, 5):
        tok = torch.arange(int(s["lens"][i]), device="cuda")
        pg = s["table"][i].long()[tok // 16]
        s["k_cache"][pg, tok % 16, :, 1] = float("-inf")
        s["v_cache"][pg[0], 0, :, 0] = float("inf")
    kept = [1, 3, 4, 6]
    for case in (s, on_split_path(s)):
        o_ref, l_ref, ob, lb = ref.paged_attention(case["q"][kept], case["k_cache"],
                                                   case["v_cache"], case["table"][kept],
                                                   case["lens"][kept], d ** -0.5, None)
        o, lse = g.paged_attention(case["q"], case["k_cache"], case["v_cache"], case["table"],
                                   case["lens"], return_lse=True)
        for i in (0, 2, 5):
            assert bool((o[i] == 0).all()) and bool((lse[i] == float("-inf")).all()), i
        ref.assert_close(o[kept], o_ref, ob, "o")
        ref.assert_close(lse[kept], l_ref, lb, "lse")


# ---- attention: both paths of every shape -----------------------------------------------------------

def path_of(case, **kw):
    """(the results, "cluster" or "split", whether an item was cut) of a call: a cluster leaves the
    workspace alone, the split path lists its items at its beginning and puts the parts of cut ones
    behind the list."""
    h_q, d = case["q"].shape[1:]
    ws = g.paged_attention_workspace(h_q, case["k_cache"].shape[2], d)
    ws.fill_(0xA5)
    got = g.paged_attention(case["q"], case["k_cache"], case["v_cache"], case["table"],
                            case["lens"], return_lse=True, workspace=ws, **kw)
    touched = ws != 0xA5
    return got, "split" if bool(touched.any()) else "cluster", bool(touched[16384:].any())


def check_on(case, path, cut=None, window=None):
    d = case["q"].shape[-1]
    o_ref, l_ref, ob, lb = ref.paged_attention(case["q"], case["k_cache"], case["v_cache"],
                                               case["table"], case["lens"], d ** -0.5, window)
    (o, lse), taken, was_cut = path_of(case, window=window)
    assert taken == path and cut in (None, was_cut)
    ref.assert_close(lse, l_ref, lb, "lse")
    ref.assert_close(o, o_ref, ob, "o")


def mixed_lengths(n, seed):
    """Empty, short and long sequences in no order."""
    gen = generator(seed)
    lens = torch.randint(1, 260, (n,), generator=gen)
    lens[::9] = 0
    lens[4::11] = torch.randint(500, 2500, (len(lens[4::11]),), generator=gen)
    return lens


@DTYPES
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(9, 1), (20, 1), (40, 2), (16, 2), (3, 1)])
def test_attention_heads_on_the_split_path(h_q, h_kv, d, dtype):
    """Groups of up to 24 query heads a key head, two items a key head among them, with blocks that
    take several whole items and items that several blocks take."""
    s = attn_inputs(mixed_lengths(110, h_q + d), h_q, h_kv, d, 16, dtype, seed=h_q + d)
    check_on(on_split_path(s), "split", cut=True)


@pytest.mark.parametrize("h_q,h_kv", [(16, 1), (40, 2)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_whole_items_of_many_heads(d, h_q, h_kv):
    """More short sequences than blocks: a block's items follow one another, with queries of their
    own, and few are cut."""
    gen = generator(d)
    lens = torch.randint(0, 60, (620,), generator=gen)
    s = attn_inputs(lens, h_q, h_kv, d, 16, torch.bfloat16, seed=d)
    check_on(on_split_path(s), "split")


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("h_q,h_kv", [(16, 1), (8, 1)])
def test_attention_one_long_sequence_of_many_heads(d, h_q, h_kv):
    s = attn_inputs([30011], h_q, h_kv, d, 16, torch.float16, seed=d)
    check_on(s, "split", cut=True)


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16),
                                     (256, torch.bfloat16)], ids=["64", "128", "256"])
@pytest.mark.parametrize("window", [None, 1, 37, 333])
@pytest.mark.parametrize("page", [1, 7, 20, 48, 100])
def test_attention_pages_and_windows_on_the_split_path(page, window, d, dtype):
    """Pages that end inside a slice, with a window that starts inside one; what lies before the
    window is NaN."""
    s = attn_inputs(mixed_lengths(160, page + d), 6, 2, d, page, dtype, seed=page + d)
    if window:
        for i, length in enumerate(s["lens"].tolist()):
            tok = torch.arange(max(0, length - window), device="cuda")
            at = (s["table"][i].long()[tok // page], tok % page)
            s["k_cache"][at], s["v_cache"][at] = float("nan"), float("nan")
    check_on(on_split_path(s), "split", window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [20, 64])
def test_attention_pages_and_windows_on_clusters(page, d):
    """The same for few short sequences, which run as clusters."""
    s = attn_inputs([170, 0, 211, 33], 6, 2, d, page, torch.bfloat16, seed=page + d, spare=0)
    check_on(s, "cluster")
    for i, before in ((0, 20), (2, 61)):
        tok = torch.arange(before, device="cuda")
        at = (s["table"][i].long()[tok // page], tok % page)
        s["k_cache"][at], s["v_cache"][at] = float("nan"), float("nan")
    check_on(s, "cluster", window=150)


@pytest.mark.parametrize("h_q,h_kv,d", [(4, 2, 128), (16, 1, 256), (16, 2, 64)])
def test_attention_refused_lengths_and_pages_on_the_split_path(h_q, h_kv, d):
    lens = mixed_lengths(40, 5)
    s = on_split_path(attn_inputs(lens, h_q, h_kv, d, 16, torch.bfloat16, seed=37))
    width = s["table"].shape[1]
    for bad in (width * 16 + 1, -1, 2 ** 31 - 1):
        t = dict(s, lens=s["lens"].clone())
        t["lens"][4] = bad                         # the reference takes such a length as 0 too
        check_on(t, "split")
        with pytest.raises(g.GemmError, match="length"):
            g.check_decode_status()
    whole, _, _ = path_of(s)
    for bad in (-1, int(s["k_cache"].shape[0]), 2 ** 31 - 1):
        t = dict(s, table=s["table"].clone())
        t["table"][4, 2] = bad
        (o, _), taken, _ = path_of(t)
        assert taken == "split"
        kept = [i for i in range(40) if i != 4]
        assert torch.equal(o[kept], whole[0][kept])
        with pytest.raises(g.GemmError, match="page"):
            g.check_decode_status()


# ---- norm without rotation, and the cache under many tokens -----------------------------------------

@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_norm_kinds_without_rotation(d, norm, weights):
    s = norm_inputs(9, 5, 2, d, 0, 1, torch.float16, seed=100 + d, weights=weights)
    s["q"][3] = 0                                  # a head of zeros stays zero
    (qr, qb), (kr, kb) = norm_refs(s, norm=norm, eps=1e-5)
    q, k = norm_call(s, norm=norm, eps=1e-5)
    ref.assert_close(q, qr, qb, "q")
    ref.assert_close(k, kr, kb, "k")
    assert bool((q[3] == 0).all())


def check_cache(kc, vc, s, slots, written, k_ref, where):
    """Both caches hold the tokens of `written` at their slots, values bit for bit, and nothing
    else."""
    page = kc.shape[1]
    kr, kb = k_ref
    at = slots[written].long().cuda()
    ref.assert_close(kc[at // page, at % page], kr[written], kb[written], f"{where}: keys")
    assert torch.equal(vc[at // page, at % page].view(torch.int16), s["v"][written].view(torch.int16))
    rest = torch.ones(kc.shape[:2], dtype=torch.bool, device="cuda")
    rest[at // page, at % page] = False
    assert bool(kc[rest].isnan().all()) and bool(vc[rest].isnan().all()), f"{where}: other places"


@DTYPES
@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
@pytest.mark.parametrize("page", [1, 16, 20])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_norm_into_the_cache_without_rotation(d, page, layout, dtype):
    """Active, inactive and refused slots; the refused ones are reported."""
    tokens = 37
    s = norm_inputs(tokens, 6, 3, d, 0, 1, dtype, seed=101)
    s["v"][5, 1, 3] = float("nan")                 # values are copied bit for bit
    pages = -(-tokens // page) + 2
    slots = torch.randperm(pages * page, generator=generator(102))[:tokens].to(torch.int32)
    slots[4] = -1
    (qr, qb), k_ref = norm_refs(s)
    for bad in (None, pages * page, -2, 2 ** 31 - 1):
        kc, vc = cache_pair(pages, page, 3, d, dtype, layout)
        at = slots.clone()
        if bad is not None:
            at[11] = bad
        q, k = norm_call(s, v=s["v"], k_cache=kc, v_cache=vc, slots=at.cuda())
        assert k is None
        ref.assert_close(q, qr, qb, "q")
        check_cache(kc, vc, s, at, [t for t in range(tokens) if t != 4 and (t != 11 or bad is None)],
                    k_ref, f"slot {bad}")
        if bad is not None:
            with pytest.raises(g.GemmError, match="cache slot"):
                g.check_decode_status()
        g.check_decode_status()


@pytest.mark.parametrize("rot", ["all", "some", "none"])
@pytest.mark.parametrize("tokens,h_q,h_k,d,page", [(3000, 32, 8, 128, 16), (3001, 32, 8, 128, 20),
                                                   (9000, 3, 1, 64, 20), (2500, 16, 2, 256, 64)])
def test_norm_of_many_tokens_into_the_cache(tokens, h_q, h_k, d, page, rot):
    """Warps take several sets of tokens, whole and in parts, each with a position and a slot of its
    own; inactive tokens and refused slots and positions lie scattered among them."""
    rot = {"all": d, "some": d // 4, "none": 0}[rot]
    s = norm_inputs(tokens, h_q, h_k, d, rot, 1, torch.bfloat16, seed=tokens + rot)
    pages = -(-tokens // page) + 3
    slots = torch.randperm(pages * page, generator=generator(103))[:tokens].to(torch.int32)
    slots[5::97] = -1
    slots[7::301] = pages * page
    lost = set(range(5, tokens, 97)) | set(range(7, tokens, 301))
    zeros = []
    (qr, qb), k_ref = norm_refs(s)
    if rot:
        zeros = list(range(11, tokens, 211))
        s["positions"][zeros] = 300                # the table has 300 rows
    kc, vc = cache_pair(pages, page, h_k, d, torch.bfloat16, "tokens")
    q, _ = norm_call(s, v=s["v"], k_cache=kc, v_cache=vc, slots=slots.cuda())
    with pytest.raises(g.GemmError, match="cache slot.*position" if rot else "cache slot"):
        g.check_decode_status()
    kept = [t for t in range(tokens) if t not in set(zeros)]
    ref.assert_close(q[kept], qr[kept], qb[kept], "q")
    assert bool((q[zeros] == 0).all())
    check_cache(kc, vc, s, slots, [t for t in kept if t not in lost], k_ref, "cache")


def test_norm_refuses_sections_past_32_bits():
    s = norm_inputs(4, 2, 1, 128, 128, 2, torch.bfloat16, seed=104)
    for sections in ((2 ** 32 + 32, 32 - 2 ** 32), (2 ** 32 + 32, 32), (2 ** 31, 64 - 2 ** 31)):
        with pytest.raises(ValueError, match="section"):
            norm_call(dict(s, sections=sections))


# ---- operands that share memory ---------------------------------------------------------------------

def test_step_refuses_outputs_that_share_memory():
    s, slots = step_inputs(3, 2, 2, 2, 2, torch.bfloat16, seed=70)
    args = [s[x] for x in ("q", "k", "v", "alpha", "beta", "state")]
    before = {x: y.clone() for x, y in s.items()}

    def refused(out=None, **change):
        with pytest.raises(g.GemmError, match="shares memory"):
            g.gated_delta_step(*(change.get(x, y) for x, y in zip(
                ("q", "k", "v", "alpha", "beta", "state"), args)), 0.5, slots, out=out)

    refused(out=s["q"])
    refused(out=s["k"])
    flat = torch.zeros(3 * 2 * 2 * 128 + 128, dtype=torch.bfloat16, device="cuda")
    shape = (3, 2, 2, 128)
    refused(out=flat[:-128].view(shape), q=flat[128:].view(shape))
    refused(out=flat[:-128].view(shape), v=flat[128:].view(shape))
    half = s["state"].view(torch.bfloat16).flatten()
    refused(out=half[:3 * 2 * 2 * 128].view(shape))
    refused(v=half[:3 * 2 * 2 * 128].view(shape))
    refused(beta=s["state"].flatten()[:12].view(3, 2, 2))
    torch.cuda.synchronize()
    for x, y in before.items():
        assert torch.equal(s[x], y), x


@pytest.mark.parametrize("tokens", [1, 4, 11])
def test_step_writes_over_its_values(tokens):
    """``out`` may be ``v`` itself, and lie beside the inputs in one buffer."""
    s, slots = step_inputs(5, tokens, 4, 4, 4, torch.float16, seed=71)
    args = [s[x] for x in ("q", "k", "v", "alpha", "beta")]
    state = s["state"].clone()
    want = g.gated_delta_step(*args, state, 0.5, slots)
    again = s["state"].clone()
    v = s["v"].clone()
    got = g.gated_delta_step(*args[:2], v, *args[3:], again, 0.5, slots, out=v)
    assert got.data_ptr() == v.data_ptr()
    assert torch.equal(got, want) and torch.equal(again, state)
    both = torch.zeros(2, 5, tokens, 4, 128, dtype=torch.float16, device="cuda")
    both[0] = s["q"]
    again = s["state"].clone()
    got = g.gated_delta_step(both[0], *args[1:], again, 0.5, slots, out=both[1])
    assert torch.equal(got, want) and torch.equal(again, state)


def test_norm_refuses_outputs_that_share_memory():
    s = norm_inputs(6, 2, 2, 128, 128, 1, torch.bfloat16, seed=72)
    kc, vc = cache_pair(2, 8, 2, 128, torch.bfloat16, "tokens")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    before = {x: s[x].clone() for x in ("q", "k", "v", "rotary", "positions", "q_weight")}

    def refused(**kw):
        with pytest.raises(g.GemmError, match="shares memory"):
            g.qk_norm_rope(**{**dict(q=s["q"], k=s["k"], q_weight=s["q_weight"],
                                     k_weight=s["k_weight"], positions=s["positions"],
                                     rotary=s["rotary"]), **kw})

    refused(q_out=s["k"])
    refused(k_out=s["q"])
    refused(q_out=s["q"], k_out=s["q"])
    same = torch.zeros(6, 2, 128, dtype=torch.bfloat16, device="cuda")
    refused(q_out=same, k_out=same)
    packed = torch.zeros(7, 2, 128, dtype=torch.bfloat16, device="cuda")
    refused(q=packed[1:], q_out=packed[:6])                    # q shifted by a token
    wide = torch.zeros(6, 5, 128, dtype=torch.bfloat16, device="cuda")
    refused(q=wide[:, :2], k=wide[:, 2:4], q_out=wide[:, 1:3])  # heads of both
    cache = dict(v=s["v"], k_cache=kc, v_cache=vc, slots=slots)
    refused(**{**cache, "v_cache": kc})
    refused(**{**cache, "q": kc[0, :6]})
    refused(**{**cache, "v": vc[1, 2:]})
    refused(**cache, q_out=vc[0, :6])
    refused(**{**cache, "slots": kc.view(torch.int32).flatten()[:6]})
    torch.cuda.synchronize()
    assert bool(kc.isnan().all()) and bool(vc.isnan().all())
    for x, y in before.items():
        assert torch.equal(s[x], y), x


@pytest.mark.parametrize("layout", ["one buffer", "heads beside each other", "pages beside each other"])
def test_norm_takes_caches_and_projections_that_only_lie_between_each_other(layout):
    """Views that interleave without sharing an element are no overlap: a projection's queries,
    keys and values normed in place, and the two caches as parts of one tensor."""
    tokens, h_q, h_k, d = 9, 4, 2, 64
    s = norm_inputs(tokens, h_q, h_k, d, d, 1, torch.bfloat16, seed=73)
    if layout == "one buffer":
        kc, vc = torch.zeros(2, 3, 4, h_k, d, dtype=torch.bfloat16, device="cuda")
    elif layout == "heads beside each other":
        both = torch.zeros(3, 4, h_k, 2 * d, dtype=torch.bfloat16, device="cuda")
        kc, vc = both[..., :d], both[..., d:]
    else:
        both = torch.zeros(3, h_k, 2, 4, d, dtype=torch.bfloat16, device="cuda")
        kc, vc = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    packed = torch.cat([s["q"], s["k"], s["v"]], 1)
    q, k, v = packed[:, :h_q], packed[:, h_q:h_q + h_k], packed[:, h_q + h_k:]
    slots = torch.randperm(12, generator=generator(74))[:tokens].to(torch.int32).cuda()
    want_q, want_k = norm_call(s)
    got, _ = g.qk_norm_rope(q, k, s["q_weight"], s["k_weight"], positions=s["positions"],
                            rotary=s["rotary"], v=v, k_cache=kc, v_cache=vc, slots=slots, q_out=q)
    assert torch.equal(packed[:, :h_q], want_q) and got.data_ptr() == packed.data_ptr()
    at = slots.long()
    assert torch.equal(kc[at // 4, at % 4], want_k)
    assert torch.equal(vc[at // 4, at % 4], s["v"])


def test_attention_refuses_outputs_that_share_memory():
    s = attn_inputs([50, 300], 4, 2, 128, 16, torch.bfloat16, seed=75)
    kept = {x: y.clone() for x, y in s.items()}

    def refused(**kw):
        with pytest.raises(g.GemmError, match="shares memory"):
            g.paged_attention(**{**dict(q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                                        page_table=s["table"], lens=s["lens"]), **kw})

    refused(out=s["v_cache"].flatten()[:2 * 4 * 128].view(2, 4, 128))
    refused(out=s["k_cache"].flatten()[-2 * 4 * 128:].view(2, 4, 128))
    flat = torch.zeros(4 * 4 * 128, dtype=torch.bfloat16, device="cuda")
    refused(q=flat[128:128 * 9].view(2, 4, 128), out=flat[:128 * 8].view(2, 4, 128))
    size = g.paged_attention_workspace(4, 2, 128).numel()
    room = torch.zeros(size + 8192, dtype=torch.uint8, device="cuda")
    refused(workspace=room, out=room[:2048].view(torch.bfloat16).view(2, 4, 128))
    refused(workspace=room, q=room[4096:4096 + 2048].view(torch.bfloat16).view(2, 4, 128))
    torch.cuda.synchronize()
    for x, y in kept.items():
        assert torch.equal(s[x].view(torch.uint8), y.view(torch.uint8)), x    # (NaN among them)
    # what lies behind the bytes that a workspace needs is not part of it
    out = room[size + 256:size + 256 + 2048].view(torch.bfloat16).view(2, 4, 128)
    assert out.data_ptr() % 16 == 0
    got = g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], out=out,
                            workspace=room)
    assert torch.equal(got, g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                              s["lens"]))


@pytest.mark.parametrize("h_q,h_kv,d", [(4, 2, 128), (16, 1, 256), (12, 12, 64)])
@pytest.mark.parametrize("lens", [[50, 0, 300, 5000], [100] * 200, [33]], ids=["few", "many", "one"])
def test_attention_writes_over_its_queries(lens, h_q, h_kv, d):
    """``out`` may be ``q`` itself: a query is read before its result is written."""
    s = attn_inputs(lens, h_q, h_kv, d, 16, torch.bfloat16, seed=76)
    for case in (s, on_split_path(s)):
        args = [case[x] for x in ("k_cache", "v_cache", "table", "lens")]
        want = g.paged_attention(case["q"], *args)
        q = case["q"].clone()
        got = g.paged_attention(q, *args, out=q)
        assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


# ---- the record of refused indices ------------------------------------------------------------------

def test_status_of_concurrent_checks_is_never_lost():
    """While one thread checks over and over, another's call on a stream of its own refuses a slot:
    it is reported by a check during the call or by the one after it, though each first check has
    an older refusal, of a position, to report and clear."""
    import threading
    step, slots = step_inputs(2, 1, 1, 1, 1, torch.bfloat16, seed=80)
    slots[1] = 99
    norm = norm_inputs(4, 1, 1, 64, 64, 1, torch.bfloat16, seed=81)
    norm["positions"][2] = -7
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g.check_decode_status()

    def bits_now(stream):
        rc, bits = g.decode_check_status(stream.cuda_stream)
        assert rc == 0
        return bits

    here = torch.cuda.current_stream()
    for turn in range(300):
        # a bit is up before the other thread starts, so that the first check has something to clear
        norm_call(norm)
        here.synchronize()
        seen = []
        go = threading.Event()

        def refuse():
            go.wait()
            for _ in range(turn % 7):
                pass
            g.gated_delta_step(*(step[x] for x in ("q", "k", "v", "alpha", "beta", "state")), 0.5, slots,
                               stream=side)

        other = threading.Thread(target=refuse)
        other.start()
        go.set()
        for _ in range(3):
            seen.append(bits_now(here))
        other.join()
        side.synchronize()
        seen.append(bits_now(side))
        assert sum(x & 4 for x in seen) == 4 and any(x & 1 for x in seen), (turn, seen)
    assert bits_now(here) == 0


def test_status_is_that_of_the_streams_device():
    """A stream's own device's record is read, whichever device is current, and the current device
    stays."""
    step, slots = step_inputs(2, 1, 1, 1, 1, torch.bfloat16, seed=82)
    slots[0] = -5
    for stream in (torch.cuda.Stream(), torch.cuda.default_stream()):
        g.gated_delta_step(*(step[x] for x in ("q", "k", "v", "alpha", "beta", "state")), 0.5, slots,
                           stream=stream)
        with pytest.raises(g.GemmError, match="state slot"):
            g.check_decode_status(stream)
        g.check_decode_status(stream.cuda_stream)
        assert torch.cuda.current_device() == 0
