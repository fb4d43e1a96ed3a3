"""The decode-step operators on the GPU against their definitions in 64 bits (tests/decode_ref.py has
the definitions and the derivation of the bounds)."""
from __future__ import annotations

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
import decode_ref as ref

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    if not torch.cuda.is_available():
        pytest.fail("the gpu tests need a CUDA device")
    g.build()
    g.load()
    yield


@pytest.fixture(autouse=True)
def no_refusals_left():
    yield
    g.check_decode_status()


def generator(seed):
    gen = torch.Generator()
    gen.manual_seed(seed)
    return gen


def normal(gen, *shape):
    return torch.randn(shape, generator=gen)


# ---- the gated delta rule, token by token --------------------------------------------------------

def step_inputs(n, tokens, h_q, h_k, h_v, dtype, seed, extra_slots=2):
    gen = generator(seed)

    def unit(*shape):
        x = normal(gen, *shape)
        return (x / x.norm(dim=-1, keepdim=True)).mul(0.99).to(dtype)

    s = dict(q=unit(n, tokens, h_q, 128), k=unit(n, tokens, h_k, 128),
             v=normal(gen, n, tokens, h_v, 128).to(dtype),
             alpha=torch.exp(-0.1 * torch.rand(n, tokens, h_v, generator=gen)),
             beta=torch.sigmoid(normal(gen, n, tokens, h_v)),
             state=0.1 * normal(gen, n + extra_slots, h_v, 128, 128))
    slots = torch.randperm(n + extra_slots, generator=gen)[:n].to(torch.int32)
    return {x: y.cuda() for x, y in s.items()}, slots.cuda()


def check_step(s, slots, scale, where, **kw):
    o_ref, s_ref, ob, sb = ref.gdn_step(**s, scale=scale, slots=slots)
    state = s["state"].clone()
    o = g.gated_delta_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], state, scale, slots, **kw)
    ref.assert_close(o, o_ref, ob, f"{where}: o")
    ref.assert_close(state, s_ref, sb, f"{where}: state")
    return o, state


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("h_q,h_k,h_v", [(1, 1, 1), (2, 2, 2), (2, 2, 6), (6, 2, 2), (4, 1, 2),
                                         (2, 1, 2), (8, 1, 1), (16, 2, 2)])
@pytest.mark.parametrize("n,tokens", [(1, 1), (5, 1), (3, 4), (2, 17)])
def test_step(n, tokens, h_q, h_k, h_v, dtype):
    s, slots = step_inputs(n, tokens, h_q, h_k, h_v, dtype, seed=n * 100 + tokens)
    check_step(s, slots, 0.73, f"{n} x {tokens}")


def test_step_many_sequences():
    """More states than any launch keeps resident; the reference is checked on a few sequences,
    the rest against a call on that sequence alone."""
    s, slots = step_inputs(600, 1, 4, 4, 8, torch.bfloat16, seed=5)
    state = s["state"].clone()
    o = g.gated_delta_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], state, 0.5, slots)
    pick = [0, 1, 299, 598, 599]
    few = {x: y[pick] if x != "state" else y for x, y in s.items()}
    o_ref, s_ref, ob, sb = ref.gdn_step(**few, scale=0.5, slots=slots[pick])
    ref.assert_close(o[pick], o_ref, ob, "o")
    at = slots[pick].long()
    ref.assert_close(state[at], s_ref[at.cpu()], sb[at.cpu()], "state")
    for i in range(0, 600, 37):
        one = s["state"].clone()
        oi = g.gated_delta_step(*(s[x][i:i + 1] for x in ("q", "k", "v", "alpha", "beta")), one,
                                0.5, slots[i:i + 1])
        assert torch.equal(oi[0], o[i]), i
        assert torch.equal(one[slots[i].long()], state[slots[i].long()]), i


def test_step_without_slots_and_out():
    s, _ = step_inputs(4, 2, 2, 2, 4, torch.float16, seed=6)
    out = torch.full((4, 2, 4, 128), NAN, dtype=torch.float16, device="cuda")
    o, _ = check_step(s, None, 1.0, "identity slots", out=out)
    assert o.data_ptr() == out.data_ptr()


def test_step_views_of_a_projection_and_padded_pool():
    """q, k, v side by side in one tensor, gates interleaved in another, a pool with space between
    its slots (whose contents stay), and one key broadcast to all sequences."""
    gen = generator(7)
    n, tokens, h = 3, 2, 2
    packed = normal(gen, n, tokens, 3 * h, 128).mul(0.08).bfloat16().cuda()
    gates = torch.rand(n, tokens, 2, h, generator=gen).cuda()
    pool = torch.full((n + 1, h * 128 * 128 + 64), 7.0, device="cuda")
    state = pool[:, :h * 128 * 128].view(n + 1, h, 128, 128)
    state.copy_(0.1 * normal(gen, n + 1, h, 128, 128))
    s = dict(q=packed[:, :, :h], k=packed[:1, :, h:2 * h].expand(n, tokens, h, 128),
             v=packed[:, :, 2 * h:], alpha=gates[:, :, 0], beta=gates[:, :, 1], state=state)
    slots = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    o_ref, s_ref, ob, sb = ref.gdn_step(**s, scale=0.73, slots=slots)
    o = g.gated_delta_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], state, 0.73, slots)
    ref.assert_close(o, o_ref, ob, "o")
    ref.assert_close(state, s_ref, sb, "state")
    assert bool((pool[:, h * 128 * 128:] == 7.0).all())


def test_step_inactive_and_refused_slots():
    s, slots = step_inputs(5, 2, 2, 2, 2, torch.bfloat16, seed=8)
    s["state"][int(slots[1])] = NAN            # belongs to an inactive sequence: never read
    for bad, status in ((-1, False), (7, True), (-2, True), (2 ** 31 - 1, True)):
        at = slots.clone()
        at[1] = bad
        keep = s["state"][int(slots[1])].clone()
        o_ref, s_ref, ob, sb = ref.gdn_step(**s, scale=0.73, slots=at)
        state = s["state"].clone()
        out = torch.full((5, 2, 2, 128), NAN, dtype=torch.bfloat16, device="cuda")
        g.gated_delta_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], state, 0.73, at, out=out)
        assert torch.equal(state[int(slots[1])].isnan(), keep.isnan())
        ref.assert_close(out, o_ref, ob, f"slot {bad}: o")
        live = [int(x) for i, x in enumerate(slots) if i != 1]
        ref.assert_close(state[live], s_ref[live], sb[live], f"slot {bad}: state")
        if status:
            with pytest.raises(g.GemmError, match="state slot"):
                g.check_decode_status()
        g.check_decode_status()                # cleared by the read


def test_step_reset_and_odd_gates():
    """alpha 0 forgets the state, beta 0 writes nothing, and gates outside 0 .. 1 are plain
    numbers."""
    s, slots = step_inputs(4, 1, 1, 1, 1, torch.bfloat16, seed=9)
    s["alpha"][:, 0, 0] = torch.tensor([0.0, 1.0, -0.5, 1.5])
    s["beta"][:, 0, 0] = torch.tensor([1.0, 0.0, -1.0, 0.5])
    _, state = check_step(s, slots, 0.73, "odd gates")
    assert torch.equal(state[int(slots[1])], s["state"][int(slots[1])])


def test_step_empty():
    s, slots = step_inputs(3, 1, 1, 1, 1, torch.bfloat16, seed=10)
    before = s["state"].clone()
    for n, tokens in ((0, 1), (3, 0)):
        o = g.gated_delta_step(*(s[x][:n, :tokens] for x in ("q", "k", "v", "alpha", "beta")),
                               s["state"], 1.0, slots[:n])
        assert tuple(o.shape) == (n, tokens, 1, 128)
    assert torch.equal(before, s["state"])


def test_step_far_slot():
    """A slot whose first element lies past 2^31 elements of the pool."""
    h_v, far = 32, 4200
    assert far * h_v * 128 * 128 > 2 ** 31
    s, _ = step_inputs(1, 1, 32, 32, h_v, torch.bfloat16, seed=11, extra_slots=0)
    pool = torch.zeros(far + 1, h_v, 128, 128, device="cuda")
    pool[far] = s["state"][0]
    o_ref, s_ref, ob, sb = ref.gdn_step(**s, scale=0.73)
    o = g.gated_delta_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], pool, 0.73,
                           torch.tensor([far], dtype=torch.int32, device="cuda"))
    ref.assert_close(o, o_ref, ob, "o")
    ref.assert_close(pool[far:], s_ref, sb, "state")


def test_step_carries_on_what_the_prefill_leaves():
    """A prompt through gated_delta_rule and the rest token by token: the definition over all of
    it, from the prompt's own final state on."""
    T, cut, h = 150, 130, 2
    s, _ = step_inputs(1, T, h, h, h, torch.bfloat16, seed=12, extra_slots=0)
    cu = torch.tensor([0, cut], dtype=torch.int32, device="cuda")
    head = [s[x][0, :cut].contiguous() for x in ("q", "k", "v", "alpha", "beta")]
    _, state = g.gated_delta_rule(*head, cu, 0.73, output_final_state=True)
    rest = {x: s[x][:, cut:] for x in ("q", "k", "v", "alpha", "beta")}
    o_ref, s_ref, ob, sb = ref.gdn_step(**rest, state=state, scale=0.73)
    for t in range(cut, T):
        o = g.gated_delta_step(*(s[x][:, t:t + 1] for x in ("q", "k", "v", "alpha", "beta")),
                               state, 0.73)
        ref.assert_close(o, o_ref[:, t - cut:t - cut + 1], ob[:, t - cut:t - cut + 1], f"token {t}")
    ref.assert_close(state, s_ref, sb, "state")


# ---- norm and rotation ----------------------------------------------------------------------------

def norm_inputs(tokens, h_q, h_k, d, rot, axes, dtype, seed, weights=True, rows=300):
    gen = generator(seed)
    s = dict(q=normal(gen, tokens, h_q, d).mul(3).to(dtype).cuda(),
             k=normal(gen, tokens, h_k, d).to(dtype).cuda(),
             v=normal(gen, tokens, h_k, d).to(dtype).cuda(),
             q_weight=(1 + 0.3 * normal(gen, d)).to(dtype).cuda() if weights else None,
             k_weight=(1 + 0.3 * normal(gen, d)).to(dtype).cuda() if weights else None,
             rotary=None, positions=None, sections=None)
    if rot:
        s["rotary"] = g.rotary_table(rows, rot)
        shape = (tokens,) if axes == 1 else (axes, tokens)
        s["positions"] = torch.randint(0, rows, shape, generator=gen, dtype=torch.int32).cuda()
        if axes > 1:
            cut = sorted(torch.randint(0, rot // 2 + 1, (axes - 1,), generator=gen).tolist())
            s["sections"] = [b - a for a, b in zip([0] + cut, cut + [rot // 2])]
    return s


def norm_refs(s, norm="rms", eps=1e-6, interleaved=False):
    return [ref.qk_norm_rope(s[x], s[x + "_weight"], norm, eps, s["positions"], s["rotary"],
                             s["sections"], interleaved) for x in "qk"]


def norm_call(s, norm="rms", eps=1e-6, interleaved=False, **kw):
    return g.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], norm=norm, eps=eps,
                          positions=s["positions"], rotary=s["rotary"], sections=s["sections"],
                          interleaved=interleaved, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d,rot,axes,interleaved", [
    (128, 128, 1, False), (128, 128, 1, True), (128, 32, 3, False), (64, 64, 2, True),
    (64, 48, 1, False), (256, 256, 4, False), (256, 64, 1, True), (96, 96, 1, False),
    (72, 16, 1, False), (8, 0, 1, False), (16, 16, 1, False), (248, 240, 3, True), (128, 0, 1, False)])
@pytest.mark.parametrize("tokens,h_q,h_k", [(1, 1, 1), (7, 6, 2), (65, 12, 4), (3, 33, 5)])
def test_norm_and_rotation(tokens, h_q, h_k, d, rot, axes, interleaved, dtype):
    s = norm_inputs(tokens, h_q, h_k, d, rot, axes, dtype, seed=d + rot + tokens)
    (qr, qb), (kr, kb) = norm_refs(s, interleaved=interleaved)
    q, k = norm_call(s, interleaved=interleaved)
    ref.assert_close(q, qr, qb, "q")
    ref.assert_close(k, kr, kb, "k")


@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("weights", [True, False])
def test_norm_kinds(norm, weights):
    s = norm_inputs(9, 4, 2, 128, 64, 1, torch.bfloat16, seed=21, weights=weights)
    s["q"][3] = 0                                  # a head of zeros stays zero
    (qr, qb), (kr, kb) = norm_refs(s, norm=norm, eps=1e-5)
    q, k = norm_call(s, norm=norm, eps=1e-5)
    ref.assert_close(q, qr, qb, "q")
    ref.assert_close(k, kr, kb, "k")
    assert bool((q[3] == 0).all())


def test_norm_in_place_on_views():
    """Queries and keys normed where they lie in a packed projection; the values beside them stay."""
    gen = generator(22)
    packed = normal(gen, 11, 4 + 2 + 2, 128).bfloat16().cuda()
    s = norm_inputs(11, 4, 2, 128, 128, 1, torch.bfloat16, seed=22)
    s["q"], s["k"] = packed[:, :4], packed[:, 4:6]
    before = packed[:, 6:].clone()
    (qr, qb), (kr, kb) = norm_refs(s)
    q, k = norm_call(s, q_out=s["q"], k_out=s["k"])
    assert q.data_ptr() == packed.data_ptr()
    ref.assert_close(packed[:, :4], qr, qb, "q")
    ref.assert_close(packed[:, 4:6], kr, kb, "k")
    assert torch.equal(packed[:, 6:], before)


def cache_pair(pages, page, h, d, dtype, layout):
    """A pair of caches full of NaN, their heads inside the page's tokens or outside them, or with
    the two interleaved in one buffer."""
    if layout == "tokens":
        return [torch.full((pages, page, h, d), NAN, dtype=dtype, device="cuda") for _ in range(2)]
    if layout == "heads":
        return [torch.full((pages, h, page, d), NAN, dtype=dtype, device="cuda").transpose(1, 2)
                for _ in range(2)]
    both = torch.full((pages, 2, page, h, d), NAN, dtype=dtype, device="cuda")
    return [both[:, 0], both[:, 1]]


@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
@pytest.mark.parametrize("page", [1, 16, 20])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_norm_into_the_cache(d, page, layout):
    tokens, h_q, h_k = 37, 6, 3
    s = norm_inputs(tokens, h_q, h_k, d, d, 1, torch.bfloat16, seed=23)
    s["v"][5, 1, 3] = NAN                          # values are copied bit for bit
    pages = -(-tokens // page) + 2
    kc, vc = cache_pair(pages, page, h_k, d, torch.bfloat16, layout)
    slots = torch.randperm(pages * page, generator=generator(24))[:tokens].to(torch.int32)
    slots[4] = -1                                  # this token's key and value go nowhere
    q, k = norm_call(s, v=s["v"], k_cache=kc, v_cache=vc, slots=slots.cuda())
    assert k is None
    (qr, qb), (kr, kb) = norm_refs(s)
    ref.assert_close(q, qr, qb, "q")
    keep = [t for t in range(tokens) if t != 4]
    at = slots[keep].long().cuda()
    ref.assert_close(kc[at // page, at % page], kr[keep], kb[keep], "keys")
    got = vc[at // page, at % page]
    assert torch.equal(got.view(torch.int16), s["v"][keep].view(torch.int16))
    touched = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    touched[at // page, at % page] = True
    assert bool(kc[~touched].isnan().all()) and bool(vc[~touched].isnan().all())


def test_norm_refused_indices():
    s = norm_inputs(6, 2, 2, 128, 128, 1, torch.bfloat16, seed=25, rows=50)
    kc, vc = cache_pair(2, 8, 2, 128, torch.bfloat16, "tokens")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    (qr, qb), (kr, kb) = norm_refs(s)
    for bad in (16, -2, 2 ** 31 - 1):
        at = slots.clone()
        at[2] = bad
        kc.fill_(NAN), vc.fill_(NAN)
        q, _ = norm_call(s, v=s["v"], k_cache=kc, v_cache=vc, slots=at)
        ref.assert_close(q, qr, qb, "q")
        assert int(kc.isnan().all(-1).all(-1).sum()) == 11 == int(vc.isnan().all(-1).all(-1).sum())
        with pytest.raises(g.GemmError, match="cache slot"):
            g.check_decode_status()
    for bad in (50, -1):
        t = dict(s, positions=s["positions"].clone())
        t["positions"][3] = bad
        kc.fill_(NAN), vc.fill_(NAN)
        q, _ = norm_call(t, v=s["v"], k_cache=kc, v_cache=vc, slots=slots)
        assert bool((q[3] == 0).all())
        keep = [0, 1, 2, 4, 5]
        ref.assert_close(q[keep], qr[keep], qb[keep], "q")
        assert bool(kc[0, 3].isnan().all()) and bool(vc[0, 3].isnan().all())
        ref.assert_close(kc[0, keep], kr[keep], kb[keep], "keys")
        _, k = norm_call(t)
        assert bool((k[3] == 0).all())
        with pytest.raises(g.GemmError, match="position"):
            g.check_decode_status()


def test_norm_strided_positions():
    """Positions of several axes as a view with space between its rows."""
    s = norm_inputs(70, 8, 2, 128, 128, 3, torch.bfloat16, seed=27)
    wide = torch.full((6, 90), -5, dtype=torch.int32, device="cuda")
    wide[::2, 7:77] = s["positions"]
    s["positions"] = wide[::2, 7:77]
    (qr, qb), (kr, kb) = norm_refs(s)
    q, k = norm_call(s)
    ref.assert_close(q, qr, qb, "q")
    ref.assert_close(k, kr, kb, "k")


@pytest.mark.parametrize("tokens,h_q,h_k,d", [(3000, 32, 8, 128), (5000, 3, 1, 64), (2500, 40, 8, 256)])
def test_norm_many_tokens(tokens, h_q, h_k, d):
    """Enough tokens that warps take several sets, whole or in parts; all against the reference."""
    s = norm_inputs(tokens, h_q, h_k, d, d // 2, 2, torch.bfloat16, seed=tokens)
    (qr, qb), (kr, kb) = norm_refs(s)
    q, k = norm_call(s)
    ref.assert_close(q, qr, qb, "q")
    ref.assert_close(k, kr, kb, "k")


def test_norm_empty_and_broadcast():
    s = norm_inputs(4, 2, 1, 128, 128, 1, torch.bfloat16, seed=26)
    t = {x: (y[:0] if x in ("q", "k", "positions") else y) for x, y in s.items()}
    q, k = norm_call(t)
    assert tuple(q.shape) == (0, 2, 128) and tuple(k.shape) == (0, 1, 128)
    kc, vc = cache_pair(2, 8, 1, 128, torch.bfloat16, "tokens")
    norm_call(t, v=s["v"][:0], k_cache=kc, v_cache=vc,
              slots=torch.zeros(0, dtype=torch.int32, device="cuda"))
    s["k"] = s["k"][:1].expand(4, 1, 128)          # one key for all tokens
    (qr, qb), (kr, kb) = norm_refs(s)
    q, k = norm_call(s)
    ref.assert_close(k, kr, kb, "k")


# ---- attention over the paged cache ----------------------------------------------------------------

def attn_inputs(lens, h_q, h_kv, d, page, dtype, seed, layout="tokens", spread=1.0, spare=1):
    """Pages in random order, every place that holds no token of any sequence NaN, and table
    entries past a sequence's pages wild."""
    gen = generator(seed)
    lens = torch.as_tensor(lens)
    n, width = len(lens), max(1, -(-int(lens.max()) // page)) + spare
    used = (lens + page - 1) // page
    total = int(used.sum()) + 1
    kc, vc = cache_pair(total, page, h_kv, d, dtype, layout)
    order = torch.randperm(total, generator=gen)
    table = torch.full((n, width), 2 ** 31 - 1, dtype=torch.int32)
    at = 0
    for i, length in enumerate(lens.tolist()):
        c = int(used[i])
        table[i, :c] = order[at:at + c]
        tok = torch.arange(length)
        pg = table[i].long()[tok // page].cuda()
        of = (tok % page).cuda()
        kc[pg, of] = normal(gen, length, h_kv, d).to(dtype).cuda()
        vc[pg, of] = normal(gen, length, h_kv, d).to(dtype).cuda()
        at += c
    q = normal(gen, n, h_q, d).mul(spread).to(dtype).cuda()
    return dict(q=q, k_cache=kc, v_cache=vc, table=table.cuda(), lens=lens.to(torch.int32).cuda())


def check_attn(s, where, scale=None, window=None, **kw):
    d = s["q"].shape[-1]
    real = d ** -0.5 if scale is None else scale
    o_ref, l_ref, ob, lb = ref.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                               s["lens"], real, window)
    out = torch.full(tuple(s["q"].shape), NAN, dtype=s["q"].dtype, device="cuda")
    o, lse = g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                               scale=scale, window=window, return_lse=True, out=out, **kw)
    assert o.data_ptr() == out.data_ptr()
    ref.assert_close(lse, l_ref, lb, f"{where}: lse")
    ref.assert_close(o, o_ref, ob, f"{where}: o")
    return o, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (3, 1), (4, 2), (8, 1), (9, 1), (32, 2), (40, 2)])
def test_attention_heads(h_q, h_kv, d, dtype):
    """Groups of 1 to 20 query heads per key head, lengths around a slice and a tile."""
    s = attn_inputs([1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0, 300], h_q, h_kv, d, 16, dtype,
                    seed=h_q + d)
    check_attn(s, f"{h_q}/{h_kv}")


@pytest.mark.parametrize("page", [1, 5, 16, 20, 64, 100, 256])
@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
def test_attention_pages_and_strides(page, layout):
    """Pages of any size, one that ends inside a slice among them, and three cache layouts."""
    s = attn_inputs([page, page + 1, 2 * page - 1, 333, 1], 4, 2, 128, page, torch.bfloat16,
                    seed=page, layout=layout)
    check_attn(s, f"pages of {page}")


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 128, 299, 5000])
def test_attention_window(window):
    """Only the last `window` tokens count; what the pages before them hold (NaN here) does not."""
    s = attn_inputs([0, 1, 16, 99, 100, 101, 300, 1000], 8, 2, 128, 16, torch.bfloat16, seed=window)
    for i, length in enumerate(s["lens"].tolist()):
        tok = torch.arange(max(0, length - window), device="cuda")
        pg = s["table"][i].long()[tok // 16]
        s["k_cache"][pg, tok % 16] = NAN
        s["v_cache"][pg, tok % 16] = NAN
    check_attn(s, f"window {window}", window=window)


@pytest.mark.parametrize("n,top", [(1, 4000), (2, 20000), (300, 40), (1100, 3), (33, 700)])
def test_attention_work_split(n, top):
    """From one sequence over all blocks to many sequences per block, empty ones between."""
    gen = generator(n)
    lens = torch.randint(0, top + 1, (n,), generator=gen)
    lens[n // 2] = top
    lens[::7] = 0 if n > 2 else top
    check_attn(attn_inputs(lens, 2, 1, 64, 16, torch.float16, seed=n), f"{n} sequences")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [5, 25, 60, 150])
def test_attention_clusters_of_each_size(n, d):
    """Short sequences: items for clusters of eight, four and two blocks, and too many for any."""
    top = {64: 128, 128: 64, 256: 32}[d] * (8 if n == 5 else 3)
    lens = torch.randint(0, top, (n,), generator=generator(n + d))
    lens[0], lens[-1] = top - 1, 0
    check_attn(attn_inputs(lens, 6, 2, d, 16, torch.bfloat16, seed=n), f"{n} sequences")


def test_attention_many_items_cut_across_blocks():
    """More items than the join lists one by one, of several tiles each, so that most blocks' ranges
    begin and end inside items; every seventh sequence is empty."""
    gen = generator(30)
    lens = torch.randint(200, 700, (270,), generator=gen)
    lens[::7] = 0
    check_attn(attn_inputs(lens, 4, 4, 64, 16, torch.bfloat16, seed=30), "1080 items")


def test_attention_strided_table():
    """A page table that is a view: every other row of a wider one, some columns in."""
    s = attn_inputs([100, 0, 333, 64], 4, 2, 128, 16, torch.bfloat16, seed=40)
    wide = torch.full((8, s["table"].shape[1] + 5), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[::2, 3:-2] = s["table"]
    s["table"] = wide[::2, 3:-2]
    check_attn(s, "strided table")


def test_attention_all_empty():
    s = attn_inputs([1, 1], 4, 2, 128, 16, torch.bfloat16, seed=31)
    s["lens"].zero_()
    o, lse = check_attn(s, "no tokens")
    assert bool((o == 0).all()) and bool((lse == float("-inf")).all())
    s["table"] = s["table"][:, :0]                 # and no pages at all
    check_attn(s, "no table")
    o = g.paged_attention(s["q"][:0], s["k_cache"], s["v_cache"], s["table"][:0], s["lens"][:0])
    assert tuple(o.shape) == (0, 4, 128)


@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_attention_flat_and_sharp(spread):
    """Equal weights, and scores so large that one token takes all the weight."""
    s = attn_inputs([700, 64, 5], 8, 2, 128, 16, torch.bfloat16, seed=32, spread=spread)
    check_attn(s, f"spread {spread}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_small_weights_beside_large_ones(d, dtype):
    """Every 16 tokens one outweighs the others e^18 to 1 and has a zero value: the results are the
    others' values."""
    s = attn_inputs([16, 100, 3001], 4, 2, d, 16, dtype, seed=d)
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    for c, fill in (("k_cache", 0.0), ("v_cache", 3e4)):
        s[c][~s[c].isnan()] = fill
    s["k_cache"][:, 5, :, 0] = 18.0
    s["v_cache"][:, 5] = 0.0
    check_attn(s, "sinks", scale=1.0)


def test_attention_scores_of_minus_infinity():
    """A key of -infinity masks its token, as an additive mask written into the cache would; the
    weights of the others stay."""
    s = attn_inputs([40, 200], 2, 1, 64, 16, torch.float16, seed=33)
    s["q"].abs_()
    s["q"].clamp_(min=0.01)
    keep = {x: y.clone() for x, y in s.items()}
    for i, t in ((0, 0), (0, 17), (1, 3), (1, 128)):
        s["k_cache"][s["table"][i, t // 16].long(), t % 16, 0] = float("-inf")
    o, lse = g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                               return_lse=True)
    # the same without the masked tokens: moved out of each sequence by the last ones
    for i, drop in ((0, (17, 0)), (1, (128, 3))):
        for t in drop:
            last = int(keep["lens"][i]) - 1
            for c in ("k_cache", "v_cache"):
                x = keep[c]
                x[keep["table"][i, t // 16].long(), t % 16] = \
                    x[keep["table"][i, last // 16].long(), last % 16]
            keep["lens"][i] -= 1
    o_ref, l_ref, ob, lb = ref.paged_attention(keep["q"], keep["k_cache"], keep["v_cache"],
                                               keep["table"], keep["lens"], 0.125, None)
    ref.assert_close(lse, l_ref, lb, "lse")
    ref.assert_close(o, o_ref, ob, "o")


def test_attention_nan_stays_in_its_head():
    """NaN in one key head's cached token reaches that head's queries and nothing else."""
    s = attn_inputs([150, 150], 4, 2, 128, 16, torch.bfloat16, seed=34)
    clean, _ = check_attn(s, "clean")
    s["v_cache"][s["table"][0, 2].long(), 3, 1] = NAN
    o = g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])
    assert bool(o[0, 2:].isnan().all())
    assert torch.equal(o[0, :2], clean[0, :2]) and torch.equal(o[1], clean[1])


def test_attention_shared_pages_and_query_views():
    """Two sequences with a common prefix share its pages; queries lie in a packed projection."""
    s = attn_inputs([100, 100], 4, 2, 128, 16, torch.bfloat16, seed=35)
    s["table"][1, :4] = s["table"][0, :4]
    packed = normal(generator(36), 2, 8, 128).bfloat16().cuda()
    s["q"] = packed[:, 2:6]
    check_attn(s, "shared prefix")


def test_attention_refused_lengths_and_pages():
    s = attn_inputs([50, 60, 70], 4, 2, 128, 16, torch.bfloat16, seed=37, spare=0)
    for bad in (81, -1, 2 ** 31 - 1):
        t = dict(s, lens=s["lens"].clone())
        t["lens"][1] = bad                         # the reference takes such a length as 0 too
        check_attn(t, f"length {bad}")
        with pytest.raises(g.GemmError, match="length"):
            g.check_decode_status()
    for bad in (-1, int(s["k_cache"].shape[0])):
        t = dict(s, table=s["table"].clone())
        t["table"][1, 2] = bad
        o = g.paged_attention(t["q"], t["k_cache"], t["v_cache"], t["table"], t["lens"])
        whole = g.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])
        assert torch.equal(o[0], whole[0]) and torch.equal(o[2], whole[2])
        with pytest.raises(g.GemmError, match="page"):
            g.check_decode_status()


def test_attention_repeats_bit_for_bit():
    """Every sum has a fixed order: calls on the same inputs give the same bits, with a workspace
    kept by the caller (its contents before the call do not matter) or without."""
    s = attn_inputs([3000, 11, 0, 777], 16, 2, 128, 16, torch.bfloat16, seed=38)
    args = (s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])
    first = g.paged_attention(*args)
    for fill in (0, 255):
        ws = g.paged_attention_workspace(16, 2, 128)
        ws.fill_(fill)
        for _ in range(3):
            assert torch.equal(g.paged_attention(*args, workspace=ws), first)


def test_attention_far_pages():
    """Pages whose first element lies past 2^31 elements of the cache."""
    page, h, d = 64, 8, 128
    pages = 2 ** 31 // (page * h * d) + 40
    kc, vc = (torch.zeros(pages, page, h, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = generator(39)
    far = torch.tensor([pages - 1, 3, pages - 7], dtype=torch.int32)
    small = [normal(gen, 3, page, h, d).bfloat16().cuda() for _ in range(2)]
    kc[far.long().cuda()], vc[far.long().cuda()] = small
    q = normal(gen, 1, 8, d).bfloat16().cuda()
    lens = torch.tensor([3 * page - 5], dtype=torch.int32, device="cuda")
    o, lse = g.paged_attention(q, kc, vc, far[None].cuda(), lens, return_lse=True)
    near = torch.arange(3, dtype=torch.int32)[None]
    o_ref, l_ref, ob, lb = ref.paged_attention(q, *small, near, lens, d ** -0.5, None)
    ref.assert_close(o, o_ref, ob, "o")
    ref.assert_close(lse, l_ref, lb, "lse")


def test_attention_recorded_and_replayed_on_other_lengths():
    """Many short sequences with cut items: eager calls on a workspace full of anything, then a
    recorded call replayed while the lengths change under it."""
    s = attn_inputs(torch.randint(300, 500, (60,), generator=generator(41)), 8, 2, 128, 16,
                    torch.bfloat16, seed=41)
    full = s["lens"].clone()
    ws = g.paged_attention_workspace(8, 2, 128)
    args = (s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])
    first = check_attn(s, "eager")
    for fill in (0, 1, 255):
        ws.fill_(fill)
        for _ in range(20):
            o, lse = g.paged_attention(*args, return_lse=True, workspace=ws)
            assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = g.paged_attention(*args, return_lse=True, workspace=ws)
    for cut in (0, 7, 290, 3):
        s["lens"].copy_(full - cut)
        s["lens"][cut % 60] = 0
        want = g.paged_attention(*args, return_lse=True)
        for _ in range(5):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


# ---- streams, graphs ---------------------------------------------------------------------------------

def decode_layer(s, step, slots, norm, kc, vc, places, table, lens, ws, **kw):
    """The three operators in a row, as a decode step runs them."""
    o1 = g.gated_delta_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], step, 0.73, slots, **kw)
    q, _ = g.qk_norm_rope(norm["q"], norm["k"], norm["q_weight"], norm["k_weight"],
                          positions=norm["positions"], rotary=norm["rotary"], v=norm["v"],
                          k_cache=kc, v_cache=vc, slots=places, **kw)
    return o1, g.paged_attention(q, kc, vc, table, lens, workspace=ws, **kw)


def layer_inputs():
    n = 5
    s, slots = step_inputs(n, 1, 2, 2, 2, torch.bfloat16, seed=51)
    norm = norm_inputs(n, 4, 2, 128, 128, 1, torch.bfloat16, seed=52)
    a = attn_inputs([33, 16, 1, 128, 200], 4, 2, 128, 16, torch.bfloat16, seed=53)
    last = a["lens"].long() - 1
    places = (a["table"].gather(1, (last // 16)[:, None])[:, 0] * 16 + last % 16).to(torch.int32)
    return s, slots, norm, a, places


def test_operators_on_a_side_stream_and_in_a_graph():
    """The chain on a stream of its own, on inputs made there, and recorded into a CUDA graph that
    is replayed on other states: the same bits as call by call."""
    s, slots, norm, a, places = layer_inputs()
    ws = g.paged_attention_workspace(4, 2, 128)
    state, kc, vc = s["state"].clone(), a["k_cache"].clone(), a["v_cache"].clone()
    first = decode_layer(s, state, slots, norm, kc, vc, places, a["table"], a["lens"], ws)
    again = decode_layer(s, state, slots, norm, kc, vc, places, a["table"], a["lens"], ws)
    torch.cuda.synchronize()

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        st2, kc2, vc2 = s["state"].clone(), a["k_cache"].clone(), a["v_cache"].clone()
    got = decode_layer(s, st2, slots, norm, kc2, vc2, places, a["table"], a["lens"], ws, stream=side)
    side.synchronize()
    for x, y in zip(got, first):
        assert torch.equal(x, y)
    # a plain stream handle in place of torch's object, with and without a workspace kept
    for kept in (ws, None):
        with torch.cuda.stream(side):
            st2, kc2, vc2 = s["state"].clone(), a["k_cache"].clone(), a["v_cache"].clone()
        got = decode_layer(s, st2, slots, norm, kc2, vc2, places, a["table"], a["lens"], kept,
                           stream=side.cuda_stream)
        side.synchronize()
        for x, y in zip(got, first):
            assert torch.equal(x, y)

    st3, kc3, vc3 = s["state"].clone(), a["k_cache"].clone(), a["v_cache"].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decode_layer(s, st3, slots, norm, kc3, vc3, places, a["table"], a["lens"], ws)
    for want in (first, again):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert torch.equal(st3, state)
    assert torch.equal(kc3.view(torch.int16), kc.view(torch.int16))
    assert torch.equal(vc3.view(torch.int16), vc.view(torch.int16))


def test_hybrid_example_decodes_what_it_would_read():
    """The example's model: the logits of tokens answered one by one (eager and recorded) are those
    of the same tokens read as a prompt.  The two differ by roundings to bfloat16 between the
    operators only: some 2^-8 of the logits' size, a few times over."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.HybridModel(seed=3)
    gen = generator(71)
    seqs = [torch.randint(0, 1024, (length,), generator=gen).cuda() for length in (40, 25, 70)]
    cut = [30, 15, 60]
    slots = torch.tensor([2, 7, 4], dtype=torch.int32, device="cuda")
    whole = [model.read(seq, 1) for seq in seqs]
    for seq, c, slot in zip(seqs, cut, slots.tolist()):
        model.read(seq[:c], slot)
    lens = torch.tensor(cut, dtype=torch.int32, device="cuda")
    token = torch.stack([seq[c] for seq, c in zip(seqs, cut)])
    got = [model.step(token, slots, lens)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = model.step(token, slots, lens)
    for t in range(1, 10):
        token.copy_(torch.stack([seq[c + t] for seq, c in zip(seqs, cut)]))
        lens.add_(1)
        graph.replay()
        got.append(logits.clone())
    for t, step in enumerate(got):
        for i, (ref_logits, c) in enumerate(zip(whole, cut)):
            want = ref_logits[c + t].float()
            err = (step[i].float() - want).abs().max()
            assert float(err) <= 2.0 ** -5 * float(want.abs().max()), (t, i, float(err))


# ---- refusals -------------------------------------------------------------------------------------------

def test_refusals_of_the_step():
    s, slots = step_inputs(2, 1, 2, 2, 4, torch.bfloat16, seed=61)
    a = [s[x] for x in ("q", "k", "v", "alpha", "beta", "state")]

    def refused(match, error=ValueError, **change):
        names = ("q", "k", "v", "alpha", "beta", "state")
        args = [change.get(n, x) for n, x in zip(names, a)]
        with pytest.raises(error, match=match):
            g.gated_delta_step(*args, 0.5, change.get("slots", slots))

    before = s["state"].clone()
    refused("float16 or bfloat16", q=a[0].float())
    refused("CUDA", q=a[0].cpu())
    refused("v must be", v=a[2].half())
    refused("k must be", k=a[1][:1])
    refused("alpha must be", alpha=a[3].double())
    refused("beta must be", beta=a[4][:, :, :1])
    refused("state must be", state=a[5].half())
    refused("contiguous within a slot", state=a[5].transpose(-1, -2))
    refused("slots must be", slots=slots.long())
    refused("slots", slots=slots.cpu())
    refused("last dimension", q=torch.cat([a[0]] * 2, -1)[..., ::2])
    refused("layout", error=g.GemmError, q=torch.cat([a[0]] * 2, 2)[:, :, :3])
    refused("aligned|multiples", error=g.GemmError, q=torch.cat([a[0]] * 2, -1)[..., 4:132])
    nine = a[0][:, :, :1].expand(2, 1, 36, 128)
    refused("8 query heads", error=g.GemmError, q=nine)
    small = dict(q=a[0][..., :64], k=a[1][..., :64], v=a[2][..., :64],
                 state=a[5][..., :64, :64].contiguous())
    refused("head_dim", error=g.GemmError, **small)
    with pytest.raises(g.GemmError, match="states"):
        g.gated_delta_step(*a[:5], s["state"][:1], 0.5)
    with pytest.raises(ValueError, match="out must be"):
        g.gated_delta_step(*a, 0.5, slots, out=torch.empty(2, 1, 2, 128, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(before, s["state"])


def test_refusals_of_the_norm():
    s = norm_inputs(4, 2, 1, 128, 128, 1, torch.bfloat16, seed=62)
    kc, vc = cache_pair(2, 8, 1, 128, torch.bfloat16, "tokens")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")

    def refused(match, error=ValueError, **kw):
        args = dict(q=s["q"], k=s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                    positions=s["positions"], rotary=s["rotary"])
        with pytest.raises(error, match=match):
            g.qk_norm_rope(**{**args, **kw})

    refused("float16 or bfloat16", q=s["q"].float())
    refused("k must be", k=s["k"].half())
    refused("q_weight must be", q_weight=s["q_weight"].float())
    refused("norm must be", norm="layer")
    refused("positions", positions=None)
    refused("rotary", rotary=None)
    refused("positions must be", positions=s["positions"].long())
    refused("sections", positions=s["positions"].expand(3, 4))
    refused("do not hold", positions=s["positions"].expand(2, 4), sections=(30, 30))
    refused("as many sections", positions=s["positions"].expand(5, 4), sections=(64, 0, 0, 0, 0))
    refused("negative section", error=g.GemmError, positions=s["positions"].expand(2, 4),
            sections=(-6, 70))
    refused("k_cache comes with", k_cache=kc)
    refused("come with k_cache", v=s["v"])
    refused("slots must be", v=s["v"], k_cache=kc, v_cache=vc, slots=slots.long())
    refused("overlap", v=s["v"], k_cache=kc[:1].expand(2, 8, 1, 128), v_cache=vc, slots=slots)
    refused("overlap", q_out=s["q"][:1].expand(4, 2, 128))
    refused("multiple of 16", error=g.GemmError, rotary=g.rotary_table(300, 24))
    wide = torch.zeros(4, 1, 264, dtype=torch.bfloat16, device="cuda")
    refused("head_dim", error=g.GemmError, q=wide, k=wide, q_weight=None, k_weight=None)
    torch.cuda.synchronize()
    assert bool(kc.isnan().all())


def test_refusals_of_the_attention():
    s = attn_inputs([5, 6], 4, 2, 128, 16, torch.bfloat16, seed=63)

    def refused(match, error=ValueError, **kw):
        args = dict(q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], page_table=s["table"],
                    lens=s["lens"])
        with pytest.raises(error, match=match):
            g.paged_attention(**{**args, **kw})

    refused("float16 or bfloat16", q=s["q"].float())
    refused("v_cache must be", v_cache=s["v_cache"].half())
    refused("v_cache must be", v_cache=s["v_cache"][:1])
    refused("page_table must be", page_table=s["table"].long())
    refused("lens must be", lens=s["lens"][:1])
    refused("lens", lens=s["lens"].cpu())
    refused("window", window=0)
    refused("out must be", out=torch.empty(2, 4, 128, device="cuda"))
    refused("workspace", workspace=torch.empty(1 << 24, dtype=torch.uint8))
    refused("workspace", error=g.GemmError,
            workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    refused("query heads", error=g.GemmError, q=s["q"][:, :3])
    refused("head_dim", error=g.GemmError, q=s["q"][..., :96],
            k_cache=s["k_cache"][..., :96], v_cache=s["v_cache"][..., :96])
