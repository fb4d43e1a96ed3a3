"""The decode-step operators on the GPU where they can go wrong: results that cancel, infinities,
sequences whose every score is masked, operands that share memory, and the kernels' less travelled
paths."""
from __future__ import annotations

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
import decode_ref as ref
from test_decode_gpu import (attn_inputs, cuda_library, generator, no_refusals_left,  # noqa: F401
                             normal)

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
