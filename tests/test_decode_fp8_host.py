"""The operators on an 8-bit cache and on 4-bit weights, host side: argument structs against the C
header, refusals of the C entry points and of the torch ones, none of which reaches a device, and the
nearest 4-bit weights."""
from __future__ import annotations

import re

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
import decode_fp8_ref as ref
import test_decode_host as host
from blackwell_tensor_core_fp16_gb300 import decode
from test_decode_host import BAD, NOT, built_library  # noqa: F401

STRUCTS = {"decode_quantize_cache_args": decode.QUANTIZE_CACHE_ARGS,
           "decode_dequantize_cache_args": decode.DEQUANTIZE_CACHE_ARGS,
           "decode_paged_attention_fp8_args": decode.PAGED_ATTENTION_FP8_ARGS,
           "decode_linear_w4_args": decode.LINEAR_W4_ARGS}


@pytest.fixture(autouse=True)
def structs(monkeypatch):
    monkeypatch.setattr(host, "STRUCTS", {**host.STRUCTS, **STRUCTS})


@pytest.mark.parametrize("name", STRUCTS)
def test_packed_struct_matches_the_header(name, tmp_path):
    host.test_packed_struct_matches_the_header(name, tmp_path)


def pack(name, **values):
    return host.pack(name, **values)


CACHE = dict(tokens=1, h_k=2, head_dim=128, pages=4, page_size=32, block_size=16,
             k=1 << 20, v=2 << 20, k_cache=3 << 20, v_cache=4 << 20, k_scale=5 << 20, v_scale=6 << 20,
             slots=7 << 20, k_cache_stride=(8192, 256, 128), v_cache_stride=(8192, 256, 128),
             k_scale_stride=(4, 2, 1), v_scale_stride=(4, 2, 1), k_stride=(256, 128),
             v_stride=(256, 128))
CACHE_REFUSALS = [
    (dict(tokens=-1), BAD, "negative"), (dict(pages=-1), BAD, "negative"), (dict(h_k=0), BAD, "head"),
    (dict(page_size=0), BAD, "page size"), (dict(block_size=0), BAD, "blocks"),
    (dict(block_size=24), BAD, "blocks"), (dict(block_size=-16), BAD, "blocks"),
    (dict(head_dim=96), NOT, "head_dim"), (dict(dtype=2), BAD, "dtype"), (dict(k=0), BAD, "null"),
    (dict(slots=0), BAD, "null"), (dict(v_scale=0), BAD, "null"), (dict(v=(1 << 20) + 8), NOT, "aligned"),
    (dict(k_cache=(3 << 20) + 8), NOT, "aligned"), (dict(tokens=2, k_stride=(260, 128)), NOT, "multiples of 8"),
    (dict(v_cache_stride=(8192, 264, 128)), NOT, "multiples of 16"),
    (dict(pages=1 << 27), NOT, "too many"), (dict(tokens=1 << 31), NOT, "too many"),
]


@pytest.mark.parametrize("change,code,match", CACHE_REFUSALS + [
    (dict(k_cache=1 << 20), BAD, "k_cache shares memory with k"),
    (dict(k_scale=4 << 20), BAD, "k_scale shares memory with v_cache"),
    (dict(v_scale=7 << 20), BAD, "v_scale shares memory with slots"),
])
def test_quantize_refusals(change, code, match):
    assert g.decode_quantize_cache(pack("decode_quantize_cache_args", **{**CACHE, **change})) == code
    assert re.search(match, g.decode_last_error())


@pytest.mark.parametrize("change,code,match", CACHE_REFUSALS + [
    (dict(k=2 << 20), BAD, "v shares memory with k"), (dict(v=3 << 20), BAD, "v shares memory with k_cache"),
])
def test_dequantize_refusals(change, code, match):
    assert g.decode_dequantize_cache(pack("decode_dequantize_cache_args", **{**CACHE, **change})) == code
    assert re.search(match, g.decode_last_error())


ATTN = dict(n=1, h_q=4, h_kv=2, head_dim=128, pages=2, page_size=32, block_size=16, table_width=1,
            workspace_bytes=1 << 30)


@pytest.mark.parametrize("change,code,match", [
    (dict(n=-1), BAD, "negative"), (dict(sinks=-1), BAD, "negative"), (dict(window=-1), BAD, "negative"),
    (dict(page_size=0), BAD, "page size"), (dict(block_size=12), BAD, "blocks"),
    (dict(dtype=7), BAD, "dtype"), (dict(h_q=3), BAD, "query heads"), (dict(h_kv=0), BAD, "key heads"),
    (dict(head_dim=96), NOT, "head_dim"), (dict(q=0), BAD, "null"), (dict(workspace=0), BAD, "null"),
    (dict(k_scale=0), BAD, "null"), (dict(o=4104), NOT, "aligned"), (dict(q_stride=(0, 4)), NOT, "multiples"),
    (dict(k_stride=(32, 8, 16)), NOT, "multiples of 16"), (dict(pages=1 << 31), NOT, "too large"),
])
def test_attention_refusals(change, code, match):
    args = pack("decode_paged_attention_fp8_args", **{**ATTN, **change})
    assert g.decode_paged_attention_fp8(args) == code
    assert re.search(match, g.decode_last_error())


W4 = dict(m=2, n=4, k=64, group=32, x=1 << 20, codes=2 << 20, scales=3 << 20, zeros=4 << 20,
          bias=5 << 20, y=6 << 20, x_stride=64, code_stride=32, scale_stride=2, zero_stride=2, y_stride=4)


@pytest.mark.parametrize("change,code,match", [
    (dict(m=-1), BAD, "negative"), (dict(dtype=3), BAD, "dtype"), (dict(activation=3), BAD, "activation"),
    (dict(group=0), BAD, "groups"), (dict(group=48), NOT, "multiples of 32"), (dict(k=80), NOT, "multiples of 32"),
    (dict(x=0), BAD, "null"), (dict(y=0), BAD, "null"), (dict(scales=0), BAD, "null"),
    (dict(codes=(2 << 20) + 8), NOT, "aligned"), (dict(x_stride=68), NOT, "x's stride"),
    (dict(code_stride=40), NOT, "codes' stride"), (dict(n=1 << 31), NOT, "too large"),
    (dict(y=1 << 20), BAD, "y shares memory with x"), (dict(bias=6 << 20), BAD, "y shares memory with bias"),
])
def test_linear_refusals(change, code, match):
    assert g.decode_linear_w4(pack("decode_linear_w4_args", **{**W4, **change})) == code
    assert re.search(match, g.decode_last_error())


@pytest.mark.parametrize("change", [
    dict(k_stride=(1 << 33, 256, 128)), dict(v_stride=(8192, 1 << 32, 128)), dict(k_stride=(-8192, 256, 128)),
    dict(k_scale_stride=(1 << 32, 2, 1)), dict(v_scale_stride=(4, 1 << 40, 1)),
])
def test_attention_refuses_strides_past_32_bits(change):
    at = {x: (y + 1) << 20 for y, x in enumerate(("q", "k_cache", "v_cache", "k_scale", "v_scale", "page_table",
                                                  "lens", "o", "workspace"))}
    base = dict(ATTN, **at, q_stride=(512, 128), k_stride=(8192, 256, 128), v_stride=(8192, 256, 128),
                k_scale_stride=(4, 2, 1), v_scale_stride=(4, 2, 1))
    assert g.decode_paged_attention_fp8(pack("decode_paged_attention_fp8_args", **{**base, **change})) == NOT
    assert "below 2^32" in g.decode_last_error()


@pytest.mark.parametrize("change", [
    dict(n=1 << 20, code_stride=4096), dict(n=3, scale_stride=1 << 31), dict(zero_stride=1 << 40),
    dict(n=2, code_stride=1 << 31), dict(code_stride=-32),
])
def test_linear_refuses_weights_past_32_bits(change):
    assert g.decode_linear_w4(pack("decode_linear_w4_args", **{**W4, **change})) == NOT
    assert "2^32" in g.decode_last_error()


def test_empty_problems_do_nothing():
    for name, values, size in (("quantize_cache", CACHE, "tokens"), ("dequantize_cache", CACHE, "tokens"),
                               ("paged_attention_fp8", ATTN, "n"), ("linear_w4", W4, "m"),
                               ("linear_w4", W4, "n")):
        args = pack(f"decode_{name}_args", **{**values, size: 0})
        assert getattr(g, f"decode_{name}")(args) == 0, name
    assert g.decode_last_error() == ""


def test_torch_refusals():
    """What the torch entry points refuse before any device is asked."""
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    codes, scale = torch.zeros(3, 16, 4, 128).to(ref.E4M3), torch.zeros(3, 2, 4, dtype=torch.uint8)
    slots = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g.quantize_cache(x, x, codes, codes, scale, scale, slots)
    with pytest.raises(ValueError, match="16-bit"):
        g.quantize_cache(x.float(), x, codes, codes, scale, scale, slots)
    with pytest.raises(TypeError, match="slots must be a tensor"):
        g.quantize_cache(x, x, codes, codes, scale, scale, [0, 1])
    with pytest.raises(ValueError, match="CUDA"):
        g.dequantize_cache(codes, codes, scale, scale, slots)
    with pytest.raises(ValueError, match="dtype"):
        g.dequantize_cache(codes, codes, scale, scale, slots, dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        g.paged_attention_fp8(x, codes, codes, scale, scale, slots[None], slots)
    w = torch.zeros(8, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="activation"):
        g.linear_w4(x[0, :, :32], w, x[0, :1], 32, activation="tanh")
    with pytest.raises(ValueError, match="CUDA"):
        g.linear_w4(x[0, :, :32], w, x[0, :1], 32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("k,group", [(128, 32), (160, 64), (96, 96), (64, 128)])
@pytest.mark.parametrize("zeros", [True, False])
def test_nearest_weights(k, group, zeros, dtype):
    """Codes stand for weights within half a step of theirs; where a zero point is rounded or a scale
    is, the ends of a group's range may be a step further (16 steps of half a rounding)."""
    gen = torch.Generator().manual_seed(k + group)
    W = torch.randn(5, k, generator=gen).to(dtype)
    W[1] = 0
    W[2] = W[2].abs() + 3                        # a range far from zero
    W[3, :7] = 40.0
    codes, scales, z = g.quantize_weight_w4(W, group, zeros)
    assert codes.shape == (5, k // 2) and scales.shape == (5, -(-k // group)) and scales.dtype == dtype
    assert (z is not None) == zeros
    eye = torch.eye(k, dtype=torch.float64)
    back, _ = ref.linear_w4(eye, codes, scales, group, z)
    step = scales.double()[:, torch.arange(k) // group]
    err = (back.T - W.double()).abs()
    half = 0.5 + (0.5 if zeros else 0.0) + 15 * ref.U[dtype]
    assert bool((err <= half * step + 1e-12).all())
    assert bool((back.T[1] == 0).all())


def test_weights_that_are_refused():
    for W in (torch.zeros(3, 5).half(), torch.zeros(4, 4), torch.zeros(4).half()):
        with pytest.raises(ValueError, match="matrix"):
            g.quantize_weight_w4(W)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("zeros", [True, False])
def test_nearest_weights_at_the_ends_of_the_range(zeros, dtype):
    """The bound of test_nearest_weights where a scale is a subnormal number, which is rounded up, so that
    no code is cut off for it, and where a group's range passes fp32's: a code's step is the scale that
    comes back, whatever its size."""
    gen = torch.Generator().manual_seed(int(zeros))
    sizes = (1e-4, 1e-5, 1e-6, 1e-7) if dtype == torch.float16 else (1e-37, 1e-38, 1e-39, 1e-40)
    normal = torch.randn(len(sizes) + 2, 256, generator=gen, dtype=torch.float64)
    W = (normal * torch.tensor(sizes + (0.0, 0.0), dtype=torch.float64)[:, None]).to(dtype)
    W[-2] = torch.finfo(dtype).max * torch.sign(normal[-2])                # one after the other, either sign
    W[-1, 3] = W[-1, 200] = torch.finfo(dtype).tiny * torch.finfo(dtype).eps      # the least number alone
    codes, scales, z = g.quantize_weight_w4(W, 128, zeros)
    assert bool(scales.isfinite().all()) and bool((scales > 0).all())
    back, _ = ref.linear_w4(torch.eye(256, dtype=torch.float64), codes, scales, 128, z)
    step = scales.double().repeat_interleave(128, 1)
    err = (back.T - W.double()).abs()
    half = 0.5 + (0.5 if zeros else 0.0) + 15 * ref.U[dtype]
    assert bool((err <= half * step).all())
    # no scale is larger than its group asks for by more than its own rounding
    top = W.double().view(len(W), 2, 128)
    need = (top.amax(-1).clamp(min=0) - top.amin(-1).clamp(max=0)) / 15 if zeros else top.abs().amax(-1) / 7
    least = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    assert bool((scales.double() <= need * (1 + ref.U[dtype]) + least).all())


def test_weights_of_a_group_wider_than_the_matrix():
    """A group may be wider than K, as in linear_w4, by any amount."""
    W = torch.randn(3, 64, generator=torch.Generator().manual_seed(1)).half()
    for zeros in (True, False):
        for one, other in zip(g.quantize_weight_w4(W, 1 << 50, zeros), g.quantize_weight_w4(W, 64, zeros)):
            assert (one is None and other is None) or torch.equal(one, other)


def test_wait_limit_and_testing_hook_refuse_what_they_do_not_have():
    assert g.decode_set_wait_timeout_ms(0) == BAD and "1 ms" in g.decode_last_error()
    assert g.decode_set_wait_timeout_ms(2000) == 0
    for mode in (-1, 2):
        assert g.decode_set_fault_injection(mode) == BAD and "fault mode" in g.decode_last_error()
    assert g.decode_set_fault_injection(0) == 0
