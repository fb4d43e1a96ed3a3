"""The operators of a decode step (C ABI in ``include/decode.h``): what a model with gated-delta-net
and attention layers runs between its dense products when every sequence has one or a few new
tokens.

* ``gated_delta_step``: the gated delta rule token by token on a pool of states;
* ``qk_norm_rope``: norm and position rotation of queries and keys, with the write of keys and
  values into a paged cache;
* ``paged_attention``: attention of one new token per sequence over that cache;
* ``quantize_cache``, ``dequantize_cache``, ``paged_attention_fp8``: the same on a cache of 8-bit codes
  with a scale for each block of tokens and head, which takes half the memory and time;
* ``linear_w4``: a linear layer with 4-bit weights (``quantize_weight_w4`` makes them).

The torch entry points check shapes, types and devices on the host and raise ``ValueError``, or
``GemmError`` with the library's message where the C call refuses.  They are asynchronous on
``stream`` (default: torch's current stream) and never synchronise, so they can be captured into a
CUDA graph.  Indices that live in device memory are checked by the kernels:
``check_decode_status`` raises if one was refused.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import ACTIVATIONS, GemmError, _build, load

DECODE_OK, DECODE_ERR_INVALID_ARG, DECODE_ERR_UNSUPPORTED, DECODE_ERR_CUDA = 0, 1, 2, 3
DECODE_NORMS = {"none": 0, "rms": 1, "l2": 2}
DECODE_STATUS = {1: "a state slot outside the pool",
                 2: "a cache slot outside the cache, or out of its block's order",
                 4: "a position outside the rotary table",
                 8: "a sequence length its page table cannot hold",
                 16: "a page number outside the cache", 32: "a copy or product that took too long"}

# The argument structs of include/decode.h, field by field (no padding on either side).
GDN_STEP_ARGS = struct.Struct("=8Q7q9q4qqif")
QK_NORM_ROPE_ARGS = struct.Struct("=12Q9q10q6qq4iiiif")
PAGED_ATTENTION_ARGS = struct.Struct("=8Qq9q2q6qif")
QUANTIZE_CACHE_ARGS = struct.Struct("=7Q5q4q6q6qii")
DEQUANTIZE_CACHE_ARGS = struct.Struct("=7Q5q4q6q6qii")
PAGED_ATTENTION_FP8_ARGS = struct.Struct("=10Qq10q2q6q6qqif")
LINEAR_W4_ARGS = struct.Struct("=6Q4q5qii")


# ---- the C ABI, one Python function per C function (args: the packed struct) ---------------------

def decode_gdn_step(args: bytes, stream: int = 0) -> int:
    return load().decode_gdn_step(args, stream)


def decode_qk_norm_rope(args: bytes, stream: int = 0) -> int:
    return load().decode_qk_norm_rope(args, stream)


def decode_paged_attention(args: bytes, stream: int = 0) -> int:
    return load().decode_paged_attention(args, stream)


def decode_paged_attention_workspace_bytes(h_q: int, h_kv: int, head_dim: int) -> int:
    out = ctypes.c_size_t(0)
    rc = load().decode_paged_attention_workspace_bytes(h_q, h_kv, head_dim, ctypes.byref(out))
    if rc != DECODE_OK:
        raise GemmError(rc, decode_last_error())
    return out.value


def decode_quantize_cache(args: bytes, stream: int = 0) -> int:
    return load().decode_quantize_cache(args, stream)


def decode_dequantize_cache(args: bytes, stream: int = 0) -> int:
    return load().decode_dequantize_cache(args, stream)


def decode_paged_attention_fp8(args: bytes, stream: int = 0) -> int:
    return load().decode_paged_attention_fp8(args, stream)


def decode_paged_attention_fp8_workspace_bytes(h_q: int, h_kv: int, head_dim: int) -> int:
    out = ctypes.c_size_t(0)
    rc = load().decode_paged_attention_fp8_workspace_bytes(h_q, h_kv, head_dim, ctypes.byref(out))
    if rc != DECODE_OK:
        raise GemmError(rc, decode_last_error())
    return out.value


def decode_linear_w4(args: bytes, stream: int = 0) -> int:
    return load().decode_linear_w4(args, stream)


def decode_last_error() -> str:
    return load().decode_last_error().decode()


def decode_check_status(stream: int = 0):
    """Returns (status, bits)."""
    bits = ctypes.c_uint32(0)
    rc = load().decode_check_status(stream, ctypes.byref(bits))
    return rc, bits.value


def decode_set_wait_timeout_ms(ms: int) -> int:
    return load().decode_set_wait_timeout_ms(ms)


def decode_set_fault_injection(mode: int) -> int:
    return load().decode_set_fault_injection(mode)


# ---- torch entry points ---------------------------------------------------------------------------
#
# Their checks, allocations and launches are in csrc/decode_binding.cpp.

def _binding():
    """The module _decode (RuntimeError if it is missing)."""
    load()
    try:
        from . import _decode
    except ImportError as e:
        raise RuntimeError(
            f"{_build.BINDING_PATH} cannot be loaded ({e}): build it first "
            "(blackwell_tensor_core_fp16_gb300.build()); there is no fallback path") from e
    return _decode


_decode = _binding()


def gated_delta_step(q, k, v, alpha, beta, state, scale: float, slots=None, out=None, stream=None):
    """The gated delta rule, token by token, on a pool of states: for each sequence i and value
    head, with S the state in slot ``slots[i]`` and for its tokens in order

        S' = alpha S;  u = beta (v - S' k);  S = S' + u k^T;  o = scale S q

    q [n, tokens, h_q, 128], k [n, tokens, h_k, 128], v [n, tokens, h_v, 128], float16 or bfloat16
    (views of a packed projection are fine: only the last dimension must be contiguous); alpha,
    beta [n, tokens, h_v] float32; state [slots, h_v, 128, 128] float32, updated in place, in the
    layout of ``gated_delta_rule``'s final_state; slots [n] int32 or None for 0 .. n - 1.  Heads as
    in ``gated_delta_rule``.  A sequence with slot -1 is inactive: its output is zero and no state
    changes.  No two sequences may share a slot.  Returns o [n, tokens, max(h_q, h_v), 128]; ``out``
    may be ``v`` itself but share no other memory with the operands."""
    return _decode.gated_delta_step(q, k, v, alpha, beta, state, scale, slots, out, stream)


def rotary_table(positions: int, rot: int, base: float = 10000.0, device="cuda"):
    """The table of ``qk_norm_rope``: float32 [positions, rot], row p with the cosines and then the
    sines of p * base^(-2 j / rot), j < rot / 2, taken in 64 bits."""
    rate = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)


def qk_norm_rope(q, k, q_weight=None, k_weight=None, norm: str = "rms", eps: float = 1e-6,
                 positions=None, rotary=None, sections=None, interleaved: bool = False, v=None,
                 k_cache=None, v_cache=None, slots=None, q_out=None, k_out=None, stream=None):
    """Norm of each query and key head, then its rotation by the token's position, in one pass:

        y = x / sqrt(mean(x^2) + eps) * weight      norm "rms" ("l2": sum in place of mean;
                                                    "none": y = x * weight)
        (a, b) -> (a cos - b sin, b cos + a sin)    for the pairs of the first ``rot`` elements

    q [tokens, h_q, d], k [tokens, h_k, d] float16 or bfloat16 (views of a packed projection are
    fine); weights [d] of the same type or None for ones.  ``rotary`` float32 [rows, rot] holds
    cosines and sines (``rotary_table``; None: no rotation) and ``positions`` int32 [tokens] the
    rows, or [axes, tokens] with ``sections`` the number of pairs of each axis.  Pair j is (j,
    rot / 2 + j), or (2 j, 2 j + 1) with ``interleaved``.

    With ``k_cache`` and ``v_cache`` [pages, page_size, h_k, d] (any strides with a dense last
    dimension), ``v`` [tokens, h_k, d] and ``slots`` int32 [tokens] (page * page_size + offset, or -1
    for none) the keys and values go to the cache and only q is returned in the pair (q, None);
    else the pair is (q, k).  ``q_out`` and ``k_out`` may be ``q`` and ``k`` themselves; what is written
    may share no other memory with the operands."""
    if norm not in DECODE_NORMS:
        raise ValueError(f"norm must be one of {sorted(DECODE_NORMS)}")
    return _decode.qk_norm_rope(q, k, q_weight, k_weight, DECODE_NORMS[norm], eps, positions, rotary,
                                sections, interleaved, v, k_cache, v_cache, slots, q_out, k_out,
                                stream)


def paged_attention_workspace(h_q: int, h_kv: int, head_dim: int, device="cuda"):
    """A workspace for ``paged_attention`` with these heads, whatever the batch and the lengths.  A
    program keeps one per stream; calls that may overlap on the GPU must not share one."""
    device = torch.device(device)
    with torch.cuda.device(device):
        size = decode_paged_attention_workspace_bytes(h_q, h_kv, head_dim)
    return torch.empty(size, dtype=torch.uint8, device=device)


def paged_attention(q, k_cache, v_cache, page_table, lens, scale: float | None = None,
                    window: int | None = None, return_lse: bool = False, out=None, workspace=None,
                    stream=None):
    """Attention of one new token per sequence over a paged cache: query head m of sequence i
    attends to the first ``lens[i]`` cached tokens (the last ``window`` of them, if given) of key
    head m // (h_q // h_kv),

        o = sum_t softmax_t(scale q . K_t) V_t,     lse = log sum_t exp(scale q . K_t)

    q [n, h_q, d] float16 or bfloat16, d 64, 128 or 256; k_cache, v_cache [pages, page_size, h_kv,
    d] of the same type (any strides with a dense last dimension); page_table [n, width] int32:
    token t lies in page ``page_table[i, t // page_size]``; lens [n] int32.  scale: default
    d ** -0.5.  A sequence of length 0, or all of whose scores are -infinity, gives zeros and lse
    -inf.  Returns o [n, h_q, d], or (o, lse [n, h_q] float32) with ``return_lse``.
    ``workspace``: from ``paged_attention_workspace``; None takes one from torch's allocator for the
    call.  A page table no wider than the lengths need lets a few short sequences run in one launch.
    ``out`` may be ``q`` itself; what is written may share no other memory with the operands."""
    return _decode.paged_attention(q, k_cache, v_cache, page_table, lens, scale, window, return_lse,
                                   out, workspace, stream)


def quantize_cache(k, v, k_cache, v_cache, k_scale, v_scale, slots, stream=None) -> None:
    """Write keys and values to their places in a paged cache of E4M3 codes with one E8M0 scale for
    each block of tokens and head: a code c under the scale e stands for c * 2^(e - 127).  For each block
    and head that new tokens go to, keys and values each on their own,

        need = the least e >= 0 with |x| <= 448 * 2^(e - 127) for all finite new elements x
        e'   = need, or max(need, e) where the block holds older tokens, of scale e
        c    = e4m3(x * 2^(127 - e')),   and where e' > e, of its other codes e4m3(c * 2^(e - e'))

    k, v [tokens, h_k, d] float16 or bfloat16, d 64, 128 or 256 (views of a packed projection are fine);
    k_cache, v_cache [pages, page_size, h_k, d] float8_e4m3fn or uint8 (strides multiples of 16, a dense
    last dimension); k_scale, v_scale [pages, blocks, h_k] uint8: blocks of page_size / blocks tokens.
    slots int32 [tokens]: page * page_size + offset, or -1 for none.

    A block's tokens fill it from its first place on, over any number of calls: what lies below a
    call's first place in a block are older tokens, what lies above is nothing.  In a call they follow
    one another in the order of their places, without a gap; one that comes up to 160 tokens after
    another of its block and does not continue it is refused (``check_decode_status``), and tokens of one
    block that are further apart leave it undefined.  An infinity or NaN is held as NaN."""
    _decode.quantize_cache(k, v, k_cache, v_cache, k_scale, v_scale, slots, stream)


def dequantize_cache(k_cache, v_cache, k_scale, v_scale, slots, dtype=torch.bfloat16, k_out=None,
                     v_out=None, stream=None):
    """The keys and values that a cache of ``quantize_cache`` holds at ``slots`` (int32 [tokens]),
    rounded once to ``dtype`` (float16 or bfloat16): a pair of tensors [tokens, h_k, d].  Slot -1 gives
    zeros.  ``k_out`` and ``v_out`` may have any strides with a dense last dimension; they may share
    no memory with each other or the operands."""
    if dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("dtype must be float16 or bfloat16")
    return _decode.dequantize_cache(k_cache, v_cache, k_scale, v_scale, slots,
                                    dtype == torch.float16, k_out, v_out, stream)


def paged_attention_fp8_workspace(h_q: int, h_kv: int, head_dim: int, device="cuda"):
    """A workspace for ``paged_attention_fp8``, as ``paged_attention_workspace`` makes one."""
    device = torch.device(device)
    with torch.cuda.device(device):
        size = decode_paged_attention_fp8_workspace_bytes(h_q, h_kv, head_dim)
    return torch.empty(size, dtype=torch.uint8, device=device)


def paged_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, lens,
                        scale: float | None = None, window: int | None = None, sinks: int = 0,
                        return_lse: bool = False, out=None, workspace=None, stream=None):
    """``paged_attention`` over a cache of ``quantize_cache``: the same operands, results and refusals,
    with the values that the codes stand for (the C header says to what precision, and for which scales).
    With a ``window`` the first ``sinks`` tokens stay visible beside the last ``window``.  ``workspace``:
    from ``paged_attention_fp8_workspace``; None takes one from torch's allocator for the call."""
    return _decode.paged_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, lens, scale,
                                       window, sinks, return_lse, out, workspace, stream)


def quantize_weight_w4(W, group: int = 128, zeros: bool = True):
    """The operands of ``linear_w4`` nearest to W [N, K] float16 or bfloat16, K even, each group of
    ``group`` neighbouring columns of a row (the last may be shorter) on its own: (codes, scales,
    zeros).  With ``zeros`` a group's range, stretched to hold 0, is dealt to the codes 0 .. 15;
    without, its largest magnitude to 7 either side of 8, and None takes the zeros' place.  W is finite."""
    if W.dim() != 2 or W.dtype not in (torch.float16, torch.bfloat16) or W.shape[1] % 2 or group < 1:
        raise ValueError("W must be a float16 or bfloat16 matrix with an even number of columns")
    n, k = W.shape
    group = min(group, max(k, 1))
    groups = -(-k // group)
    w = torch.nn.functional.pad(W.float(), (0, groups * group - k)).view(n, groups, group)
    # (in 64 bits: a range of bfloat16 may pass fp32's)
    if zeros:
        low, high = w.amin(-1).clamp(max=0).double(), w.amax(-1).clamp(min=0).double()
        scale = (high - low) / 15
    else:
        scale = w.abs().amax(-1).double() / 7
    # a scale that is a subnormal number is rounded up: down, it could leave the largest weights out of the
    # codes' reach by half of theirs
    info = torch.finfo(W.dtype)
    least = info.tiny * info.eps
    scale = torch.where(scale < info.tiny, torch.ceil(scale / least) * least, scale).to(W.dtype)
    by = torch.where(scale > 0, scale.float(), 1.0)
    zero = torch.round(-low / by).clamp(0, 15).float() if zeros else torch.full_like(by, 8)
    code = torch.round(w / by[..., None] + zero[..., None]).clamp(0, 15).to(torch.uint8)
    code = code.view(n, groups * group)[:, :k]
    return (code[:, 0::2] | code[:, 1::2] << 4).contiguous(), scale, \
        zero.to(torch.uint8) if zeros else None


def linear_w4(x, codes, scales, group: int = 128, zeros=None, bias=None, activation: str = "none",
              out=None, stream=None):
    """act(x @ W.T + bias) with 4-bit weights, for few tokens:

        W[j, c] = scales[j, c // group] * (code[j, c] - zeros[j, c // group])

    x [tokens, K] float16 or bfloat16; codes uint8 [N, K / 2]: column 2 c in byte c's lower half, column
    2 c + 1 in its upper; scales [N, ceil(K / group)] of x's type; zeros uint8 of the same shape, or None
    for 8 everywhere; bias [N] of x's type.  K and group are multiples of 32.  Rows of all but bias may
    be strided (x by multiples of 8, codes of 16 elements).  No weight is rounded: groups' sums and their
    scaling are fp32.  activation: "none", "relu" or "gelu".  Returns [tokens, N] in x's type.

    Takes less time than ``linear`` with 16-bit weights up to 64 tokens (14336 x 4096 weights: 18 and 25
    us), of small weights up to some 256 (4096 x 4096: 17 and 19); for more, ``linear`` is faster (2048
    tokens, 14336 x 4096: 419 and 151), with the weights in 16 bits."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return _decode.linear_w4(x, codes, scales, group, zeros, bias, ACTIVATIONS[activation], out, stream)


def check_decode_status(stream=None) -> None:
    """Synchronise ``stream`` and raise GemmError if a kernel of this module refused an index on the
    stream's device since the last check there.  A device's streams and threads share the record,
    and a refusal is reported to whichever check comes first after it."""
    if stream is None:
        stream = torch.cuda.current_stream()
    if hasattr(stream, "cuda_stream"):
        # (a default stream's handle does not say whose it is)
        with torch.cuda.device(stream.device):
            rc, bits = decode_check_status(int(stream.cuda_stream))
    else:
        rc, bits = decode_check_status(int(stream))
    if rc != DECODE_OK:
        raise GemmError(rc, decode_last_error())
    if bits:
        raise GemmError(DECODE_ERR_INVALID_ARG,
                        "refused: " + "; ".join(w for b, w in DECODE_STATUS.items() if bits & b))
