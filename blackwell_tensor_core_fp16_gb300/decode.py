"""The operators of a decode step (C ABI in ``include/decode.h``): what a model with gated-delta-net
and attention layers runs between its dense products when every sequence has one or a few new
tokens.

* ``gated_delta_step``: the gated delta rule token by token on a pool of states;
* ``qk_norm_rope``: norm and position rotation of queries and keys, with the write of keys and
  values into a paged cache;
* ``paged_attention``: attention of one new token per sequence over that cache.

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

from . import GemmError, _build, load

DECODE_OK, DECODE_ERR_INVALID_ARG, DECODE_ERR_UNSUPPORTED, DECODE_ERR_CUDA = 0, 1, 2, 3
DECODE_NORMS = {"none": 0, "rms": 1, "l2": 2}
DECODE_STATUS = {1: "a state slot outside the pool", 2: "a cache slot outside the cache",
                 4: "a position outside the rotary table",
                 8: "a sequence length its page table cannot hold",
                 16: "a page number outside the cache"}

# The argument structs of include/decode.h, field by field (no padding on either side).
GDN_STEP_ARGS = struct.Struct("=8Q7q9q4qqif")
QK_NORM_ROPE_ARGS = struct.Struct("=12Q9q10q6qq4iiiif")
PAGED_ATTENTION_ARGS = struct.Struct("=8Qq9q2q6qif")


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


def decode_last_error() -> str:
    return load().decode_last_error().decode()


def decode_check_status(stream: int = 0):
    """Returns (status, bits)."""
    bits = ctypes.c_uint32(0)
    rc = load().decode_check_status(stream, ctypes.byref(bits))
    return rc, bits.value


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
