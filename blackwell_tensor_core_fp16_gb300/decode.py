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

from . import GemmError, load

DECODE_OK, DECODE_ERR_INVALID_ARG, DECODE_ERR_UNSUPPORTED, DECODE_ERR_CUDA = 0, 1, 2, 3
DECODE_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
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


# ---- checks that the torch entry points share ---------------------------------------------------
#
# A call on a few tokens takes a few microseconds on the GPU, so the entry points test all of their
# operands in one expression and look for the one at fault (_explain) only when it fails.

def _explain(device, *operands):
    """Raises ValueError for the first operand (name, tensor, dtype, shape) that is not what it
    has to be."""
    for name, t, dtype, shape in operands:
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    raise ValueError("operands must be CUDA tensors on one device")


def _dense(name, shape, stride):
    """Refuses a tensor whose last dimension is not contiguous."""
    if stride[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _written(name, t):
    """Refuses a tensor that is written and whose elements may share memory (its strides are not
    those of a dense tensor's permuted and padded dimensions)."""
    reach = t.shape[-1]
    for s, n in sorted((s, n) for s, n in zip(t.stride()[:-1], t.shape[:-1]) if n > 1):
        if s < reach:
            raise ValueError(f"{name}'s elements overlap")
        reach = s * (n - 1) + reach


def _half_dtype(q):
    code = DECODE_DTYPES.get(q.dtype)
    if code is None:
        raise ValueError("16-bit operands must be float16 or bfloat16")
    if not q.is_cuda:
        raise ValueError("operands must be CUDA tensors")
    return code


def _call(function, args, index, stream):
    """The C call on device ``index`` and the given stream."""
    if stream is None:
        handle = _current_stream(index)
    else:
        handle = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == index:
        rc = function(args, handle)
    else:
        with torch.cuda.device(index):
            rc = function(args, handle)
    if rc != DECODE_OK:
        raise GemmError(rc, decode_last_error())


# torch.cuda.current_stream(i).cuda_stream without the Stream object in between (0.1 for 3 us)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _empty(shape, dtype, device, stream):
    """New memory that belongs to the stream the call runs on."""
    if stream is not None and hasattr(stream, "cuda_stream"):
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


# ---- torch entry points ---------------------------------------------------------------------------

def gated_delta_step(q, k, v, alpha, beta, state, scale: float, slots=None, out=None, stream=None):
    """The gated delta rule, token by token, on a pool of states: for each sequence i and value
    head, with S the state in slot ``slots[i]`` and for its tokens in order

        S' = alpha S;  u = beta (v - S' k);  S = S' + u k^T;  o = scale S q

    q [n, tokens, h_q, 128], k [n, tokens, h_k, 128], v [n, tokens, h_v, 128], float16 or bfloat16
    (views of a packed projection are fine: only the last dimension must be contiguous); alpha,
    beta [n, tokens, h_v] float32; state [slots, h_v, 128, 128] float32, updated in place, in the
    layout of ``gated_delta_rule``'s final_state; slots [n] int32 or None for 0 .. n - 1.  Heads as
    in ``gated_delta_rule``.  A sequence with slot -1 is inactive: its output is zero and no state
    changes.  No two sequences may share a slot.  Returns o [n, tokens, max(h_q, h_v), 128]."""
    code = _half_dtype(q)
    dt, qs, ks, vs, ss = q.dtype, q.shape, k.shape, v.shape, state.shape
    if len(qs) != 4 or len(ks) != 4 or len(vs) != 4 or len(ss) != 4:
        raise ValueError("q, k and v must be [n, tokens, heads, head_dim], state [slots, h_v, d, d]")
    n, tokens, h_q, d = qs
    h_k, h_v, n_slots, index = ks[2], vs[2], ss[0], q.get_device()
    shape = (n, tokens, h_q if h_q > h_v else h_v, d)
    if out is None:
        out = _empty(shape, dt, q.device, stream)
    if not (k.dtype is dt and v.dtype is dt and out.dtype is dt and alpha.dtype is torch.float32
            and beta.dtype is torch.float32 and state.dtype is torch.float32
            and ks == (n, tokens, h_k, d) and vs == (n, tokens, h_v, d) and out.shape == shape
            and alpha.shape == beta.shape == (n, tokens, h_v) and ss == (n_slots, h_v, d, d)
            and k.get_device() == v.get_device() == out.get_device() == alpha.get_device()
            == beta.get_device() == state.get_device() == index
            and (slots is None or (slots.dtype is torch.int32 and slots.shape == (n,)
                                   and slots.get_device() == index))):
        _explain(q.device, ("k", k, dt, (n, tokens, h_k, d)), ("v", v, dt, (n, tokens, h_v, d)),
                 ("alpha", alpha, torch.float32, (n, tokens, h_v)),
                 ("beta", beta, torch.float32, (n, tokens, h_v)),
                 ("state", state, torch.float32, (n_slots, h_v, d, d)),
                 ("out", out, dt, shape), *([] if slots is None else [
                     ("slots", slots, torch.int32, (n,))]))
    q_stride, k_stride, v_stride, state_stride = q.stride(), k.stride(), v.stride(), state.stride()
    a_stride, b_stride = alpha.stride(), beta.stride()
    for name, size, stride in (("q", qs, q_stride), ("k", ks, k_stride), ("v", vs, v_stride),
                               ("alpha", alpha.shape, a_stride), ("beta", beta.shape, b_stride)):
        if stride[-1] != 1:
            _dense(name, size, stride)
    if state_stride[1:] != (d * d, d, 1) and (h_v > 1 or state_stride[2:] != (d, 1)):
        raise ValueError("state must be contiguous within a slot")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if slots is not None and not slots.is_contiguous():
        raise ValueError("slots must be contiguous")
    args = GDN_STEP_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), beta.data_ptr(),
        state.data_ptr(), 0 if slots is None else slots.data_ptr(), out.data_ptr(),
        n, tokens, h_q, h_k, h_v, d, n_slots, *q_stride[:3], *k_stride[:3], *v_stride[:3],
        *a_stride[:2], *b_stride[:2], state_stride[0], code, scale)
    _call(load().decode_gdn_step, args, index, stream)
    return out


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
    else the pair is (q, k).  ``q_out`` and ``k_out`` may be ``q`` and ``k`` themselves."""
    code = _half_dtype(q)
    dt, qs, ks, device, index = q.dtype, q.shape, k.shape, q.device, q.get_device()
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    if norm not in DECODE_NORMS:
        raise ValueError(f"norm must be one of {sorted(DECODE_NORMS)}")
    tokens, h_q, d = qs
    h_k = ks[1]
    if not (k.dtype is dt and ks == (tokens, h_k, d) and k.get_device() == index
            and (q_weight is None or (q_weight.dtype is dt and q_weight.shape == (d,)
                                      and q_weight.get_device() == index))
            and (k_weight is None or (k_weight.dtype is dt and k_weight.shape == (d,)
                                      and k_weight.get_device() == index))):
        _explain(device, ("k", k, dt, (tokens, h_k, d)),
                 *((name, w, dt, (d,)) for name, w in (("q_weight", q_weight),
                                                       ("k_weight", k_weight)) if w is not None))
    qw_ptr = kw_ptr = 0
    if q_weight is not None:
        if not q_weight.is_contiguous():
            raise ValueError("q_weight must be contiguous")
        qw_ptr = q_weight.data_ptr()
    if k_weight is not None:
        if not k_weight.is_contiguous():
            raise ValueError("k_weight must be contiguous")
        kw_ptr = k_weight.data_ptr()

    rot = axes = rows = position_stride = position_ptr = table_ptr = 0
    sec = (0, 0, 0, 0)
    if rotary is not None:
        if rotary.dim() != 2 or not rotary.is_contiguous():
            raise ValueError("rotary must be a contiguous [rows, rot] table")
        rows, rot = rotary.shape
        if positions is None or positions.dim() not in (1, 2):
            raise ValueError("a rotation needs positions [tokens] or [axes, tokens]")
        ps, p_stride = positions.shape, positions.stride()
        axes = 1 if len(ps) == 1 else ps[0]
        if not (positions.dtype is torch.int32 and rotary.dtype is torch.float32
                and ps[-1] == tokens and positions.get_device() == rotary.get_device() == index):
            _explain(device, ("rotary", rotary, torch.float32, (rows, rot)),
                     ("positions", positions, torch.int32, (*ps[:-1], tokens)))
        if p_stride[-1] != 1:
            _dense("positions", ps, p_stride)
        if len(ps) == 2:
            if sections is None or len(sections) != axes or not 1 <= axes <= 4:
                raise ValueError("positions of 1 to 4 axes need as many sections")
            position_stride = p_stride[0]
            sec = (*(int(x) for x in sections), *(0,) * (4 - axes))
            if sum(sec) != rot // 2:
                raise ValueError(f"sections {list(sections)} do not hold rot / 2 = {rot // 2} pairs")
        elif sections is not None:
            raise ValueError("sections need positions [axes, tokens]")
        position_ptr, table_ptr = positions.data_ptr(), rotary.data_ptr()
    elif positions is not None or sections is not None:
        raise ValueError("positions and sections need a rotary table")

    pages = page_size = v_ptr = kc_ptr = vc_ptr = slot_ptr = ko_ptr = 0
    v_stride, kc_stride, vc_stride, ko_stride = (0, 0), (0, 0, 0), (0, 0, 0), (0, 0)
    if k_cache is not None:
        if v is None or v_cache is None or slots is None or k_cache.dim() != 4 or k_out is not None:
            raise ValueError("k_cache comes with v, v_cache and slots, [pages, page_size, h_k, d], "
                             "and without k_out")
        cs = k_cache.shape
        pages, page_size = cs[0], cs[1]
        if not (v.dtype is dt and k_cache.dtype is dt and v_cache.dtype is dt
                and slots.dtype is torch.int32 and v.shape == (tokens, h_k, d)
                and cs == v_cache.shape == (pages, page_size, h_k, d) and slots.shape == (tokens,)
                and v.get_device() == k_cache.get_device() == v_cache.get_device()
                == slots.get_device() == index):
            _explain(device, ("v", v, dt, (tokens, h_k, d)),
                     ("k_cache", k_cache, dt, (pages, page_size, h_k, d)),
                     ("v_cache", v_cache, dt, (pages, page_size, h_k, d)),
                     ("slots", slots, torch.int32, (tokens,)))
        if not slots.is_contiguous():
            raise ValueError("slots must be contiguous")
        v_stride, kc_stride, vc_stride = v.stride(), k_cache.stride(), v_cache.stride()
        for name, t, stride in (("v", v, v_stride), ("k_cache", k_cache, kc_stride),
                                ("v_cache", v_cache, vc_stride)):
            if stride[-1] != 1:
                _dense(name, t.shape, stride)
        if not k_cache.is_contiguous():
            _written("k_cache", k_cache)
        if not v_cache.is_contiguous():
            _written("v_cache", v_cache)
        v_ptr, kc_ptr, vc_ptr = v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
        slot_ptr = slots.data_ptr()
    else:
        if v is not None or v_cache is not None or slots is not None:
            raise ValueError("v, v_cache and slots come with k_cache")
        if k_out is None:
            k_out = _empty((tokens, h_k, d), dt, device, stream)
            ko_stride = (h_k * d, d)
        else:
            ko_stride = _output("k_out", k_out, dt, (tokens, h_k, d), device)
        ko_ptr = k_out.data_ptr()
    if q_out is None:
        q_out = _empty((tokens, h_q, d), dt, device, stream)
        qo_stride = (h_q * d, d)
    else:
        qo_stride = _output("q_out", q_out, dt, (tokens, h_q, d), device)
    q_stride, k_stride = q.stride(), k.stride()
    if q_stride[-1] != 1:
        _dense("q", qs, q_stride)
    if k_stride[-1] != 1:
        _dense("k", ks, k_stride)
    args = QK_NORM_ROPE_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v_ptr, qw_ptr, kw_ptr, position_ptr, table_ptr,
        q_out.data_ptr(), ko_ptr, kc_ptr, vc_ptr, slot_ptr,
        tokens, h_q, h_k, d, rot, axes, rows, pages, page_size,
        *q_stride[:2], *k_stride[:2], *v_stride[:2], *qo_stride[:2], *ko_stride[:2],
        *kc_stride[:3], *vc_stride[:3], position_stride, *sec, code, DECODE_NORMS[norm],
        bool(interleaved), eps)
    _call(load().decode_qk_norm_rope, args, index, stream)
    return q_out, k_out


def _output(name, t, dtype, shape, device):
    """Strides of an output that the caller gave."""
    if not (t.dtype is dtype and t.shape == shape and t.device == device):
        _explain(device, (name, t, dtype, shape))
    stride = t.stride()
    if stride[-1] != 1:
        _dense(name, shape, stride)
    _written(name, t)
    return stride


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
    d ** -0.5.  A sequence of length 0 gives zeros and lse -inf.  Returns o [n, h_q, d], or (o,
    lse [n, h_q] float32) with ``return_lse``.  ``workspace``: from ``paged_attention_workspace``;
    None takes one from torch's allocator for the call."""
    code = _half_dtype(q)
    dt, qs, cs, ts = q.dtype, q.shape, k_cache.shape, page_table.shape
    device, index = q.device, q.get_device()
    if len(qs) != 3 or len(cs) != 4 or len(ts) != 2:
        raise ValueError("q must be [n, h_q, d], the caches [pages, page_size, h_kv, d] and "
                         "page_table [n, width]")
    n, h_q, d = qs
    pages, page_size, h_kv, _ = cs
    if out is None:
        out = _empty(qs, dt, device, stream)
    if not (k_cache.dtype is dt and v_cache.dtype is dt and out.dtype is dt
            and page_table.dtype is torch.int32 and lens.dtype is torch.int32
            and cs == v_cache.shape and cs[3] == d and ts[0] == n and lens.shape == (n,)
            and out.shape == qs
            and k_cache.get_device() == v_cache.get_device() == page_table.get_device()
            == lens.get_device() == out.get_device() == index):
        _explain(device, ("k_cache", k_cache, dt, (pages, page_size, h_kv, d)),
                 ("v_cache", v_cache, dt, (pages, page_size, h_kv, d)),
                 ("page_table", page_table, torch.int32, (n, ts[1])),
                 ("lens", lens, torch.int32, (n,)), ("out", out, dt, (n, h_q, d)))
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("window must be at least 1")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if not lens.is_contiguous():
        raise ValueError("lens must be contiguous")
    q_stride, k_stride, v_stride = q.stride(), k_cache.stride(), v_cache.stride()
    t_stride = page_table.stride()
    for name, size, stride in (("q", qs, q_stride), ("k_cache", cs, k_stride),
                               ("v_cache", cs, v_stride), ("page_table", ts, t_stride)):
        if stride[-1] != 1:
            _dense(name, size, stride)
    lse = _empty((n, h_q), torch.float32, device, stream) if return_lse else None
    if workspace is None:
        with torch.cuda.device(device):
            size = decode_paged_attention_workspace_bytes(h_q, h_kv, d)
        workspace = _empty(size, torch.uint8, device, stream)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    args = PAGED_ATTENTION_ARGS.pack(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
        lens.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, n, h_q, h_kv, d, pages, page_size, ts[1],
        t_stride[0], window, *q_stride[:2], *k_stride[:3], *v_stride[:3], code,
        d ** -0.5 if scale is None else scale)
    _call(load().decode_paged_attention, args, index, stream)
    return (out, lse) if return_lse else out


def check_decode_status(stream=None) -> None:
    """Synchronise ``stream`` and raise GemmError if a kernel of this module refused an index
    since the last check."""
    if stream is None:
        stream = torch.cuda.current_stream()
    rc, bits = decode_check_status(
        int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))
    if rc != DECODE_OK:
        raise GemmError(rc, decode_last_error())
    if bits:
        raise GemmError(DECODE_ERR_INVALID_ARG,
                        "refused: " + "; ".join(w for b, w in DECODE_STATUS.items() if bits & b))
