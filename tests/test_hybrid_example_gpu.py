"""The hybrid example's model against its own definition in 64 bits."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
from test_decode_gpu import cuda_library, generator, no_refusals_left  # noqa: F401

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def definition(model, tokens, d, moved=()):
    """(logits [tokens, vocab], the attention layer's rotated keys [tokens, h_kv, d]) of one sequence in
    64 bits on the CPU.  ``moved``: tokens whose keys are rotated as if they stood one place further
    on (a mistake, for the test of the bound)."""
    w = {x: getattr(model, x).double().cpu() for x in
         ("embed", "head", "gdn_in", "gdn_gates", "gdn_out", "attn_in", "attn_out")}
    T, group = len(tokens), model.h_v // model.h_k
    x = w["embed"][tokens.cpu()]
    y = (x @ w["gdn_in"].T).view(T, -1, d)
    qk = y[:, :2 * model.h_k] / (y[:, :2 * model.h_k].pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    gates = x @ w["gdn_gates"].T
    alpha = torch.exp(-torch.nn.functional.softplus(gates[:, :model.h_v] - 2))
    beta = torch.sigmoid(gates[:, model.h_v:])
    o = torch.empty(T, model.h_v, d, dtype=torch.float64)
    for j in range(model.h_v):
        S = torch.zeros(d, d, dtype=torch.float64)
        q, k, v = qk[:, j // group], qk[:, model.h_k + j // group], y[:, 2 * model.h_k + j]
        for t in range(T):
            S = alpha[t, j] * S
            S = S + torch.outer(beta[t, j] * (v[t] - S @ k[t]), k[t])
            o[t, j] = d ** -0.5 * (S @ q[t])
    x = x + o.view(T, -1) @ w["gdn_out"].T

    y = (x @ w["attn_in"].T).view(T, -1, d)
    n = model.h_q + model.h_kv
    qk = y[:, :n] / (y[:, :n].pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    at = torch.arange(T, dtype=torch.float64)[:, None].expand(T, n).clone()
    at[list(moved), model.h_q:] += 1
    angle = at[..., None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    z = torch.complex(qk[..., :d // 2], qk[..., d // 2:]) * torch.polar(torch.ones_like(angle), angle)
    qk = torch.cat([z.real, z.imag], -1)
    keys = qk[:, model.h_q:]
    k = keys.repeat_interleave(model.h_q // model.h_kv, 1)
    v = y[:, n:].repeat_interleave(model.h_q // model.h_kv, 1)
    s = torch.einsum("qhd,khd->hqk", qk[:, :model.h_q], k) * d ** -0.5
    s = s.masked_fill(torch.ones(T, T).triu(1).bool(), float("-inf"))
    o = torch.einsum("hqk,khd->qhd", s.softmax(-1), v)
    x = x + o.reshape(T, -1) @ w["attn_out"].T
    return x @ w["head"].T, keys


def test_hybrid_example_against_its_definition():
    """Prompt and answers, eager: the logits, and the keys in the cache, which show the rotation more
    plainly.  Fourteen roundings to bfloat16 lie between a token and its logits (projections,
    norms, mixers, residuals, the head), nine between it and its key, each of 2^-9.3 of its values'
    size in the mean square and with a gain of about one: 2^-7.4 and 2^-7.7 of the results' size,
    and the bound is 2^-6 for both.  Keys rotated by one place too many are further off than that."""
    module = example()
    model = module.HybridModel(seed=5)
    gen = generator(72)
    seqs = [torch.randint(0, 1024, (length,), generator=gen).cuda() for length in (48, 20, 77)]
    cut = [40, 5, 60]
    slots = torch.tensor([2, 7, 4], dtype=torch.int32, device="cuda")
    want = [definition(model, seq, module.D) for seq in seqs]
    got = [[model.read(seq[:c], slot)] for seq, c, slot in zip(seqs, cut, slots.tolist())]
    lens = torch.tensor(cut, dtype=torch.int32, device="cuda")
    for t in range(8):
        logits = model.step(torch.stack([seq[c + t] for seq, c in zip(seqs, cut)]), slots, lens)
        for i in range(3):
            got[i].append(logits[i:i + 1])
        lens.add_(1)

    def off(x, ref):
        """The error of each token, of its size."""
        x, ref = x.double().cpu().flatten(1), ref.flatten(1)
        return (x - ref).pow(2).mean(-1).sqrt() / ref.pow(2).mean(-1).sqrt()

    for i, (c, slot) in enumerate(zip(cut, slots.tolist())):
        logits, keys = (x[:c + 8] for x in want[i])
        at = torch.arange(c + 8, device="cuda")
        place = model.places(torch.full_like(at, slot), at).long()
        cached = model.k_cache.flatten(0, 1)[place]
        assert float(off(torch.cat(got[i]), logits).max()) <= 2.0 ** -6, i
        assert float(off(cached, keys).max()) <= 2.0 ** -6, i
        moved = definition(model, seqs[i], module.D, moved=[3, c + 2])[1][:c + 8]
        assert (off(cached, moved) > 2.0 ** -6).nonzero().flatten().tolist() == [3, c + 2], i
