"""A decode step's operators on few bits, run together: projection, norm and rotation, cache write,
attention, projection, each held to its own definition on what the one before it gave, and the hybrid
example with them."""
from __future__ import annotations

import subprocess
import sys

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
import decode_fp8_ref as ref
from test_decode_gpu import cuda_library, generator, no_refusals_left, normal  # noqa: F401
from test_hybrid_example_gpu import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_steps_of_an_attention_layer(dtype):
    """Prompts of three sequences and four steps of each, one of them inactive in the last two."""
    gen = generator(51)
    hidden, h_q, h_kv, d, page, block = 256, 6, 2, 64, 16, 8
    W_in = (normal(gen, (h_q + 2 * h_kv) * d, hidden) * hidden ** -0.5).to(dtype).cuda()
    W_out = (normal(gen, hidden, h_q * d) * (h_q * d) ** -0.5).to(dtype).cuda()
    w_in, w_out = (g.quantize_weight_w4(W, 64, zeros) for W, zeros in ((W_in, True), (W_out, False)))
    rotary = g.rotary_table(256, d)
    table = torch.randperm(30, generator=gen).to(torch.int32).view(3, 10).cuda()
    kc, vc = (torch.zeros(30, page, h_kv, d, dtype=torch.uint8, device="cuda").view(ref.E4M3)
              for _ in range(2))
    ks, vs = (torch.zeros(30, page // block, h_kv, dtype=torch.uint8, device="cuda") for _ in range(2))
    ws = g.paged_attention_fp8_workspace(h_q, h_kv, d)
    window, sinks = 40, 4

    def layer(x, seq, pos, active):
        codes, scales, zeros = w_in
        y = g.linear_w4(x, codes, scales, 64, zeros=zeros)
        want, bound = ref.linear_w4(x, codes, scales, 64, zeros)
        ref.assert_close(y, want, bound, "projection")
        y = y.view(len(x), -1, d)
        q, k = g.qk_norm_rope(y[:, :h_q], y[:, h_q:h_q + h_kv], positions=pos, rotary=rotary)
        v = y[:, h_q + h_kv:]
        slots = (table[seq.long(), (pos // page).long()] * page + pos % page).to(torch.int32)
        slots = torch.where(active, slots, torch.full_like(slots, -1))
        before = [t.clone() for t in (kc, vc, ks, vs)]
        g.quantize_cache(k, v, kc, vc, ks, vs, slots)
        for t, c, s, old_c, old_s in ((k, kc, ks, before[0], before[2]), (v, vc, vs, before[1], before[3])):
            codes64, scale64 = ref.quantize_cache(t, old_c, old_s, slots)
            assert torch.equal(c.float().double().cpu(), codes64) and torch.equal(s.cpu(), scale64)
        lens = torch.where(active, pos + 1, torch.zeros_like(pos)).to(torch.int32)
        rows = table[seq.long()].contiguous()
        o, lse = g.paged_attention_fp8(q, kc, vc, ks, vs, rows, lens, window=window, sinks=sinks,
                                       return_lse=True, workspace=ws)
        want = ref.paged_attention(q, kc, vc, ks, vs, rows, lens, d ** -0.5, window, sinks)
        ref.assert_close(o, want[0], want[2], "attention")
        ref.assert_close(lse, want[1], want[3], "lse")
        codes, scales, zeros = w_out
        out = g.linear_w4(o.view(len(x), -1), codes, scales, 64, activation="gelu")
        want, bound = ref.linear_w4(o.view(len(x), -1), codes, scales, 64, activation="gelu")
        ref.assert_close(out, want, bound, "output")

    counts = [70, 1, 33]
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(counts)).cuda()
    pos = torch.cat([torch.arange(c) for c in counts]).to(torch.int32).cuda()
    layer(normal(gen, sum(counts), hidden).to(dtype).cuda(), seq, pos, torch.ones_like(seq, dtype=torch.bool))
    pos = torch.tensor(counts, dtype=torch.int32, device="cuda")
    for step in range(4):
        active = torch.tensor([True, step < 2, True], device="cuda")
        layer((normal(gen, 3, hidden) * 2 ** step).to(dtype).cuda(), torch.arange(3).cuda(), pos, active)
        pos = pos + active.to(torch.int32)
    k, v = g.dequantize_cache(kc, vc, ks, vs, torch.arange(30 * page, dtype=torch.int32, device="cuda"), dtype)
    for t, c, s in ((k, kc, ks), (v, vc, vs)):
        assert torch.equal(t.cpu(), ref.values(c, s).flatten(0, 1).to(dtype))


@pytest.mark.parametrize("cache,weights,window", [("e4m3", 16, None), ("16 bits", 4, None), ("e4m3", 4, 24)])
def test_hybrid_example_on_few_bits(cache, weights, window):
    """Prompts and a step that is recorded and replayed: the same tokens as the eager steps."""
    module = example()
    gen = generator(52)
    prompts = [torch.randint(0, 1024, (length,), generator=gen).cuda() for length in (40, 1, 70)]
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")

    def answers(recorded):
        model = module.HybridModel(seed=3, cache=cache, weights=weights, window=window,
                                   sinks=2 if window else 0)
        token = torch.stack([model.read(p, int(s))[-1].argmax() for p, s in zip(prompts, slots)])
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        out = [token.clone()]

        def one():
            logits = model.step(token, slots, lens)
            token.copy_(logits.argmax(-1))
            lens.add_(1)
            return logits

        assert bool(one().isfinite().all())
        out.append(token.clone())
        if recorded:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
        for _ in range(10):
            graph.replay() if recorded else one()
            out.append(token.clone())
        return torch.stack(out)

    assert torch.equal(answers(False), answers(True))


def test_hybrid_example_command():
    out = subprocess.run([sys.executable, example().__file__, "--cache", "e4m3", "--weights", "4"],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert "32 steps of 4 sequences" in out.stdout
