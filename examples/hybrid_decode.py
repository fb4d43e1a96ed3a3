"""A small hybrid model, one gated-delta-net layer and one attention layer, reading prompts and
answering token by token with this library's operators:

    python examples/hybrid_decode.py

Both layers go linear -> qk_norm_rope -> mixer -> linear.  The delta-rule layer's queries and keys get
unit length; its mixer is ``gated_delta_rule`` for a prompt, whose final state goes to the sequence's
slot of a pool, and ``gated_delta_step`` for new tokens.  The attention layer's get an RMS norm and
the rotation, keys and values go to the paged cache in the same pass, and its mixer is
``paged_attention``, for a prompt with one row per token (all rows share the sequence's pages and
each sees the tokens up to its own).  A decode step of the whole batch is recorded into one CUDA
graph: lengths, positions and cache places live in device memory.

Weights are random: the example shows the calls, not a language.
"""
from __future__ import annotations

import os
import sys
import time

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blackwell_tensor_core_fp16_gb300 as g  # noqa: E402

D = 128              # head dimension of both layers


class HybridModel:
    """Weights, and the states and caches of up to ``slots`` sequences."""

    def __init__(self, hidden=512, vocab=1024, gdn_heads=(2, 4), attn_heads=(4, 2), slots=8,
                 pages=64, page_size=16, max_len=512, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).to(dtype)

        self.h_k, self.h_v = gdn_heads             # delta rule: query and key heads, value heads
        self.h_q, self.h_kv = attn_heads
        self.embed, self.head = weight(vocab, hidden), weight(vocab, hidden)
        self.gdn_in = weight((2 * self.h_k + self.h_v) * D, hidden)
        self.gdn_gates = weight(2 * self.h_v, hidden)
        self.gdn_out = weight(hidden, self.h_v * D)
        self.attn_in = weight((self.h_q + 2 * self.h_kv) * D, hidden)
        self.attn_out = weight(hidden, self.h_q * D)
        self.q_weight, self.k_weight = (torch.ones(D, dtype=dtype, device="cuda") for _ in range(2))
        self.rotary = g.rotary_table(max_len, D)
        self.state = torch.zeros(slots, self.h_v, D, D, device="cuda")
        self.k_cache, self.v_cache = (torch.zeros(pages, page_size, self.h_kv, D, dtype=dtype,
                                                  device="cuda") for _ in range(2))
        # every slot has pages of its own here; a server would hand them out as lengths grow
        per_slot = pages // slots
        self.page_table = torch.arange(slots * per_slot, dtype=torch.int32,
                                       device="cuda").view(slots, per_slot)
        self.workspace = g.paged_attention_workspace(self.h_q, self.h_kv, D)

    def places(self, slot, positions):
        """Where tokens at ``positions`` of the sequences in ``slot`` lie in the cache."""
        size = self.k_cache.shape[1]
        page = self.page_table[slot.long(), (positions // size).long()]
        return (page * size + positions % size).to(torch.int32)

    def _gdn_inputs(self, x):
        """q, k (unit length), v, alpha, beta of x [tokens, hidden]."""
        y = g.linear(x, self.gdn_in).view(len(x), -1, D)
        q, k = g.qk_norm_rope(y[:, :self.h_k], y[:, self.h_k:2 * self.h_k], norm="l2")
        gates = g.linear(x, self.gdn_gates).float()
        alpha = torch.exp(-F.softplus(gates[:, :self.h_v] - 2))
        beta = torch.sigmoid(gates[:, self.h_v:])
        return q, k, y[:, 2 * self.h_k:], alpha, beta

    def _attention(self, x, positions, places, table, lens):
        y = g.linear(x, self.attn_in).view(len(x), -1, D)
        q, _ = g.qk_norm_rope(y[:, :self.h_q], y[:, self.h_q:self.h_q + self.h_kv], self.q_weight,
                              self.k_weight, positions=positions, rotary=self.rotary,
                              v=y[:, self.h_q + self.h_kv:], k_cache=self.k_cache,
                              v_cache=self.v_cache, slots=places)
        o = g.paged_attention(q, self.k_cache, self.v_cache, table, lens, workspace=self.workspace)
        return x + g.linear(o.view(len(x), -1), self.attn_out)

    def read(self, tokens, slot):
        """Logits [tokens, vocab] of one prompt (int64 [tokens]), whose state and keys go to ``slot``."""
        T = len(tokens)
        x = self.embed[tokens]
        q, k, v, alpha, beta = self._gdn_inputs(x)
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        o, final = g.gated_delta_rule(q, k, v.contiguous(), alpha, beta, cu, D ** -0.5,
                                      output_final_state=True)
        self.state[slot] = final[0]
        x = x + g.linear(o.view(T, -1), self.gdn_out)
        at = torch.arange(T, dtype=torch.int32, device="cuda")
        slots = torch.full_like(at, slot)
        x = self._attention(x, at, self.places(slots, at), self.page_table[slot].expand(T, -1), at + 1)
        return g.linear(x, self.head)

    def step(self, tokens, slots, lens):
        """Logits [n, vocab] of one new token of each sequence (int64 [n]); ``lens`` int32 [n] counts
        the tokens before it.  Only tensors' contents change between calls, so a call can be
        recorded."""
        x = self.embed[tokens]
        q, k, v, alpha, beta = self._gdn_inputs(x)
        o = g.gated_delta_step(q[:, None], k[:, None], v[:, None], alpha[:, None], beta[:, None],
                               self.state, D ** -0.5, slots)
        x = x + g.linear(o.view(len(x), -1), self.gdn_out)
        x = self._attention(x, lens, self.places(slots, lens), self.page_table[slots.long()], lens + 1)
        return g.linear(x, self.head)


def main():
    model = HybridModel()
    n, steps = 4, 32
    slots = torch.tensor([5, 0, 3, 6], dtype=torch.int32, device="cuda")
    prompts = [torch.randint(0, 1024, (length,), device="cuda") for length in (17, 64, 1, 33)]
    token = torch.stack([model.read(p, int(s))[-1].argmax() for p, s in zip(prompts, slots.tolist())])
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    answers = [token.clone()]

    # one eager step settles the kernels' attributes; then the step is recorded once and replayed
    def one():
        token.copy_(model.step(token, slots, lens).argmax(-1))
        lens.add_(1)

    one()
    answers.append(token.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(steps):
        graph.replay()
        answers.append(token.clone())
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    g.check_decode_status()
    for i, answer in enumerate(torch.stack(answers, 1).tolist()):
        print(f"sequence {i}: {answer}")
    print(f"{steps} steps of {n} sequences: {took / steps * 1e6:.0f} us a step")


if __name__ == "__main__":
    main()
