"""A wait of the 4-bit linear layer's kernels that runs out, without a GPU fault: with
decode_set_fault_injection(1) the codes of a block's second stage, or the operands of its second chunk, are never
announced.  With a limit of 200 ms the kernel stops issuing, waits for what is in flight and returns; the status word
says so, and the next call is right."""
from __future__ import annotations

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
from test_decode_fp8_gpu import check_linear, weights
from test_decode_gpu import cuda_library, generator, no_refusals_left, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def settings():
    yield
    g.decode_set_fault_injection(0)
    g.decode_set_wait_timeout_ms(2000)


@pytest.mark.parametrize("m,n,k,group", [
    (3, 9000, 4096, 128),          # few tokens, several stages of each of several items a block
    (2, 128, 65536, 64),           # the columns shared out in a cluster
    (20, 1000, 4096, 128),         # more tokens, in a cluster; sums of two chunks
    (40, 20000, 1024, 32),         # sums of one chunk, more blocks than the GPU holds
])
def test_wait_runs_out_and_the_next_call_is_right(m, n, k, group):
    gen = generator(m + n)
    x = (0.2 * normal(gen, m, k)).bfloat16().cuda()
    s = weights(gen, n, k, group, torch.bfloat16, True, False)
    want = check_linear(x, s, "before")
    for _ in range(2):
        assert g.decode_set_wait_timeout_ms(200) == 0
        assert g.decode_set_fault_injection(1) == 0
        g.linear_w4(x, **s)
        assert g.decode_set_fault_injection(0) == 0
        assert g.decode_set_wait_timeout_ms(2000) == 0
        with pytest.raises(g.GemmError, match="took too long"):
            g.check_decode_status()
        for _ in range(4):
            assert torch.equal(g.linear_w4(x, **s), want)
        g.check_decode_status()


def test_one_stage_or_chunk_has_no_second():
    """The hook touches nothing where a block has one stage, or one chunk."""
    gen = generator(1)
    assert g.decode_set_fault_injection(1) == 0
    for m in (2, 20):
        x = (0.2 * normal(gen, m, 128)).half().cuda()
        check_linear(x, weights(gen, 64, 128, 128, torch.float16, True, True), f"{m} tokens")
    g.check_decode_status()
