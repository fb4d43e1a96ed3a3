"""Operands that share memory: the check of strided tensors against sets of bytes, and the refusals
of the C entry points, none of which reaches a device."""
from __future__ import annotations

import os
import subprocess

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
from blackwell_tensor_core_fp16_gb300 import _build
from test_decode_host import NORM, STEP, built_library, pack  # noqa: F401

BRUTE_FORCE = r"""
#include "overlap.h"
#include <cstdio>
#include <random>
#include <set>

int main()
{
    std::mt19937 gen(1);
    auto draw = [&](int lo, int hi) { return static_cast<int64_t>(lo + gen() % (hi - lo + 1)); };
    const char* const base = reinterpret_cast<const char*>(0x10000);
    int meet = 0, apart = 0, wrong = 0;
    for (int n = 0; n < 200000; ++n) {
        std::set<int64_t> bytes[2];
        int64_t at[2], row[2], size[2][3], stride[2][3];
        const int64_t common = draw(1, 24);
        for (int k = 0; k < 2; ++k) {
            at[k] = 2 * draw(0, 40), row[k] = draw(1, 4);
            for (int d = 0; d < 3; ++d) {
                size[k][d] = draw(0, 40) == 0 ? 0 : draw(1, 4);
                stride[k][d] = draw(0, 2) ? draw(0, 3) * common : draw(0, 24);
            }
            for (int64_t a = 0; a < size[k][0]; ++a)
                for (int64_t b = 0; b < size[k][1]; ++b)
                    for (int64_t c = 0; c < size[k][2]; ++c)
                        for (int64_t e = 0; e < 2 * row[k]; ++e)
                            bytes[k].insert(at[k] + e + 2 * (a * stride[k][0] + b * stride[k][1] +
                                                             c * stride[k][2]));
        }
        bool want = false;
        for (const int64_t x : bytes[0]) want = want || bytes[1].count(x);
        const decode::Operand a("a", base + at[0], 2, row[0], size[0], stride[0]);
        const decode::Operand b("b", base + at[1], 2, row[1], size[1], stride[1]);
        wrong += overlap(a, b) != want || overlap(b, a) != want || !same(a, a);
        (want ? meet : apart)++;
    }
    std::printf("%d %d %d\n", meet, apart, wrong);
    // what never ends by itself is cut off and counts as shared: far fewer steps than elements
    const int64_t many[2] = {1 << 20, 1 << 20}, in[2] = {1 << 21, 2}, out[2] = {(1 << 21) + 2, 6};
    overlap(decode::Operand("a", base, 1, 1, many, in), decode::Operand("b", base + 1, 1, 1, many, out));
    return 0;
}
"""


def test_overlap_of_strided_tensors(tmp_path):
    (tmp_path / "brute.cpp").write_text(BRUTE_FORCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", f"-I{_build.CSRC}", "-o",
                    str(tmp_path / "brute"), str(tmp_path / "brute.cpp")], check=True)
    run = subprocess.run([str(tmp_path / "brute")], capture_output=True, text=True, check=True,
                         timeout=60)
    meet, apart, wrong = map(int, run.stdout.split())
    assert wrong == 0 and meet > 50000 and apart > 50000


# The addresses below are made up: what is not refused would run on them.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses stay off a GPU")


# Addresses far apart for every pointer, so that only the ones a case moves share memory.
def apart(name, sizes, **values):
    from test_decode_host import fields
    pointers = [f for f, code, _ in fields(name) if code == "Q"]
    return pack(name, **{**sizes, **{f: (x + 1) << 32 for x, f in enumerate(pointers)}, **values})


STEP_STRIDES = dict(q_stride=(256, 256, 128), k_stride=(256, 256, 128), v_stride=(512, 512, 128),
                    alpha_stride=(4, 4), beta_stride=(4, 4), state_stride=4 * 128 * 128)


@no_gpu
@pytest.mark.parametrize("change,match", [
    (dict(o=1 << 32, q=1 << 32), "o shares memory with q"),
    (dict(o=(1 << 32) + 256, q=1 << 32), "o shares memory with q"),
    (dict(o=1 << 40, k=(1 << 40) + 768), "o shares memory with k"),
    (dict(o=1 << 40, v=(1 << 40) + 16), "o shares memory with v"),
    (dict(o=1 << 40, alpha=(1 << 40) + 512), "o shares memory with alpha"),
    (dict(o=1 << 40, beta=(1 << 40) + 512), "o shares memory with beta"),
    (dict(o=1 << 40, slots=(1 << 40) + 512), "o shares memory with slots"),
    (dict(state=1 << 40, q=(1 << 40) + 512), "state shares memory with q"),
    (dict(o=1 << 40, state=(1 << 40) - 4 * 4 * 128 * 128 + 64), "shares memory with"),
])
def test_step_refuses_shared_memory(change, match):
    args = apart("decode_gdn_step_args", {**STEP, **STEP_STRIDES}, **change)
    assert g.decode_gdn_step(args) == g.GDN_ERR_INVALID_ARG
    assert match in g.decode_last_error()


@no_gpu
@pytest.mark.parametrize("change,match", [
    (dict(q_out=1 << 40, k=1 << 40), "q_out shares memory with k"),
    (dict(q_out=1 << 40, q=(1 << 40) + 256), "q_out shares memory with q"),
    (dict(q_out=1 << 40, q=1 << 40, q_stride=(512, 256)), "q_out shares memory with q"),
    (dict(k_cache=1 << 40, v_cache=1 << 40), "shares memory with"),
    (dict(k_cache=1 << 40, k=(1 << 40) + 512), "k_cache shares memory with k"),
    (dict(v_cache=1 << 40, v=(1 << 40) + 512), "v_cache shares memory with v"),
    (dict(v_cache=1 << 40, slots=(1 << 40) + 512), "v_cache shares memory with slots"),
    (dict(k_cache=1 << 40, table=(1 << 40) + 512), "k_cache shares memory with table"),
    (dict(k_cache=1 << 40, positions=(1 << 40) + 512), "k_cache shares memory with positions"),
    (dict(q_out=1 << 40, q_weight=1 << 40), "q_out shares memory with q_weight"),
    (dict(q_out=1 << 40, k_weight=1 << 40), "q_out shares memory with k_weight"),
])
def test_norm_refuses_shared_memory(change, match):
    sizes = {**NORM, "tokens": 4, "q_stride": (256, 128), "k_stride": (128, 128), "v_stride": (128, 128),
             "q_out_stride": (256, 128), "k_cache_stride": (2048, 128, 128),
             "v_cache_stride": (2048, 128, 128)}
    args = apart("decode_qk_norm_rope_args", sizes, **change)
    assert g.decode_qk_norm_rope(args) == g.GDN_ERR_INVALID_ARG
    assert match in g.decode_last_error()
