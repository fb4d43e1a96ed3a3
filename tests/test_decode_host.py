"""The decode-step operators' host side: the packed argument structs against the C header, and the
refusals of the C entry points, none of which reaches a device."""
from __future__ import annotations

import os
import re
import shutil
import struct
import subprocess

import pytest

import blackwell_tensor_core_fp16_gb300 as g
from blackwell_tensor_core_fp16_gb300 import _build, decode

HEADER = next(h for h in _build.HEADERS if h.endswith("decode.h"))
STRUCTS = {"decode_gdn_step_args": decode.GDN_STEP_ARGS,
           "decode_qk_norm_rope_args": decode.QK_NORM_ROPE_ARGS,
           "decode_paged_attention_args": decode.PAGED_ATTENTION_ARGS}


@pytest.fixture(scope="session", autouse=True)
def built_library():
    g.build()
    return g.load()


def fields(name):
    """(field, its struct code, its count) of a header struct, in order."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1)
    for line in filter(None, (x.strip() for x in body.split(";"))):
        base, names = re.match(r"((?:const )?\w+(?:\s*\*)?)\s*(.*)", line, re.S).groups()
        code = "Q" if "*" in base else {"int64_t": "q", "int32_t": "i", "float": "f"}[base]
        for item in names.split(","):
            m = re.match(r"\s*(\w+)(?:\[(\w+)\])?", item)
            count = {None: 1, "DECODE_MAX_AXES": 4}.get(m.group(2)) or int(m.group(2))
            yield m.group(1), code, count


@pytest.mark.parametrize("name", STRUCTS)
def test_packed_struct_matches_the_header(name, tmp_path):
    """The binding's format has the header's fields in their order, and the C compiler lays them
    out without padding."""
    codes = "".join(code * count for _, code, count in fields(name))
    fmt = STRUCTS[name].format.lstrip("=")
    assert "".join(c * int(k or 1) for k, c in re.findall(r"(\d*)([A-Za-z])", fmt)) == codes
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    src = tmp_path / "layout.c"
    lines = "".join(f'printf("%zu ", offsetof({name}, {f}));' for f, _, _ in fields(name))
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "{HEADER}"\n'
                   f'int main(void) {{ {lines} printf("%zu", sizeof({name})); return 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", f"-I{include}", "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want, at = [], 0
    for _, code, count in fields(name):
        want.append(at)
        at += struct.calcsize("=" + code) * count
    assert got == want + [at] and at == STRUCTS[name].size


def pack(name, **values):
    """A struct of plausible values (pointers 4096, dense strides left 0) with some replaced."""
    out = []
    for field, code, count in fields(name):
        x = values.get(field, 4096 if code == "Q" else 1.0 if code == "f" else 0)
        x = list(x) if isinstance(x, (list, tuple)) else [x] * count
        assert len(x) == count, field
        out += x
    return STRUCTS[name].pack(*out)


STEP = dict(n=1, tokens=1, h_q=2, h_k=2, h_v=4, head_dim=128, n_slots=1)
NORM = dict(tokens=1, h_q=2, h_k=1, head_dim=128, rot=64, axes=1, table_rows=8, pages=2,
            page_size=16, norm=1)
ATTN = dict(n=1, h_q=4, h_kv=2, head_dim=128, pages=2, page_size=16, table_width=1,
            workspace_bytes=1 << 30)
BAD, NOT = g.GDN_ERR_INVALID_ARG, g.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,code,match", [
    (dict(n=-1), BAD, "negative"), (dict(tokens=-1), BAD, "negative"), (dict(h_v=0), BAD, "heads"),
    (dict(dtype=2), BAD, "dtype"), (dict(h_v=3), BAD, "layout"), (dict(h_q=3), BAD, "layout"),
    (dict(head_dim=64), NOT, "head_dim"), (dict(h_q=36), NOT, "8 query heads"),
    (dict(q=0), BAD, "null"), (dict(state=0), BAD, "null"), (dict(slots=0, n=2), BAD, "states"),
    (dict(v=4104), NOT, "aligned"), (dict(tokens=2, k_stride=(0, 12, 0)), NOT, "multiples"),
    (dict(n_slots=2, state_stride=64), BAD, "state_stride"), (dict(n=1 << 40), NOT, "too many"),
])
def test_step_refusals(change, code, match):
    args = pack("decode_gdn_step_args", **{**STEP, **change})
    assert g.decode_gdn_step(args) == code
    assert re.search(match, g.decode_last_error())


@pytest.mark.parametrize("change,code,match", [
    (dict(tokens=-1), BAD, "negative"), (dict(h_q=0, h_k=0), BAD, "heads"),
    (dict(dtype=-1), BAD, "dtype"), (dict(norm=3), BAD, "norm"), (dict(head_dim=12), NOT, "head_dim"),
    (dict(head_dim=264), NOT, "head_dim"), (dict(rot=24), NOT, "rot"), (dict(rot=144), NOT, "rot"),
    (dict(axes=0), BAD, "axes"), (dict(axes=5), BAD, "axes"),
    (dict(axes=2, sections=(10, 10, 0, 0)), BAD, "sections"),
    (dict(axes=2, sections=(-1, 33, 0, 0)), BAD, "negative section"),
    (dict(v=0), BAD, "together"), (dict(slots=0), BAD, "together"), (dict(page_size=0), BAD, "pages"),
    (dict(pages=1 << 30), BAD, "pages"), (dict(q_out=0), BAD, "null"), (dict(positions=0), BAD, "null"),
    (dict(k=4100), NOT, "aligned"), (dict(tokens=2, q_stride=(4, 0)), NOT, "multiples"),
    (dict(v_cache_stride=(4, 0, 0)), NOT, "multiples"), (dict(tokens=1 << 31), NOT, "too many"),
])
def test_norm_refusals(change, code, match):
    args = pack("decode_qk_norm_rope_args", **{**NORM, **change})
    assert g.decode_qk_norm_rope(args) == code
    assert re.search(match, g.decode_last_error())


@pytest.mark.parametrize("change,code,match", [
    (dict(n=-1), BAD, "negative"), (dict(page_size=0), BAD, "page size"), (dict(dtype=7), BAD, "dtype"),
    (dict(h_q=3), BAD, "query heads"), (dict(h_kv=0), BAD, "key heads"), (dict(window=-1), BAD, "neg"),
    (dict(head_dim=96), NOT, "head_dim"), (dict(q=0), BAD, "null"), (dict(workspace=0), BAD, "null"),
    (dict(o=4104), NOT, "aligned"), (dict(q_stride=(0, 4)), NOT, "multiples"),
    (dict(k_stride=(8, 4, 8)), NOT, "multiples"), (dict(pages=1 << 31), NOT, "too large"),
])
def test_attention_refusals(change, code, match):
    args = pack("decode_paged_attention_args", **{**ATTN, **change})
    assert g.decode_paged_attention(args) == code
    assert re.search(match, g.decode_last_error())


def test_empty_problems_do_nothing():
    assert g.decode_gdn_step(pack("decode_gdn_step_args", **{**STEP, "n": 0})) == 0
    assert g.decode_gdn_step(pack("decode_gdn_step_args", **{**STEP, "tokens": 0})) == 0
    assert g.decode_qk_norm_rope(pack("decode_qk_norm_rope_args", **{**NORM, "tokens": 0})) == 0
    assert g.decode_paged_attention(pack("decode_paged_attention_args", **{**ATTN, "n": 0})) == 0
    assert g.decode_last_error() == ""


def test_unknown_names_of_the_package_still_raise():
    with pytest.raises(AttributeError):
        g.no_such_operator
    assert callable(g.gated_delta_step) and callable(g.paged_attention)
