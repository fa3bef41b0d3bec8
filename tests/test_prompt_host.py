"""The prompt attention without a GPU: the header's symbols, the struct's layout and
the refusals of the C entry points (all before any CUDA call)."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

from mla_attention_decode_gb300 import build, prompt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mla_prompt.h")
OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3
FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return prompt.load_library()


def args(**kw):
    d = dict(q_nope=FAKE, q_pe=FAKE, k_nope=FAKE, k_pe=FAKE, v=FAKE, qo_indptr=FAKE, kv_indptr=FAKE, prefix=None, out=FAKE, lse=FAKE,
             q_nope_token_stride=2048, q_nope_head_stride=128, q_pe_token_stride=1024, q_pe_head_stride=64,
             k_nope_token_stride=4096, k_nope_head_stride=256, k_pe_token_stride=576, v_token_stride=4096, v_head_stride=256,
             out_token_stride=2048, out_head_stride=128, num_q=10, num_kv=20, batch=2, heads=16, causal=1, sm_scale=0.07)
    d.update(kw)
    return prompt.mla_prompt_args(**d)


def test_library_exports_every_declared_symbol(lib):
    names = set(re.findall(r"MLA_API\s+[\w\s\*]+?\b(mla_\w+)\s*\(", open(HEADER).read()))
    assert names == {"mla_prompt_fwd", "mla_prompt_workspace_bytes"}
    for name in names:
        assert hasattr(lib, name), name


def test_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    s = prompt.mla_prompt_args
    lines = f'  printf("all %zu\\n", sizeof({s.__name__}));\n'
    lines += "".join(f'  printf("{f} %zu\\n", offsetof({s.__name__}, {f}));\n' for f, _ in s._fields_)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mla_prompt.h"\nint main(void) {\n' + lines + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    assert int(got["all"]) == ctypes.sizeof(s)
    for f, _ in s._fields_:
        assert int(got[f]) == getattr(s, f).offset, f


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), OK), (dict(num_q=0), OK), (dict(batch=0, q_nope=None, out=None), OK),
    (dict(num_q=-1), INVALID), (dict(num_kv=-1), INVALID), (dict(num_q=1 << 30), INVALID), (dict(batch=-1), INVALID),
    (dict(batch=65537), INVALID), (dict(heads=0), UNSUPPORTED), (dict(heads=129), UNSUPPORTED), (dict(causal=2), INVALID),
    (dict(sm_scale=0.0), INVALID), (dict(sm_scale=-1.0), INVALID), (dict(sm_scale=math.inf), INVALID),
    (dict(sm_scale=math.nan), INVALID), (dict(qo_indptr=None), INVALID), (dict(kv_indptr=FAKE + 2), INVALID),
    (dict(prefix=FAKE + 1), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 8), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(out_token_stride=12), INVALID), (dict(out_head_stride=0), INVALID), (dict(q_nope=FAKE + 8), INVALID),
    (dict(q_nope=None), INVALID), (dict(q_nope_token_stride=-2048), INVALID), (dict(q_nope_head_stride=4), INVALID),
    (dict(q_nope_token_stride=1 << 39), INVALID)])
def test_refusals(lib, kw, status):
    a = args(**kw)
    assert lib.mla_prompt_fwd(ctypes.addressof(a), FAKE, 1 << 30, None) == status


def test_refusals_of_the_workspace(lib):
    a = args()
    n = lib.mla_prompt_workspace_bytes(ctypes.addressof(a))
    assert n >= 256
    assert lib.mla_prompt_fwd(ctypes.addressof(a), None, n, None) == INVALID
    assert lib.mla_prompt_fwd(ctypes.addressof(a), FAKE + 128, n, None) == INVALID
    assert lib.mla_prompt_fwd(ctypes.addressof(a), FAKE, n - 1, None) == TOO_SMALL
    assert lib.mla_prompt_fwd(None, FAKE, n, None) == INVALID
    assert lib.mla_prompt_workspace_bytes(None) == 0
    bad = args(heads=0)
    assert lib.mla_prompt_workspace_bytes(ctypes.addressof(bad)) == 0
