"""The cache operators without a GPU: the header's symbols, the struct layouts,
the rotation plan, the refusals of the C entry points (all before any CUDA
call) and of the Python layer."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

from mla_attention_decode_gb300 import binding, build, cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mla_cache.h")
OK, INVALID, UNSUPPORTED, TOO_SMALL = 0, 1, 2, 3
FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return cache.load_library()


def desc(**kw):
    d = dict(kv=FAKE, kv_scale=FAKE, kv_dtype=1, page_size=64, num_pages=10, num_layers=1)
    d.update(kw)
    return cache.mla_cache(**d)


def test_library_exports_every_declared_symbol(lib):
    names = sorted(set(re.findall(r"MLA_API\s+[\w\s\*]+?\b(mla_\w+)\s*\(", open(HEADER).read())))
    assert {"mla_rope_plan", "mla_cache_append", "mla_cache_gather", "mla_cache_slots", "mla_cache_copy_pages",
            "mla_cache_fork", "mla_cache_resize", "mla_cache_free", "mla_cache_compact",
            "mla_cache_workspace_bytes"} == set(names)
    for name in names:
        assert hasattr(lib, name), name
    assert binding.mla_status_string(cache.MLA_ERR_OUT_OF_PAGES) != "unknown status"


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = [cache.mla_cache, cache.mla_rope, cache.mla_norm, cache.mla_append_args, cache.mla_page_table]
    lines = ""
    for s in structs:
        n = s.__name__
        lines += f'  printf("{n} %zu\\n", sizeof({n}));\n'
        lines += "".join(f'  printf("{n}.{f} %zu\\n", offsetof({n}, {f}));\n' for f, _ in s._fields_)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mla_cache.h"\nint main(void) {\n' + lines +
                   "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines())
    for s in structs:
        assert int(got[s.__name__]) == ctypes.sizeof(s), s.__name__
        for f, _ in s._fields_:
            assert int(got[f"{s.__name__}.{f}"]) == getattr(s, f).offset, (s.__name__, f)


@pytest.mark.parametrize("freq", [1.0, 1e-4, 0.0, -0.3, 2 * math.pi, 100.0, 1e-12])
def test_rope_plan_counts_turns(lib, freq):
    """turn = freq / 2 pi mod 1 in units of 2^-64: off by the fp64 quotient's
    rounding (2^-53 of its magnitude) and half a unit."""
    r = cache.MLARope(inv_freq=[freq] * 32).rope
    turns = freq / (2 * math.pi)
    off = (r.turn[0] / 2.0 ** 64 - turns) % 1.0
    assert min(off, 1.0 - off) <= 2.0 ** -52 * max(1.0, abs(turns))


def test_rope_plan_axes(lib):
    r = cache.MLARope(sections=(8, 12, 12), interleaved=False, scale=1.5)
    assert r.num_axes == 3 and list(r.rope.axis) == [0] * 8 + [1] * 12 + [2] * 12
    assert r.rope.interleaved == 0 and r.rope.scale == 1.5
    assert cache.MLARope().num_axes == 1


def test_rope_plan_refusals(lib):
    with pytest.raises(ValueError):
        cache.MLARope(inv_freq=[1.0] * 31)
    with pytest.raises(ValueError):
        cache.MLARope(sections=(8, 8))
    with pytest.raises(ValueError):
        cache.MLARope(sections=(16, 16), axis_of_pair=[0] * 32)
    for bad in (dict(inv_freq=[math.nan] * 32), dict(inv_freq=[math.inf] * 32), dict(scale=math.inf),
                dict(axis_of_pair=[8] * 32), dict(axis_of_pair=[-1] + [0] * 31)):
        with pytest.raises(binding.MLAError) as e:
            cache.MLARope(**bad)
        assert e.value.status == INVALID
    assert lib.mla_rope_plan(None, None, 1, 0, 1.0, FAKE) == INVALID


@pytest.mark.parametrize("field,value,status", [
    ("kv_dtype", 3, UNSUPPORTED), ("kv_dtype", -1, UNSUPPORTED), ("page_size", 0, UNSUPPORTED),
    ("page_size", 48, UNSUPPORTED), ("num_pages", -1, INVALID), ("num_pages", 1 << 26, UNSUPPORTED),
    ("num_layers", 0, INVALID), ("kv", 0, INVALID), ("kv", FAKE + 8, INVALID), ("kv_scale", 0, INVALID),
    ("kv_scale", FAKE + 2, INVALID), ("reserved", 1, INVALID)])
def test_cache_refusals(lib, field, value, status):
    c = desc(**{field: value})
    assert lib.mla_cache_gather(ctypes.addressof(c), 0, FAKE, 1, FAKE, 576, None, None) == status
    assert lib.mla_cache_copy_pages(ctypes.addressof(c), FAKE, FAKE, 1, None, None) == status
    assert lib.mla_cache_workspace_bytes(ctypes.addressof(c), 1) == 0


@pytest.mark.parametrize("kw", [
    dict(kv_dtype=2, scale_stride=17), dict(kv_dtype=2, scale_stride=18, kv_scale=FAKE + 8),
    dict(num_layers=2, kv_layer_bytes=640 * 576 - 16), dict(num_layers=2, kv_layer_bytes=640 * 576 + 8),
    dict(num_layers=2, kv_layer_bytes=640 * 576, scale_layer_bytes=2),
    dict(kv_dtype=2, scale_stride=18, num_layers=2, kv_layer_bytes=640 * 288, scale_layer_bytes=640 * 18 - 16)])
def test_cache_layer_refusals(lib, kw):
    d = desc(**kw)
    assert lib.mla_cache_gather(ctypes.addressof(d), 0, FAKE, 1, FAKE, 576, None, None) == INVALID


def append_args(**kw):
    a = dict(kv_lat=FAKE, kv_pe=FAKE, slots=FAKE, positions=FAKE, q_lat=0, q_pe=FAKE, q_out=FAKE, kv_lat_stride=576,
             kv_pe_stride=576, position_stride=1, q_pe_token_stride=16 * 192, q_pe_head_stride=192, num_tokens=1)
    a.update(kw)
    return bytes(cache.mla_append_args(**a))


@pytest.mark.parametrize("kw", [
    dict(num_tokens=-1), dict(num_tokens=(1 << 27) + 1), dict(layer=1), dict(layer=-1), dict(kv_lat=FAKE + 8),
    dict(kv_pe=FAKE + 2), dict(kv_pe=0), dict(slots=0), dict(slots=FAKE + 2), dict(kv_lat_stride=580),
    dict(kv_pe_stride=577), dict(positions=0), dict(q_out=0), dict(q_out=FAKE + 8), dict(q_pe=FAKE + 2),
    dict(q_pe=0), dict(q_pe_head_stride=65), dict(q_lat=FAKE + 2, q_lat_token_stride=8192, q_lat_head_stride=512),
    dict(q_lat=FAKE, q_lat_token_stride=8192, q_lat_head_stride=513), dict(kv_lat=0)])
def test_append_refusals(lib, kw):
    c, rope = desc(), cache.MLARope()
    assert lib.mla_cache_append(ctypes.addressof(c), rope.address, None, append_args(**kw), None, None) == INVALID


def test_append_norm_and_error_word_refusals(lib):
    d = desc()
    c = ctypes.addressof(d)
    for kw in (dict(apply=16), dict(weight_fp32=2), dict(eps=-1.0), dict(eps=math.nan)):
        n = cache.mla_norm(**kw)
        assert lib.mla_cache_append(c, None, ctypes.addressof(n), append_args(), None, None) == INVALID, kw
    n = cache.mla_norm(apply=1)
    n.weight[0] = FAKE + 8
    assert lib.mla_cache_append(c, None, ctypes.addressof(n), append_args(), None, None) == INVALID
    assert lib.mla_cache_append(c, None, None, append_args(), FAKE + 2, None) == INVALID
    assert lib.mla_cache_append(c, None, None, None, None, None) == INVALID


def test_empty_calls_are_noops(lib):
    d = desc()
    c = ctypes.addressof(d)
    assert lib.mla_cache_append(c, None, None, append_args(num_tokens=0), None, None) == OK
    assert lib.mla_cache_gather(c, 0, None, 0, None, 576, None, None) == OK
    assert lib.mla_cache_copy_pages(c, None, None, 0, None, None) == OK
    assert lib.mla_cache_free(c, None, None, 0, None, None) == OK
    t = bytes(cache.mla_page_table(page_indptr=FAKE))
    assert lib.mla_cache_slots(c, t, None, 0, None, None, 0, None, None) == OK


def test_gather_slots_copy_free_refusals(lib):
    d = desc()
    c = ctypes.addressof(d)
    for args in ((1, FAKE, 1, FAKE, 576), (0, 0, 1, FAKE, 576), (0, FAKE, 1, FAKE + 8, 576), (0, FAKE, 1, FAKE, 575),
                 (0, FAKE, 1, FAKE, 568), (0, FAKE, -1, FAKE, 576)):
        assert lib.mla_cache_gather(c, *args, None, None) == INVALID, args
    t = bytes(cache.mla_page_table(page_indptr=FAKE, kv_indices=FAKE, last_page_len=FAKE, batch=2, num_indices=4))
    assert lib.mla_cache_slots(c, t, None, 5, FAKE, None, 0, None, None) == INVALID
    assert lib.mla_cache_slots(c, t, FAKE, 5, None, None, 0, None, None) == INVALID
    for bad in (dict(page_indptr=0), dict(kv_indices=0), dict(last_page_len=0), dict(batch=-1), dict(batch=65537),
                dict(page_indptr=FAKE + 2)):
        kw = dict(page_indptr=FAKE, kv_indices=FAKE, last_page_len=FAKE, batch=2, num_indices=4)
        kw.update(bad)
        assert lib.mla_cache_slots(c, bytes(cache.mla_page_table(**kw)), FAKE, 5, FAKE, None, 0, None, None) == INVALID
    assert lib.mla_cache_copy_pages(c, None, FAKE, 1, None, None) == INVALID
    assert lib.mla_cache_copy_pages(c, FAKE, FAKE, -1, None, None) == INVALID
    assert lib.mla_cache_free(c, FAKE + 4, FAKE, 1, None, None) == INVALID
    assert lib.mla_cache_free(c, FAKE, None, 1, None, None) == INVALID


def test_table_and_compact_refusals(lib):
    d = desc()
    c = ctypes.addressof(d)
    need = lib.mla_cache_workspace_bytes(c, 2)
    assert need > 0
    tab = lambda at, **kw: bytes(cache.mla_page_table(**{**dict(  # noqa: E731
        page_indptr=at, kv_indices=at + 256, last_page_len=at + 512, batch=2, num_indices=4), **kw}))
    a, b = tab(FAKE), tab(FAKE + 4096)
    for fn in (lib.mla_cache_fork, lib.mla_cache_resize):
        assert fn(c, FAKE, a, FAKE, b, FAKE, need - 1, None) == TOO_SMALL
        assert fn(c, FAKE, a, FAKE, a, FAKE, need, None) == INVALID            # in place
        assert fn(c, FAKE, a, None, b, FAKE, need, None) == INVALID
        assert fn(c, None, a, FAKE, b, FAKE, need, None) == INVALID
        assert fn(c, FAKE + 4, a, FAKE, b, FAKE, need, None) == INVALID
        assert fn(c, FAKE, a, FAKE, b, FAKE + 16, need, None) == INVALID
        assert fn(c, FAKE, None, FAKE, b, FAKE, need, None) == INVALID
    assert lib.mla_cache_resize(c, FAKE, a, FAKE, tab(FAKE + 4096, batch=1), FAKE, need, None) == INVALID
    assert lib.mla_cache_compact(c, FAKE, FAKE, FAKE, FAKE, 4, None, FAKE, 16, None) == TOO_SMALL
    assert lib.mla_cache_compact(c, None, FAKE, FAKE, FAKE, 4, None, FAKE, need, None) == INVALID
    assert lib.mla_cache_compact(c, FAKE, FAKE, None, FAKE, 4, None, FAKE, need, None) == INVALID
    assert lib.mla_cache_compact(c, FAKE, FAKE, FAKE, FAKE, -1, None, FAKE, need, None) == INVALID
    assert lib.mla_cache_workspace_bytes(c, -1) == 0


def test_python_layer_refuses_host_tensors(lib):
    with pytest.raises(ValueError):
        cache.MLACachePool(torch.zeros(64, 576, dtype=torch.bfloat16), "bf16", 64)
    with pytest.raises(ValueError):
        cache.MLANorm(kv_lat=torch.ones(512))
    assert cache.MLANorm(kv_lat=True, q_pe=True).norm.apply == 0b1001


@pytest.mark.parametrize("kw,status", [
    (dict(kv_dtype=2, scale_stride=34, scale_width=18), OK), (dict(kv_dtype=2, scale_stride=34, scale_width=34), OK),
    (dict(kv_dtype=2, scale_stride=34, scale_width=17), INVALID),
    (dict(kv_dtype=2, scale_stride=34, scale_width=35), INVALID),
    (dict(kv_dtype=2, scale_stride=34, scale_width=-1), INVALID), (dict(kv_dtype=1, scale_width=18), INVALID),
    (dict(kv_dtype=0, kv_scale=0, scale_width=18), INVALID), (dict(reserved2=1), INVALID)])
def test_scale_width_refusals(lib, kw, status):
    """Scale rows are 18 bytes or more of their stride; other formats have none."""
    d = desc(**kw)
    assert lib.mla_cache_copy_pages(ctypes.addressof(d), None, None, 0, None, None) == status
    assert (lib.mla_cache_workspace_bytes(ctypes.addressof(d), 1) > 0) == (status == OK)


def test_extension_tells_the_full_torch_version(lib):
    """Development builds of one release differ in what follows its three numbers."""
    assert cache._ext.torch_version == torch.__version__ and open(build.EXT_TORCH).read() == torch.__version__
    assert cache.EXT_TORCH_PATH == build.EXT_TORCH


def test_extension_for_another_torch_is_refused(lib, tmp_path, monkeypatch):
    """Before it is loaded where the build says so, by its own word otherwise."""
    release = torch.__version__.split("+")[0]
    monkeypatch.setattr(cache, "_lib", None)
    said = tmp_path / "built_for"
    said.write_text(release + ".dev20260101")
    monkeypatch.setattr(cache, "EXT_TORCH_PATH", str(said))
    monkeypatch.setattr(cache, "_load_extension", lambda: pytest.fail("loaded"))
    with pytest.raises(RuntimeError, match="build it again"):
        cache.load_library()
    monkeypatch.setattr(cache, "EXT_TORCH_PATH", str(tmp_path / "none"))
    other = type("Other", (), {"torch_version": release + "a0"})
    monkeypatch.setattr(cache, "_load_extension", lambda: other)
    with pytest.raises(RuntimeError, match="build it again"):
        cache.load_library()
    assert cache._lib is None


@pytest.mark.parametrize("freq", [1.0, 0.3, 1e-4, 3.7e-9, 1e-13, 100.0, 2 * math.pi * 0.75])
def test_rope_plan_of_negative_frequencies(lib, freq):
    """A pair that turns the other way turns by exactly the opposite angle, and a
    small frequency keeps its precision: the quotient's rounding (2^-52 of it) and
    half a unit."""
    there, back = cache.MLARope(inv_freq=[freq] * 32).rope, cache.MLARope(inv_freq=[-freq] * 32).rope
    assert (there.turn[3] + back.turn[3]) % 2 ** 64 == 0
    turns = (freq / (2 * math.pi)) % 1.0
    assert abs(there.turn[3] - turns * 2.0 ** 64) <= 2.0 ** 64 * 2.0 ** -52 * max(turns, freq / 6) + 1
