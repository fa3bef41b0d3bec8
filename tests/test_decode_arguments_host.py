"""What the Python decoders say of tensors that are not what they must be, without a GPU: every
check comes before any CUDA call (types, sizes and strides first, then where a tensor is)."""
import ctypes

import pytest
import torch

from mla_attention_decode_gb300 import binding, build, cache

FAKE = 1 << 20  # never dereferenced: the checks fail first


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def arguments(kv_dtype, paged, q_len=1):
    """A call's arguments as they must be, but in host memory, and its plan: three sequences of 300, 0 and 70 rows."""
    bf16, i32 = torch.bfloat16, torch.int32
    if paged:
        plan = binding.mla_decode_plan_paged([0, 5, 5, 7], [44, 0, 6], 64, 9, kv_dtype, num_sms=152)
        rows, table = 9 * 64, dict(indptr=torch.zeros(4, dtype=i32), indices=torch.zeros(7, dtype=i32), last=torch.zeros(3, dtype=i32))
    else:
        plan = binding.mla_decode_plan_multi([0, 300, 300, 370], q_len, kv_dtype, num_sms=152)
        rows, table = 370, dict(indptr=torch.zeros(4, dtype=i32), indices=None, last=None)
    kv = torch.zeros(rows, 288 if kv_dtype == "mxfp4" else 576, dtype=bf16 if kv_dtype == "bf16" else torch.uint8)
    scale = {"bf16": None, "fp8": torch.ones(1), "fp8_row": torch.ones(rows),
             "mxfp4": torch.zeros(rows, 18, dtype=torch.uint8)}[kv_dtype]
    n = 3 * q_len
    return plan, dict(q=torch.zeros(n, 16, 576, dtype=bf16), kv=kv, scale=scale, **table, qo=torch.zeros(4, dtype=i32),
                      out=torch.zeros(n, 16, 512, dtype=bf16), lse=torch.zeros(n, 16), sm_scale=1 / 24, stream=None)


def call(plan, args):
    ext = cache.extension()
    core = ext.decode_core(ctypes.addressof(plan), FAKE, 1 << 30, 0)
    return ext.decode(core, *args.values())


def refused(plan, args, match):
    with pytest.raises(ValueError, match=match):
        call(plan, args)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "fp8_row", "mxfp4"])
@pytest.mark.parametrize("paged", [False, True])
def test_types_sizes_and_strides(kv_dtype, paged):
    plan, ok = arguments(kv_dtype, paged)
    refused(plan, ok, "^q is on cuda:0")  # as they must be but for where they are
    indptr = "kv_page_indptr" if paged else "kv_indptr"
    cases = [("q", ok["q"].half(), "q is bf16"), ("q", ok["q"].transpose(0, 1), "q is contiguous"), ("q", 5, "q is a tensor"),
             ("kv", ok["kv"].float(), "kv is "), ("kv", ok["kv"][:-1], "kv has "), ("kv", ok["kv"].t(), "kv is contiguous"),
             ("indptr", ok["indptr"].long(), indptr + " is int32"), ("indptr", ok["indptr"][:3], indptr + " has 3 "),
             ("indptr", torch.zeros(8, dtype=torch.int32)[::2], indptr + " is contiguous"),
             ("qo", ok["qo"].long(), "qo_indptr is int32"), ("qo", ok["qo"][:2], "qo_indptr has 2 "),
             ("out", ok["out"].float(), "out is bf16"), ("out", ok["out"][:2], "out has "),
             ("out", torch.zeros(3, 16, 576, dtype=torch.bfloat16)[..., :512], "out is contiguous"),
             ("lse", ok["lse"].double(), "lse is fp32"), ("lse", ok["lse"][:2], "lse has "),
             ("lse", torch.zeros(16, 3).t(), "lse is contiguous")]
    if paged:
        cases += [("indices", ok["indices"].long(), "kv_indices is int32"), ("indices", ok["indices"][:6], "kv_indices has 6 "),
                  ("last", ok["last"].short(), "kv_last_page_len is int32"), ("last", ok["last"][:2], "kv_last_page_len has 2 ")]
    if kv_dtype == "fp8":
        cases += [("scale", torch.ones(1).double(), "kv_scale is fp32"), ("scale", torch.ones(0), "kv_scale is fp32")]
    if kv_dtype == "mxfp4":
        cases += [("scale", ok["scale"].short(), "kv_scale is e8m0"), ("scale", ok["scale"][:-1], "kv_scale is e8m0"),
                  ("scale", ok["scale"][:, :17], "kv_scale is e8m0"), ("scale", ok["scale"].flatten(), "kv_scale is e8m0"),
                  ("scale", torch.zeros(18, ok["scale"].shape[0], dtype=torch.uint8).t(), "kv_scale is e8m0")]
    if kv_dtype == "fp8_row":
        cases += [("scale", ok["scale"].half(), "kv_scale is fp32"), ("scale", ok["scale"][:-1], "kv_scale is fp32")]
    # what is checked later is left out (None: null) or empty, so that the case is reached
    order = list(ok)
    for name, bad, match in cases:
        args = {k: None if k not in ("sm_scale", "stream") and order.index(k) < order.index(name) else v for k, v in ok.items()}
        refused(plan, {**args, name: bad}, match)


@pytest.mark.parametrize("name,match", [("q", "^q is on cuda:0, the call's device$"), ("kv", "^kv is on cuda:0, the call's device$"),
                                        ("scale", "^kv_scale is on cuda:0, the call's device$"),
                                        ("indptr", "kv_page_indptr is on cuda:0, the call's device, or in pinned host memory"),
                                        ("indices", "kv_indices is on"), ("last", "kv_last_page_len is on"), ("qo", "qo_indptr is on"),
                                        ("out", "out is on"), ("lse", "lse is on")])
def test_host_memory_that_is_not_pinned(name, match):
    plan, ok = arguments("bf16" if name == "q" else "fp8_row", True)
    refused(plan, {k: v if k in (name, "sm_scale", "stream") else None for k, v in ok.items()}, match)


@pytest.mark.parametrize("q_len", [2, 5])
def test_sizes_with_several_tokens(q_len):
    """Indices a sequence, output rows a token."""
    plan, ok = arguments("fp8_row", False, q_len)
    for name, bad, match in (("indptr", ok["indptr"][:3], "kv_indptr has 3 "), ("qo", ok["qo"][:2], "qo_indptr has 2 "),
                             ("out", ok["out"][1:], "out has "), ("lse", ok["lse"][1:], "lse has ")):
        refused(plan, {k: bad if k == name else (v if k in ("sm_scale", "stream") else None) for k, v in ok.items()}, match)
    none = {k: v if k in ("sm_scale", "stream") else None for k, v in ok.items()}
    refused(plan, {**none, "qo": ok["qo"][:3]}, "qo_indptr is on")  # (only its first three are read)
