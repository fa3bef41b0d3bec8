"""Decoder objects without a GPU: copies of one that has been called, which plan and workspace a call goes
by, and calls without the compiled extension."""
import copy
import ctypes
import pickle

import pytest
import torch

from mla_attention_decode_gb300 import binding, build, cache


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


class Extension:
    """In place of the compiled one: its cores are those of the real one, its calls say which core they got."""

    def __init__(self):
        self.real, self.made, self.called = cache.extension(), [], []

    def decode_core(self, plan, workspace, nbytes, device):
        core = self.real.decode_core(plan, workspace, nbytes, 0)
        self.made.append((plan, workspace, nbytes, core))
        return core

    def decode(self, core, *args):
        self.called.append(core)
        return 0, "out", "lse"


class Workspace:
    """A workspace that says it is in device memory."""
    is_cuda, device = True, torch.device("cuda:0")

    def __init__(self, n):
        self.n = n

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.n

    def element_size(self):
        return 1


def decoder(monkeypatch, paged=False):
    ext = Extension()
    monkeypatch.setattr(cache, "extension", lambda: ext)
    dec = binding.PagedMLADecoder([0, 3], [5], 64, 4, "fp8", device="cpu", num_sms=152) if paged else \
        binding.MLADecoder([0, 300, 700], "fp8_row", device="cpu", num_sms=152)
    dec.workspace = Workspace(1 << 20)
    return ext, dec


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda d: pickle.loads(pickle.dumps(d))], ids=["copy", "deepcopy", "pickle"])
def test_a_decoder_that_was_called_can_be_copied(monkeypatch, paged, how):
    ext, dec = decoder(monkeypatch, paged)
    args = [None] * (6 if paged else 4)
    assert dec(*args) == ("out", "lse")
    other = how(dec)
    assert other.plan.as_dict() == dec.plan.as_dict() and other.kv_dtype == dec.kv_dtype
    other(*args), dec(*args)
    assert len(ext.made) == 2 and ext.called == [ext.made[0][3], ext.made[1][3], ext.made[0][3]]
    assert ext.made[1][0] == ctypes.addressof(other.plan)


def test_a_call_goes_by_the_plan_and_the_workspace_of_its_time(monkeypatch):
    """Also when another thread replaces the plan between the two lines of a call that look at it."""
    ext, dec = decoder(monkeypatch)
    args = [None] * 4
    dec(*args), dec(*args)
    assert len(ext.made) == 1
    first = dec.plan
    dec.plan = binding.mla_decode_plan([0, 10], "fp8_row", num_sms=152)
    dec(*args)
    dec.workspace = Workspace(1 << 21)
    dec(*args)
    assert [m[0] for m in ext.made] == [ctypes.addressof(p) for p in (first, dec.plan, dec.plan)] and ext.made[2][2] == 1 << 21

    class Decoder(type(dec)):
        """Its plan is replaced by `raced` right after it has been read for the third time."""
        raced = None

        @property
        def plan(self):
            plan = self.__dict__["plan"]
            if self.raced is not None:
                self.__dict__["plan"], self.raced = self.raced, None
            return plan

    racer = Decoder.__new__(Decoder)
    racer.__dict__.update({k: v for k, v in dec.__dict__.items() if k != "_made"})
    racer.raced = binding.mla_decode_plan([0, 20], "fp8_row", num_sms=152)
    held = racer.__dict__["plan"]
    racer(*args)
    racer(*args)  # the replaced plan's own core
    made = [m[0] for m in ext.made[3:]]
    assert made == [ctypes.addressof(held), ctypes.addressof(racer.plan)] and ext.called[-1] is ext.made[-1][3]


@pytest.mark.parametrize("error", [RuntimeError, ImportError])
@pytest.mark.parametrize("kv_dtype,scale,stride", [("bf16", None, 0), ("fp8", torch.ones(1), 0), ("fp8_row", torch.ones(300), 4),
                                                   ("fp8_row", torch.ones(300, 3)[:, 1], 12), ("mxfp4", torch.ones(300, 20), 20)])
@pytest.mark.parametrize("paged", [False, True])
def test_without_the_extension_a_decoder_calls_the_library(monkeypatch, error, kv_dtype, scale, stride, paged):
    def missing():
        raise error("not built")

    calls = []
    monkeypatch.setattr(cache, "extension", missing)
    for name in ("mla_decode_fwd", "mla_decode_fwd_paged"):
        monkeypatch.setattr(binding, name, lambda *a, _n=name, **kw: calls.append((_n, a, kw)))
    if paged:
        dec, table = binding.PagedMLADecoder([0, 3], [5], 64, 4, kv_dtype, device="cpu", num_sms=152), ("indptr", "indices", "last")
    else:
        dec, table = binding.MLADecoder([0, 256], kv_dtype, device="cpu", num_sms=152), ("indptr",)
    out, lse = dec("q", "kv", *table, "qo", kv_scale=scale, sm_scale=0.5, stream=7)
    assert out.shape == (1, 16, 512) and out.dtype == torch.bfloat16 and lse.shape == (1, 16) and lse.dtype == torch.float32
    name, a, kw = calls[0]
    assert name == ("mla_decode_fwd_paged" if paged else "mla_decode_fwd") and kw == dict(sm_scale=0.5, scale_stride=stride, stream=7)
    assert a[:2] == ("q", "kv") and a[2] is scale and a[3:] == (*table, "qo", out, lse, dec.plan, dec.workspace)
    mine = torch.zeros(1, 16, 512), torch.zeros(1, 16)
    assert dec("q", "kv", *table, "qo", kv_scale=scale, out=mine[0], lse=mine[1]) == mine
    if kv_dtype == "fp8_row":
        for bad in (torch.ones(255), torch.ones(300).double(), torch.ones(300, 1)):
            with pytest.raises(ValueError):
                dec("q", "kv", *table, "qo", kv_scale=bad)
