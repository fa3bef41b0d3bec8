"""The Python decoders with pinned host buffers, with tensors that are not what they must be, and without the
compiled extension."""
import pytest
import torch

from mla_attention_decode_gb300 import binding, build, cache, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def arguments(dtype):
    lens = [1000, 0, 64, 3000, 1]
    inp = synth.make_inputs(lens, "fp8" if dtype == "fp8_row" else dtype, seed=17)
    scale = {"bf16": None, "fp8": inp.kv_scale, "mxfp4": inp.block_scales,
             "fp8_row": torch.rand(inp.kv.shape[0], generator=torch.Generator("cpu").manual_seed(1)) * 0.02}[dtype]
    return binding.MLADecoder(inp.kv_indptr, dtype, device=DEV), inp, inp.kv.to(DEV), None if scale is None else scale.to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp8_row", "mxfp4"])
def test_pinned_host_buffers(dtype):
    dec, inp, kv, scale = arguments(dtype)
    want = dec(inp.q.to(DEV), kv, inp.kv_indptr.to(DEV), inp.qo_indptr.to(DEV), kv_scale=scale)
    q = inp.q.to(DEV) if dtype == "bf16" else inp.q.pin_memory()
    got = [torch.zeros_like(t, device="cpu").pin_memory() for t in want]
    dec(q, kv, inp.kv_indptr.pin_memory(), inp.qo_indptr.pin_memory(), kv_scale=scale, out=got[0], lse=got[1])
    torch.cuda.synchronize()
    assert dec.poll_error() == 0 and all(torch.equal(a, b.cpu()) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp8_row", "mxfp4"])
def test_without_the_extension(dtype, monkeypatch):
    dec, inp, kv, scale = arguments(dtype)
    args = (inp.q.to(DEV), kv, inp.kv_indptr.to(DEV), inp.qo_indptr.to(DEV))
    want = dec(*args, kv_scale=scale)

    def missing():
        raise RuntimeError("not built")

    monkeypatch.setattr(cache, "extension", missing)
    dec._made = None
    got = dec(*args, kv_scale=scale)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and dec.poll_error() == 0


def test_refusals():
    dec, inp, kv, scale = arguments("fp8_row")
    ok = dict(q=inp.q.to(DEV), kv=kv, kv_indptr=inp.kv_indptr.to(DEV), qo_indptr=inp.qo_indptr.to(DEV), kv_scale=scale,
              out=torch.zeros(5, 16, 512, dtype=torch.bfloat16, device=DEV), lse=torch.zeros(5, 16, device=DEV))
    dec(**ok)
    for name, bad in (("q", ok["q"].half()), ("q", inp.q), ("kv", kv[:-1]), ("kv", kv.cpu()), ("kv_indptr", ok["kv_indptr"].long()),
                      ("kv_indptr", inp.kv_indptr), ("qo_indptr", ok["qo_indptr"][:4]), ("kv_scale", scale.cpu()),
                      ("kv_scale", scale.cpu().pin_memory()), ("kv", kv.cpu().pin_memory()), ("out", ok["out"][:4]),
                      ("out", ok["out"].float()), ("out", torch.zeros(5, 16, 520, dtype=torch.bfloat16, device=DEV)[..., :512]),
                      ("lse", ok["lse"][:4]), ("lse", torch.zeros(16, 5, device=DEV).t())):
        with pytest.raises(ValueError):
            dec(**{**ok, name: bad})
    assert dec.poll_error() == 0
