"""The e4m3 format with a scale per row without a GPU: plans, and the refusals of
the C entry points (all before any CUDA call)."""
import ctypes

import pytest

from mla_attention_decode_gb300 import binding, build, cache

FAKE = 1 << 20  # never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED = 0, 1, 2
ROW = binding.MLA_KV_FP8_ROW


@pytest.fixture(scope="module")
def lib():
    build.build()
    return cache.load_library()


def desc(**kw):
    d = dict(kv=FAKE, kv_scale=FAKE, kv_dtype=ROW, page_size=64, num_pages=10, num_layers=1, scale_stride=4)
    d.update(kw)
    return cache.mla_cache(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(scale_stride=12, scale_width=4), OK), (dict(scale_stride=12), OK), (dict(num_pages=0, kv=0, kv_scale=0), OK),
    (dict(num_layers=2, kv_layer_bytes=640 * 576, scale_layer_bytes=640 * 4), OK),
    (dict(kv_scale=0), INVALID), (dict(kv_scale=FAKE + 4), INVALID), (dict(scale_stride=0), INVALID),
    (dict(scale_stride=2), INVALID), (dict(scale_stride=6), INVALID), (dict(scale_stride=-4), INVALID),
    (dict(scale_stride=12, scale_width=8), INVALID), (dict(scale_stride=12, scale_width=12), INVALID),
    (dict(scale_width=18), INVALID), (dict(scale_width=-4), INVALID),
    (dict(num_layers=2, kv_layer_bytes=640 * 576, scale_layer_bytes=640 * 4 - 4), INVALID),
    (dict(num_layers=2, kv_layer_bytes=640 * 576, scale_layer_bytes=640 * 4 + 2), INVALID),
    (dict(num_layers=2, kv_layer_bytes=640 * 288, scale_layer_bytes=640 * 4), INVALID),
    (dict(kv_dtype=3), UNSUPPORTED), (dict(kv_dtype=5), UNSUPPORTED)])
def test_cache_descriptions(lib, kw, status):
    d = desc(**kw)
    assert lib.mla_cache_copy_pages(ctypes.addressof(d), None, None, 0, None, None) == status
    assert (lib.mla_cache_workspace_bytes(ctypes.addressof(d), 1) > 0) == (status == OK)


@pytest.mark.parametrize("scale,stride", [(None, 4), (FAKE + 2, 4), (FAKE, 0), (FAKE, 2), (FAKE, 6), (FAKE, -4)])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_refusals(lib, scale, stride, paged):
    P = FAKE
    if paged:
        plan = binding.mla_decode_plan_paged([0, 2, 3], [7, 64], 64, 4, "fp8_row", num_sms=152)
        rc = lib.mla_decode_fwd_paged(P, P, scale, stride, P, P, P, P, P, None, 1 / 24, ctypes.byref(plan), P, 1 << 30, None)
    else:
        plan = binding.mla_decode_plan([0, 300, 700], "fp8_row", num_sms=152)
        rc = lib.mla_decode_fwd(P, P, scale, stride, P, P, P, None, 1 / 24, ctypes.byref(plan), P, 1 << 30, None)
    assert rc == INVALID


@pytest.mark.parametrize("lens", [[5], [0, 300, 8192, 1], [2000] * 64])
@pytest.mark.parametrize("q_len", [1, 2, 4])
def test_plans_are_those_of_one_scale_for_all(lens, q_len):
    """Tiles, ranges and fusion do not depend on where the scales are (the cost model's bytes a row
    differ by less than 1%, which these layouts do not notice)."""
    ind = [0]
    for n in lens:
        ind.append(ind[-1] + n)
    a, b = (binding.mla_decode_plan_multi(ind, q_len, dt, num_sms=152) if q_len > 1 else
            binding.mla_decode_plan(ind, dt, num_sms=152) for dt in ("fp8", "fp8_row"))
    a.kv_dtype = ROW
    assert a.as_dict() == b.as_dict() and list(a.first_row) == list(b.first_row)


def test_formats_that_do_not_exist_are_refused(lib):
    for code in (3, 5, -1):
        for plan in (lambda: binding.mla_decode_plan([0, 5], code, num_sms=152),
                     lambda: binding.mla_decode_plan_multi([0, 5], 2, code, num_sms=152),
                     lambda: binding.mla_decode_plan_paged([0, 1], [5], 8, 3, code, num_sms=152)):
            with pytest.raises(binding.MLAError) as e:
                plan()
            assert e.value.status == binding.MLA_ERR_UNSUPPORTED
    plan = binding.mla_decode_plan([0, 300], "fp8_row", num_sms=152)
    plan.mx_scores = 1  # of the 4-bit format only
    assert lib.mla_decode_fwd(FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE, None, 1 / 24, ctypes.byref(plan), FAKE, 1 << 30, None) == INVALID
