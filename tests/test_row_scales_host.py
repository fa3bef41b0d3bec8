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
@pytest.mark.parametrize("q_len", [1, 2])
def test_plans_are_those_of_one_scale_for_all(lens, q_len):
    """Tiles, ranges and fusion do not depend on where the scales are (the cost model's bytes a row
    differ by less than 1%, which these layouts do not notice)."""
    ind = [0]
    for n in lens:
        ind.append(ind[-1] + n)
    a, b = (binding.mla_decode_plan_multi(ind, q_len, dt, num_sms=152) if q_len > 1 else
            binding.mla_decode_plan(ind, dt, num_sms=152) for dt in ("fp8", "fp8_row"))
    a.kv_dtype = ROW
    assert a.as_dict() == b.as_dict()
    assert q_len == 2 or list(a.first_row) == list(b.first_row)


@pytest.mark.parametrize("q_len", [2, 3, 4, 5, 15, 16])
@pytest.mark.parametrize("splits", [0, 1, 17])
def test_pairs_of_tokens_plan_as_entries(q_len, splits):
    """The unit list is that of the rows which each pair's later token sees; two slots a unit."""
    lens = [0, 1, 2, 5, 129, 300, 4000, 9000]
    ind = [0]
    for n in lens:
        ind.append(ind[-1] + n)
    plan = binding.mla_decode_plan_multi(ind, q_len, "fp8_row", num_sms=7, num_splits=splits)
    assert (plan.tokens_fused, plan.q_len, plan.batch) == (2, q_len, len(lens) * q_len)
    pairs = (q_len + 1) // 2
    rows = [0]
    for n in lens:
        for i in range(pairs):  # the later token is q_len - 1 - 2 (pairs - 1 - i)
            rows.append(rows[-1] + max(0, n - 2 * (pairs - 1 - i)))
    ref = binding.mla_decode_plan(rows, "fp8", num_sms=7, num_splits=splits)  # (a unit boundary of the same weight)
    assert plan.schedule == ref.schedule and plan.total_tiles == ref.total_tiles
    assert [c for c in range(256) if plan.first_row[c] >= 0] == [c for c in range(256) if ref.first_row[c] >= 0] or ref.late_tiles
    if plan.late_tiles == ref.late_tiles == 0:
        assert plan.num_work == 2 * ref.num_work and plan.splits_max == ref.splits_max
        # the same tiles, of entries that begin where their sequence does
        starts = [(rows[e], ind[e // pairs]) for e in range(len(rows) - 1) if rows[e + 1] > rows[e]]
        for got, want in zip(plan.first_row, ref.first_row):
            if want >= 0:
                own, begin = max(x for x in starts if x[0] <= want)
                assert got == want - own + begin


def test_fused_plans_are_checked(lib):
    """What the planner does not make is refused: an odd number of slots, a fused plan of another format."""
    def fwd(plan):
        return lib.mla_decode_fwd(FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE, None, 1 / 24, ctypes.byref(plan), FAKE + 8, 1 << 30, None)
    for field, value in (("num_work", 3), ("q_len", 1), ("q_len", 17), ("tokens_fused", 3), ("kv_dtype", 1), ("kv_dtype", 2), ("batch", 7)):
        plan = binding.mla_decode_plan_multi([0, 300, 700], 4, "fp8_row", num_sms=152)
        setattr(plan, field, value)
        assert fwd(plan) == INVALID, field


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


@pytest.mark.parametrize("lens", [[8192] * 64, [5000 - 37 * i for i in range(100)], [2000] * 40])
def test_ranges_of_tiles_weigh_a_unit_boundary_as_one_tile(lens):
    """One token a sequence: balanced ranges with one empty position between sequences, the
    late blocks one fewer; every tile is some block's."""
    ind = [0]
    for n in lens:
        ind.append(ind[-1] + n)
    plan = binding.mla_decode_plan(ind, "fp8_row", num_sms=152)
    assert (plan.schedule, plan.unit_cost, plan.late_tiles) == (1, 1, 1)
    assert plan.total_tiles == sum(-(-n // 128) for n in lens) and plan.grid == 152
    assert plan.num_work >= len(lens) and min(plan.first_row[:152]) >= 0
    pairs = binding.mla_decode_plan_multi(ind, 2, "fp8_row", num_sms=152)
    assert pairs.schedule == 0 or (pairs.unit_cost, pairs.late_tiles) == (2, 1)


@pytest.mark.parametrize("page", [4, 8, 16, 64, 128])
def test_paged_plans_say_where_blocks_begin(page):
    """From pages of 8 rows on, the first row of each block's first tile, counted over the pages."""
    lens = [5000 - 37 * i for i in range(100)] + [0, 1]
    counts, at, ind = [-(-n // page) for n in lens], [0], [0]
    for n, c in zip(lens, counts):
        at.append(at[-1] + c)
        ind.append(ind[-1] + n)
    last = [n - (c - 1) * page if c else 0 for n, c in zip(lens, counts)]
    plan = binding.mla_decode_plan_paged(at, last, page, at[-1], "fp8_row", num_sms=152)
    if page < 8:
        assert set(plan.first_row) == {-1}
        return
    flat = binding.mla_decode_plan(ind, "fp8_row", num_sms=152)
    for got, want in zip(plan.first_row, flat.first_row):
        if want < 0:
            assert got == -1
            continue
        b = max(i for i in range(len(lens)) if ind[i] <= want and lens[i])
        assert got == at[b] * page + want - ind[b]
