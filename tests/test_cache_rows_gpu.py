"""Rows of the latent cache on the GPU: append, gather and slots against fp64.

Tolerances.  The kernels compute in fp32 and round once.  Relative error of a
normed value before that rounding: sum of 512 squares as 16 products a lane and
5 shuffles, at most 21 roundings of 2^-24 and half of it after the square root;
the reciprocal root 2 ulp (2^-22); three products: below 2^-19.9 in all, taken
as 2^-19.  A rotated pair adds the angle's error (2 pi 2^-33, 2^-24 pi from its
conversion to fp32, 2 ulp of the functions) and two roundings, relative to
|a| + |b|: within the same 2^-19 (|a| + |b|).  Then one rounding: half a step,
2^-8 relative (bf16), 2^-4 relative or 2^-10 absolute (e4m3 normal, subnormal),
half the distance of neighbours (e2m1: 1/4 below 2, 1/2 below 4, 1 up to 6)."""
import numpy as np
import pytest
import torch

from mla_attention_decode_gb300 import binding, build, cache, synth
from cache_reference import WIDTH, dequant, rms, rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
NOISE = 2.0 ** -19
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def new_pool(kv_dtype, rows, page_size=1, layers=1, stride=18, fill=None, scale=0.011):
    """A pool over storage filled with `fill` (or random bytes without NaN codes)."""
    g = gen(rows + 7 * layers)
    if kv_dtype == "bf16":
        kv = torch.randn(layers, rows, 576, generator=g).to(torch.bfloat16)
    else:
        kv = torch.randint(0, 120, (layers, rows, WIDTH[kv_dtype]), generator=g, dtype=torch.uint8)
    sc = None
    if kv_dtype == "fp8":
        sc = torch.full((1,), scale, device=DEV)
    elif kv_dtype == "mxfp4":
        sc = torch.randint(120, 130, (layers, rows, stride), generator=g, dtype=torch.uint8).to(DEV)
    return cache.MLACachePool(kv.to(DEV), kv_dtype, page_size, kv_scale=sc)


def expected(x_lat, x_pe, weights, positions, freq, axes, inter, scale, which):
    """(latent, position part) in fp64 and the magnitude |a| + |b| of each position column's pair."""
    lat, pe = x_lat.double(), x_pe.double()
    if which + "_lat" in weights:
        lat = rms(lat, weights[which + "_lat"], EPS)
    if which + "_pe" in weights:
        pe = rms(pe, weights[which + "_pe"], EPS)
    a = pe.abs()
    if inter:
        mag = (a[..., 0::2] + a[..., 1::2]).repeat_interleave(2, -1)
    else:
        mag = torch.cat([a[..., :32] + a[..., 32:]] * 2, -1)
    return lat, rotate(pe, positions, freq, axes, inter, scale), mag * abs(scale)


def check_bf16(got, ref, noise, what):
    err = (got.double() - ref).abs()
    bound = 2.0 ** -8 * (ref.abs() + noise) + noise
    assert torch.all(err <= bound), f"{what}: {float((err - bound).max())} over the bound"


def check_row(kv_dtype, kv, sc, ref, noise, what):
    """Cache rows (CPU) hold ref [n, 576] (fp64), each rounded once."""
    if kv_dtype == "bf16":
        return check_bf16(kv, ref, noise, what)
    if kv_dtype == "fp8":
        s = float(sc)
        y = (ref / s).clamp(-448, 448)
        n = noise / s + y.abs() * 2.0 ** -23
        err = (dequant("fp8", kv, 1.0) - y).abs()
        assert torch.all(err <= torch.maximum(2.0 ** -4 * (y.abs() + n), torch.tensor(2.0 ** -10)) + n), what
        return None
    e = sc[:, :18].double() - 127
    amax = ref.abs().view(-1, 18, 32).amax(-1)
    tol = noise.view(-1, 18, 32).amax(-1)
    top = 6 * torch.exp2(e)
    assert torch.all(amax - tol <= top), f"{what}: a block clips"
    assert torch.all((amax + tol > top / 2) | (sc[:, :18] == 0) | (amax == 0)), f"{what}: a block's scale is too large"
    step = torch.exp2(e).repeat_interleave(32, 1)
    y = ref.abs() / step
    half = torch.where(y < 2, 0.25, torch.where(y < 4, 0.5, 1.0)).double()
    err = (dequant("mxfp4", kv, sc) - ref).abs()
    assert torch.all(err <= half * step * (1 + 2.0 ** -20) + noise), what


CASES = [
    # kv, page, tokens, interleaved, axes, normed parts, queries, fp32 weights
    ("bf16", 1, 1, True, 1, ("kv_lat",), "pe", False),
    ("bf16", 16, 77, False, 3, ("kv_lat", "kv_pe", "q_lat", "q_pe"), "full", False),
    ("bf16", 64, 5, True, 4, (), "full", False),
    ("fp8", 64, 1, True, 1, ("kv_lat",), "pe", False),
    ("fp8", 1, 130, False, 2, ("kv_lat", "q_pe"), "pe", True),
    ("fp8", 8, 33, True, 1, (), "none", False),
    ("fp8", 2, 9, False, 1, ("kv_lat", "kv_pe", "q_lat", "q_pe"), "full", True),
    ("mxfp4", 64, 1, True, 1, ("kv_lat",), "pe", False),
    ("mxfp4", 4, 61, False, 3, ("kv_lat", "kv_pe"), "none", True),
    ("mxfp4", 1, 300, True, 2, (), "full", False),
]


@pytest.mark.parametrize("kv_dtype,page,t,inter,axes,normed,q,fp32", CASES)
@pytest.mark.parametrize("fused", [False, True])
def test_append(kv_dtype, page, t, inter, axes, normed, q, fp32, fused):
    """Keys and queries against fp64; rows and columns that are not written stay.
    fused: inputs are columns of wider projections, as they come in use."""
    g = gen(t)
    pages = -(-t // page) + 3
    pool = new_pool(kv_dtype, pages * page, page, layers=2)
    wide = torch.randn(t, 1536 + 576, generator=g).to(torch.bfloat16)
    kv_a = wide[:, 1536:] if fused else wide[:, 1536:].contiguous()
    qb = torch.randn(t, 16, 128 + 64, generator=g).to(torch.bfloat16)
    q_pe = qb[..., 128:] if fused else qb[..., 128:].contiguous()
    # heads before tokens, as a batched product leaves them
    q_lat = torch.randn(16, t, 512, generator=g).to(torch.bfloat16).transpose(0, 1)
    if not fused:
        q_lat = q_lat.contiguous()
    q0 = torch.randn(t, 16, 576, generator=g).to(torch.bfloat16)
    wt = torch.float32 if fp32 else torch.bfloat16
    weights = {n: (1 + 0.2 * torch.randn(512 if n.endswith("lat") else 64, generator=g)).to(wt) for n in normed}
    pos = torch.randint(-5, 1 << 20, (t, axes), generator=g, dtype=torch.int32)
    freq = [10000.0 ** (-i / 32) for i in range(32)]
    axis = [i % axes for i in range(32)]
    scale = 1.0 if axes == 1 else 0.75
    slots = torch.randperm(pages * page, generator=g)[:t].to(torch.int32)
    rope = cache.MLARope(inv_freq=freq, axis_of_pair=axis, interleaved=inter, scale=scale)
    norm = cache.MLANorm(eps=EPS, **{n: w.to(DEV) for n, w in weights.items()})
    before = pool.kv.cpu().clone()
    sc_before = None if kv_dtype != "mxfp4" else pool.kv_scale.cpu().clone()

    def dev(x):  # the same strides on the device
        if not fused:
            return x.to(DEV)
        base = {kv_a: wide, q_pe: qb}.get(x)
        return base.to(DEV)[..., base.shape[-1] - x.shape[-1]:] if base is not None else \
            x.transpose(0, 1).to(DEV).transpose(0, 1)

    kv_d, q_out = dev(kv_a), q0.to(DEV)
    kw = {} if q == "none" else dict(q_pe=dev(q_pe), q_out=q_out)
    if q == "full":
        kw["q_lat"] = dev(q_lat)
    pool.append(kv_d[:, :512], kv_d[:, 512:], slots.to(DEV), rope, pos.to(DEV), norm=norm, layer=1, **kw)
    assert pool.poll_error() == 0
    after = pool.kv.cpu()
    at = slots.long()
    assert torch.equal(after[0].view(torch.uint8), before[0].view(torch.uint8)), "the other layer"
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(after[1][rest].view(torch.uint8), before[1][rest].view(torch.uint8)), "other rows"
    lat, pe, mag = expected(kv_a[:, :512], kv_a[:, 512:], weights, pos, freq, axis, inter, scale, "kv")
    ref, noise = torch.cat([lat, pe], 1), NOISE * torch.cat([lat.abs(), mag], 1)
    sc = None if kv_dtype == "bf16" else (pool.kv_scale.cpu() if kv_dtype == "fp8" else pool.kv_scale.cpu()[1, at])
    check_row(kv_dtype, after[1, at], sc, ref, noise, "keys")
    if sc_before is not None:
        sc_after = pool.kv_scale.cpu()
        assert torch.equal(sc_after[0], sc_before[0]) and torch.equal(sc_after[1, rest], sc_before[1, rest])
    q_got = q_out.cpu()
    lat, pe, mag = expected(q_lat, q_pe, weights, pos, freq, axis, inter, scale, "q")
    if q == "none":
        assert torch.equal(q_got, q0)
        return
    check_bf16(q_got[..., 512:], pe, NOISE * mag, "queries, position part")
    if q == "full":
        check_bf16(q_got[..., :512], lat, NOISE * lat.abs(), "queries, latent part")
    else:
        assert torch.equal(q_got[..., :512], q0[..., :512])


@pytest.mark.parametrize("inter", [True, False])
def test_append_in_place_queries(inter):
    """q_pe and q_lat may be the columns of q_out: the same bits as out of place."""
    g = gen(3)
    t = 21
    q0 = torch.randn(t, 16, 576, generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.randint(0, 9999, (t,), generator=g, dtype=torch.int32).to(DEV)
    pool = new_pool("bf16", 4)
    rope = cache.MLARope(interleaved=inter)
    norm = cache.MLANorm(q_lat=True, q_pe=True)
    a, b = torch.zeros_like(q0), q0.clone()
    pool.append(None, None, None, rope, pos, norm=norm, q_pe=q0[..., 512:], q_lat=q0[..., :512], q_out=a)
    pool.append(None, None, None, rope, pos, norm=norm, q_pe=b[..., 512:], q_lat=b[..., :512], q_out=b)
    assert torch.equal(a, b) and not torch.equal(a, q0)
    c = q0.clone()
    pool.append(None, None, None, rope, pos, norm=norm, q_pe=c[..., 512:], q_out=c)
    assert torch.equal(c[..., 512:], a[..., 512:]) and torch.equal(c[..., :512], q0[..., :512])
    assert pool.poll_error() == 0


@pytest.mark.parametrize("inter", [True, False])
def test_rotation_at_far_positions(inter):
    """Positions up to the ends of int32: the angle modulo one turn is exact to
    2^-33 turns plus the frequency's own fp64 rounding (2^31 * 2^-54 turns at
    most), where an fp32 angle would be off by whole turns."""
    pos = torch.tensor([0, 1, -1, 12345678, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 99999999], dtype=torch.int32)
    freq = [10000.0 ** (-i / 32) for i in range(32)]
    g = gen(11)
    kv = torch.randn(8, 576, generator=g).to(torch.bfloat16)
    pool = new_pool("bf16", 8)
    pool.append(kv.to(DEV)[:, :512], kv.to(DEV)[:, 512:], torch.arange(8, dtype=torch.int32, device=DEV),
                cache.MLARope(inv_freq=freq, interleaved=inter), pos.to(DEV))
    # the fp64 product of the reference is itself off by 2^31 * 2^-53 radians
    _, ref, mag = expected(kv[:, :512], kv[:, 512:], {}, pos.view(-1, 1), freq, [0] * 32, inter, 1.0, "kv")
    check_bf16(pool.kv.cpu()[0][:, 512:], ref, NOISE * mag, "far positions")
    assert torch.equal(pool.kv.cpu()[0][:, :512], kv[:, :512])


@pytest.mark.parametrize("kv_dtype", ["fp8", "mxfp4"])
def test_append_stores_as_the_quantisers_do(kv_dtype):
    """No norm and no rotation: nothing but the storage rounding is left, and the
    bytes are those of the generators (borders and ties included)."""
    g = gen(5)
    n = 70
    x = torch.randn(n, 576, generator=g) * torch.exp2(torch.randint(-30, 30, (n, 1), generator=g).float())
    x[0] = 0
    x[1, 32:64] = 0
    # ties of e2m1 under a block scale of 1 (largest value 6), and magnitudes at the scale's border
    x[2, :16] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
    x[3, :32], x[4, :32] = 1.5, 1.5078125
    x[5] = torch.linspace(-600, 600, 576)
    x[6] = torch.arange(576) * 2.0 ** -133  # subnormal
    x = x.to(torch.bfloat16)
    if kv_dtype == "fp8":
        want, scale = synth.quantize_fp8(x)
        pool = new_pool("fp8", n, scale=float(scale))
        # another scale, so that values saturate and fall among the subnormals
        small = new_pool("fp8", n, scale=1.0)
        small.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], torch.arange(n, dtype=torch.int32, device=DEV))
        ref = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(small.kv.cpu()[0], ref)
    else:
        want, bytes_ = synth.quantize_mxfp4(x)
        pool = new_pool("mxfp4", n)
    pool.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], torch.arange(n, dtype=torch.int32, device=DEV))
    assert torch.equal(pool.kv.cpu()[0], want)
    if kv_dtype == "mxfp4":
        assert torch.equal(pool.kv_scale.cpu()[0], bytes_)


@pytest.mark.parametrize("scale", [1.0, 0.011, 1 / 3, 0.99999994, 1.0000001, 5.7e-3, 448.0, 3.1e-7, 2.0 ** -61, 2.0 ** -59,
                                   2.0 ** 59 * 1.1, 2.0 ** 61, 7e20, 1e-30, 3e38, 1.2e-38])
def test_e4m3_of_every_bf16_value(scale):
    """Every bf16 value (infinities, NaN and subnormals among them) is stored as
    e4m3 of the correctly rounded quotient, whatever the scale."""
    bits = torch.arange(65536, dtype=torch.int32)
    x = torch.cat([bits, torch.zeros(114 * 576 - 65536, dtype=torch.int32)]).to(torch.int16).view(torch.bfloat16).view(114, 576)
    s = torch.tensor([scale], dtype=torch.float32)
    pool = new_pool("fp8", 114, scale=scale)
    assert torch.equal(pool.kv_scale.cpu(), s)
    pool.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], torch.arange(114, dtype=torch.int32, device=DEV))
    want = (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)
    got = pool.kv.cpu()[0].view(torch.float8_e4m3fn)
    nan = torch.isnan(want.float())
    assert torch.equal(torch.isnan(got.float()), nan)
    assert torch.equal(got.view(torch.uint8)[~nan], want.view(torch.uint8)[~nan])


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "mxfp4"])
def test_append_infinities_and_nan(kv_dtype):
    """bf16 keeps them; e4m3 saturates infinities and keeps NaN; an MXFP4 block
    that holds one reads back as NaN, and no other block does."""
    x = torch.ones(3, 576)
    x[0, 5], x[0, 40], x[1, 530], x[2, 575] = float("inf"), float("-inf"), float("nan"), float("inf")
    x = x.to(torch.bfloat16)
    pool = new_pool(kv_dtype, 3, scale=0.5)
    slots = torch.arange(3, dtype=torch.int32, device=DEV)
    pool.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], slots)
    y = pool.gather(slots).cpu().float()
    if kv_dtype == "bf16":
        assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(x.float()))
    elif kv_dtype == "fp8":
        assert y[0, 5] == 224 and y[0, 40] == -224 and torch.isnan(y[1, 530]) and int(torch.isnan(y).sum()) == 1
    else:
        bad = torch.zeros(3, 18, dtype=torch.bool)
        bad[0, 0] = bad[0, 1] = bad[1, 16] = bad[2, 17] = True
        assert torch.equal(torch.isnan(y), bad.repeat_interleave(32, 1))
        assert torch.all(y[~torch.isnan(y)] == 1)
        assert torch.equal(pool.kv_scale.cpu()[0] == 255, bad)


def test_zero_rows_and_one_large_value():
    """A row of zeros norms to zeros; one large value among zeros to sqrt(512)."""
    x = torch.zeros(2, 576)
    x[1, 100] = 2.0 ** 60
    pool = new_pool("bf16", 2)
    pool.append(x.to(torch.bfloat16).to(DEV)[:, :512], x.to(torch.bfloat16).to(DEV)[:, 512:],
                torch.arange(2, dtype=torch.int32, device=DEV), norm=cache.MLANorm(kv_lat=True, kv_pe=True))
    y = pool.kv.cpu()[0].double()
    assert torch.all(y[0] == 0) and int((y[1] != 0).sum()) == 1
    assert abs(float(y[1, 100]) - 512 ** 0.5) <= 2.0 ** -8 * 512 ** 0.5 * (1 + 2.0 ** -10)


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "mxfp4"])
def test_skipped_and_bad_slots(kv_dtype):
    """-1 stores nothing and is no error; a slot outside the cache stores nothing and is one."""
    g = gen(2)
    x = torch.randn(6, 576, generator=g).to(torch.bfloat16).to(DEV)
    pool = new_pool(kv_dtype, 8, page_size=4)
    before = pool.kv.clone()
    slots = torch.tensor([-1, 2, -1, 7, -1, -1], dtype=torch.int32, device=DEV)
    pool.append(x[:, :512], x[:, 512:], slots)
    assert pool.poll_error() == 0
    changed = (pool.kv != before).any(-1)[0].cpu()
    assert changed.nonzero().flatten().tolist() == [2, 7]
    before = pool.kv.clone()
    for bad in (8, -2, 2 ** 31 - 1, -2 ** 31):
        pool.append(x[:1, :512], x[:1, 512:], torch.tensor([bad], dtype=torch.int32, device=DEV))
        assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX and pool.poll_error() == 0
        assert torch.equal(pool.kv, before)
        out = torch.full((1, 576), 3.0, dtype=torch.bfloat16, device=DEV)
        pool.gather(torch.tensor([bad], dtype=torch.int32, device=DEV), out=out)
        assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX
        assert torch.all(out == 3)


@pytest.mark.parametrize("stride", [18, 19, 32])
def test_mxfp4_scale_rows_of_any_stride(stride):
    """Only the first 18 bytes of a scale row are read and written."""
    g = gen(8)
    x = torch.randn(40, 576, generator=g).to(torch.bfloat16)
    pool = new_pool("mxfp4", 40, stride=stride)
    pad = pool.kv_scale[..., 18:].clone()
    slots = torch.randperm(40, generator=g).to(torch.int32).to(DEV)
    pool.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], slots)
    want, by = synth.quantize_mxfp4(x)
    assert torch.equal(pool.kv[0][slots.long()].cpu(), want)
    assert torch.equal(pool.kv_scale[0][slots.long(), :18].cpu(), by)
    assert torch.equal(pool.kv_scale[..., 18:], pad)
    assert torch.equal(pool.gather(slots).cpu().double(), dequant("mxfp4", want, by))


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("n", [1, 3, 1000])
def test_gather(kv_dtype, n):
    g = gen(n)
    pool = new_pool(kv_dtype, 384, page_size=16, layers=2)
    slots = torch.randint(0, 384, (n,), generator=g, dtype=torch.int32)
    slots[n // 2] = -1 if n > 1 else slots[0]
    buf = torch.full((n, 592), 7.0, dtype=torch.bfloat16, device=DEV)
    out = pool.gather(slots.to(DEV), out=buf[:, 8:584], layer=1)
    assert pool.poll_error() == 0 and out.data_ptr() == buf[:, 8:].data_ptr()
    at = slots.long().clamp(min=0)
    sc = None if kv_dtype == "bf16" else (0.011 if kv_dtype == "fp8" else pool.kv_scale.cpu()[1, at])
    ref = dequant(kv_dtype, pool.kv.cpu()[1, at], np.float32(sc) if kv_dtype == "fp8" else sc)
    got = buf.cpu().double()
    keep = slots >= 0
    # e4m3: the product in fp32, then bf16: two roundings
    err = (got[keep, 8:584] - ref[keep]).abs()
    assert torch.all(err <= (2.0 ** -8 + 2.0 ** -23) * ref[keep].abs() if kv_dtype == "fp8" else err == 0)
    assert torch.all(got[~keep] == 7) and torch.all(got[:, :8] == 7) and torch.all(got[:, 584:] == 7)


def test_gather_every_code():
    """Every e4m3 byte, and every e2m1 code under every scale byte, exactly (scale 1; 6 * 2^127 is infinite)."""
    kv = torch.arange(256, dtype=torch.uint8).repeat(9)[:4 * 576].view(4, 576)
    pool = cache.MLACachePool(kv.to(DEV), "fp8", 1, kv_scale=torch.ones(1, device=DEV))
    slots = torch.arange(4, dtype=torch.int32, device=DEV)
    got, ref = pool.gather(slots).cpu().double(), dequant("fp8", kv, 1.0)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))
    n = 256
    packed = torch.tensor([(2 * j) % 16 | ((2 * j + 1) % 16) << 4 for j in range(288)], dtype=torch.uint8).repeat(n, 1)
    sc = torch.arange(256, dtype=torch.uint8).view(n, 1).repeat(1, 18)
    pool = cache.MLACachePool(packed.to(DEV), "mxfp4", 1, kv_scale=sc.to(DEV))
    got = pool.gather(torch.arange(n, dtype=torch.int32, device=DEV)).cpu()
    ref = dequant("mxfp4", packed, sc).float().to(torch.bfloat16)  # exact but for overflow
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[:255].float(), ref[:255].float())


@pytest.mark.parametrize("page", [1, 4, 64, 256])
@pytest.mark.parametrize("batch", [1, 2, 37])
def test_slots(page, batch):
    g = gen(page + batch)
    lens = torch.randint(0, 700, (batch,), generator=g).tolist()
    lens[batch // 2] = 5
    counts = [-(-n // page) for n in lens]
    total = sum(counts)
    perm = torch.randperm(total + 5, generator=g)[:total].to(torch.int32)
    indptr = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32)
    last = torch.tensor([n - (c - 1) * page if c else 0 for n, c in zip(lens, counts)], dtype=torch.int32)
    new = [int(torch.randint(0, n + 1, (1,), generator=g)) for n in lens]
    new[batch // 2] = 5
    qo = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32)
    pool = new_pool("bf16", (total + 5) * page, page)
    t = int(qo[-1]) + 3  # a padded batch
    rows = torch.full((t, 2), -9, dtype=torch.int32, device=DEV)
    slots, _ = pool.slots((indptr.to(DEV), perm.to(DEV), last.to(DEV)), qo.to(DEV), t, rows=rows[:, 1])
    assert pool.poll_error() == 0
    want_s, want_r = [], []
    for b in range(batch):
        for r in range(lens[b] - new[b], lens[b]):
            want_s.append(int(perm[int(indptr[b]) + r // page]) * page + r % page)
            want_r.append(r)
    assert slots.tolist() == want_s + [-1] * 3
    assert rows[:, 1].tolist() == want_r + [0] * 3 and torch.all(rows[:, 0] == -9)


def test_slots_bad_tables():
    """Tables that disagree with each other give -1 and the error, and no read outside them."""
    pool = new_pool("bf16", 64, 16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    for indptr, idx, last, qo in (([0, 1], [0], [5], [0, 6]),        # more new tokens than rows
                                  ([0, 1], [4], [5], [0, 5]),        # a page out of range
                                  ([0, 1], [-1], [5], [0, 5]),
                                  ([0, 2], [0], [5], [0, 5]),        # past the table
                                  ([-1, 1], [0], [5], [0, 5]),
                                  ([0, 1], [0], [17], [0, 5]),       # more rows than a page has
                                  ([0, 1], [0], [0], [0, 5]),
                                  ([0, 0], [0], [0], [0, 1])):       # an empty sequence with a token
        slots, _ = pool.slots((i32(indptr), i32(idx), i32(last)), i32(qo), qo[-1])
        assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX, (indptr, idx, last, qo)
        assert slots[0] == -1


def test_rows_past_32_bit_offsets():
    """A cache of 4.9 GB: rows near its end are written and read where they belong."""
    rows = 4_250_000
    pool = cache.MLACachePool(torch.zeros(rows, 576, dtype=torch.bfloat16, device=DEV), "bf16", 1)
    g = gen(9)
    x = torch.randn(5, 576, generator=g).to(torch.bfloat16)
    slots = torch.tensor([rows - 1, 0, 3_800_000, 1_864_136, rows - 2], dtype=torch.int32, device=DEV)
    pool.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], slots)
    assert torch.equal(pool.kv[slots.long()].cpu(), x)
    assert torch.equal(pool.gather(slots).cpu(), x)
    assert int((pool.kv[:, 0] != 0).sum()) == 5
    assert pool.poll_error() == 0


def test_layers_with_scales_and_strides_of_their_own():
    """An e4m3 cache whose layers have a scale each and lie apart in a wider tensor."""
    g = gen(12)
    big = torch.zeros(3, 50, 576, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.tensor([0.5, 0.01, 2.0], device=DEV)
    pool = cache.MLACachePool(big[:, :48], "fp8", 16, kv_scale=scale)
    x = torch.randn(20, 576, generator=g).to(torch.bfloat16)
    slots = torch.randperm(48, generator=g)[:20].to(torch.int32)
    for layer in (2, 0, 1):
        pool.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], slots.to(DEV), layer=layer)
    assert pool.poll_error() == 0
    raw = big.view(torch.uint8).cpu()
    for layer in range(3):
        want = (x.float() / scale[layer].cpu()).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(raw[layer, slots.long()], want.view(torch.uint8))
        got = pool.gather(slots.to(DEV), layer=layer).cpu()
        assert torch.equal(got, (want.float() * scale[layer].cpu()).to(torch.bfloat16))
    assert torch.all(raw[:, 48:] == 0), "rows of no layer"


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8", "mxfp4"])
def test_allocated_layers_fit_the_decode(kv_dtype):
    """Every layer of an allocated pool meets the decode's alignments, whatever its rows."""
    pool = cache.MLACachePool.allocate(kv_dtype, 13, 1, num_layers=3, device=DEV)
    for layer in range(3):
        assert pool.kv[layer].data_ptr() % 32 == 0
        if kv_dtype == "mxfp4":
            assert pool.kv_scale[layer].data_ptr() % 16 == 0
    assert pool.num_pages == 13 and pool.num_layers == 3


@pytest.mark.parametrize("how", ["stream", "handle"])
def test_memory_made_on_the_calls_stream(how):
    """Without out= the result belongs to the stream that the call names, as a torch stream or a handle."""
    pool = new_pool("bf16", 64, 16)
    table = (torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV),
             torch.tensor([9], dtype=torch.int32, device=DEV))
    qo = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    named = s if how == "stream" else s.cuda_stream
    slots, _ = pool.slots(table, qo, 9, stream=named)
    rows = pool.gather(slots, stream=named)
    indices, refs, live = pool.compact(table[1], stream=named)
    s.synchronize()
    assert slots.tolist() == list(range(32, 41)) and torch.equal(rows, pool.kv[0, 32:41])
    assert int(live) == 0 and pool.poll_error(named) == binding.MLA_ERR_DEVICE_INDEX  # page 2 is free


def test_another_stream_and_a_graph():
    """The calls on a stream of their own, then captured and replayed with new inputs."""
    g = gen(4)
    x = torch.randn(9, 576, generator=g).to(torch.bfloat16).to(DEV)
    slots = torch.arange(9, dtype=torch.int32, device=DEV)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    rope, norm = cache.MLARope(), cache.MLANorm(kv_lat=True)
    pool = new_pool("fp8", 16)
    pool.append(x[:, :512], x[:, 512:], slots, rope, pos, norm=norm)
    ref = pool.gather(slots).clone()
    pool.kv.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pool.append(x[:, :512], x[:, 512:], slots, rope, pos, norm=norm, stream=s)
    out = pool.gather(slots, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.append(x[:, :512], x[:, 512:], slots, rope, pos, norm=norm)
        pool.gather(slots, out=out)
    y = torch.randn(9, 576, generator=g).to(torch.bfloat16).to(DEV)
    pool.append(y[:, :512], y[:, 512:], slots, rope, pos + 3, norm=norm)
    want = pool.gather(slots).clone()
    x.copy_(y)
    pos += 3
    pool.kv.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and pool.poll_error() == 0


def test_python_refusals():
    pool = new_pool("bf16", 64, 16)
    x = torch.zeros(4, 576, dtype=torch.bfloat16, device=DEV)
    slots = torch.zeros(4, dtype=torch.int32, device=DEV)
    pos = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    q = torch.zeros(4, 16, 576, dtype=torch.bfloat16, device=DEV)
    ok = dict(kv_lat=x[:, :512], kv_pe=x[:, 512:], slots=slots, rope=cache.MLARope(), positions=pos)
    pool.append(**ok)
    for bad in (dict(kv_lat=x[:, :511]), dict(kv_lat=x[:, :512].float()), dict(kv_pe=None), dict(kv_pe=x[:3, 512:]),
                dict(slots=slots.long()), dict(slots=slots[:3]), dict(slots=slots.cpu()), dict(positions=None),
                dict(positions=pos.long()), dict(positions=pos[:3]), dict(rope=cache.MLARope(sections=(16, 8, 8))),
                dict(q_pe=q[..., 512:]), dict(q_out=q), dict(q_pe=q[..., 512:], q_out=q.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(kv_lat=None), dict(kv_lat=None, kv_pe=None)):
        with pytest.raises(ValueError):
            pool.append(**{**ok, **bad})
    for kv, dt, page, sc in ((x, "bf16", 3, None), (x, "fp8", 1, None), (x.view(torch.uint8)[:, :576], "fp8", 1, torch.ones(1, device=DEV)),
                             (x, "bf16", 1, torch.ones(1, device=DEV)),
                             (torch.zeros(4, 288, dtype=torch.uint8, device=DEV), "mxfp4", 1, torch.zeros(4, 17, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            cache.MLACachePool(kv, dt, page, kv_scale=sc)
    for call in (lambda: pool.gather([0, 1]), lambda: pool.gather(slots, out=x.float()),
                 lambda: pool.gather(slots, out=x[:3]), lambda: pool.slots((slots, slots), slots, 1),
                 lambda: pool.slots((slots[:1], slots, slots[:1]), slots[:1], 1), lambda: pool.free(slots.view(2, 2)),
                 lambda: pool.slots((slots[:2], slots, slots[:1]), slots[:2], -1),
                 lambda: pool.copy_pages(slots, slots[:2]), lambda: pool.free(slots[::2]),
                 lambda: pool.fork(pool.table(1, 4), slots, pool.table(2, 4)),
                 lambda: pool.resize(pool.table(1, 4), None, pool.table(1, 4)),
                 lambda: pool.compact(slots, out=(slots, pool.refs[:2], slots[:1]))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(binding.MLAError):  # rows that overlap
        pool.gather(slots, out=x[:1].expand(4, 576))
    with pytest.raises(ValueError):
        cache.MLANorm(kv_lat=torch.ones(64, device=DEV))
    with pytest.raises(ValueError):
        cache.MLANorm(kv_lat=torch.ones(512, device=DEV), kv_pe=torch.ones(64, device=DEV).bfloat16())
    with pytest.raises(binding.MLAError) as e:
        pool.append(**{**ok, "layer": 1})
    assert e.value.status == binding.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [1.0, 0.011, 1 / 3, 448.0, 2.0 ** -59, 2.0 ** 59, 2.0 ** 61, 1e-30])
def test_e4m3_keeps_the_sign_of_zero(scale):
    """Zeros, and what rounds to them, keep their sign, among ordinary values, among
    values past the range, and where the quotient is a division."""
    x = torch.zeros(6, 576)
    x[0], x[1, ::2], x[2, 1::3] = -0.0, -0.0, -0.0
    x[3] = torch.where(torch.arange(576) % 5 == 0, torch.tensor(-0.0), torch.linspace(-3, 3, 576) * scale)
    x[4] = torch.where(torch.arange(576) % 2 == 0, torch.tensor(-0.0), torch.tensor(1e30))
    x[5] = -scale * 2.0 ** -11 * (torch.arange(576) % 3)
    x = x.to(torch.bfloat16)
    pool = new_pool("fp8", 6, scale=scale)
    pool.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], torch.arange(6, dtype=torch.int32, device=DEV))
    want = (x.float() / torch.tensor([scale], dtype=torch.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert int((want.view(torch.uint8) == 0x80).sum()) > 1200
    assert torch.equal(pool.kv.cpu()[0], want.view(torch.uint8))


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_mxfp4_keeps_the_sign_of_zero(sign):
    """The bytes of the generators for zeros of either sign, in blocks of zeros and among values."""
    x = torch.full((3, 576), 0.0 * sign)
    x[1, ::2] = 1.25
    x[2] = sign * torch.linspace(0, 0.2, 576)
    x[2, ::32] = 6.0
    x = x.to(torch.bfloat16)
    want, scales = synth.quantize_mxfp4(x)
    pool = new_pool("mxfp4", 3)
    pool.append(x.to(DEV)[:, :512], x.to(DEV)[:, 512:], torch.arange(3, dtype=torch.int32, device=DEV))
    assert torch.equal(pool.kv.cpu()[0], want) and torch.equal(pool.kv_scale.cpu()[0], scales)


@pytest.mark.parametrize("layer", [2, -1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 62])
def test_layers_out_of_range(layer):
    """No number that is not a layer's is taken for one, whatever its low 32 bits."""
    pool = new_pool("bf16", 8, layers=2)
    before = pool.kv.clone()
    x = torch.ones(2, 576, dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    for call in (lambda: pool.append(x[:, :512], x[:, 512:], slots, layer=layer), lambda: pool.gather(slots, layer=layer)):
        with pytest.raises(binding.MLAError) as e:
            call()
        assert e.value.status == binding.MLA_ERR_INVALID_ARG
    assert torch.equal(pool.kv, before) and pool.poll_error() == 0


@pytest.mark.parametrize("batch", [2047, 2048, 2049, 3000])
def test_slots_of_many_sequences(batch):
    """Batches on both sides of what is staged on chip, with empty sequences, sequences
    without new tokens and a padded tail."""
    g = gen(batch)
    page = 4
    lens = torch.randint(0, 12, (batch,), generator=g)
    new = torch.minimum(torch.randint(0, 5, (batch,), generator=g), lens)
    lens[0], new[0], lens[-1], new[-1] = 3, 0, 9, 9
    lens[7], new[7] = 0, 0
    counts = (lens + page - 1) // page
    indptr = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    qo = torch.cat([new.new_zeros(1), new.cumsum(0)])
    total = int(indptr[-1])
    perm = torch.randperm(total + 9, generator=g)[:total]
    last = torch.where(counts > 0, lens - (counts - 1) * page, counts)
    seq = torch.repeat_interleave(torch.arange(batch), new)
    row = lens[seq] - new[seq] + torch.arange(seq.numel()) - qo[seq]
    want = perm[indptr[seq] + row // page] * page + row % page
    pool = new_pool("bf16", (total + 9) * page, page)
    t = seq.numel() + 5
    i32 = lambda v: v.to(torch.int32).to(DEV)  # noqa: E731
    rows = torch.full((t,), -9, dtype=torch.int32, device=DEV)
    slots, _ = pool.slots((i32(indptr), i32(perm), i32(last)), i32(qo), t, rows=rows)
    assert pool.poll_error() == 0
    assert slots.tolist() == want.tolist() + [-1] * 5 and rows.tolist() == row.tolist() + [0] * 5
