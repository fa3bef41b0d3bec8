"""The e4m3 cache with a scale per row ("fp8_row") on the GPU: append, gather, the
page operators and the decode, against fp64.

Tolerances of the decode, per output of head h and feature j, with w_t the exact
softmax weights and v_t = code_t s_t:
  * the output's rounding to bf16                               2^-8 |out|
  * a weight times its row's scale enters P.V as two e4m3 terms: each keeps 4 bits,
    so 2^-8 w_t |v_t|, or half of e4m3's smallest step, 2^-10, where that is more;
    the reference of the weights lies 4 (log2) below the largest score of
    the rows so far and scales are taken relative to a power of two S at most twice
    the largest scale, so that is 2^-14 w_max |code_t| S in the output
  * the query enters the scores as two e4m3 terms: exact for a bf16 query down to
    half the smallest step, 2^-10 where the head's largest is 224 or more: a score
    moves by at most d = sum_c |k_c| max|q| 2^-10 / 224 / 24, weights by 2 d of themselves
  * fp32 sums of products and weights, exponentials (2^-22)     2^-14 w_t |v_t|
and of the log of the sum: d, 2^-22 of its size and 2e-5 for the sums."""
import pytest
import torch

from mla_attention_decode_gb300 import binding, build, cache
from test_cache_rows_gpu import EPS, NOISE, expected, check_bf16, gen

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def values(codes, scales):
    """Codes [n, 576] and scales [n] (CPU) in fp64."""
    return codes.view(torch.float8_e4m3fn).double() * scales.double().unsqueeze(-1)


def stored(y):
    """Rows y (fp32) as codes and scales, by the definition."""
    amax = y.abs().amax(-1)
    s = (amax / 448).clamp(min=2.0 ** -64)
    return (y / s.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def random_cache(g, n, spread=0.5):
    y = torch.randn(n, 576, generator=g)
    codes, s = stored(y)
    return codes, s * torch.exp(spread * torch.randn(n, generator=g))


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("page,t,inter,axes,normed,q,layers,stride", [
    (64, 1, True, 1, ("kv_lat",), "pe", 1, 1), (1, 130, False, 2, ("kv_lat", "q_pe"), "pe", 2, 1),
    (8, 33, True, 1, (), "none", 1, 3), (2, 9, False, 3, ("kv_lat", "kv_pe", "q_lat", "q_pe"), "full", 2, 3),
    (16, 700, False, 4, ("kv_lat", "kv_pe"), "pe", 1, 2)])
def test_append(page, t, inter, axes, normed, q, layers, stride):
    g = gen(t + page)
    rows = (-(-t // page) + 3) * page
    codes0 = torch.randint(0, 120, (layers, rows, 576), generator=g, dtype=torch.uint8)
    wide0 = torch.rand(layers, rows, stride, generator=g) + 0.5
    wide = wide0.to(DEV)
    pool = cache.MLACachePool(codes0.to(DEV), "fp8_row", page, kv_scale=wide[:, :, 0])
    kv_a = torch.randn(t, 640, generator=g).to(torch.bfloat16)
    kv_a *= torch.exp2(torch.randint(-20, 20, (t, 1), generator=g).float())
    qb = torch.randn(t, 16, 192, generator=g).to(torch.bfloat16)
    q_lat = torch.randn(t, 16, 512, generator=g).to(torch.bfloat16)
    weights = {n: (1 + 0.2 * torch.randn(512 if n.endswith("lat") else 64, generator=g)).to(torch.bfloat16) for n in normed}
    pos = torch.randint(-5, 1 << 20, (t, axes), generator=g, dtype=torch.int32)
    freq, axis = [10000.0 ** (-i / 32) for i in range(32)], [i % axes for i in range(32)]
    slots = torch.randperm(rows, generator=g)[:t].to(torch.int32)
    slots[t // 2:t // 2 + 1] = -1
    rope = cache.MLARope(inv_freq=freq, axis_of_pair=axis, interleaved=inter)
    norm = cache.MLANorm(eps=EPS, **{n: w.to(DEV) for n, w in weights.items()})
    dev = kv_a.to(DEV)
    q_out = torch.zeros(t, 16, 576, dtype=torch.bfloat16, device=DEV)
    more = {} if q == "none" else dict(q_pe=qb.to(DEV)[..., 128:], q_out=q_out)
    if q == "full":
        more["q_lat"] = q_lat.to(DEV)
    layer = layers - 1
    pool.append(dev[:, 64:576], dev[:, 576:], slots.to(DEV), rope, pos.to(DEV), norm, layer=layer, **more)
    assert pool.poll_error() == 0
    lat, pe, mag = expected(kv_a[:, 64:576], kv_a[:, 576:], weights, pos, freq, axis, inter, 1.0, "kv")
    if "kv_pe" in weights:  # the rotated pair's magnitudes after the norm
        mag = torch.full_like(mag, 0.0) + pe.abs().amax(-1, keepdim=True) * 2
    y = torch.cat([lat, pe], -1)
    noise = torch.cat([lat.abs(), mag], -1) * NOISE
    keep = slots >= 0
    at = slots[keep].long()
    got, s = pool.kv[layer].cpu(), pool.kv_scale[layer].cpu()
    y, noise = y[keep], noise[keep]
    amax = y.abs().amax(-1)
    assert torch.all((s[at].double() - amax / 448).abs() <= (noise.amax(-1) + amax * 2.0 ** -24) / 448)
    # codes under the stored scale: half a step of e4m3 (2^-4 relative, 2^-10 absolute), the quotient's rounding
    x, n = y / s[at].double().unsqueeze(-1), noise / s[at].double().unsqueeze(-1)
    n = n + x.abs() * 2.0 ** -23
    err = (got[at].view(torch.float8_e4m3fn).double() - x.clamp(-448, 448)).abs()
    assert torch.all(err <= torch.maximum(2.0 ** -4 * (x.abs() + n), torch.tensor(2.0 ** -10)) + n)
    # what is not written stays, scales in other columns too
    left = torch.ones(rows, dtype=torch.bool)
    left[at] = False
    assert torch.equal(got[left], codes0[layer][left])
    now = wide.cpu()
    assert torch.equal(now[layer][left], wide0[layer][left]) and torch.equal(now[:, :, 1:], wide0[:, :, 1:])
    if layers > 1:
        assert torch.equal(pool.kv[0].cpu(), codes0[0]) and torch.equal(now[0], wide0[0])
    if q != "none":
        _, ref, mag = expected(q_lat, qb[..., 128:], weights, pos, freq, axis, inter, 1.0, "q")
        check_bf16(q_out[..., 512:].cpu(), ref, (mag + ref.abs().amax(-1, keepdim=True) * 2) * NOISE, "queries")


def odd_rows():
    """Rows whose storage is decided by the definition alone: bf16 values as they are."""
    g = gen(5)
    x = torch.randn(64, 576, generator=g) * torch.exp2(torch.randint(-40, 40, (64, 1), generator=g).float())
    x[1] = 0
    x[2] = -0.0
    x[3] = torch.linspace(-1, 1, 576)
    x[4] = 0
    x[4, 17] = -3e38
    x[5] = 1e-39                       # subnormal: under the smallest scale
    x[6] = 2.0 ** -64 * 448 * torch.randn(576, generator=g)
    x[7, :] = 448
    x[7, 1::2] = torch.exp2(-torch.arange(288).float() % 24)
    x[8] = torch.randn(576, generator=g) * 1e37
    x[9, 575] = 1e6                    # one large value in the position part
    return x.to(torch.bfloat16)


def test_append_stores_what_the_division_gives():
    """Bit for bit: the scale the largest magnitude over 448, the codes e4m3 of the quotient."""
    x = odd_rows()
    pool = cache.MLACachePool.allocate("fp8_row", 64, 1)
    xd = x.to(DEV)
    pool.append(xd[:, :512], xd[:, 512:], torch.arange(64, dtype=torch.int32, device=DEV))
    codes, s = stored(x.float())
    assert torch.equal(pool.kv_scale[0].cpu(), s) and torch.equal(pool.kv[0].cpu(), codes)
    assert torch.equal(pool.gather(torch.arange(64, dtype=torch.int32, device=DEV)).cpu(),
                       (codes.view(torch.float8_e4m3fn).float() * s.unsqueeze(-1)).to(torch.bfloat16))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("column", [0, 300, 511, 512, 575])
def test_append_of_rows_that_are_not_finite(bad, column):
    x = torch.randn(3, 576, generator=gen(1)).to(torch.bfloat16)
    x[1, column] = bad
    pool = cache.MLACachePool.allocate("fp8_row", 1, 4)
    xd = x.to(DEV)
    pool.append(xd[:, :512], xd[:, 512:], torch.arange(3, dtype=torch.int32, device=DEV))
    codes, s = stored(x.float()[[0, 2]])
    got = pool.kv_scale[0].cpu()
    assert torch.isnan(got[1]) and torch.equal(got[[0, 2]], s)
    assert torch.equal(pool.kv[0].cpu()[[0, 2]], codes) and torch.all(pool.kv[0, 1] == 0)
    assert torch.all(torch.isnan(pool.gather(torch.tensor([1], dtype=torch.int32, device=DEV))))


@pytest.mark.parametrize("n", [1, 9, 1000])
def test_gather(n):
    g = gen(n)
    codes, s = random_cache(g, 384, 3.0)
    wide = torch.zeros(2, 384, 5)
    wide[1, :, 0] = s
    pool = cache.MLACachePool(torch.stack([codes.flip(0), codes]).to(DEV), "fp8_row", 16, kv_scale=wide.to(DEV)[..., 0])
    slots = torch.randint(0, 384, (n,), generator=g, dtype=torch.int32)
    want = (codes.view(torch.float8_e4m3fn).float() * s.unsqueeze(-1)).to(torch.bfloat16)
    out = torch.full((n + 2, 584), 7.0, dtype=torch.bfloat16, device=DEV)
    bad = torch.cat([slots, torch.tensor([-1, 384], dtype=torch.int32)]).to(DEV)
    pool.gather(bad, out=out[:, :576], layer=1)
    assert torch.equal(out[:n, :576].cpu(), want[slots.long()])
    assert torch.all(out[n:] == 7.0) and torch.all(out[:, 576:] == 7.0)
    assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX
    assert torch.equal(pool.gather(slots.to(DEV), layer=1).cpu(), want[slots.long()]) and pool.poll_error() == 0


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("page", [1, 2, 8, 64, 256])
@pytest.mark.parametrize("layers,stride", [(1, 1), (3, 1), (2, 4)])
def test_page_operators_move_scales(page, layers, stride):
    """Copies, forks, cuts and compaction take a row's scale with its codes; other columns stay."""
    g, pages = gen(page * 7 + layers), 24
    rows = pages * page
    codes = torch.randint(0, 256, (layers, rows, 576), generator=g, dtype=torch.uint8)
    wide = torch.rand(layers, rows, stride, generator=g)
    dev = wide.to(DEV)
    pool = cache.MLACachePool(codes.to(DEV), "fp8_row", page, kv_scale=dev[:, :, 0])

    def rows_of(r):
        r = torch.as_tensor(r)
        return torch.cat([pool.kv.cpu()[:, r], dev.cpu()[:, r, :1].contiguous().view(torch.uint8).view(layers, r.numel(), 4)], -1)

    def page_rows(p, n=page):
        return torch.arange(n) + int(p) * page

    before = {p: rows_of(page_rows(p)) for p in range(pages)}
    pool.copy_pages(torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.tensor([22, 23], dtype=torch.int32, device=DEV))
    assert torch.equal(rows_of(page_rows(22)), before[0]) and torch.equal(rows_of(page_rows(23)), before[1])
    lens = torch.tensor([2 * page + max(1, page // 2), page, 0, max(1, page // 4)], dtype=torch.int32, device=DEV)
    table = pool.resize(pool.table(4, 0), lens, pool.table(4, 8))
    forks = pool.fork(table, torch.tensor([0, 0, 3], dtype=torch.int32, device=DEV), pool.table(3, 8))
    indptr, indices = forks[0].tolist(), forks[1].tolist()
    src = table[1].tolist()
    for n, (b, parent) in enumerate(((0, [0, 1, 2]), (0, [0, 1, 2]), (3, [4]))):
        mine = indices[indptr[n]:indptr[n + 1]]
        used = max(1, page // 2) if b == 0 else max(1, page // 4)
        for k, p in enumerate(mine):
            m = used if k == len(mine) - 1 else page
            assert torch.equal(rows_of(page_rows(p, m)), rows_of(page_rows(src[parent[k]], m)))
    # the first sequence ends; compaction moves what is left, scales with it
    want = [rows_of(page_rows(p)) for n in range(3) for p in indices[indptr[n]:indptr[n + 1]]]
    pool.free(table[1][:5])
    used = forks[1][:indptr[3]]
    at, _, _ = pool.compact(used)
    for p, w in zip(at.tolist(), want):
        assert torch.equal(rows_of(page_rows(p)), w)
    assert pool.poll_error() == 0
    assert torch.equal(dev.cpu()[:, :, 1:], wide[:, :, 1:])


# ------------------------------------------------------------------ decode
def reference(q, codes, scales, spans, q_len=1, sm=1 / 24):
    """Sequences as lists of rows: out, lse, tolerance of out, tolerance of lse, in fp64."""
    out, lse, tol, tol_lse = [], [], [], []
    k_all = values(codes, scales)
    for b, rows in enumerate(spans):
        for i in range(q_len):
            n = len(rows) - (q_len - 1 - i)
            if n <= 0:
                out.append(torch.zeros(16, 512).double()), lse.append(torch.full((16,), -torch.inf).double())
                tol.append(torch.zeros(16, 512).double()), tol_lse.append(torch.zeros(16).double())
                continue
            at = torch.as_tensor(rows[:n])
            k, qq = k_all[at], q[b * q_len + i].double()
            a = qq @ k.T * sm
            l = torch.logsumexp(a, -1)
            w, v = torch.exp(a - l.unsqueeze(-1)), k[:, :512]
            ref = w @ v
            d = ((k.abs().sum(-1)).unsqueeze(0) * qq.abs().amax(-1, keepdim=True) * 2.0 ** -10 / 224 * abs(sm)).amax(-1)
            span = 2 * scales[at].double().max() * codes[at][:, :512].view(torch.float8_e4m3fn).double().abs()
            wv = w @ v.abs()
            t = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -14 + 2 * d.unsqueeze(-1)) * wv
            # the smallest step, in the rows where it is more than 2^-8 of the weight
            small = (w.unsqueeze(-1) * v.abs() * 2.0 ** -8 < 2.0 ** -14 * w.amax(-1).view(-1, 1, 1) * span).double() \
                if n * 16 * 512 <= 1 << 24 else torch.ones(1, 1, 1)
            t = t + 2.0 ** -14 * w.amax(-1, keepdim=True) * (small * span).sum(1)
            out.append(ref), lse.append(l), tol.append(t)
            tol_lse.append(d + 2.0 ** -22 * l.abs() + 2e-5)
    return [torch.stack(x) for x in (out, lse, tol, tol_lse)]


def check(got, lse, ref):
    out, l, t, tl = ref
    got, lse = got.double().cpu(), lse.double().cpu()
    assert torch.all(torch.isfinite(got))
    err = (got - out).abs()
    assert torch.all(err <= t), f"{float((err - t).max())} over the bound, largest error {float(err.max())}"
    assert torch.equal(torch.isinf(lse), torch.isinf(l))
    fin = torch.isfinite(l)
    assert torch.all((lse - l).abs()[fin] <= tl[fin]), float((lse - l).abs()[fin].max())


def indptr_of(lens):
    return torch.cat([torch.zeros(1), torch.tensor(lens).cumsum(0)]).to(torch.int32)


def poisoned(codes, s, total):
    """Room for `total` rows, all NaN (codes and scales) but the first."""
    c = torch.full((total, 576), 0x7f, dtype=torch.uint8)
    x = torch.full((total,), float("nan"))
    c[:codes.shape[0]], x[:codes.shape[0]] = codes, s
    return c, x


@pytest.mark.parametrize("lens,splits", [([1], 0), ([5, 0, 130, 1, 128, 257, 1000], 0), ([0, 0], 0), ([129, 3000, 64], 3),
                                         ([4097] * 3 + [17], 0), ([33] * 200, 0)])
@pytest.mark.parametrize("q_len", [1, 2, 3, 4, 5, 8, 15, 16])
def test_decode(lens, splits, q_len):
    g = gen(sum(lens) + q_len)
    ind = indptr_of(lens)
    codes, s = random_cache(g, max(1, sum(lens)))
    c, x = poisoned(codes, s, max(1, sum(lens)) + 130)
    # queries that no sequence has (behind the last; between two) are NaN
    q = torch.randn(len(lens) * (q_len + 1) + 1, 16, 576, generator=g).to(torch.bfloat16)
    qo = (torch.arange(len(lens) + 1) * (q_len + 1)).to(torch.int32)
    owned = (torch.arange(len(lens)).view(-1, 1) * (q_len + 1) + torch.arange(q_len)).flatten()
    q0, q = q[owned].clone(), torch.full_like(q, float("nan"))
    q[owned] = q0
    dec = binding.MLADecoder(ind, "fp8_row", num_splits=splits, q_len=q_len)
    assert dec.plan.tokens_fused == (2 if q_len > 1 else 0) and dec.plan.batch == len(lens) * q_len
    out, lse = dec(q.to(DEV), c.to(DEV), ind.to(DEV), qo.to(DEV), kv_scale=x.to(DEV))
    assert dec.poll_error() == 0
    spans = [list(range(int(a), int(e))) for a, e in zip(ind[:-1], ind[1:])]
    check(out, lse, reference(q0, codes, s, spans, q_len))


@pytest.mark.parametrize("q_len", [1, 2, 5])
@pytest.mark.parametrize("sms", [0, 3])
def test_decode_rows_that_begin_further_on(q_len, sms):
    """The first sequence begins at a row of its own, with rows of nobody before it; few blocks
    (many units each) and all of them."""
    g, base, lens = gen(31), 777, [1500, 0, 129, 1, 4000, 640]
    ind = indptr_of(lens) + base
    codes, s = random_cache(g, base + sum(lens))
    codes[:base], s[:base] = 127, float("nan")
    q = torch.randn(len(lens) * q_len, 16, 576, generator=g).to(torch.bfloat16)
    qo = (torch.arange(len(lens) + 1) * q_len).to(torch.int32)
    dec = binding.MLADecoder(ind, "fp8_row", q_len=q_len, num_sms=sms)
    out, lse = dec(q.to(DEV), codes.to(DEV), ind.to(DEV), qo.to(DEV), kv_scale=s.to(DEV))
    assert dec.poll_error() == 0
    check(out, lse, reference(q, codes, s, [list(range(int(a), int(e))) for a, e in zip(ind[:-1], ind[1:])], q_len))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[130, 0, 64, 5, 1000, 257, 128, 1], [3000, 1, 2047]])
def test_decode_pages(page, lens):
    """Pages at random places; every row that no sequence owns holds NaN codes and NaN scales;
    scales every third column of a wider tensor."""
    g = gen(page + len(lens))
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3
    perm = torch.randperm(pages, generator=g)[:sum(counts)]
    at = indptr_of(counts)
    spans = []
    for b, n in enumerate(lens):
        mine = perm[int(at[b]):int(at[b + 1])]
        spans.append([int(mine[r // page]) * page + r % page for r in range(n)])
    codes, s = poisoned(torch.zeros(0, 576, dtype=torch.uint8), torch.zeros(0), pages * page)
    owned = torch.tensor([r for x in spans for r in x])
    codes[owned], s[owned] = random_cache(g, owned.numel())
    last = torch.tensor([n - (c - 1) * page if c else 0 for n, c in zip(lens, counts)], dtype=torch.int32)
    q = torch.randn(len(lens), 16, 576, generator=g).to(torch.bfloat16)
    qo = torch.arange(len(lens) + 1, dtype=torch.int32)
    wide = torch.full((pages * page, 3), float("nan"))
    wide[:, 1] = s
    dec = binding.PagedMLADecoder(at, last, page, pages, "fp8_row")
    out, lse = dec(q.to(DEV), codes.to(DEV), at.to(DEV), perm.to(torch.int32).to(DEV), last.to(DEV), qo.to(DEV),
                   kv_scale=wide.to(DEV)[:, 1])
    assert dec.poll_error() == 0
    check(out, lse, reference(q, codes, s, spans))


@pytest.mark.parametrize("scale", ["wide", "rising", "falling", "zeros", "large", "small"])
def test_decode_scales_of_all_sizes(scale):
    """Rows whose scales lie far apart, in either order over the tiles; zero; near the ends of the range."""
    g, n = gen(9), 700
    codes, s = random_cache(g, n)
    q = torch.randn(1, 16, 576, generator=g)
    if scale == "wide":
        s = s * torch.exp2(torch.randint(-20, 1, (n,), generator=g).float())
    elif scale in ("rising", "falling"):
        s = s * torch.exp2(torch.linspace(-12, 0, n) if scale == "rising" else torch.linspace(0, -12, n))
    elif scale == "zeros":
        s[::3] = 0
        s[:200] = 0
    else:  # scores and outputs of ordinary size all the same
        f = 2.0 ** 100 if scale == "large" else 2.0 ** -60
        s, q = s * f, q / f
    q = q.to(torch.bfloat16)
    ind, qo = torch.tensor([0, n], dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    for splits in (1, 0):
        dec = binding.MLADecoder(ind, "fp8_row", num_splits=splits)
        out, lse = dec(q.to(DEV), codes.to(DEV), ind.to(DEV), qo.to(DEV), kv_scale=s.to(DEV))
        assert dec.poll_error() == 0
        check(out, lse, reference(q, codes, s, [list(range(n))]))


@pytest.mark.parametrize("q_len", [2, 3, 4, 7])
@pytest.mark.parametrize("scale", [float("nan"), 2.0 ** 120, 0.0])
def test_scales_of_rows_that_a_token_does_not_see(q_len, scale):
    """The last q_len - 1 rows hold any scale: the first token's output is the same, bit for bit,
    and so is every token's that the rows behind it leave."""
    g, lens = gen(17), [300, 129, 128, 2500, q_len]
    ind = indptr_of(lens)
    codes, s = random_cache(g, sum(lens))
    q = torch.randn(len(lens) * q_len, 16, 576, generator=g).to(torch.bfloat16).to(DEV)
    qo = (torch.arange(len(lens) + 1) * q_len).to(torch.int32).to(DEV)
    dec = binding.MLADecoder(ind, "fp8_row", q_len=q_len)
    full, full_lse = (x.clone() for x in dec(q, codes.to(DEV), ind.to(DEV), qo, kv_scale=s.to(DEV)))
    for seen in range(1, q_len):  # tokens that keep every row they see
        c, x = codes.clone(), s.clone()
        for e in ind[1:].tolist():
            c[e - (q_len - seen):e] = 0 if scale != scale else 120
            x[e - (q_len - seen):e] = scale
        out, lse = dec(q, c.to(DEV), ind.to(DEV), qo, kv_scale=x.to(DEV))
        keep = torch.arange(len(lens) * q_len, device=DEV) % q_len < seen
        assert torch.equal(out[keep], full[keep]) and torch.equal(lse[keep], full_lse[keep]), seen
        if scale != scale:
            assert torch.all(torch.isnan(out[~keep].float())) and torch.all(torch.isnan(lse[~keep]))


@pytest.mark.parametrize("n,bad", [(1, 0), (300, 299), (300, 0), (900, 500)])
def test_decode_of_a_row_that_is_not_finite(n, bad):
    """A row with scale NaN in one sequence reaches that sequence's output, and no other."""
    g = gen(n)
    codes, s = random_cache(g, 2 * n)
    s[bad] = float("nan")
    q = torch.randn(2, 16, 576, generator=g).to(torch.bfloat16)
    ind, qo = torch.tensor([0, n, 2 * n], dtype=torch.int32), torch.tensor([0, 1, 2], dtype=torch.int32)
    dec = binding.MLADecoder(ind, "fp8_row")
    out, lse = dec(q.to(DEV), codes.to(DEV), ind.to(DEV), qo.to(DEV), kv_scale=s.to(DEV))
    assert torch.all(torch.isnan(out[0])) and torch.all(torch.isnan(lse[0]))
    ref = reference(q[1:], codes, s, [list(range(n, 2 * n))])
    check(out[1:], lse[1:], ref)


def test_decode_pages_at_the_far_end_of_a_long_cache():
    """Rows whose bytes lie past 2^31 and 2^32 from the cache's start."""
    rows = (1 << 32) // 576 + 5000
    page = 64
    pages = rows // page
    kv = torch.zeros(pages * page, 576, dtype=torch.uint8, device=DEV)
    scale = torch.zeros(pages * page, dtype=torch.float32, device=DEV)
    pool = cache.MLACachePool(kv, "fp8_row", page, kv_scale=scale)
    g = gen(3)
    mine = torch.tensor([pages - 1, 0, (1 << 31) // (576 * page), pages - 2], dtype=torch.int32)
    n = 3 * page + 11
    slots = (mine.repeat_interleave(page).long() * page + torch.arange(page).repeat(4))[:n]
    x = torch.randn(n, 576, generator=g).to(torch.bfloat16)
    xd = x.to(DEV)
    pool.append(xd[:, :512], xd[:, 512:], slots.to(torch.int32).to(DEV))
    codes, s = stored(x.float())
    assert torch.equal(kv[slots.to(DEV)].cpu(), codes) and torch.equal(scale[slots.to(DEV)].cpu(), s)
    q = torch.randn(1, 16, 576, generator=g).to(torch.bfloat16)
    at, last = torch.tensor([0, 4], dtype=torch.int32), torch.tensor([11], dtype=torch.int32)
    dec = binding.PagedMLADecoder(at, last, page, pages, "fp8_row")
    out, lse = dec(q.to(DEV), kv, at.to(DEV), mine.to(DEV), last.to(DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                   kv_scale=scale)
    assert dec.poll_error() == 0 and pool.poll_error() == 0
    check(out, lse, reference(q, codes, s, [list(range(n))]))


def test_decode_reports_a_bad_page():
    """A page index outside the cache: page 0 is read instead, and the error word says so."""
    codes, s = random_cache(gen(2), 256)
    at, last = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([64], dtype=torch.int32)
    q = torch.randn(1, 16, 576, generator=gen(2)).to(torch.bfloat16)
    dec = binding.PagedMLADecoder(at, last, 64, 4, "fp8_row")
    args = [last.to(DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)]
    out, lse = dec(q.to(DEV), codes.to(DEV), at.to(DEV), torch.tensor([1, 4, 2], dtype=torch.int32, device=DEV), *args,
                   kv_scale=s.to(DEV))
    assert dec.poll_error() == binding.MLA_ERR_DEVICE_INDEX
    rows = [r for p in (1, 0, 2) for r in range(64 * p, 64 * p + 64)]
    check(out, lse, reference(q, codes, s, [rows]))


@pytest.mark.parametrize("page", [16, 64, 128])
def test_decode_reports_pages_that_are_not_the_plan(page):
    """Sequences that begin elsewhere in the table than the plan says: the error word says so, or
    (pages of 128 rows: the same tiles as the plan's) the result is that of the device's table; the
    next call of the same decoder, with the plan's, is right."""
    codes, s = random_cache(gen(3), 8 * page)
    at, last = torch.tensor([0, 3, 7], dtype=torch.int32), torch.tensor([page, 5], dtype=torch.int32)
    q = torch.randn(2, 16, 576, generator=gen(3)).to(torch.bfloat16)
    dec = binding.PagedMLADecoder(at, last, page, 8, "fp8_row")
    table = torch.tensor([6, 1, 4, 0, 3, 7, 2], dtype=torch.int32)
    qo = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    moved = torch.tensor([0, 4, 7], dtype=torch.int32)
    for device_at in (moved, at):
        out, lse = dec(q.to(DEV), codes.to(DEV), device_at.to(DEV), table.to(DEV), last.to(DEV), qo, kv_scale=s.to(DEV))
        error = dec.poll_error()
        assert error == (binding.MLA_ERR_DEVICE_INDEX if page < 128 and device_at is moved else 0)
        if error == 0:
            ends = [int(device_at[1]), 7]
            spans = [[int(table[i]) * page + r for i in range(a, e) for r in range(n if i == e - 1 else page)]
                     for a, e, n in zip([0, ends[0]], ends, last.tolist())]
            check(out, lse, reference(q, codes, s, spans))


@pytest.mark.parametrize("page", [2, 16, 64])
def test_replayed_decode_follows_the_table(page):
    """A captured call, replayed after the page table, the rows and their scales have changed in
    place just before it on the same stream."""
    g, lens = gen(page), [700, 64, 1000]
    counts = [-(-n // page) for n in lens]
    at, pages = indptr_of(counts), sum(counts)
    last = torch.tensor([n - (c - 1) * page for n, c in zip(lens, counts)], dtype=torch.int32)
    q = torch.randn(3, 16, 576, generator=g).to(torch.bfloat16)
    qo = torch.arange(4, dtype=torch.int32, device=DEV)
    dec = binding.PagedMLADecoder(at, last, page, pages, "fp8_row")
    codes, s = random_cache(g, pages * page)
    kv, sc, table = codes.to(DEV), s.to(DEV), torch.zeros(pages, dtype=torch.int32, device=DEV)
    args = (q.to(DEV), kv, at.to(DEV), table, last.to(DEV), qo)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dec(*args, kv_scale=sc)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = dec(*args, kv_scale=sc)
    for turn in range(3):
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        codes, s = random_cache(g, pages * page)
        new = perm.to(DEV), codes.to(DEV), s.to(DEV)
        table.copy_(new[0]), kv.copy_(new[1]), sc.copy_(new[2])
        graph.replay()
        assert dec.poll_error() == 0
        spans = [[int(perm[int(at[b]) + r // page]) * page + r % page for r in range(n)] for b, n in enumerate(lens)]
        check(out, lse, reference(q, codes, s, spans))


def test_decode_static_and_stages_agree():
    """The entry point without a workspace, and the two stages apart, give the decode's bits."""
    lens = [700, 0, 64, 2000]
    ind = indptr_of(lens)
    codes, s = random_cache(gen(4), sum(lens))
    q = torch.randn(4, 16, 576, generator=gen(4)).to(torch.bfloat16)
    dec = binding.MLADecoder(ind, "fp8_row")
    a = [q.to(DEV), codes.to(DEV), s.to(DEV), ind.to(DEV), torch.arange(5, dtype=torch.int32, device=DEV)]
    out, lse = dec(a[0], a[1], a[3], a[4], kv_scale=a[2])
    for form in ("static", "stages"):
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        if form == "static":
            binding.mla_decode_fwd_static(*a, o, l, dec.plan, scale_stride=4)
        else:
            binding.mla_decode_split(*a, o, l, dec.plan, dec.workspace, scale_stride=4)
            binding.mla_decode_combine(o, l, dec.plan, dec.workspace)
        assert torch.equal(o, out) and torch.equal(l, lse), form


# ------------------------------------------------------------------ as used
def test_a_conversation():
    """A prompt appended, read back and decoded over, then four steps of one token each, the
    steps captured once and replayed; every step against fp64 of what the cache holds."""
    g, page, lens = gen(11), 16, [37, 150, 16]
    pool = cache.MLACachePool.allocate("fp8_row", 40, page, num_layers=2)
    rope, norm = cache.MLARope(interleaved=False), cache.MLANorm(kv_lat=True)
    tables = [pool.table(3, 24), pool.table(3, 24)]
    pool.resize(pool.table(3, 0), torch.tensor(lens, dtype=torch.int32, device=DEV), tables[0])
    qo = indptr_of(lens).to(DEV)
    slots, pos = pool.slots(tables[0], qo, sum(lens), rows=torch.empty(sum(lens), dtype=torch.int32, device=DEV))
    x = torch.randn(sum(lens), 576, generator=g).to(torch.bfloat16).to(DEV)
    for layer in range(2):
        pool.append(x[:, :512], x[:, 512:], slots, rope, pos, norm, layer=layer)
    back = pool.gather(slots, layer=1)
    codes, s = pool.kv[1].cpu(), pool.kv_scale[1].cpu()
    assert torch.equal(back.cpu(), values(codes, s)[slots.cpu().long()].float().to(torch.bfloat16))
    one = torch.arange(4, dtype=torch.int32, device=DEV)
    new_lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    xs, qs = torch.zeros(3, 576, dtype=torch.bfloat16, device=DEV), torch.zeros(3, 16, 576, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    for step in range(4):
        a, b = tables[step % 2], tables[(step + 1) % 2]
        new_lens.copy_(torch.tensor([n + step + 1 for n in lens]))
        now = [n + step + 1 for n in lens]
        counts = [-(-n // page) for n in now]
        dec = binding.PagedMLADecoder(indptr_of(counts), [n - (c - 1) * page for n, c in zip(now, counts)], page, 40, "fp8_row")
        xs.copy_(torch.randn(3, 576, generator=g))
        qs.copy_(torch.randn(3, 16, 576, generator=g))
        outs = []
        torch.cuda.synchronize()
        pool.resize(a, new_lens, b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            at, _ = pool.slots(b, one, 3, rows=pos)
            for layer in range(2):
                pool.append(xs[:, :512], xs[:, 512:], at, rope, pos, norm, layer=layer)
                outs.append(dec(qs, pool.kv[layer], *b, one, kv_scale=pool.kv_scale[layer]))
        for _ in range(2):  # the same step twice: the same rows again
            graph.replay()
        torch.cuda.synchronize()
        assert dec.poll_error() == 0 and pool.poll_error() == 0
        indptr, idx = b[0].tolist(), b[1].tolist()
        spans = [[idx[indptr[i] + r // page] * page + r % page for r in range(n)] for i, n in enumerate(now)]
        for layer in range(2):
            codes, s = pool.kv[layer].cpu(), pool.kv_scale[layer].cpu()
            check(outs[layer][0], outs[layer][1], reference(qs.cpu(), codes, s, spans))


def test_a_decoder_whose_plan_or_workspace_is_replaced():
    """A call goes by the objects that the decoder has then, not by those that it was made with."""
    codes, s = random_cache(gen(7), 900)
    q = torch.randn(2, 16, 576, generator=gen(7)).to(torch.bfloat16)
    qo = torch.tensor([0, 1, 2], dtype=torch.int32)
    dec = binding.MLADecoder([0, 300, 600], "fp8_row")
    for ind in ([0, 300, 600], [0, 1, 900], [0, 0, 130]):
        new = binding.MLADecoder(ind, "fp8_row")
        dec.plan, dec.workspace = new.plan, new.workspace
        del new
        ind = torch.tensor(ind, dtype=torch.int32)
        out, lse = dec(q.to(DEV), codes.to(DEV), ind.to(DEV), qo.to(DEV), kv_scale=s.to(DEV))
        spans = [list(range(int(a), int(e))) for a, e in zip(ind[:-1], ind[1:])]
        check(out, lse, reference(q, codes, s, spans))
        assert dec.poll_error() == 0


def test_another_stream():
    codes, s = random_cache(gen(6), 500)
    ind, qo = torch.tensor([0, 500], dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    q = torch.randn(1, 16, 576, generator=gen(6)).to(torch.bfloat16)
    dec = binding.MLADecoder(ind, "fp8_row")
    args = [q.to(DEV), codes.to(DEV), ind.to(DEV), qo.to(DEV)]
    sd = s.to(DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = dec(*args, kv_scale=sd, stream=side)
    side.synchronize()
    check(out, lse, reference(q, codes, s, [list(range(500))]))


def test_python_refusals():
    kv = torch.zeros(64, 576, dtype=torch.uint8, device=DEV)
    for bad in (None, torch.ones(1, device=DEV), torch.ones(64, dtype=torch.float64, device=DEV), torch.ones(64),
                torch.ones(64, 1, device=DEV)):
        with pytest.raises(ValueError):
            cache.MLACachePool(kv, "fp8_row", 16, kv_scale=bad)
    for bad in (torch.ones(65, device=DEV)[1:], torch.ones(1, device=DEV).expand(64)):  # alignment, one scale for all rows
        with pytest.raises(binding.MLAError):
            cache.MLACachePool(kv, "fp8_row", 16, kv_scale=bad)
    dec = binding.MLADecoder([0, 64], "fp8_row")
    q, ind = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device=DEV), torch.tensor([0, 64], dtype=torch.int32, device=DEV)
    for bad in (torch.ones(64, 1, device=DEV), torch.ones(64, dtype=torch.bfloat16, device=DEV), torch.ones(63, device=DEV)):
        with pytest.raises(ValueError):
            dec(q, kv, ind, ind, kv_scale=bad)
    for bad in (None, torch.ones(1, device=DEV).expand(64)):
        with pytest.raises(binding.MLAError):
            dec(q, kv, ind, ind, kv_scale=bad)
