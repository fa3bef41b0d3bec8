"""Attention of a prompt on the GPU against fp64.

Tolerances, per output of token i, head h and column c, with w_j the exact weights:
  * the output's rounding to bf16                    2^-8 |out|
  * a weight enters the product with v as bf16       2^-8 sum_j w_j |v_j|
  * fp32 sums of 192 products (each at most 24 roundings of 2^-24 deep or one after
    the other: 192 2^-24 of the sum of magnitudes M_j), the scaled subtraction and
    the exponential (2^-22, and 2^-23 of the largest score in log2 units): a weight
    moves by d = 2 (192 2^-24 max_j M_j + 2^-21 + 2^-22 max_j |s_j|) of itself, and so
    does the sum that it is divided by; sums of up to n weights: n 2^-24 of themselves
and of the log of the sum half of that, 2^-23 of its size and 2^-21 for the logarithm."""
import ctypes
import math

import pytest
import torch

from mla_attention_decode_gb300 import binding, build, cache, prompt

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
SM = 1 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def indptr(lens, first=0):
    return torch.tensor([first] + lens).cumsum(0).to(torch.int32)


def inputs(g, tq, tk, heads, layout="fused"):
    """fused: columns of wider projections, as they come in use; plain: contiguous; heads: heads before tokens."""
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    if layout == "fused":
        qb, q, kvb, rows = r(tq, heads, 192), r(tq, heads, 576), r(tk, heads, 256), r(tk, 576)
        return dict(q_nope=qb.to(DEV)[..., :128], q_pe=q.to(DEV)[..., 512:], k_nope=kvb.to(DEV)[..., :128],
                    k_pe=rows.to(DEV)[:, 512:], v=kvb.to(DEV)[..., 128:])
    if layout == "plain":
        return dict(q_nope=r(tq, heads, 128).to(DEV), q_pe=r(tq, heads, 64).to(DEV), k_nope=r(tk, heads, 128).to(DEV),
                    k_pe=r(tk, 64).to(DEV), v=r(tk, heads, 128).to(DEV))
    return dict(q_nope=r(heads, tq, 128).to(DEV).transpose(0, 1), q_pe=r(heads, tq, 64).to(DEV).transpose(0, 1),
                k_nope=r(heads, tk, 128).to(DEV).transpose(0, 1), k_pe=r(tk, 72).to(DEV)[:, 8:],
                v=r(heads, tk, 128).to(DEV).transpose(0, 1))


def reference(x, qo, kv, causal=True, prefix=None, sm=SM):
    """out, lse and their tolerances in fp64 (on the GPU, by plain products); rows of no document: NaN."""
    tq, heads = x["q_nope"].shape[:2]
    out = torch.full((tq, heads, 128), math.nan, dtype=torch.float64, device=DEV)
    lse = torch.full((tq, heads), math.nan, dtype=torch.float64, device=DEV)
    tol, tol_lse = out.clone(), lse.clone()
    d = {k: t.double() for k, t in x.items()}
    for b in range(len(qo) - 1):
        qs, ks = slice(int(qo[b]), int(qo[b + 1])), slice(int(kv[b]), int(kv[b + 1]))
        n, m = qs.stop - qs.start, ks.stop - ks.start
        i, j = torch.arange(n, device=DEV).view(n, 1), torch.arange(m, device=DEV).view(1, m)
        seen = torch.ones(n, m, dtype=torch.bool, device=DEV)
        if causal:
            seen = (j <= m - n + i) | (j < (0 if prefix is None else int(prefix[b])))
        for h in range(heads):
            a = d["q_nope"][qs, h] @ d["k_nope"][ks, h].T + d["q_pe"][qs, h] @ d["k_pe"][ks].T
            big = d["q_nope"][qs, h].abs() @ d["k_nope"][ks, h].abs().T + d["q_pe"][qs, h].abs() @ d["k_pe"][ks].abs().T
            s = torch.where(seen, a * sm, -math.inf)
            l = torch.logsumexp(s, 1) if m else torch.full((n,), -math.inf, device=DEV, dtype=torch.float64)
            w = torch.exp(s - torch.where(torch.isinf(l), 0.0, l).unsqueeze(1))
            v = d["v"][ks, h]
            out[qs, h], lse[qs, h] = w @ v, l
            top = torch.where(seen, s.abs(), 0.0).amax(1) if m else torch.zeros(n, device=DEV)
            mag = torch.where(seen, big, 0.0).amax(1) * sm if m else torch.zeros(n, device=DEV)
            dd = 2 * (192 * 2.0 ** -24 * mag + 2.0 ** -21 + 2.0 ** -22 * top * 1.4427) + m * 2.0 ** -24
            tol[qs, h] = 2.0 ** -8 * out[qs, h].abs() + (2.0 ** -8 + 2 * dd).unsqueeze(1) * (w @ v.abs())
            tol_lse[qs, h] = dd + 2.0 ** -23 * torch.where(torch.isinf(l), 0.0, l).abs() + 2.0 ** -21
    return out, lse, tol, tol_lse


def check(got, lse, ref):
    out, l, t, tl = ref
    own = ~torch.isnan(l)
    err = (got.double() - out).abs()[own.unsqueeze(-1).expand_as(out)]
    bound = t[own.unsqueeze(-1).expand_as(out)]
    assert torch.all(err <= bound), f"{float((err - bound).max())} over the bound, largest error {float(err.max())}"
    inf = torch.isinf(l)
    assert torch.equal(torch.isinf(lse) & (lse < 0) & own, inf)
    fin = own & ~inf
    assert torch.all((lse.double() - l).abs()[fin] <= tl[fin]), float((lse.double() - l).abs()[fin].max())


def run(x, qo, kv, causal=True, prefix=None, sm=SM, **kw):
    p = prompt.MLAPrompt(x["q_nope"].shape[0], x["k_nope"].shape[0], len(qo) - 1, heads=x["q_nope"].shape[1], causal=causal,
                         sm_scale=sm)
    pf = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV)
    out, lse = p(**x, qo_indptr=qo.to(DEV), kv_indptr=kv.to(DEV), prefix=pf, **kw)
    assert p.poll_error() == 0
    return out, lse


@pytest.mark.parametrize("n", [1, 2, 17, 127, 128, 129, 200, 255, 256, 257, 511, 700])
@pytest.mark.parametrize("context", [0, 1, 300])
def test_lengths(n, context):
    """One document, causal, its tokens after a context."""
    x = inputs(gen(n + context), n, n + context, 2)
    qo, kv = indptr([n]), indptr([n + context])
    check(*run(x, qo, kv), reference(x, qo, kv))


@pytest.mark.parametrize("layout", ["fused", "plain", "heads"])
@pytest.mark.parametrize("mask", ["causal", "prefix", "full"])
@pytest.mark.parametrize("heads", [1, 3, 16])
def test_documents(layout, mask, heads):
    """Documents of many lengths side by side, empty ones and ones with more tokens than keys among them."""
    nq, nk = [5, 0, 300, 129, 1, 64, 260], [5, 7, 300, 640, 0, 40, 1300]
    x = inputs(gen(heads), sum(nq), sum(nk), heads, layout)
    qo, kv = indptr(nq), indptr(nk)
    prefix = [0, 9, 100, 640, 3, -4, 999] if mask == "prefix" else None
    out, lse = run(x, qo, kv, mask != "full", prefix)
    check(out, lse, reference(x, qo, kv, mask != "full", prefix))


@pytest.mark.parametrize("nq,nk", [(300, 100), (300, 172), (130, 1), (513, 129), (256, 128)])
def test_more_tokens_than_keys(nq, nk):
    """The first tokens see nothing: whole query tiles without a key tile."""
    x = inputs(gen(nq), nq, nk, 2)
    qo, kv = indptr([nq]), indptr([nk])
    check(*run(x, qo, kv), reference(x, qo, kv))
    check(*run(x, qo, kv, prefix=[nk // 2]), reference(x, qo, kv, prefix=[nk // 2]))


def test_128_heads():
    x = inputs(gen(128), 150, 200, 128)
    qo, kv = indptr([100, 50]), indptr([120, 80])
    check(*run(x, qo, kv), reference(x, qo, kv))


@pytest.mark.parametrize("nk", [1, 63, 127, 128, 129, 384, 1025])
def test_every_key_seen(nk):
    x = inputs(gen(nk), 300, nk, 2)
    qo, kv = indptr([300]), indptr([nk])
    check(*run(x, qo, kv, causal=False), reference(x, qo, kv, causal=False))


def test_many_short_documents():
    g = gen(4)
    nq = torch.randint(0, 6, (1500,), generator=g).tolist()
    nk = [n + int(c) for n, c in zip(nq, torch.randint(0, 9, (1500,), generator=g))]
    x = inputs(g, sum(nq), sum(nk), 1)
    qo, kv = indptr(nq), indptr(nk)
    check(*run(x, qo, kv), reference(x, qo, kv))


def test_rows_of_no_document_stay():
    """Tokens before the first document and behind the last keep what out and lse held; strided out."""
    x = inputs(gen(1), 400, 500, 2)
    qo, kv = torch.tensor([30, 140, 350], dtype=torch.int32), torch.tensor([7, 200, 480], dtype=torch.int32)
    wide = torch.full((400, 2, 264), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((400, 2), 7.0, device=DEV)
    out, _ = run(x, qo, kv, out=wide[..., 8:136], lse=lse)
    check(out, lse, reference(x, qo, kv))
    for t in (out, lse):
        assert torch.all(t[:30] == 7.0) and torch.all(t[350:] == 7.0)
    assert torch.all(wide[..., :8] == 7.0) and torch.all(wide[..., 136:] == 7.0)


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
def test_what_lies_outside_a_document_does_not_reach_it(poison):
    """Keys, values and queries of no document are NaN or infinite; so are the keys (not the
    values) that the causal order hides from all tokens but the last."""
    nq, nk = [100, 130], [100, 250]
    x = inputs(gen(2), 300, 500, 2, "plain")
    qo, kv = torch.tensor([20, 120, 250], dtype=torch.int32), torch.tensor([10, 110, 360], dtype=torch.int32)
    for k in ("q_nope", "q_pe"):
        x[k][:20] = poison
        x[k][250:] = poison
    for k in ("k_nope", "k_pe", "v"):
        x[k][:10] = poison
        x[k][360:] = poison
    clean = {k: torch.nan_to_num(t, 0.0, 0.0, 0.0) for k, t in x.items()}
    ref = reference(clean, qo, kv)
    check(*run(x, qo, kv), ref)
    x["k_nope"][109] = poison
    x["k_pe"][359] = poison
    out, lse = run(x, qo, kv)
    for t in [*ref]:  # the last token of each document sees the poison
        t[119] = t[249] = math.nan
    check(out, lse, ref)
    if math.isnan(poison):
        assert torch.all(torch.isnan(out[[119, 249]])) and torch.all(torch.isnan(lse[[119, 249]]))


@pytest.mark.parametrize("kind", ["peaked", "rising", "falling", "flat", "scaled"])
def test_scores_of_all_sizes(kind):
    """Maxima that rise over the key tiles (what was summed is rescaled), fall, dominate or vanish."""
    n, m = 260, 900
    x = inputs(gen(3), n, m, 2, "plain")
    sm = SM
    if kind == "peaked":
        x["q_nope"] = (x["q_nope"].float() * 30).to(torch.bfloat16)
    elif kind in ("rising", "falling"):
        f = torch.linspace(0, 60, m, device=DEV)
        f = f if kind == "rising" else f.flip(0)
        x["q_pe"][..., 0], x["k_pe"][:, 0] = 8.0, f.to(torch.bfloat16)
    elif kind == "flat":
        x["q_nope"] = torch.zeros_like(x["q_nope"])
        x["q_pe"] = torch.zeros_like(x["q_pe"])
    else:
        sm = 1e-3
    qo, kv = indptr([n]), indptr([m])
    for causal in (True, False):
        check(*run(x, qo, kv, causal, sm=sm), reference(x, qo, kv, causal, sm=sm))


@pytest.mark.parametrize("tq,tk", [(1, 0), (300, 0), (0, 5), (0, 0)])
def test_nothing_to_see(tq, tk):
    x = inputs(gen(1), tq, tk, 2, "plain")
    out, lse = run(x, indptr([tq]), indptr([tk]))
    assert out.shape == (tq, 2, 128) and torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("qo,kv", [([0, 50, 40, 90], [0, 50, 60, 90]), ([0, 50, 60, 101], [0, 50, 60, 90]),
                                   ([-1, 50, 60, 90], [0, 50, 60, 90]), ([0, 50, 60, 90], [0, 50, 40, 90]),
                                   ([0, 50, 60, 90], [0, 50, 60, 101]), ([0, 50, 60, 90], [-5, 50, 60, 90]),
                                   ([0, 1 << 30, 60, 90], [0, 50, 60, 90])])
def test_bounds_that_do_not_fit_are_reported(qo, kv):
    """The error word says so, the documents whose bounds fit are computed or left, nothing else is touched."""
    x = inputs(gen(1), 100, 100, 2, "plain")
    p = prompt.MLAPrompt(100, 100, 3, heads=2)
    out, lse = torch.full((100, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((100, 2), 7.0, device=DEV)
    a, b = torch.tensor(qo, dtype=torch.int32, device=DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
    p(**x, qo_indptr=a, kv_indptr=b, out=out, lse=lse)
    assert p.poll_error() == binding.MLA_ERR_DEVICE_INDEX and p.poll_error() == 0
    good = [d for d in range(3) if 0 <= qo[d] <= qo[d + 1] <= 100 and 0 <= kv[d] <= kv[d + 1] <= 100]
    fits = torch.zeros(100, dtype=torch.bool, device=DEV)
    for d in good:
        fits[qo[d]:qo[d + 1]] = True
    assert torch.all(out[~fits] == 7.0) and torch.all(lse[~fits] == 7.0)
    p(**x, qo_indptr=indptr([50, 10, 30]).to(DEV), kv_indptr=indptr([50, 10, 30]).to(DEV))
    assert p.poll_error() == 0


def test_same_bits_again_and_from_a_graph():
    """Replays of one captured call over other inputs and other bounds: the bits of plain calls; two graphs
    that share a workspace, and a call on another stream."""
    g = gen(8)
    sets = [inputs(g, 700, 900, 4, "plain") for _ in range(2)]
    bounds = [(indptr([300, 400]), indptr([500, 400])), (indptr([1, 650]), indptr([40, 700]))]
    p = prompt.MLAPrompt(700, 900, 2, heads=4)
    want = []
    for x, (qo, kv) in zip(sets, bounds):
        o, l = torch.zeros(700, 4, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(700, 4, device=DEV)
        p(**x, qo_indptr=qo.to(DEV), kv_indptr=kv.to(DEV), out=o, lse=l)
        want.append((o, l))
    live = {k: t.clone() for k, t in sets[0].items()}
    qo, kv = bounds[0][0].to(DEV), bounds[0][1].to(DEV)
    outs = [(torch.zeros(700, 4, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(700, 4, device=DEV)) for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for o, l in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            p(**live, qo_indptr=qo, kv_indptr=kv, out=o, lse=l)
    for k in (1, 0, 1):
        for n, t in sets[k].items():
            live[n].copy_(t)
        qo.copy_(bounds[k][0])
        kv.copy_(bounds[k][1])
        for (o, l), graph in zip(outs, graphs):
            o.zero_(), l.zero_()
            graph.replay()
        for o, l in outs:
            assert torch.equal(o, want[k][0]) and torch.equal(l, want[k][1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, l = torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])
    torch.cuda.synchronize()
    p(**sets[0], qo_indptr=bounds[0][0].to(DEV), kv_indptr=bounds[0][1].to(DEV), out=o, lse=l, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(l, want[0][1])
    assert p.poll_error() == 0


def test_a_prompt_in_chunks_over_the_cache():
    """A prompt in three chunks, each appended to a row-scaled cache, its context read back and up-projected,
    and the chunk attended: against fp64 of the same keys and values; then one more token by the decode, whose
    absorbed form over the same rows gives the same attention."""
    g, heads, page, total = gen(21), 16, 16, 700
    pool = cache.MLACachePool.allocate("fp8_row", 60, page)
    rope, norm = cache.MLARope(interleaved=True), cache.MLANorm(kv_lat=True)
    w = (torch.randn(512, heads * 256, generator=g) / 22).to(torch.bfloat16).to(DEV)
    kv_a = torch.randn(total, 576, generator=g).to(torch.bfloat16).to(DEV)
    qb = torch.randn(total, heads, 192, generator=g).to(torch.bfloat16).to(DEV)
    q = torch.zeros(total, heads, 576, dtype=torch.bfloat16, device=DEV)
    tables = [pool.table(1, 60), pool.table(1, 60)]
    done = 0
    for step, n in enumerate((257, 300, 143)):
        a, b = tables[step % 2], tables[(step + 1) % 2]
        end = done + n
        pool.resize(a, torch.tensor([end], dtype=torch.int32, device=DEV), b)
        new = slice(done, end)
        ind = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        slots, pos = pool.slots(b, ind, n, rows=torch.empty(n, dtype=torch.int32, device=DEV))
        pool.append(kv_a[new, :512], kv_a[new, 512:], slots, rope, pos, norm, q_pe=qb[new, :, 128:], q_out=q[new])
        context = torch.tensor([0, end], dtype=torch.int32, device=DEV)
        rows = pool.gather(pool.slots(b, context, end)[0])
        kv_b = (rows[:, :512] @ w).view(end, heads, 256)
        x = dict(q_nope=qb[new, :, :128], q_pe=q[new, :, 512:], k_nope=kv_b[..., :128], k_pe=rows[:, 512:], v=kv_b[..., 128:])
        out, lse = run(x, ind.cpu(), context.cpu())
        check(out, lse, reference(x, ind.cpu(), context.cpu()))
        done = end
    assert pool.poll_error() == 0
    # the last token again, absorbed: q_nope W_uk over the latent columns, and the output up-projected.  The prompt's
    # keys and values are bf16 products (2^-8 of each of 128 terms of a score, random signs, and of each value); the
    # decode's query is rounded to bf16 and its rows are the codes themselves.
    wk = w.view(512, heads, 256)
    q1 = torch.zeros(1, heads, 576, dtype=torch.bfloat16, device=DEV)
    q1[0, :, :512] = torch.einsum("hd,chd->hc", qb[-1, :, :128].float(), wk[..., :128].float()).to(torch.bfloat16)
    q1[0, :, 512:] = q[-1, :, 512:]
    dec = binding.PagedMLADecoder([0, -(-total // page)], [total - (-(-total // page) - 1) * page], page, 60, "fp8_row")
    table = tables[1]
    o, l = dec(q1, pool.kv[0], *table, torch.tensor([0, 1], dtype=torch.int32, device=DEV), kv_scale=pool.kv_scale[0], sm_scale=SM)
    assert dec.poll_error() == 0
    up = torch.einsum("hc,chd->hd", o[0].float(), wk[..., 128:].float())
    assert torch.all((l[0] - lse[-1]).abs() <= 0.02)
    assert torch.linalg.norm(up - out[-1].float()) <= 0.02 * torch.linalg.norm(up)


def test_an_object_is_made_for_a_cuda_device():
    with pytest.raises(ValueError):
        prompt.MLAPrompt(1, 1, 1, device="cpu")


def test_python_refusals():
    x = inputs(gen(1), 10, 12, 2, "plain")
    qo, kv = indptr([10]).to(DEV), indptr([12]).to(DEV)
    p = prompt.MLAPrompt(10, 12, 1, heads=2)
    ok = dict(**x, qo_indptr=qo, kv_indptr=kv)
    p(**ok)
    for k, bad in (("q_nope", x["q_nope"].float()), ("q_pe", x["q_pe"][..., :32]), ("k_nope", x["k_nope"].cpu()),
                   ("v", x["v"][:11]), ("k_pe", x["k_pe"].view(12, 64).t().contiguous().t()), ("qo_indptr", qo.long()),
                   ("kv_indptr", kv[:1]), ("prefix", torch.zeros(2, dtype=torch.int32, device=DEV)),
                   ("out", torch.zeros(10, 2, 128, device=DEV)), ("lse", torch.zeros(10, 2, dtype=torch.bfloat16, device=DEV)),
                   ("lse", torch.zeros(2, 10, device=DEV).t())):
        with pytest.raises(ValueError):
            p(**{**ok, k: bad})
    with pytest.raises(ValueError):
        prompt.MLAPrompt(9, 12, 1, heads=2)(**ok)
    odd = torch.zeros(10, 2, 132, dtype=torch.bfloat16, device=DEV)
    for k, bad in (("q_nope", odd[..., :128]), ("q_nope", odd[..., 4:]), ("out", odd[..., :128]),
                   ("v", torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV).expand(12, 2, 128))):
        with pytest.raises(binding.MLAError):
            p(**{**ok, k: bad})


@pytest.mark.parametrize("n,context", [(1, 0), (1, 12000), (17, 5000), (130, 4000), (256, 1100), (300, 2500)])
@pytest.mark.parametrize("heads", [1, 16])
def test_few_tokens_after_a_long_context(n, context, heads):
    """The keys dealt to several CTAs and their results joined."""
    x = inputs(gen(n + heads), n, n + context, heads)
    qo, kv = indptr([n]), indptr([n + context])
    check(*run(x, qo, kv), reference(x, qo, kv))


@pytest.mark.parametrize("mask", ["causal", "prefix", "full"])
def test_uneven_documents_share_the_split(mask):
    """Documents far shorter than the average that decides the split: shares without a key tile, documents without
    keys; rows of no document stay."""
    nq, nk = [3, 0, 5, 1, 40], [6003, 30, 5, 1, 3500]
    x = inputs(gen(5), sum(nq) + 9, sum(nk) + 50, 2)
    qo, kv = indptr(nq, 4), indptr(nk, 11)
    prefix = [6000, 9, 2, 0, 10000] if mask == "prefix" else None
    out, lse = torch.full((x["q_nope"].shape[0], 2, 128), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((x["q_nope"].shape[0], 2), 7.0, device=DEV)
    run(x, qo, kv, mask != "full", prefix, out=out, lse=lse)
    check(out, lse, reference(x, qo, kv, mask != "full", prefix))
    for t in (out, lse):
        assert torch.all(t[:4] == 7.0) and torch.all(t[4 + sum(nq):] == 7.0)


def test_split_and_unsplit_calls():
    """An object made for more rows gives the bits of one made for these, and so does the C entry point; a NaN in
    one share reaches its rows' results; bounds that do not fit."""
    n, m = 20, 6000
    x = inputs(gen(6), n, m, 2)
    qo, kv = indptr([n]), indptr([m])
    ref = reference(x, qo, kv)
    args = dict(**x, qo_indptr=qo.to(DEV), kv_indptr=kv.to(DEV))
    a, b = prompt.MLAPrompt(n, m, 1, heads=2), prompt.MLAPrompt(5 * n, 2 * m, 9, heads=2)
    o1, l1 = a(**args)
    o2, l2 = b(**args)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    check(o1, l1, ref)
    lib, o3, l3 = prompt.load_library(), torch.zeros_like(o1), torch.zeros_like(l1)
    s = [x[k].stride(i) for k, d in (("q_nope", 2), ("q_pe", 2), ("k_nope", 2), ("k_pe", 1), ("v", 2)) for i in range(d)]
    p = [x[k].data_ptr() for k in ("q_nope", "q_pe", "k_nope", "k_pe", "v")]
    ws = torch.zeros(a.workspace.numel(), dtype=torch.uint8, device=DEV)
    g = prompt.mla_prompt_args(*p, args["qo_indptr"].data_ptr(), args["kv_indptr"].data_ptr(), None, o3.data_ptr(), l3.data_ptr(),
                               *s, 256, 128, n, m, 1, 2, 1, SM)
    torch.cuda.synchronize()
    need = int(lib.mla_prompt_workspace_bytes(ctypes.addressof(g)))
    assert need == a.workspace.numel()
    assert lib.mla_prompt_fwd(ctypes.addressof(g), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(o3, o1) and torch.equal(l3, l1)
    x["k_nope"][3000] = math.nan  # every token sees it
    o, l = a(**args)
    assert torch.all(torch.isnan(o)) and torch.all(torch.isnan(l))
    o.fill_(7.0), l.fill_(7.0)
    a(**{**args, "kv_indptr": torch.tensor([0, m + 1], dtype=torch.int32, device=DEV)}, out=o, lse=l)
    assert a.poll_error() == binding.MLA_ERR_DEVICE_INDEX and torch.all(o == 7.0) and torch.all(l == 7.0)
