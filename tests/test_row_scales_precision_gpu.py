"""What the row-scaled decode keeps of weights and scales that lie far apart, against fp64.

With w_t the exact softmax weights of a token and head, s_t the rows' scales, u_t = w_t s_t
and U the largest u_t of a block of 32 rows, the tolerance of an output sum_t u_t code_t is
  * its rounding to bf16                                     2^-8 |out|
  * a weight times its row's scale enters P.V as two e4m3 terms that keep 4 bits each, under
    a power of two that leaves the block's largest at 2^7 or more and the second term 2^5
    up: half of the smallest step, 2^-10, is 2^-22 of U      max(2^-8 u_t, 2^-22 U) |code_t|
  * n rows take n / 32 accumulations in fp32, each off by at most 2^-23 of the sum of
    magnitudes; the exponentials and the sum of the weights  (n 2^-28 + 2^-16) u_t |code_t|
  * the query enters the scores as two e4m3 terms under a power of two (the largest that leaves
    its magnitude at 448 or less; half of it is allowed too, so twice the error): with e_c
    what they leave of column c, row t's score moves by at most d_t = 2 / 24 sum_c e_c |k_tc|
    and its weight by d_t + sum_r w_r d_r of itself (twice that: second order)
and of the log of the sum sum_r w_r d_r, 2^-22 of its size and 2e-5."""
import pytest
import torch

from mla_attention_decode_gb300 import binding, build
from test_row_scales_gpu import indptr_of, stored, values

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def reference(q, codes, scales, rows):
    """One token's 16 heads over cache rows `rows`: out, lse and their tolerances."""
    code = codes[rows].view(torch.float8_e4m3fn).double()
    s = scales[rows].double()
    k, qq = code * s.unsqueeze(1), q.double()
    a = qq @ k.T / 24
    l = torch.logsumexp(a, -1)
    w = torch.softmax(a, -1)  # (not exp(a - l): where scores pass 2^53, l has no room for the log of a sum)
    x = qq * torch.exp2(torch.floor(torch.log2(448 / qq.abs().amax(-1, keepdim=True))))
    hi = x.to(torch.float8_e4m3fn).double()
    left = (x - hi - (x - hi).to(torch.float8_e4m3fn).double()).abs() * (qq.abs().amax(-1, keepdim=True) / x.abs().amax(-1, keepdim=True))
    d = 2 / 24 * (left @ k.abs().T)
    mean = (w * d).sum(-1, keepdim=True)
    u = w * s
    out = u @ code[:, :512]
    top = torch.nn.functional.pad(u, (0, -len(rows) % 32)).view(16, -1, 32).amax(-1).repeat_interleave(32, 1)[:, :len(rows)]
    t = torch.maximum(2.0 ** -8 * u, 2.0 ** -22 * top) + u * (len(rows) * 2.0 ** -28 + 2.0 ** -16)
    t = t + 2 * torch.where(w > 0, u * (d + mean), 0.0)
    return out, l, 2.0 ** -8 * out.abs() + t @ code[:, :512].abs(), mean.squeeze(1) + 2.0 ** -22 * l.abs() + 2e-5


def check(path, q, codes, s, lens):
    """Each sequence one unit, over the layout that `path` names: ("rows", tokens) or ("pages", rows a page)."""
    kind, n = path
    q_len = n if kind == "rows" else 1
    qo = (torch.arange(len(lens) + 1) * q_len).to(torch.int32).to(DEV)
    start = [0] + torch.tensor(lens).cumsum(0).tolist()
    if kind == "rows":
        ind = indptr_of(lens)
        dec = binding.MLADecoder(ind, "fp8_row", num_splits=1, q_len=q_len)
        out, lse = dec(q.to(DEV), codes.to(DEV), ind.to(DEV), qo, kv_scale=s.to(DEV))
    else:
        counts = [-(-x // n) for x in lens]
        at, pages = indptr_of(counts), sum(counts)
        perm = torch.randperm(pages, generator=torch.Generator("cpu").manual_seed(n))
        kv, sc = torch.zeros(pages * n, 576, dtype=torch.uint8), torch.zeros(pages * n)
        for b, x in enumerate(lens):
            r = torch.arange(x)
            to = perm[int(at[b]) + r // n] * n + r % n
            kv[to], sc[to] = codes[start[b]:start[b] + x], s[start[b]:start[b] + x]
        last = torch.tensor([x - (c - 1) * n for x, c in zip(lens, counts)], dtype=torch.int32)
        dec = binding.PagedMLADecoder(at, last, n, pages, "fp8_row", num_splits=1)
        out, lse = dec(q.to(DEV), kv.to(DEV), at.to(DEV), perm.to(torch.int32).to(DEV), last.to(DEV), qo, kv_scale=sc.to(DEV))
    assert dec.poll_error() == 0
    out, lse = out.double().cpu(), lse.double().cpu()
    for b, x in enumerate(lens):
        for i in range(q_len):
            ref, l, t, tl = reference(q[b * q_len + i], codes, s, torch.arange(start[b], start[b] + x - (q_len - 1 - i)))
            err, size = (out[b * q_len + i] - ref).abs(), ref.abs().amax(-1, keepdim=True)
            assert torch.all(err <= t), f"sequence {b}, token {i}: off by {float((err / size).max()):.2e} of the largest output"
            assert torch.all((lse[b * q_len + i] - l).abs() <= tl)


PATHS = [("rows", 1), ("rows", 2), ("rows", 3), ("pages", 1), ("pages", 16), ("pages", 64)]


@pytest.mark.parametrize("path", PATHS, ids=lambda p: f"{p[0]}{p[1]}")
@pytest.mark.parametrize("k", [6, 12, 16, 20, 60])
def test_rows_of_large_scale_without_weight(path, k):
    """Every 50th row (the first or the last among them) is 2^k times as large as the others; for half of the
    heads its score is so low that it has no weight, for the other half it has all of it."""
    g, q_len = torch.Generator("cpu").manual_seed(k), path[1] if path[0] == "rows" else 1
    lens = [700, 651, 1501]
    y = torch.randn(sum(lens), 576, generator=g) * 2.0 ** -k
    y[:, :512] = (y[:, :512] / 2 + 2.0 ** -k)
    y[:, 575] = 0
    at = torch.cat([torch.arange(0, 700, 50), torch.arange(700, 1351, 50), torch.arange(1351, 2852, 50)])
    y[at] = 0
    y[at, :512] = 0.25 * torch.randn(at.numel(), 512, generator=g)
    y[at, 575] = -24
    codes, s = stored(y)
    q = torch.zeros(3 * q_len, 16, 576)
    q[..., 512:575] = 3 * 2.0 ** k * torch.randn(3 * q_len, 16, 63, generator=g)
    q[:, ::2, 575], q[:, 1::2, 575] = 8 * 2.0 ** k, -8 * 2.0 ** k
    check(path, q.to(torch.bfloat16), codes, s, lens)


@pytest.mark.parametrize("path", PATHS, ids=lambda p: f"{p[0]}{p[1]}")
@pytest.mark.parametrize("n,spread", [(8192, 0), (8192, 1), (32768, 0), (32768, 1)])
@pytest.mark.parametrize("gap", [9, 11, 12, 13, 15])
def test_one_row_far_above_a_long_tail(path, n, spread, gap):
    """A row whose score lies `gap` nats above the others' (the first row, one among them, one near the
    end): together they weigh as much as it does, or nearly, one by one next to nothing."""
    g, q_len = torch.Generator("cpu").manual_seed(n + gap), path[1] if path[0] == "rows" else 1
    lens = [n, 1000, n - 77]
    total = sum(lens)
    f = torch.exp(0.3 * torch.randn(total, 1, generator=g))  # the rows' sizes
    y = torch.cat([f * (1 + 0.5 * torch.randn(total, 512, generator=g)), torch.randn(total, 64, generator=g)], 1)
    y[:, 575] = 0
    at = torch.tensor([0, n + 517, total - 20])
    y[at, :512] -= 2 * f[at]
    y[at, 575] = 0.375 * gap
    codes, s = stored(y)
    q = torch.zeros(3 * q_len, 16, 576)
    q[..., 512:575] = spread * 24 / 63 ** 0.5 * torch.randn(3 * q_len, 16, 63, generator=g)
    q[..., 575] = 64
    check(path, q.to(torch.bfloat16), codes, s, lens)


@pytest.mark.parametrize("q_len", [1, 2])
def test_a_scale_of_minus_zero_is_zero(q_len):
    g = torch.Generator("cpu").manual_seed(3)
    codes, s = stored(torch.randn(700, 576, generator=g))
    s[::7] = 0
    q = torch.randn(2 * q_len, 16, 576, generator=g).to(torch.bfloat16).to(DEV)
    ind, qo = indptr_of([300, 400]).to(DEV), (torch.arange(3) * q_len).to(torch.int32).to(DEV)
    dec = binding.MLADecoder(ind.cpu(), "fp8_row", q_len=q_len)
    want = [t.clone() for t in dec(q, codes.to(DEV), ind, qo, kv_scale=s.to(DEV))]
    s[::7] = -0.0
    got = dec(q, codes.to(DEV), ind, qo, kv_scale=s.to(DEV))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.all(torch.isfinite(got[0]))


@pytest.mark.parametrize("path", PATHS, ids=lambda p: f"{p[0]}{p[1]}")
def test_scores_that_rise_far_from_tile_to_tile(path):
    """Each sequence's scores rise by 12 nats over every 200 rows (the reference rises and what was summed is
    rescaled, again and again), and then fall as far."""
    g, q_len = torch.Generator("cpu").manual_seed(5), path[1] if path[0] == "rows" else 1
    lens = [2600, 700, 1500]
    total = sum(lens)
    y = torch.cat([1 + 0.5 * torch.randn(total, 512, generator=g), torch.randn(total, 64, generator=g)], 1)
    at = torch.cat([torch.arange(n).float() for n in lens])
    half = torch.cat([torch.full((n,), n / 2) for n in lens])
    y[:, 575] = 12 * (half - (at - half).abs()) / 200 * 24 / 512
    codes, s = stored(y)
    q = torch.zeros(3 * q_len, 16, 576)
    q[..., 512:575] = torch.randn(3 * q_len, 16, 63, generator=g)
    q[..., 575] = 512
    check(path, q.to(torch.bfloat16), codes, s, lens)
