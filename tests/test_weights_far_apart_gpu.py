"""A long tail of rows that one by one weigh next to nothing under one row far above them, in the caches
without a scale per row, against fp64; each sequence one unit.  Tolerances of e4m3 as in
test_row_scales_precision_gpu, the weights alone in place of their products with scales.  Of MXFP4 the same
but for what a weight loses: a row's largest block scale 2^G (of its 18 blocks; with block-scaled
scores, whose rows are laid out by them, of the 16 of the values) enters its weight and its values
are relative to it; both terms are relative to the unit's largest weight times the largest 2^G, 16
or more in e4m3, and the second is 2^4 up: half of the smallest step, 2^-10, is 2^-18 of that."""
import pytest
import torch

from mla_attention_decode_gb300 import binding, build, synth
from test_row_scales_gpu import indptr_of
from test_row_scales_precision_gpu import PATHS, reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def sink(n, spread, gap, q_len):
    """Three sequences of n, 1000 and n - 77 rows; in each one row whose score lies `gap` nats above the others',
    which spread by `spread`: fp32 rows and queries."""
    g = torch.Generator("cpu").manual_seed(int(n + gap))
    lens = [n, 1000, n - 77]
    total = sum(lens)
    y = torch.cat([1 + 0.5 * torch.randn(total, 512, generator=g), torch.randn(total, 64, generator=g)], 1)
    y[:, 575] = 0
    at = torch.tensor([0, n + 517, total - 20])
    y[at, :512] -= 2
    y[at, 575] = 0.375 * gap
    q = torch.zeros(3 * q_len, 16, 576)
    q[..., 512:575] = spread * 24 / 63 ** 0.5 * torch.randn(3 * q_len, 16, 63, generator=g)
    q[..., 575] = 64
    return y, q.to(torch.bfloat16), lens


def decode(path, kv_dtype, q, kv, scale, lens, **more):
    """The layout that `path` names: ("rows", tokens) or ("pages", rows a page)."""
    kind, n = path
    q_len = n if kind == "rows" else 1
    qo = (torch.arange(len(lens) + 1) * q_len).to(torch.int32).to(DEV)
    if kind == "rows":
        ind = indptr_of(lens)
        dec = binding.MLADecoder(ind, kv_dtype, num_splits=1, q_len=q_len, **more)
        out, lse = dec(q.to(DEV), kv.to(DEV), ind.to(DEV), qo, kv_scale=scale.to(DEV))
    else:
        counts = [-(-x // n) for x in lens]
        at, pages = indptr_of(counts), sum(counts)
        perm = torch.randperm(pages, generator=torch.Generator("cpu").manual_seed(n))
        to = torch.cat([perm[int(at[b]) + torch.arange(x) // n] * n + torch.arange(x) % n for b, x in enumerate(lens)])
        laid = torch.zeros(pages * n, kv.shape[1], dtype=torch.uint8)
        laid[to] = kv
        if scale.dim() == 2:
            scale, rows = torch.full((pages * n, scale.shape[1]), 127, dtype=torch.uint8), scale
            scale[to] = rows
        last = torch.tensor([x - (c - 1) * n for x, c in zip(lens, counts)], dtype=torch.int32)
        dec = binding.PagedMLADecoder(at, last, n, pages, kv_dtype, num_splits=1, **more)
        out, lse = dec(q.to(DEV), laid.to(DEV), at.to(DEV), perm.to(torch.int32).to(DEV), last.to(DEV), qo, kv_scale=scale.to(DEV))
    assert dec.poll_error() == 0
    return out.double().cpu(), lse.double().cpu()


@pytest.mark.parametrize("path", PATHS, ids=lambda p: f"{p[0]}{p[1]}")
@pytest.mark.parametrize("n,spread", [(8192, 0), (8192, 1), (32768, 1)])
@pytest.mark.parametrize("gap", [5, 7, 8, 9, 11, 13])
def test_e4m3(path, n, spread, gap):
    q_len = path[1] if path[0] == "rows" else 1
    y, q, lens = sink(n, spread, gap, q_len)
    scale = torch.tensor([0.0125])
    codes = (y / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    out, lse = decode(path, "fp8", q, codes, scale, lens)
    start = [0, n, n + 1000]
    for b, x in enumerate(lens):
        for i in range(q_len):
            rows = torch.arange(start[b], start[b] + x - (q_len - 1 - i))
            ref, l, t, tl = reference(q[b * q_len + i], codes, scale.expand(sum(lens)), rows)
            err = (out[b * q_len + i] - ref).abs()
            assert torch.all(err <= t), f"sequence {b}, token {i}: off by {float((err / ref.abs().max()).max()):.2e} of the largest output"
            assert torch.all((lse[b * q_len + i] - l).abs() <= tl)


E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


@pytest.mark.parametrize("path,more", [(p, {}) for p in [("rows", 1), ("rows", 2), ("pages", 1), ("pages", 16), ("pages", 64)]] +
                         [(p, dict(mx_block_scaled=True)) for p in [("rows", 1), ("pages", 64), ("pages", 128)]],
                         ids=lambda v: f"{v[0]}{v[1]}" if isinstance(v, tuple) else ("scaled" if v else "converted"))
@pytest.mark.parametrize("n", [2048, 8192])
@pytest.mark.parametrize("top", [2, 3, 4, 6])  # e2m1 values; times 64 / 24 nats
def test_mxfp4(path, more, n, top):
    q_len = path[1] if path[0] == "rows" else 1
    y, q, lens = sink(n, 0, top / 0.375, q_len)
    y[:, 512:575] = 0
    packed, scales = synth.quantize_mxfp4(y.to(torch.bfloat16))
    out, lse = decode(path, "mxfp4", q, packed, scales, lens, **more)
    nib = torch.stack([packed & 15, packed >> 4], -1).flatten(1).long()
    v = E2M1[nib] * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    start = [0, n, n + 1000]
    for b, x in enumerate(lens):
        for i in range(q_len):
            rows = torch.arange(start[b], start[b] + x - (q_len - 1 - i))
            a = q[b * q_len + i].double() @ v[rows].T / 24
            w, l = torch.softmax(a, -1), torch.logsumexp(a, -1)
            size = torch.exp2(scales[rows, :16 if more else 18].double().amax(-1) - 127)
            code, u = v[rows, :512] / size.unsqueeze(1), w * size
            ref = u @ code
            t = torch.maximum(2.0 ** -8 * u, 2.0 ** -18 * w.amax(-1, keepdim=True) * size.max()) + u * (len(rows) * 2.0 ** -28 + 2.0 ** -16)
            err = (out[b * q_len + i] - ref).abs()
            assert torch.all(err <= 2.0 ** -8 * ref.abs() + t @ code.abs()), \
                f"sequence {b}, token {i}: off by {float((err / ref.abs().max()).max()):.2e} of the largest output"
            assert torch.all((lse[b * q_len + i] - l).abs() <= 2.0 ** -22 * l.abs() + 2e-5)
