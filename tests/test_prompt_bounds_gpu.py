"""Prompts of which one document's bounds do not fit: the others' results, with keys shared out
over several blocks and not; tolerances as in test_prompt_gpu."""
import pytest
import torch

from mla_attention_decode_gb300 import binding, build, prompt
from test_prompt_gpu import DEV, check, gen, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def call(x, qo, kv):
    """One call into buffers of 7.0; its error word is that of bounds that do not fit."""
    tq, heads = x["q_nope"].shape[:2]
    p = prompt.MLAPrompt(tq, x["k_nope"].shape[0], len(qo) - 1, heads=heads)
    out = torch.full((tq, heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((tq, heads), 7.0, device=DEV)
    p.workspace[256:].fill_(0x40)  # what a call before left of its partial results: 3.0 and the like
    a, b = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (qo, kv))
    p(**x, qo_indptr=a, kv_indptr=b, out=out, lse=lse)
    assert p.poll_error() == binding.MLA_ERR_DEVICE_INDEX and p.poll_error() == 0
    return out, lse


def documents(x, qo, kv):
    """The documents whose bounds fit, and how many of them claim each token."""
    tq, tk = x["q_nope"].shape[0], x["k_nope"].shape[0]
    fit = [b for b in range(len(qo) - 1) if 0 <= qo[b] <= qo[b + 1] <= tq and 0 <= kv[b] <= kv[b + 1] <= tk]
    claims = torch.zeros(tq, dtype=torch.int32, device=DEV)
    for b in fit:
        claims[qo[b]:qo[b + 1]] += 1
    return fit, claims


@pytest.mark.parametrize("tq,tk,qo,kv", [
    (100, 100, [0, 1 << 30, 60, 90], [0, 50, 60, 90]), (100, 100, [0, 50, 60, 90], [0, 50, 40, 90]),
    (100, 100, [0, 50, 60, 101], [0, 50, 60, 90]), (100, 100, [0, 50, 60, 90], [-5, 50, 60, 90]),
    (1000, 1200, [0, 1000, 200, 700], [0, 1000, 1100, 1200]), (900, 900, [600, 900, 0, 300], [0, 300, 300, 900]),
    # the keys shared out
    (100, 9000, [0, 1 << 30, 60, 90], [0, 3000, 3000, 9000]), (100, 9000, [0, 50, 60, 90], [0, 5000, 4000, 9000]),
    (300, 9000, [20, 300, 10, 20], [0, 4000, 4000, 9000]), (40, 9000, [-1, 10, 20, 30], [0, 10, 20, 9000])])
def test_other_documents_are_computed(tq, tk, qo, kv):
    x = inputs(gen(tq + tk), tq, tk, 2, "plain")
    out, lse = call(x, qo, kv)
    fit, claims = documents(x, qo, kv)
    assert torch.all(out[claims == 0] == 7.0) and torch.all(lse[claims == 0] == 7.0)
    for b in fit:
        ref = reference(x, qo[b:b + 2], kv[b:b + 2])
        for t in ref:
            t[claims > 1] = float("nan")
        check(out, lse, ref)


@pytest.mark.parametrize("bad", [0, 17, 40, 49])
@pytest.mark.parametrize("bound", [-3, 1 << 30])
@pytest.mark.parametrize("tk", [3000, 12000])
def test_documents_of_a_larger_batch_are_computed_or_left(bad, bound, tk):
    """50 documents of two tokens, one bound of the tokens wrong: right rows, or rows as they were."""
    n = 50
    x = inputs(gen(bad), 2 * n, tk, 1, "plain")
    qo, kv = [2 * b for b in range(n + 1)], [tk // n * b for b in range(n + 1)]
    qo[bad] = bound
    out, lse = call(x, qo, kv)
    fit, claims = documents(x, qo, kv)
    assert int(claims.max()) == 1 and torch.all(out[claims == 0] == 7.0) and torch.all(lse[claims == 0] == 7.0)
    left = torch.all(torch.all(out == 7.0, -1), -1) & torch.all(lse == 7.0, -1)
    for b in fit:
        ref = reference(x, qo[b:b + 2], kv[b:b + 2])
        for t in ref:
            t[left] = float("nan")
        if not torch.all(left[qo[b]:qo[b + 1]]):
            check(out, lse, ref)
