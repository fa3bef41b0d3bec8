"""More operators of the latent cache, measured: a cache in e4m3 with a scale per row, and the attention of a prompt.

The cache ("fp8_row") holds rows of 576 columns (512 latent, 64 position) as e4m3 codes with one fp32 scale
a row, chosen when the row is written: s = max(max|y| / 448, 2^-64).  Measured are

  append  norms and position rotation of keys and queries, and the key rows' store as codes and scales
  gather  rows of the cache as bf16, through the page table
  decode  attention of one query token a sequence (or a few) over the cache, contiguous or in pages
  prompt  attention of a prompt's own tokens, head by head, from the up-projected keys and values: documents
          side by side, each causal, causal with a prefix that every token sees, or all to all

Every case is plain values; lengths of a ragged batch follow from them (see ``lengths``).
"""
import math

import numpy as np
import torch

own = False

HEADS, LAT, PE, ROW = 16, 512, 64, 576
NOPE = 128                      # a head's columns of keys without position, and of values
EPS = 1e-6
SM_DECODE, SM_PROMPT = 1 / 24, 1 / math.sqrt(NOPE + PE)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a batch of 64: once per layer and token
        dict(name="step_append_b64", op="append", tokens=64, page=64, pages=70, q=True, norms="kv", axes=1, interleaved=True),
        # a prompt's rows in one call, with every norm and three position axes
        dict(name="prompt_append", op="append", tokens=8190, page=16, pages=600, q=True, norms="all", axes=3,
             interleaved=False),
        # the cached context of a small batch as bf16, for a prompt's next chunk
        dict(name="gather_b4", op="gather", batch=4, length=1024, spread=333, page=64),
        # the cached context of a large batch as bf16
        dict(name="gather_b32", op="gather", batch=32, length=8192, spread=1000, page=16),
        # one token each of four short conversations: latency
        dict(name="decode_b4", op="decode", batch=4, length=1024, spread=200, page=64, q_len=1),
        # one token each of 64 long conversations in a contiguous cache
        dict(name="decode_b64", op="decode", batch=64, length=8192, spread=1, page=0, q_len=1),
        # the same with drafted tokens: two tokens a sequence are checked in one step
        dict(name="decode_draft_b32", op="decode", batch=32, length=4096, spread=999, page=0, q_len=2),
        # small pages, ragged lengths
        dict(name="decode_pages_b33", op="decode", batch=33, length=2500, spread=777, page=16, q_len=1),
        # a short question: latency
        dict(name="prompt_short", op="prompt", batch=1, tokens=17, t_spread=1, context=0, c_spread=1, heads=16, mask="causal"),
        # documents side by side, each with a prefix that all of its tokens see
        dict(name="prompt_documents", op="prompt", batch=7, tokens=1100, t_spread=901, context=0, c_spread=1, heads=16,
             mask="prefix"),
        # the next chunk of four prompts whose first 4096 tokens or so are cached
        dict(name="prompt_chunk", op="prompt", batch=4, tokens=509, t_spread=77, context=4096, c_spread=999, heads=16,
             mask="causal"),
        # a long prompt in one call
        dict(name="prompt_long", op="prompt", batch=1, tokens=8190, t_spread=1, context=0, c_spread=1, heads=16,
             mask="causal"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "gather", "decode", "decode", "prompt", "prompt", "prompt"))
    page = 1 << rng.randint(0, 8)
    if op == "append":
        tokens = _between(rng, 1, 8190)
        return dict(op=op, tokens=tokens, page=page, pages=-(-tokens // page) + rng.randint(0, 64), q=rng.random() < 0.7,
                    norms=rng.choice(("none", "kv", "all")), axes=rng.choice((1, 2, 3, 4)),
                    interleaved=rng.random() < 0.5)
    if op == "gather":
        batch = _between(rng, 1, 64)
        return dict(op=op, batch=batch, length=_between(rng, 1, 200000 // batch), spread=_between(rng, 1, 999), page=page)
    if op == "decode":
        batch, paged = _between(rng, 1, 64), rng.random() < 0.6
        return dict(op=op, batch=batch, length=_between(rng, 1, min(30000, 400000 // batch)), spread=_between(rng, 1, 999),
                    page=page if paged else 0, q_len=1 if paged else rng.choice((1, 1, 2, 2, 3, 5)))
    batch, heads = _between(rng, 1, 24), rng.choice((16, 16, 16, 1, 5, 32))
    tokens = _between(rng, 1, 5000 // batch + 1)
    context = rng.choice((0, 0, _between(rng, 1, 12000 // batch)))
    if heads == 32:
        tokens, context = tokens // 2 + 1, context // 2
    return dict(op=op, batch=batch, tokens=tokens, t_spread=_between(rng, 1, tokens), context=context,
                c_spread=_between(rng, 1, context + 1), heads=heads, mask=rng.choice(("causal", "causal", "prefix", "full")))


def lengths(case):
    """The lengths of a ragged batch: ``length`` less up to ``spread`` rows, none below one (or the query tokens)."""
    return [max(case.get("q_len", 1), case["length"] - (b * 37) % case["spread"]) for b in range(case["batch"])]


def documents(case):
    """(query tokens, keys, prefix) of each document of a prompt: its own tokens follow its cached context."""
    got = []
    for b in range(case["batch"]):
        n = max(1, case["tokens"] - (b * 37) % case["t_spread"])
        k = n + max(0, case["context"] - (b * 53) % case["c_spread"])
        got.append((n, k, (k * (1 + b % 4)) // 5 if case["mask"] == "prefix" else 0))
    return got


def _pairs(case):
    """Visible (query, key) pairs of a head."""
    total = 0
    for n, k, prefix in documents(case):
        seen = np.full(n, k) if case["mask"] == "full" else np.maximum(k - n + 1 + np.arange(n), prefix)
        total += int(seen.sum())
    return total


def work(case):
    op = case["op"]
    if op == "append":
        t = case["tokens"]
        return {"bytes": t * (ROW * 2 + ROW + 4 + 4 + 4 * case["axes"]) + (t * HEADS * PE * 4 if case["q"] else 0),
                "flops": t * 8.0 * (ROW + (HEADS * PE if case["q"] else 0))}
    if op == "gather":
        n = sum(lengths(case))
        return {"bytes": n * (ROW + 4 + ROW * 2 + 4), "flops": float(n * ROW)}
    if op == "decode":
        n, t = sum(lengths(case)), case["batch"] * case["q_len"]
        return {"bytes": n * (ROW + 4) + t * HEADS * (ROW + LAT) * 2, "flops": 2.0 * n * case["q_len"] * HEADS * (ROW + LAT)}
    docs = documents(case)
    q, k, h = sum(d[0] for d in docs), sum(d[1] for d in docs), case["heads"]
    return {"bytes": q * h * (NOPE + PE + NOPE) * 2 + k * (h * 2 * NOPE + PE) * 2 + q * h * 4,
            "flops": 2.0 * (NOPE + PE + NOPE) * _pairs(case) * h}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(v):
    at = [0]
    for n in v:
        at.append(at[-1] + n)
    return at


def _cache(g, rows):
    """A cache in use: rows of about unit size, some larger and some smaller, as codes and scales."""
    y = _randn(g, min(rows, 1 << 16), ROW)
    base = (y * (448 / y.abs().amax(1, keepdim=True))).to(torch.float8_e4m3fn).view(torch.uint8)
    data = torch.empty(rows, ROW, dtype=torch.uint8, device="cuda")
    for at in range(0, rows, base.shape[0]):  # the same block again, its rows turned by some columns
        part = data[at:at + base.shape[0]]
        part.copy_(base[:part.shape[0]].roll(at // base.shape[0], 1))
    return data, torch.exp(0.3 * _randn(g, rows)) * (3.2 / 448)


def _axes_of_pairs(axes):
    """The 32 pairs dealt to the axes in runs: 32 / 16+16 / 8+12+12 / 8+8+8+8."""
    runs = {1: (32,), 2: (16, 16), 3: (8, 12, 12), 4: (8, 8, 8, 8)}[axes]
    return [a for a, n in enumerate(runs) for _ in range(n)]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "append":
        t, rows = case["tokens"], case["pages"] * case["page"]
        s["kv_a"] = _randn(g, t, ROW).to(torch.bfloat16)                     # latent and position part side by side
        s["q_b"] = _randn(g, t, HEADS, NOPE + PE).to(torch.bfloat16)         # a head's columns, then its position part
        s["q"] = _randn(g, t, HEADS, ROW).to(torch.bfloat16)                 # the queries that the decode reads
        s["positions"] = torch.randint(0, 100000, (t, case["axes"]), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"] = [10000.0 ** (-i / 32) for i in range(32)]
        s["axis_of_pair"] = _axes_of_pairs(case["axes"])
        s["weights"] = {k: (1 + 0.1 * _randn(g, n)).to(torch.bfloat16)
                        for k, n in (("kv_lat", LAT), ("kv_pe", PE), ("q_pe", PE))}
        s["cache"], s["scale"] = _cache(g, rows)
        s["slots"] = torch.randperm(rows, generator=g, device="cuda")[:t].to(torch.int32)
        if own:
            from mla_attention_decode_gb300 import cache
            s["pool"] = cache.MLACachePool(s["cache"], "fp8_row", case["page"], kv_scale=s["scale"])
            s["rope"] = cache.MLARope(inv_freq=s["inv_freq"], axis_of_pair=s["axis_of_pair"],
                                      interleaved=case["interleaved"])
            names = {"none": (), "kv": ("kv_lat",), "all": ("kv_lat", "kv_pe", "q_pe")}[case["norms"]]
            s["norm"] = cache.MLANorm(eps=EPS, **{n: s["weights"][n] for n in names})
    elif op in ("gather", "decode"):
        lens, page = lengths(case), case["page"]
        if page:  # pages at random places of a cache with a few more
            counts = [-(-n // page) for n in lens]
            pages = sum(counts) + 7
            s["page_indptr"] = _ints(_cum(counts))
            s["last"] = _ints([n - (c - 1) * page for n, c in zip(lens, counts)])
            s["indices"] = torch.randperm(pages, generator=g, device="cuda")[:sum(counts)].to(torch.int32)
            s["cache"], s["scale"] = _cache(g, pages * page)
        else:
            s["kv_indptr"] = _ints(_cum(lens))
            s["cache"], s["scale"] = _cache(g, sum(lens))
        if op == "gather":
            s["qo_indptr"], s["total"] = _ints(_cum(lens)), sum(lens)
        else:
            t = case["batch"] * case["q_len"]
            s["q"] = _randn(g, t, HEADS, ROW).to(torch.bfloat16)
            s["qo_indptr"] = _ints([b * case["q_len"] for b in range(case["batch"] + 1)])
            s["lens"] = _ints(lens)
            if own:
                from mla_attention_decode_gb300 import binding
                if page:
                    s["decoder"] = binding.PagedMLADecoder(_cum(counts), s["last"].cpu(), page, pages, "fp8_row")
                else:
                    s["decoder"] = binding.MLADecoder(_cum(lens), "fp8_row", q_len=case["q_len"])
        if own and op == "gather":
            from mla_attention_decode_gb300 import cache
            s["pool"] = cache.MLACachePool(s["cache"], "fp8_row", page, kv_scale=s["scale"])
    else:
        docs, h = documents(case), case["heads"]
        tq, tk = sum(d[0] for d in docs), sum(d[1] for d in docs)
        s["q_b"] = _randn(g, tq, h, NOPE + PE).to(torch.bfloat16)            # the query projection
        s["q"] = _randn(g, tq, h, ROW).to(torch.bfloat16)                    # its rotated part in the last 64 columns
        s["kv_b"] = _randn(g, tk, h, 2 * NOPE).to(torch.bfloat16)            # the up-projection: keys, then values
        s["rows"] = _randn(g, tk, ROW).to(torch.bfloat16)                    # rows of the cache: the position part is theirs
        s["qo_indptr"], s["kv_indptr"] = _ints(_cum([d[0] for d in docs])), _ints(_cum([d[1] for d in docs]))
        s["prefix"] = _ints([d[2] for d in docs]) if case["mask"] == "prefix" else None
        s["most"] = max(d[0] for d in docs), max(d[1] for d in docs)
        if own:
            from mla_attention_decode_gb300 import prompt
            s["prompt"] = prompt.MLAPrompt(tq, tk, case["batch"], heads=h, causal=case["mask"] != "full")
    return s


# ------------------------------------------------------------------ the plain forms
def _norm(x, w, on):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float() if on else x


def _rotate(x, s, interleaved):
    """x [t, ..., 64] turned pair by pair; the angles in 64 bits (positions may be far)."""
    freq = torch.tensor(s["inv_freq"], dtype=torch.float64, device=x.device)
    axis = torch.tensor(s["axis_of_pair"], device=x.device)
    angle = s["positions"][:, axis].double() * freq
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (PE // 2,)
    cos, sin = angle.cos().float().view(shape), angle.sin().float().view(shape)
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_append(s, case):
    every, inter, w = case["norms"] == "all", case["interleaved"], s["weights"]
    x = s["kv_a"].float()
    y = torch.cat([_norm(x[:, :LAT], w["kv_lat"], case["norms"] != "none"),
                   _rotate(_norm(x[:, LAT:], w["kv_pe"], every), s, inter)], -1)
    scale = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -64)
    at = s["slots"].long()
    s["cache"][at] = (y / scale.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["scale"][at] = scale
    if case["q"]:
        s["q"][..., LAT:] = _rotate(_norm(s["q_b"][..., NOPE:].float(), w["q_pe"], every), s, inter).to(torch.bfloat16)


def _slots(s, page, at, rows):
    """Where rows `rows` of sequences `at` lie in the cache."""
    if page:
        return s["indices"][(s["page_indptr"][at] + rows // page).long()].long() * page + rows % page
    return (s["kv_indptr"][at] + rows).long()


def _plain_gather(s, case):
    qo = s["qo_indptr"].long()
    seq = torch.repeat_interleave(torch.arange(case["batch"], device=qo.device), qo[1:] - qo[:-1])
    at = _slots(s, case["page"], seq, torch.arange(seq.numel(), device=qo.device) - qo[seq])
    rows = s["cache"][at].view(torch.float8_e4m3fn).float() * s["scale"][at].unsqueeze(1)
    return {"slots": at.int(), "rows": rows.to(torch.bfloat16)}


def _softmax(scores, seen):
    """Softmax over the last dimension of what is seen; rows of zeros where nothing is."""
    scores = scores.masked_fill_(~seen, -math.inf)
    most = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(total.clamp(min=1e-30)), (total.log() + most).squeeze(-1)


def _plain_decode(s, case):
    b, t, lens = case["batch"], case["q_len"], s["lens"].long()
    rows = torch.arange(max(lengths(case)), device=lens.device)
    at = _slots(s, case["page"], torch.arange(b, device=lens.device).unsqueeze(1),
                torch.minimum(rows, lens.unsqueeze(1) - 1))                              # [b, rows]
    k = s["cache"][at].view(torch.float8_e4m3fn).float() * s["scale"][at].unsqueeze(-1)
    q = s["q"].float().view(b, t * HEADS, ROW)
    scores = (q @ k.transpose(1, 2)).view(b, t, HEADS, -1) * SM_DECODE
    limit = lens.view(b, 1) - (t - 1) + torch.arange(t, device=lens.device)              # rows that a token sees
    p, lse = _softmax(scores, (rows < limit.unsqueeze(-1)).unsqueeze(2))
    out = p.view(b, t * HEADS, -1) @ k[..., :LAT]
    return {"out": out.view(b * t, HEADS, LAT).to(torch.bfloat16), "lse": lse.reshape(b * t, HEADS)}


def _plain_prompt(s, case):
    qo, kv, (nq, nk), h = s["qo_indptr"].long(), s["kv_indptr"].long(), s["most"], case["heads"]
    i, j = torch.arange(nq, device=qo.device), torch.arange(nk, device=qo.device)
    n, m = (qo[1:] - qo[:-1]).unsqueeze(1), (kv[1:] - kv[:-1]).unsqueeze(1)
    mine = i < n                                                                         # [documents, nq]
    at_q = (qo[:-1].unsqueeze(1) + torch.minimum(i, n - 1)).clamp(min=0)
    at_k = (kv[:-1].unsqueeze(1) + torch.minimum(j, m - 1)).clamp(min=0)
    q = torch.cat([s["q_b"][..., :NOPE], s["q"][..., LAT:]], -1)[at_q].float().transpose(1, 2)
    k_pe = s["rows"][:, LAT:].unsqueeze(1).expand(-1, h, -1)
    k = torch.cat([s["kv_b"][..., :NOPE], k_pe], -1)[at_k].float().transpose(1, 2)
    v = s["kv_b"][..., NOPE:][at_k].float().transpose(1, 2)
    seen = (j < m).unsqueeze(1)                                                          # [documents, 1, nk]
    if case["mask"] != "full":
        before = j <= (m - n + i).unsqueeze(-1)                                          # [documents, nq, nk]
        if case["mask"] == "prefix":
            before |= j < s["prefix"].view(-1, 1, 1)
        seen = seen & before
    p, lse = _softmax((q @ k.transpose(2, 3)) * SM_PROMPT, seen.unsqueeze(1))
    out = (p @ v).transpose(1, 2)[mine]
    return {"out": out.to(torch.bfloat16), "lse": lse.transpose(1, 2)[mine]}


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "append":
        if own:
            with_q = dict(q_pe=s["q_b"][..., NOPE:], q_out=s["q"]) if case["q"] else {}
            s["pool"].append(s["kv_a"][:, :LAT], s["kv_a"][:, LAT:], s["slots"], s["rope"], s["positions"],
                             norm=s["norm"], **with_q)
        else:
            _plain_append(s, case)
        return {"q": s["q"], "codes": s["cache"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    if op == "gather":
        if own:
            slots, _ = s["pool"].slots((s["page_indptr"], s["indices"], s["last"]), s["qo_indptr"], s["total"])
            return {"slots": slots, "rows": s["pool"].gather(slots)}
        return _plain_gather(s, case)
    if op == "decode":
        if own:
            table = (s["page_indptr"], s["indices"], s["last"]) if case["page"] else (s["kv_indptr"],)
            out, lse = s["decoder"](s["q"], s["cache"], *table, s["qo_indptr"], kv_scale=s["scale"])
            return {"out": out, "lse": lse}
        return _plain_decode(s, case)
    if own:
        out, lse = s["prompt"](s["q_b"][..., :NOPE], s["q"][..., LAT:], s["kv_b"][..., :NOPE], s["rows"][:, LAT:],
                               s["kv_b"][..., NOPE:], s["qo_indptr"], s["kv_indptr"], prefix=s["prefix"])
        return {"out": out, "lse": lse}
    return _plain_prompt(s, case)


# ------------------------------------------------------------------ the definition in 64 bits
def _turned(x, pos, s, inter):
    """Each pair as a complex number times exp(i pos f), in 64 bits."""
    first = torch.arange(32, device=x.device) * (2 if inter else 1)
    second = first + (1 if inter else 32)
    angle = torch.stack([pos[:, a].double() * f for a, f in zip(s["axis_of_pair"], s["inv_freq"])], 1)
    unit = torch.polar(torch.ones_like(angle), angle).view(x.shape[0], *([1] * (x.dim() - 2)), 32)
    z = torch.complex(x[..., first], x[..., second]) * unit
    y = torch.empty_like(x)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _unit(x, w):
    return w.double() * x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def _exact_append(s, case):
    w, inter, at = s["weights"], case["interleaved"], s["slots"].long()
    row, q = s["kv_a"].double(), s["q"].double()
    if case["norms"] != "none":
        row[:, :LAT] = _unit(row[:, :LAT], w["kv_lat"])
    if case["norms"] == "all":
        row[:, LAT:] = _unit(row[:, LAT:], w["kv_pe"])
    row[:, LAT:] = _turned(row[:, LAT:], s["positions"], s, inter)
    if case["q"]:
        pe = s["q_b"][..., NOPE:].double()
        q[..., LAT:] = _turned(_unit(pe, w["q_pe"]) if case["norms"] == "all" else pe, s["positions"], s, inter)
    codes, scale = s["cache"].view(torch.float8_e4m3fn).double(), s["scale"].double()
    top = torch.maximum(row.max(1).values, -row.min(1).values)
    scale[at] = torch.maximum(top / 448, torch.full_like(top, 2.0 ** -64))
    codes[at] = row / scale[at].view(-1, 1)
    return {"q": q, "codes": codes, "scale": scale}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "append":
        return _exact_append(s, case)
    if op == "prompt":
        out, lse, at_q, at_k = [], [], 0, 0
        for n, k, prefix in documents(case):
            own_q, own_k = slice(at_q, at_q + n), slice(at_k, at_k + k)
            at_q, at_k = at_q + n, at_k + k
            pos = torch.arange(k - n, k, device="cuda").view(n, 1)
            key = torch.arange(k, device="cuda").view(1, k)
            hidden = (key > pos) & (key >= prefix) & (case["mask"] != "full")
            heads, logs = [], []
            for h in range(case["heads"]):
                a = s["q_b"][own_q, h, :NOPE].double() @ s["kv_b"][own_k, h, :NOPE].double().T
                a += s["q"][own_q, h, LAT:].double() @ s["rows"][own_k, LAT:].double().T
                a = torch.where(hidden, -math.inf, a * SM_PROMPT)
                logs.append(torch.logsumexp(a, 1))
                heads.append(torch.exp(a - logs[-1].unsqueeze(1)) @ s["kv_b"][own_k, h, NOPE:].double())
            out.append(torch.stack(heads, 1))
            lse.append(torch.stack(logs, 1))
        return {"out": torch.cat(out), "lse": torch.cat(lse)}
    lens, page, at = lengths(case), case["page"], []
    if page:
        indptr, indices = s["page_indptr"].tolist(), s["indices"].cpu()
        for b, n in enumerate(lens):
            r = torch.arange(n)
            at.append((indices[indptr[b]:indptr[b + 1]].long()[r // page] * page + r % page).cuda())
    else:
        start = _cum(lens)
        at = [torch.arange(start[b], start[b] + n, device="cuda") for b, n in enumerate(lens)]
    value = lambda rows: s["cache"][rows].view(torch.float8_e4m3fn).double() * s["scale"][rows].double().view(-1, 1)
    if op == "gather":
        return {"slots": None, "rows": value(torch.cat(at))}
    out, lse = [], []
    for b, rows in enumerate(at):
        k = value(rows)
        for i in range(case["q_len"]):
            n = lens[b] - (case["q_len"] - 1 - i)
            a = (k[:n] @ s["q"][b * case["q_len"] + i].double().T) * SM_DECODE
            out.append(torch.softmax(a, 0).T @ k[:n, :LAT])
            lse.append(torch.logsumexp(a, 0))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}
