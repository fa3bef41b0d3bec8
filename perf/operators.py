"""The operators around the latent cache, measured: what each case is, its plain form and its definition.

The library decodes over a latent cache of 576-wide rows (512 latent columns, 64 position columns)
in bf16, e4m3 (one fp32 scale) or MXFP4 (e2m1 with an e8m0 byte per 32 elements), in pages.  The
operators here write that cache, read it back and manage its pages:

  append   norms of keys and of each query head, the position rotation (one or several axes), and
           the key row's store in the cache's format, in one pass
  step     a batch's page tables grown by a few rows, the new rows appended, the tables cut back
  gather   rows of the cache as bf16, through the page table
  copy     pages copied in every layer
  fork     sequences forked (full pages shared, a part-filled last page copied), the forks freed
  compact  the live pages moved to the front of the cache, page table and counts rewritten

Every case is plain values; lengths of a ragged batch follow from them (see ``lengths``).
"""
import math

import torch

own = False

HEADS, LAT, PE, ROW, BLOCK = 16, 512, 64, 576, 32
EPS = 1e-6
ROW_BYTES = {"bf16": 1152, "fp8": 576, "mxfp4": 288}
SCALE_BYTES = {"bf16": 0, "fp8": 0, "mxfp4": 18}
KINDS = ("bf16", "fp8", "mxfp4")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a batch of 4 with contexts of 1024: the smallest call, once per layer and token
        dict(name="step_append_fp8_b4", op="append", tokens=4, kv="fp8", page=64, pages=68, q="pe", norms="kv",
             axes=1, interleaved=True),
        # a prompt's rows in one call: every norm, three position axes, the queries' latent part too
        dict(name="prompt_append_bf16", op="append", tokens=8190, kv="bf16", page=16, pages=600, q="full",
             norms="all", axes=3, interleaved=False),
        # drafted tokens of a batch of 64: tables grown by 4 rows, rows appended, tables cut back
        dict(name="draft_step_bf16_b64", op="step", batch=64, length=1024, spread=64, grow=4, kv="bf16", page=16,
             axes=1, interleaved=True),
        # a chunk of a prompt per sequence into a 4-bit cache, read back in bf16 for the chunk's own attention
        dict(name="chunk_step_mxfp4_b7", op="step", batch=7, length=2000, spread=700, grow=1021, kv="mxfp4", page=64,
             axes=3, interleaved=False),
        # the cached context of a small batch as bf16
        dict(name="gather_fp8_b4", op="gather", batch=4, length=1024, spread=333, kv="fp8", page=64),
        # the cached context of the largest 4-bit batch as bf16
        dict(name="gather_mxfp4_b32", op="gather", batch=32, length=8192, spread=1000, kv="mxfp4", page=64),
        # a few pages copied in one layer: the latency of the call
        dict(name="copy_fp8_8_pages", op="copy", n=8, layers=1, kv="fp8", page=64, pages=256),
        # a prefix's pages duplicated in every layer
        dict(name="copy_mxfp4_4001_pages", op="copy", n=4001, layers=6, kv="mxfp4", page=64, pages=9000),
        # 3 samples of each of 4 prompts
        dict(name="fork_bf16_b4x3", op="fork", batch=4, children=3, length=1024, spread=333, layers=1, kv="bf16",
             page=64),
        # 8 samples of each of 64 long prompts, in every layer of a stack
        dict(name="fork_fp8_b64x8", op="fork", batch=64, children=8, length=8192, spread=777, layers=12, kv="fp8",
             page=64),
        # a small cache with a few holes
        dict(name="compact_fp8_small", op="compact", pages=515, live=300, moved=40, layers=1, kv="fp8", page=64),
        # a large cache of several layers, half empty
        dict(name="compact_bf16_large", op="compact", pages=20011, live=11000, moved=4500, layers=2, kv="bf16",
             page=64),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "step", "gather", "copy", "fork", "compact"))
    kv = rng.choice(KINDS)
    page = 1 << rng.randint(0, 8)
    axes, inter = rng.choice((1, 2, 3, 4)), rng.random() < 0.5
    if op == "append":
        kv = rng.choice(("bf16", "fp8"))
        tokens = _between(rng, 1, 8190)
        return dict(op=op, tokens=tokens, kv=kv, page=page, pages=-(-tokens // page) + rng.randint(0, 64),
                    q=rng.choice(("none", "pe", "full")), norms=rng.choice(("none", "kv", "all")), axes=axes,
                    interleaved=inter)
    if op == "step":
        batch = _between(rng, 1, 128)
        return dict(op=op, batch=batch, length=_between(rng, 1, 4096), spread=_between(rng, 1, 999),
                    grow=_between(rng, 1, max(1, 7147 // batch)), kv=kv, page=page, axes=axes, interleaved=inter)
    if op == "gather":
        batch = _between(rng, 1, 64)
        return dict(op=op, batch=batch, length=_between(rng, 1, 200000 // batch), spread=_between(rng, 1, 999), kv=kv,
                    page=page)
    # the page operators: about 0.8 GB of rows moved at most
    each = page * (ROW_BYTES[kv] + SCALE_BYTES[kv])
    layers = _between(rng, 1, 12)
    if op == "copy":
        n = _between(rng, 1, min(50000, max(1, 460_000_000 // (each * layers))))
        return dict(op=op, n=n, layers=layers, kv=kv, page=page, pages=2 * n + rng.randint(0, 100))
    if op == "fork":
        page = max(page, 2)
        batch, children = _between(rng, 1, 64), _between(rng, 1, 8)
        return dict(op=op, batch=batch, children=children, length=_between(rng, 1, 8192), spread=_between(rng, 1, 999),
                    layers=_between(rng, 1, 4), kv=kv, page=page)
    pages = _between(rng, 2, min(60000, max(4, 1_600_000_000 // (each * layers))))
    live = rng.randint(1, pages - 1)
    return dict(op=op, pages=pages, live=live, moved=rng.randint(0, min(live, pages - live)), layers=layers, kv=kv,
                page=page)


def lengths(case):
    """The lengths of a ragged batch: ``length`` less up to ``spread`` rows, none below one."""
    return [max(1, case["length"] - (b * 37) % case["spread"]) for b in range(case["batch"])]


def _fork_copies(case):
    """Rows that the forks own a copy of: those of the parents' part-filled last pages."""
    return case["children"] * sum(n % case["page"] for n in lengths(case))


def work(case):
    op, kv = case["op"], case["kv"]
    row = ROW_BYTES[kv] + SCALE_BYTES[kv]
    if op == "append":
        t = case["tokens"]
        parts = {"none": 0, "pe": PE, "full": ROW}[case["q"]]
        moved = t * (ROW * 2 + row + 4 + 4 * case["axes"]) + t * HEADS * parts * 4
        return {"bytes": moved, "flops": t * 8.0 * (ROW + HEADS * parts)}
    if op == "step":
        t = case["batch"] * case["grow"]
        tables = sum(-(-n // case["page"]) + -(-(n + case["grow"]) // case["page"]) for n in lengths(case)) * 4 * 2
        # the rows in, the rows stored, the queries' position part; the rows read back (stored and bf16) where the cache has 4 bits
        moved = t * (ROW * 2 + row + HEADS * PE * 4 + 12) + (t * (row + ROW * 2) if kv == "mxfp4" else 0) + tables
        return {"bytes": moved, "flops": t * 8.0 * (ROW + HEADS * PE)}
    if op == "gather":
        n = sum(lengths(case))
        return {"bytes": n * (row + ROW * 2 + 4), "flops": float(n * ROW)}
    if op == "copy":
        return {"bytes": 2 * case["n"] * case["layers"] * case["page"] * row + 8 * case["n"], "flops": 0}
    if op == "fork":
        entries = sum(-(-n // case["page"]) for n in lengths(case))
        return {"bytes": 2 * _fork_copies(case) * case["layers"] * row + 4 * entries * (1 + 3 * case["children"]),
                "flops": 0}
    return {"bytes": 2 * case["moved"] * case["layers"] * case["page"] * row + 8 * case["pages"] + 8 * case["live"],
            "flops": 0}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _cache(g, kv, layers, rows):
    """A cache in use: rows of about unit size in the cache's format, (rows, scales, bytes per scale row)."""
    if kv == "bf16":
        base = _randn(g, 1 << 16, ROW).to(torch.bfloat16)
        scale = None
    elif kv == "fp8":
        base = (_randn(g, 1 << 16, ROW) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scale = torch.full((1,), 0.0109375, device="cuda")
    else:
        base = torch.randint(0, 256, (1 << 16, ROW // 2), generator=g, device="cuda", dtype=torch.uint8)
        scale = torch.randint(123, 128, (layers, rows, ROW // BLOCK), generator=g, device="cuda", dtype=torch.uint8)
    data = torch.empty(layers, rows, base.shape[1], dtype=base.dtype, device="cuda")
    flat = data.view(-1, base.shape[1])
    for at in range(0, flat.shape[0], base.shape[0]):  # the same block again, its rows turned by some columns
        part = flat[at:at + base.shape[0]]
        part.copy_(base[:part.shape[0]].roll(at // base.shape[0], 1))
    return data, scale


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cum(v):
    at = [0]
    for n in v:
        at.append(at[-1] + n)
    return at


def _axes_of_pairs(axes):
    """The 32 pairs dealt to the axes in runs: 32 / 16+16 / 8+12+12 / 8+8+8+8."""
    runs = {1: (32,), 2: (16, 16), 3: (8, 12, 12), 4: (8, 8, 8, 8)}[axes]
    return [a for a, n in enumerate(runs) for _ in range(n)]


def _tokens(s, g, case, t, far):
    """What a layer's projections leave for t tokens, and their positions (1 to `axes` of them a token)."""
    s["kv_a"] = _randn(g, t, ROW).to(torch.bfloat16)                          # latent and position part side by side
    s["q_b"] = _randn(g, t, HEADS, 128 + PE).to(torch.bfloat16)               # a head's 128 columns, then its position part
    s["q"] = _randn(g, t, HEADS, ROW).to(torch.bfloat16)                      # the queries that the decode reads
    s["positions"] = torch.randint(0, far, (t, case["axes"]), generator=g, device="cuda", dtype=torch.int32)
    s["inv_freq"] = [10000.0 ** (-i / 32) for i in range(32)]
    s["axis_of_pair"] = _axes_of_pairs(case["axes"])
    s["weights"] = {k: (1 + 0.1 * _randn(g, n)).to(torch.bfloat16)
                    for k, n in (("kv_lat", LAT), ("kv_pe", PE), ("q_lat", LAT), ("q_pe", PE))}


def _handles(s, case, refs=None):
    """What a program of the framework keeps: the pool over its cache, the rotation and the norms."""
    from mla_attention_decode_gb300 import cache
    s["pool"] = cache.MLACachePool(s["cache"], case["kv"], case["page"], kv_scale=s["scale"], refs=refs)
    if "inv_freq" in s:
        s["rope"] = cache.MLARope(inv_freq=s["inv_freq"], axis_of_pair=s["axis_of_pair"],
                                  interleaved=case["interleaved"])
        names = {"none": (), "kv": ("kv_lat",), "all": ("kv_lat", "kv_pe", "q_lat", "q_pe")}[case.get("norms", "kv")]
        if case.get("q") == "none":
            names = [n for n in names if n.startswith("kv")]
        elif case.get("q", "pe") == "pe":
            names = [n for n in names if n != "q_lat"]
        s["norm"] = cache.MLANorm(eps=EPS, **{n: s["weights"][n] for n in names})


def _table(s, g, case, spare, extra=0):
    """Sequences of lengths(case) on pages at random places of a cache with `spare` more pages."""
    lens, page = lengths(case), case["page"]
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    at = _cum(counts)
    s["page_indptr"], s["last"] = _ints(at), _ints([n - (c - 1) * page for n, c in zip(lens, counts)])
    s["indices"] = torch.randperm(pages, generator=g, device="cuda")[:at[-1]].to(torch.int32)
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["refs"][s["indices"].long()] = 1
    s["lens"] = _ints(lens)
    s["cache"], s["scale"] = _cache(g, case["kv"], case.get("layers", 1), pages * page)
    return lens, at


def prepare(case, seed):
    g, op, page = _gen(seed), case["op"], case["page"]
    s = {"case": case}
    if op == "append":
        t, rows = case["tokens"], case["pages"] * page
        _tokens(s, g, case, t, 100000)
        s["cache"], s["scale"] = _cache(g, case["kv"], 1, rows)
        s["slots"] = torch.randperm(rows, generator=g, device="cuda")[:t].to(torch.int32)
        if case["q"] == "full":
            s["q_abs"] = _randn(g, t, HEADS, LAT).to(torch.bfloat16)
    elif op == "step":
        lens, grow = lengths(case), case["grow"]
        more = [-(-(n + grow) // page) for n in lens]
        _table(s, g, case, sum(more) + 5)
        t = case["batch"] * grow
        _tokens(s, g, case, t, 100000)
        s["grown"] = _ints([n + grow for n in lens])
        s["qo_indptr"] = _ints([b * grow for b in range(case["batch"] + 1)])
        s["entries"] = sum(more)
        if own:
            s["table2"] = [torch.empty_like(s["page_indptr"]), s["indices"].new_empty(sum(more)), torch.empty_like(s["last"])]
            s["table3"] = [torch.empty_like(s["page_indptr"]), torch.empty_like(s["indices"]), torch.empty_like(s["last"])]
    elif op == "gather":
        lens, _ = _table(s, g, case, 7)
        s["qo_indptr"], s["total"] = _ints(_cum(lens)), sum(lens)
    elif op == "copy":
        n = case["n"]
        s["cache"], s["scale"] = _cache(g, case["kv"], case["layers"], case["pages"] * page)
        at = torch.randperm(case["pages"], generator=g, device="cuda")[:2 * n].to(torch.int32)
        s["src"], s["dst"] = at[:n].contiguous(), at[n:].contiguous()
    elif op == "fork":
        lens, children = lengths(case), case["children"]
        _, at = _table(s, g, case, children * sum(n % page > 0 for n in lens) + 3)
        s["parents"] = _ints([b for b in range(case["batch"]) for _ in range(children)])
        s["entries"] = children * at[-1]
        if own:
            s["table2"] = [_ints([0] * (len(lens) * children + 1)), s["indices"].new_empty(s["entries"]),
                           _ints([0] * (len(lens) * children))]
    else:
        n, live, moved = case["pages"], case["live"], case["moved"]
        s["cache"], s["scale"] = _cache(g, case["kv"], case["layers"], n * page)
        at = torch.cat([torch.randperm(live, generator=g, device="cuda")[:live - moved],
                        live + torch.randperm(n - live, generator=g, device="cuda")[:moved]])
        s["refs"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["refs"][at] = 1
        twice = at[::5]  # some pages are two sequences'
        s["refs"][twice] += 1
        at = torch.cat([at, twice])
        s["indices"] = at[torch.randperm(at.numel(), generator=g, device="cuda")].to(torch.int32)
    if own:
        _handles(s, case, s.get("refs"))
        if op == "compact":
            s["out"] = (torch.empty_like(s["indices"]), torch.empty_like(s["refs"]), _ints([0]))
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


def _e2m1(v):
    """Codes of the nearest e2m1 values, ties to the even code."""
    m = v.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    return (code + 8 * (v < 0)).to(torch.uint8)


def _store(s, kv, slots, y):
    """Rows y (fp32) into the cache's first layer at rows `slots`, in its format."""
    at = slots.long()
    if kv == "bf16":
        s["cache"][0, at] = y.to(torch.bfloat16)
    elif kv == "fp8":
        s["cache"][0, at] = (y / s["scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        blocks = y.view(-1, ROW // BLOCK, BLOCK)
        amax = blocks.abs().amax(-1)
        # the smallest power of two with amax <= 6 * 2^e, from amax's own exponent (exact)
        frac, ex = torch.frexp(amax)
        e = torch.where(amax > 0, ex - 3 + (frac > 0.75), torch.zeros_like(ex)).clamp(-127, 127)
        codes = _e2m1(torch.ldexp(blocks, -e.unsqueeze(-1))).view(-1, ROW)
        s["cache"][0, at] = codes[:, 0::2] | (codes[:, 1::2] << 4)
        s["scale"][0, at] = (e + 127).to(torch.uint8)


def _values(s, kv, slots):
    """Rows `slots` of the cache's first layer, in 32 bits."""
    at = slots.long()
    if kv == "bf16":
        return s["cache"][0, at].float()
    if kv == "fp8":
        return s["cache"][0, at].view(torch.float8_e4m3fn).float() * s["scale"]
    grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], device=at.device)
    grid = torch.cat([grid, -grid])
    packed = s["cache"][0, at]
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(1)
    scale = torch.ldexp(torch.ones((), device=at.device), s["scale"][0, at].int() - 127)
    return (grid[codes.int()].view(-1, ROW // BLOCK, BLOCK) * scale.unsqueeze(-1)).view(-1, ROW)


def _plain_append(s, case, slots, positions, norms, q):
    s = dict(s, positions=positions)
    all_, inter, w = norms == "all", case["interleaved"], s["weights"]
    x = s["kv_a"].float()
    lat = _norm(x[:, :LAT], w["kv_lat"], norms != "none")
    pe = _rotate(_norm(x[:, LAT:], w["kv_pe"], all_), s, inter)
    _store(s, case["kv"], slots, torch.cat([lat, pe], -1))
    if q != "none":
        s["q"][..., LAT:] = _rotate(_norm(s["q_b"][..., 128:].float(), w["q_pe"], all_), s, inter).to(torch.bfloat16)
        if q == "full":
            s["q"][..., :LAT] = _norm(s["q_abs"].float(), w["q_lat"], all_).to(torch.bfloat16)


def _row_slots(indptr, indices, last, qo_indptr, page):
    """Row in the cache, and place in its sequence, of the last qo_indptr[b + 1] - qo_indptr[b] rows of each sequence."""
    indptr, last, qo = indptr.long(), last.long(), qo_indptr.long()
    counts, n = indptr[1:] - indptr[:-1], qo[1:] - qo[:-1]
    length = torch.where(counts > 0, (counts - 1) * page + last, torch.zeros_like(counts))
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n)
    row = length[seq] - n[seq] + torch.arange(seq.numel(), device=n.device) - qo[seq]
    slots = indices.long()[indptr[seq] + row // page] * page + row % page
    return slots.int(), row.int()


def _plain_resize(s, table, lens, page):
    """The table for the new lengths: pages kept, the lowest free ones added, those past the end given back."""
    indptr, indices = table[0].long(), table[1]
    old, new = indptr[1:] - indptr[:-1], (lens.long() + page - 1) // page
    at = torch.cat([new.new_zeros(1), new.cumsum(0)])
    seq = torch.repeat_interleave(torch.arange(new.numel(), device=new.device), new)
    j = torch.arange(seq.numel(), device=new.device) - at[seq]
    kept = j < old[seq]
    out = torch.empty(seq.numel(), dtype=torch.int32, device=new.device)
    out[kept] = indices[(indptr[seq] + j)[kept]]
    fresh = (s["refs"] == 0).nonzero().squeeze(1)[:int((~kept).sum())]
    out[~kept] = fresh.int()
    s["refs"][fresh] = 1
    seq = torch.repeat_interleave(torch.arange(old.numel(), device=old.device), old)
    gone = (torch.arange(seq.numel(), device=old.device) - indptr[seq]) >= new[seq]
    s["refs"].index_add_(0, indices[gone].long(), indices.new_full((int(gone.sum()),), -1))
    last = torch.where(new > 0, lens.long() - (new - 1) * page, torch.zeros_like(new))
    return at.int(), out, last.int()


def _plain_step(s, case):
    page, kv = case["page"], case["kv"]
    grown = _plain_resize(s, (s["page_indptr"], s["indices"]), s["grown"], page)
    slots, row = _row_slots(*grown, s["qo_indptr"], page)
    positions = s["positions"].clone()
    positions[:, 0] = row
    _plain_append(s, case, slots, positions, "kv", "pe")
    rows = _values(s, kv, slots).to(torch.bfloat16) if kv == "mxfp4" else None
    cut = _plain_resize(s, grown, s["lens"], page)
    return grown, slots, rows, cut


def _plain_fork(s, case):
    page, parents = case["page"], s["parents"].long()
    indptr, last = s["page_indptr"].long(), s["last"].long()
    counts = (indptr[1:] - indptr[:-1])[parents]
    at = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    seq = torch.repeat_interleave(torch.arange(counts.numel(), device=counts.device), counts)
    j = torch.arange(seq.numel(), device=counts.device) - at[seq]
    out = s["indices"][indptr[parents[seq]] + j].clone()
    part = (counts > 0) & (last[parents] < page)
    mine = (j == counts[seq] - 1) & part[seq]
    src = out[mine].long()
    dst = (s["refs"] == 0).nonzero().squeeze(1)[:src.numel()]
    out[mine] = dst.int()
    s["refs"].index_add_(0, out.long(), torch.ones_like(out))
    used = torch.arange(page, device=src.device) < last[parents[seq[mine]]].unsqueeze(1)
    rows_in, rows_out = ((p.unsqueeze(1) * page + torch.arange(page, device=src.device))[used] for p in (src, dst))
    s["cache"][:, rows_out] = s["cache"][:, rows_in]
    if case["kv"] == "mxfp4":
        s["scale"][:, rows_out] = s["scale"][:, rows_in]
    table = at.int(), out, s["last"][parents]
    held = s["refs"].clone()
    s["refs"].index_add_(0, out.long(), -torch.ones_like(out))  # the forks have ended
    return table, held


def _pages(s, page):
    return [x.view(x.shape[0], -1, page, x.shape[-1]) for x in (s["cache"], s["scale"]) if x is not None and x.dim() == 3]


def _plain_compact(s, case):
    alive = s["refs"] > 0
    live = alive.sum()
    at = torch.arange(alive.numel(), device=alive.device)
    src, dst = (alive & (at >= live)).nonzero().squeeze(1), (~alive & (at < live)).nonzero().squeeze(1)
    place = at.clone()
    place[src] = dst
    refs = torch.where(at < live, s["refs"], torch.zeros_like(s["refs"]))
    refs[dst] = s["refs"][src]
    for x in _pages(s, case["page"]):
        x[:, dst] = x[:, src]
    return place[s["indices"].long()].int(), refs, live.int().view(1)


def _cache_out(s, kv):
    """The cache as a result: e4m3 as the values it holds, the rest as it is stored."""
    return s["cache"].view(torch.float8_e4m3fn) if kv == "fp8" else s["cache"]


def run(s):
    case = s["case"]
    op, kv, page = case["op"], case["kv"], case["page"]
    if op == "append":
        if own:
            with_q = {} if case["q"] == "none" else dict(q_pe=s["q_b"][..., 128:], q_out=s["q"])
            if case["q"] == "full":
                with_q["q_lat"] = s["q_abs"]
            s["pool"].append(s["kv_a"][:, :LAT], s["kv_a"][:, LAT:], s["slots"], s["rope"], s["positions"],
                             norm=s["norm"], **with_q)
        else:
            _plain_append(s, case, s["slots"], s["positions"], case["norms"], case["q"])
        return {"q": s["q"], "cache": _cache_out(s, kv)}
    if op == "step":
        if own:
            pool, t2, t3 = s["pool"], s["table2"], s["table3"]
            pool.resize((s["page_indptr"], s["indices"], s["last"]), s["grown"], out=t2)
            slots, _ = pool.slots(t2, s["qo_indptr"], s["kv_a"].shape[0], rows=s["positions"][:, 0])
            pool.append(s["kv_a"][:, :LAT], s["kv_a"][:, LAT:], slots, s["rope"], s["positions"], norm=s["norm"],
                        q_pe=s["q_b"][..., 128:], q_out=s["q"])
            rows = pool.gather(slots) if kv == "mxfp4" else None
            pool.resize(t2, s["lens"], out=t3)
        else:
            t2, slots, rows, t3 = _plain_step(s, case)
        return {"grown": list(t2), "slots": slots, "rows": rows, "cut": list(t3), "refs": s["refs"], "q": s["q"],
                "cache": None if kv == "mxfp4" else _cache_out(s, kv)}
    if op == "gather":
        table = (s["page_indptr"], s["indices"], s["last"])
        if own:
            slots, _ = s["pool"].slots(table, s["qo_indptr"], s["total"])
            return {"slots": slots, "rows": s["pool"].gather(slots)}
        slots, _ = _row_slots(*table, s["qo_indptr"], page)
        return {"slots": slots, "rows": _values(s, kv, slots).to(torch.bfloat16)}
    if op == "copy":
        if own:
            s["pool"].copy_pages(s["src"], s["dst"])
        else:
            for x in _pages(s, page):
                x[:, s["dst"].long()] = x[:, s["src"].long()]
        return {"cache": s["cache"], "scale": s["scale"] if kv == "mxfp4" else None}
    if op == "fork":
        if own:
            t2 = s["pool"].fork((s["page_indptr"], s["indices"], s["last"]), s["parents"], out=s["table2"])
            held = s["refs"].clone()
            s["pool"].free(t2[1])
        else:
            t2, held = _plain_fork(s, case)
        return {"table": list(t2), "held": held, "refs": s["refs"], "cache": s["cache"],
                "scale": s["scale"] if kv == "mxfp4" else None}
    if own:
        s["pool"].compact(s["indices"], out=s["out"])
        at, refs, live = s["out"]
    else:
        at, refs, live = _plain_compact(s, case)
    return {"indices": at, "refs": refs, "live": live, "cache": s["cache"],
            "scale": s["scale"] if kv == "mxfp4" else None}


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


def _exact_append(s, case, slots, pos, norms, q_mode):
    """The queries and the rows, unrounded."""
    w, inter = s["weights"], case["interleaved"]
    row = s["kv_a"].double()
    if norms != "none":
        row[:, :LAT] = _unit(row[:, :LAT], w["kv_lat"])
    if norms == "all":
        row[:, LAT:] = _unit(row[:, LAT:], w["kv_pe"])
    row[:, LAT:] = _turned(row[:, LAT:], pos, s, inter)
    q = s["q"].double()
    if q_mode != "none":
        pe = s["q_b"][..., 128:].double()
        q[..., LAT:] = _turned(_unit(pe, w["q_pe"]) if norms == "all" else pe, pos, s, inter)
    if q_mode == "full":
        q[..., :LAT] = _unit(s["q_abs"].double(), w["q_lat"]) if norms == "all" else s["q_abs"].double()
    return q, row


def _exact_cache(s, case, slots, row):
    """The first layer's values after the rows are stored; the new rows as they are before their rounding."""
    if case["kv"] == "bf16":
        c = s["cache"].double()
        c[0, slots.long()] = row
    else:
        c = s["cache"].view(torch.float8_e4m3fn).double()
        c[0, slots.long()] = (row / s["scale"].double()).clamp(-448, 448)
    return c


def exact(case, seed):
    op, kv, page = case["op"], case["kv"], case["page"]
    if op in ("copy", "fork", "compact"):
        return None  # whole numbers and copies: nothing is computed
    s = prepare(case, seed)
    if op == "append":
        q, row = _exact_append(s, case, s["slots"], s["positions"], case["norms"], case["q"])
        return {"q": q, "cache": _exact_cache(s, case, s["slots"], row)}
    indptr, indices, last = (s[k].tolist() for k in ("page_indptr", "indices", "last"))
    lens, slots = lengths(case), []
    if op == "gather":
        for b, n in enumerate(lens):
            r = torch.arange(n)
            slots.append(torch.tensor(indices[indptr[b]:indptr[b + 1]])[r // page] * page + r % page)
        at = torch.cat(slots).cuda()
        if kv == "bf16":
            return {"slots": None, "rows": s["cache"][0, at].double()}
        if kv == "fp8":
            return {"slots": None, "rows": s["cache"][0, at].view(torch.float8_e4m3fn).double() * s["scale"].double()}
        code = torch.stack([s["cache"][0, at] % 16, s["cache"][0, at] // 16], -1).view(-1, ROW).long()
        e, m = (code % 8) // 2, code % 2  # sign, two exponent bits, one mantissa bit
        mag = torch.where(e == 0, 0.5 * m, torch.exp2((e - 1).double()) * (1 + 0.5 * m))
        block = torch.exp2(s["scale"][0, at].double() - 127).repeat_interleave(BLOCK, 1)
        return {"slots": None, "rows": torch.where(code >= 8, -mag, mag) * block}
    # a step: the fresh pages by hand, the lowest free ones in order of sequence and place
    free = [p for p, r in enumerate(s["refs"].tolist()) if r == 0]
    pos, at = s["positions"].clone(), []
    for b, n in enumerate(lens):
        mine = indices[indptr[b]:indptr[b + 1]]
        while len(mine) * page < n + case["grow"]:
            mine.append(free.pop(0))
        at += [mine[r // page] * page + r % page for r in range(n, n + case["grow"])]
        pos[b * case["grow"]:(b + 1) * case["grow"], 0] = torch.arange(n, n + case["grow"], device=pos.device)
    at = torch.tensor(at, device="cuda")
    q, row = _exact_append(s, case, at, pos, "kv", "pe")
    # which 4-bit value a number next to a border becomes is not a question of distance: no value there
    cache = None if kv == "mxfp4" else _exact_cache(s, case, at, row)
    return {"grown": None, "slots": None, "rows": None, "cut": None, "refs": None, "q": q, "cache": cache}
