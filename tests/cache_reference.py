"""Plain forms of the cache operators for their tests: fp64 torch on the CPU and
Python lists.  Shares no code with the CUDA path."""
import math

import torch

LAT, PE, ROW, BLOCK = 512, 64, 576, 32
WIDTH = {"bf16": 576, "fp8": 576, "mxfp4": 288}


# ------------------------------------------------------------------ rows
def rotate(x, positions, inv_freq, axis_of_pair, interleaved, scale=1.0):
    """x [T, ..., 64] (fp64), positions [T, axes]."""
    y = x.clone()
    for i in range(32):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        # the angle modulo one turn with exact integers (a position times an fp64 frequency)
        ang = [math.fmod(int(p) * inv_freq[i], 2 * math.pi) for p in positions[:, axis_of_pair[i]].tolist()]
        c = torch.tensor([math.cos(v) for v in ang], dtype=torch.float64).view(-1, *([1] * (x.dim() - 2)))
        s = torch.tensor([math.sin(v) for v in ang], dtype=torch.float64).view(-1, *([1] * (x.dim() - 2)))
        y[..., a] = scale * (x[..., a] * c - x[..., b] * s)
        y[..., b] = scale * (x[..., a] * s + x[..., b] * c)
    return y


def rms(x, weight, eps):
    w = 1.0 if weight is True else weight.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def e2m1_values():
    pos = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(pos + [-v for v in pos], dtype=torch.float64)


def dequant(kv_dtype, kv, scale):
    """Cache rows [n, width] (CPU) -> fp64 [n, 576]; scale: a number (fp8) or e8m0 bytes [n, >= 18] (mxfp4)."""
    if kv_dtype == "bf16":
        return kv.double()
    if kv_dtype == "fp8":
        return kv.view(torch.float8_e4m3fn).double() * float(scale)
    codes = torch.stack([kv & 15, kv >> 4], -1).flatten(1).long()
    e = scale[:, :18].double() - 127
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64), e)
    s = torch.where(scale[:, :18] == 255, torch.full_like(s, math.nan), s)
    return e2m1_values()[codes] * s.repeat_interleave(BLOCK, 1)


# ------------------------------------------------------------------ pages
class PoolModel:
    """The pages of a cache as lists: ``refs`` and, per page, a list of row tags."""

    def __init__(self, num_pages, page_size):
        self.n, self.p = num_pages, page_size
        self.refs = [0] * num_pages
        self.rows = [[None] * page_size for _ in range(num_pages)]

    def free_pages(self, k):
        got = [i for i, r in enumerate(self.refs) if r == 0][:k]
        return got if len(got) == k else None

    def pages_of(self, length):
        return -(-length // self.p)

    def fork(self, seqs, parents):
        """seqs: list of (pages, length).  Returns the forks, or None where pages are short."""
        need = [1 if seqs[q][1] % self.p else 0 for q in parents]
        fresh = self.free_pages(sum(need))
        if fresh is None:
            return None
        out = []
        for q in parents:
            pages, length = list(seqs[q][0]), seqs[q][1]
            shared = pages
            if length % self.p:
                new = fresh.pop(0)
                self.rows[new][:length % self.p] = self.rows[pages[-1]][:length % self.p]
                self.refs[new] = 1
                shared, pages = pages[:-1], pages[:-1] + [new]
            for g in shared:
                self.refs[g] += 1
            out.append((pages, length))
        return out

    def resize(self, seqs, lengths):
        plan, need = [], 0
        for (pages, length), want in zip(seqs, lengths):
            keep, r0 = min(len(pages), self.pages_of(want)), min(length, want)
            cow = want != length and r0 % self.p != 0 and self.refs[pages[keep - 1]] > 1
            first = keep - cow
            plan.append((first, cow, r0))
            need += self.pages_of(want) - first
        fresh = self.free_pages(need)
        if fresh is None:
            return None
        out, gone = [], []
        for (pages, length), want, (first, cow, r0) in zip(seqs, lengths, plan):
            new = [fresh.pop(0) for _ in range(self.pages_of(want) - first)]
            if cow:
                self.rows[new[0]][:r0 % self.p] = self.rows[pages[first]][:r0 % self.p]
            for g in new:
                self.refs[g] = 1
            gone += pages[first:]
            out.append((pages[:first] + new, want))
        for g in gone:
            self.refs[g] -= 1
        return out

    def free(self, pages):
        for g in pages:
            self.refs[g] -= 1

    def compact(self):
        """Returns the new number of each page."""
        live = sum(r > 0 for r in self.refs)
        holes = [i for i in range(live) if self.refs[i] == 0]
        movers = [i for i in range(live, self.n) if self.refs[i] > 0]
        place = list(range(self.n))
        for s, d in zip(movers, holes):
            place[s] = d
            self.refs[d], self.refs[s] = self.refs[s], 0
            self.rows[d] = list(self.rows[s])
        return place, live


def table_of(seqs, page_size, capacity=None, device="cpu"):
    """(page_indptr, kv_indices, last_page_len) of a list of (pages, length)."""
    at, idx, last = [0], [], []
    for pages, length in seqs:
        idx += pages
        at.append(len(idx))
        last.append(length - (len(pages) - 1) * page_size if pages else 0)
    idx += [-7] * ((capacity or len(idx)) - len(idx))
    make = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    return make(at), make(idx), make(last)


def seqs_of(table, page_size):
    """The reverse of table_of."""
    at, idx, last = (t.tolist() for t in table)
    return [(idx[a:b], (b - a - 1) * page_size + last[i] if b > a else 0)
            for i, (a, b) in enumerate(zip(at[:-1], at[1:]))]
