"""Pages of the latent cache on the GPU: copy, fork, resize, free and compact
against a model of lists, the refusals that leave everything as it was, and a
run of them with the decode as they are used."""
import numpy as np
import pytest
import torch

from mla_attention_decode_gb300 import binding, build, cache, synth
from cache_reference import PoolModel, WIDTH, seqs_of, table_of
from test_parity_gpu import CODES, assert_parity, gate_terms, orc  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DTYPES = ["bf16", "fp8", "mxfp4"]


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def new_pool(kv_dtype, pages, page, layers=1, stride=18, max_batch=4096):
    """A pool whose bytes are all random (copies are of bytes: any code will do)."""
    g = gen(pages * page + layers)
    rows, width = pages * page, WIDTH[kv_dtype] * (2 if kv_dtype == "bf16" else 1)
    kv = torch.randint(0, 256, (layers, rows, width), generator=g, dtype=torch.uint8).to(DEV)
    if kv_dtype == "bf16":
        kv = kv.view(torch.bfloat16)
    sc = None
    if kv_dtype == "fp8":
        sc = torch.ones(1, device=DEV)
    elif kv_dtype == "mxfp4":
        sc = torch.randint(0, 256, (layers, rows, stride), generator=g, dtype=torch.uint8).to(DEV)
    return cache.MLACachePool(kv, kv_dtype, page, kv_scale=sc, max_batch=max_batch)


def bytes_of(pool):
    """[layers, pages, page, row and scale bytes] on the CPU."""
    kv = pool.kv.view(torch.uint8).cpu().view(pool.num_layers, pool.num_pages, pool.page_size, -1)
    if pool.kv_dtype != binding.MLA_KV_MXFP4:
        return kv
    sc = pool.kv_scale.cpu().view(pool.num_layers, pool.num_pages, pool.page_size, -1)
    return torch.cat([kv, sc], -1)


def bytes_row(pool, page, r):
    """One row's bytes (and scale bytes) in every layer."""
    at = page * pool.page_size + r
    parts = [pool.kv.view(torch.uint8)[:, at].cpu()]
    if pool.kv_dtype == binding.MLA_KV_MXFP4:
        parts.append(pool.kv_scale[:, at].cpu())
    return torch.cat(parts, -1)


@pytest.mark.parametrize("kv_dtype", DTYPES)
@pytest.mark.parametrize("page", [1, 2, 8, 64, 256])
@pytest.mark.parametrize("layers,stride", [(1, 18), (3, 32)])
def test_copy_pages(kv_dtype, page, layers, stride):
    pool = new_pool(kv_dtype, 40, page, layers, stride)
    before = bytes_of(pool)
    src, dst = [3, 3, 7, 39, 12, 0], [1, 20, 2, 38, 12, 39 - 4]
    pool.copy_pages(i32(src), i32(dst))
    assert pool.poll_error() == 0
    want = before.clone()
    want[:, dst] = before[:, src]
    assert torch.equal(bytes_of(pool), want)


def test_copy_pages_odd_scale_stride():
    """Scale rows of 19 bytes and pages of one row: copies of single bytes."""
    # a layer of 33 x 19 bytes in a tensor of 48 x 19 a layer
    kv = torch.randint(0, 256, (2, 33, 288), dtype=torch.uint8, device=DEV)
    sc = torch.randint(0, 256, (2, 48, 19), dtype=torch.uint8, device=DEV)
    pool = cache.MLACachePool(kv, "mxfp4", 1, kv_scale=sc[:, :33])
    kv0, sc0 = kv.clone(), sc.clone()
    pool.copy_pages(i32([32, 5, 8]), i32([0, 1, 31]))
    kv0[:, [0, 1, 31]], sc0[:, [0, 1, 31]] = kv0[:, [32, 5, 8]], sc0[:, [32, 5, 8]]
    assert pool.poll_error() == 0
    assert torch.equal(kv, kv0) and torch.equal(sc, sc0)


def test_copy_pages_bad_index():
    pool = new_pool("fp8", 6, 4)
    before = bytes_of(pool)
    pool.copy_pages(i32([0, 6, 1, -1]), i32([5, 1, -3, 2]))
    assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX
    want = before.clone()
    want[:, 5] = before[:, 0]
    assert torch.equal(bytes_of(pool), want)


def test_copy_past_32_bit_offsets():
    """Pages more than 4 GB apart, in a cache of 3 layers of 4.7 GB."""
    pool = cache.MLACachePool(torch.zeros(3, 64 * 64000, 576, dtype=torch.bfloat16, device=DEV), "bf16", 64)
    pool.kv[:, -64:] = torch.arange(64, device=DEV).view(1, 64, 1).to(torch.bfloat16) + \
        100 * torch.arange(3, device=DEV).view(3, 1, 1).to(torch.bfloat16)
    pool.copy_pages(i32([63999]), i32([1]))
    assert pool.poll_error() == 0
    assert torch.equal(pool.kv[:, 64:128], pool.kv[:, -64:])
    assert torch.all(pool.kv[:, :64] == 0) and torch.all(pool.kv[:, 128:192] == 0)


def check_state(pool, model, table, seqs, tags_to_bytes):
    """The device's tables, counts and rows are the model's."""
    assert pool.refs.tolist() == model.refs
    got = seqs_of(table, pool.page_size)
    assert got == seqs
    now = bytes_of(pool)
    for pages, length in seqs:
        for j, pg in enumerate(pages):
            for r in range(min(pool.page_size, length - j * pool.page_size)):
                tag = model.rows[pg][r]
                if tag is not None:
                    assert torch.equal(now[:, pg, r], tags_to_bytes[tag]), (pg, r)


@pytest.mark.parametrize("kv_dtype,page,layers,pages", [
    ("bf16", 4, 2, 90), ("fp8", 1, 1, 90), ("mxfp4", 8, 3, 90), ("fp8", 16, 1, 90),
    # past what one CTA, the deciding cluster, and a kernel of its own for the counts go over
    ("fp8", 4, 1, 16385), ("mxfp4", 2, 2, 32800), ("mxfp4", 2, 1, 70001)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_random_life_of_a_pool(kv_dtype, page, layers, pages, seed):
    """Grow, write, fork, truncate, free and compact in random order: tables,
    counts and every live row follow the model; pages never handed out twice.
    In a large cache others hold all but 90 pages, at random places."""
    rng = np.random.RandomState(seed)
    pool, model = new_pool(kv_dtype, pages, page, layers), PoolModel(pages, page)
    others = rng.permutation(pages)[90:]
    for g in others:
        model.refs[g] = 1
    pool.refs[torch.from_numpy(others).to(DEV)] = 1
    seqs, table = [([], 0)] * 3, table_of([([], 0)] * 3, page, 1, DEV)
    tags, tags_to_bytes = 0, {}

    def run(call, want, batch):
        """`want`: the model's sequences, or None where it found too few pages."""
        nonlocal seqs, table
        cap = 1000
        out = pool.table(batch, cap)
        out[1].fill_(-7)
        call(out)
        if want is None:
            assert pool.poll_error() == cache.MLA_ERR_OUT_OF_PAGES
            assert torch.all(out[0] == 0) and torch.all(out[2] == 0)
            return False
        assert pool.poll_error() == 0
        assert torch.all(out[1][int(out[0][-1]):] == -7), "entries past the table"
        seqs, table = want, out
        return True

    for _ in range(30):
        op = rng.choice(["resize", "resize", "fork", "drop", "compact"])
        if op == "resize":
            lengths = [max(0, n + int(rng.randint(-2 * page, 4 * page + 1))) if rng.rand() < 0.7 else n for _, n in seqs]
            old = [n for _, n in seqs]
            want = model.resize(seqs, lengths)
            if run(lambda out: pool.resize(table, i32(lengths), out), want, len(seqs)):
                new = [max(0, n - m) for n, m in zip(lengths, old)]
                qo = [0] + np.cumsum(new).tolist()
                if qo[-1]:
                    slots, _ = pool.slots(table, i32(qo), qo[-1])
                    x = torch.randint(0, 256, (layers, qo[-1], bytes_of(pool).shape[-1]), dtype=torch.uint8)
                    kv = pool.kv.view(torch.uint8)
                    kv[:, slots.long()] = x[..., :kv.shape[-1]].to(DEV)
                    if pool.kv_scale is not None and pool.kv_scale.dim() == 3:
                        pool.kv_scale[:, slots.long()] = x[..., kv.shape[-1]:].to(DEV)
                    for b, (pgs, n) in enumerate(seqs):
                        for i in range(new[b]):
                            r = n - new[b] + i
                            assert model.refs[pgs[r // page]] == 1, "a shared page is written"
                            model.rows[pgs[r // page]][r % page] = tags
                            tags_to_bytes[tags] = x[:, qo[b] + i]
                            tags += 1
        elif op == "fork":
            parents = rng.randint(0, len(seqs), rng.randint(1, 4)).tolist()
            old = seqs
            if run(lambda out: pool.fork(table, i32(parents), out), model.fork(seqs, parents), len(parents)):
                # the parents end: the forks go on
                gone = [g for pgs, _ in old for g in pgs]
                model.free(gone)
                pool.free(i32(gone))
        elif op == "drop" and len(seqs) > 1:
            lengths = [0 if i == 0 else n for i, (_, n) in enumerate(seqs)]
            run(lambda out: pool.resize(table, i32(lengths), out), model.resize(seqs, lengths), len(seqs))
        elif op == "compact":
            place, live = model.compact()
            n = int(table[0][-1])
            idx, _, got_live = pool.compact(table[1][:n].contiguous())
            assert int(got_live) == live
            table = (table[0], idx, table[2])
            seqs = [([place[g] for g in pgs], n) for pgs, n in seqs]
        assert pool.poll_error() == 0
        check_state(pool, model, table, seqs, tags_to_bytes)


def test_truncating_into_a_shared_page_copies_it():
    """A fork truncated to the middle of a shared full page and grown again
    writes into a page of its own; rows past the cut are not copied."""
    page = 8
    pool = new_pool("fp8", 10, page)
    t0 = pool.resize(pool.table(1, 0), i32([20]), pool.table(1, 3))
    t1 = pool.fork(t0, i32([0]), pool.table(1, 3))
    assert seqs_of(t0, page) == [([0, 1, 2], 20)] and seqs_of(t1, page) == [([0, 1, 3], 20)]
    assert pool.refs.tolist() == [2, 2, 1, 1] + [0] * 6
    before = bytes_of(pool)
    t2 = pool.resize(t1, i32([13]), pool.table(1, 3))
    assert seqs_of(t2, page) == [([0, 4], 13)]
    assert pool.refs.tolist() == [2, 1, 1, 0, 1] + [0] * 5
    now = bytes_of(pool)
    assert torch.equal(now[:, 4, :5], before[:, 1, :5]) and torch.equal(now[:, 4, 5:], before[:, 4, 5:])
    t3 = pool.resize(t2, i32([14]), pool.table(1, 3))
    assert seqs_of(t3, page) == [([0, 4], 14)]
    assert pool.poll_error() == 0


def test_calls_that_cannot_be_met_change_nothing():
    page = 4
    pool = new_pool("bf16", 8, page)
    t0 = pool.resize(pool.table(2, 0), i32([10, 7]), pool.table(2, 5))
    refs, data = pool.refs.clone(), bytes_of(pool)
    tries = [
        (lambda o: pool.resize(t0, i32([10, 40]), o), 99, cache.MLA_ERR_OUT_OF_PAGES),
        (lambda o: pool.resize(t0, i32([2 ** 31 - 1, 2 ** 31 - 1]), o), 99, binding.MLA_ERR_DEVICE_INDEX),
        (lambda o: pool.resize(t0, i32([10, 9]), o), 5, binding.MLA_ERR_DEVICE_INDEX),      # no room in the table
        (lambda o: pool.resize(t0, i32([10, -1]), o), 99, binding.MLA_ERR_DEVICE_INDEX),
        (lambda o: pool.fork(t0, i32([0, 2]), o), 99, binding.MLA_ERR_DEVICE_INDEX),        # no such parent
        (lambda o: pool.fork(t0, i32([-1, 0]), o), 99, binding.MLA_ERR_DEVICE_INDEX),
        (lambda o: pool.fork((i32([0, 3, 9]), t0[1], t0[2]), i32([0, 1]), o), 99, binding.MLA_ERR_DEVICE_INDEX),
        (lambda o: pool.fork((t0[0], t0[1], i32([5, 1])), i32([0, 1]), o), 99, binding.MLA_ERR_DEVICE_INDEX),
    ]
    for call, room, status in tries:
        out = pool.table(2, room)
        for x in out:
            x.fill_(-7)
        call(out)
        assert pool.poll_error() == status
        assert out[0].tolist() == [0, 0, 0] and out[2].tolist() == [0, 0] and torch.all(out[1] == -7)
        assert torch.equal(pool.refs, refs) and torch.equal(bytes_of(pool), data)
    big = pool.table(4, 99)
    pool.fork(t0, i32([0, 1, 0, 1]), big)  # 4 part-filled pages, 3 free
    assert pool.poll_error() == cache.MLA_ERR_OUT_OF_PAGES and torch.equal(pool.refs, refs)
    small = new_pool("bf16", 8, page, max_batch=1)
    with pytest.raises(binding.MLAError) as e:
        small.fork(small.table(1, 0), i32([0] * 5000), small.table(5000, 9))
    assert e.value.status == binding.MLA_ERR_WORKSPACE_TOO_SMALL


def test_bad_page_numbers_are_skipped():
    page = 4
    pool = new_pool("fp8", 8, page)
    pool.refs[:3] = i32([1, 1, 1])
    t = (i32([0, 3]), i32([0, 8, 2]), i32([4]))
    out = pool.fork(t, i32([0]), pool.table(1, 3))
    assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX
    assert out[1].tolist() == [0, -1, 2] and pool.refs.tolist() == [2, 1, 2, 0, 0, 0, 0, 0]
    # a part-filled last page that does not exist
    t = (i32([0, 2]), i32([0, -5]), i32([3]))
    out = pool.fork(t, i32([0]), pool.table(1, 3))
    assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX
    assert out[1].tolist()[:2] == [0, -1] and pool.refs.tolist()[:3] == [3, 1, 2]
    idx, _, live = pool.compact(i32([0, 5, -1, 9, 2]))
    assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX
    assert idx.tolist() == [0, -1, -1, -1, 2] and int(live) == 3


def test_free_counts():
    pool = new_pool("fp8", 6, 4)
    pool.refs.copy_(i32([3, 1, 0, 2, 1, 1]))
    pool.free(i32([0, 3, 0, -1, 5]))
    assert pool.poll_error() == 0 and pool.refs.tolist() == [1, 1, 0, 1, 1, 0]
    pool.free(i32([1, 1, 1, 2, 6, -2]))  # more often than held; out of range
    assert pool.poll_error() == binding.MLA_ERR_DEVICE_INDEX
    assert pool.refs.tolist() == [1, 0, 0, 1, 1, 0]


def test_empty_batches_and_pools():
    pool = new_pool("mxfp4", 4, 2)
    out = pool.resize(pool.table(0, 0), i32([]), pool.table(0, 0))
    assert out[0].tolist() == [0]
    out = pool.fork(pool.table(3, 0), i32([1, 1]), pool.table(2, 0))  # forks of empty sequences
    assert out[0].tolist() == [0, 0, 0] and out[2].tolist() == [0, 0]
    idx, _, live = pool.compact(i32([]))
    assert int(live) == 0 and pool.refs.tolist() == [0] * 4
    pool.refs.fill_(1)
    before = bytes_of(pool)
    idx, _, live = pool.compact(i32([3, 1]))
    assert int(live) == 4 and idx.tolist() == [3, 1] and torch.equal(bytes_of(pool), before)
    none = cache.MLACachePool.allocate("bf16", 0, 16)
    assert int(none.compact(i32([]))[2]) == 0
    none.resize(none.table(1, 0), i32([1]), none.table(1, 4))
    assert none.poll_error() == cache.MLA_ERR_OUT_OF_PAGES
    assert pool.poll_error() == 0


@pytest.mark.parametrize("pages", [31, 32, 33, 1000, 70001, 300007])
@pytest.mark.parametrize("share", [0.1, 0.5, 0.97])
def test_many_pages(pages, share):
    """Compaction and fresh pages over long lists of pages against numpy."""
    rng = np.random.RandomState(pages)
    kv = torch.arange(pages, dtype=torch.int32, device=DEV).view(torch.uint8).view(pages, 4).repeat(1, 72)
    sc = kv[:, :18].contiguous()
    pool = cache.MLACachePool(kv, "mxfp4", 1, kv_scale=sc)
    refs = (rng.rand(pages) < share) * rng.randint(1, 4, pages)
    pool.refs.copy_(torch.from_numpy(refs.astype(np.int32)))
    alive = np.nonzero(refs)[0]
    live = alive.size
    holes, movers = np.nonzero(refs[:live] == 0)[0], alive[alive >= live]
    place = np.arange(pages)
    place[movers] = holes
    # fresh pages first: the lowest free ones
    want = min(pages - live, 500)
    t = pool.resize(pool.table(2, 0), i32([want // 3, want - want // 3]), pool.table(2, want))
    free = np.nonzero(refs == 0)[0][:want]
    assert t[1].tolist() == free.tolist() and torch.all(pool.refs[torch.from_numpy(free).to(DEV)] == 1)
    pool.resize(t, i32([0, 0]), pool.table(2, 0))
    assert pool.refs.tolist() == refs.tolist()
    out = (torch.empty(live, dtype=torch.int32, device=DEV), torch.full((pages,), -1, dtype=torch.int32, device=DEV), i32([0]))
    kv0 = kv.clone()
    pool.compact(torch.from_numpy(alive.astype(np.int32)).to(DEV), out=out)
    assert pool.poll_error() == 0
    assert int(out[2]) == live and out[0].tolist() == place[alive].tolist()
    new = np.zeros(pages, dtype=np.int64)
    new[place[alive]] = refs[alive]
    assert out[1].tolist() == new.tolist() and pool.refs.tolist() == refs.tolist()
    kv0[torch.from_numpy(holes).to(DEV)] = kv0[torch.from_numpy(movers).to(DEV)]
    assert torch.equal(kv, kv0) and torch.equal(pool.kv_scale, kv0[:, :18])


def test_long_tables_of_many_sequences():
    """Thousands of sequences over pages of one row, some empty, forked and cut."""
    rng = np.random.RandomState(0)
    lens = rng.randint(0, 40, 3000).tolist()
    pages = 2 * sum(lens) + 10
    pool = new_pool("fp8", pages, 1)
    t0 = pool.resize(pool.table(3000, 0), i32(lens), pool.table(3000, sum(lens)))
    assert t0[1].tolist() == list(range(sum(lens)))
    parents = rng.randint(0, 3000, 2500).tolist()
    t1 = pool.fork(t0, i32(parents), pool.table(2500, sum(lens[p] for p in parents)))
    at = np.cumsum([0] + lens)
    want = [list(range(at[p], at[p + 1])) for p in parents]
    assert [s[0] for s in seqs_of(t1, 1)] == want
    counts = np.ones(pages, dtype=np.int64)
    counts[sum(lens):] = 0
    for w in want:
        counts[w] += 1
    assert pool.refs.tolist() == counts.tolist()
    t2 = pool.resize(t0, i32([n // 2 for n in lens]), pool.table(3000, sum(lens)))
    assert [s[0] for s in seqs_of(t2, 1)] == [list(range(at[i], at[i] + n // 2)) for i, n in enumerate(lens)]
    assert pool.poll_error() == 0


def test_long_tables_with_part_filled_pages():
    """Tables of over 131072 entries whose sequences end inside a page: forks copy
    it, and so does a cut into a shared page."""
    rng = np.random.RandomState(1)
    page, n = 2, 600
    lens = rng.randint(300, 700, n).tolist()
    cnt = [-(-x // page) for x in lens]
    pool = new_pool("mxfp4", 3 * sum(cnt) + 10, page)
    t0 = pool.resize(pool.table(n, 0), i32(lens), pool.table(n, sum(cnt)))
    at = np.cumsum([0] + cnt)
    pages = [list(range(at[i], at[i + 1])) for i in range(n)]
    assert [s[0] for s in seqs_of(t0, page)] == pages
    before = bytes_of(pool)
    t1 = pool.fork(t0, i32(list(range(n))), pool.table(n, sum(cnt)))
    fresh, want = sum(cnt), []
    for i in range(n):
        row = list(pages[i])
        if lens[i] % 2:
            row[-1], fresh = fresh, fresh + 1
        want.append(row)
    assert [s[0] for s in seqs_of(t1, page)] == want
    now = bytes_of(pool)
    odd = [i for i in range(n) if lens[i] % 2]
    assert torch.equal(now[:, [want[i][-1] for i in odd], 0], before[:, [pages[i][-1] for i in odd], 0])
    assert torch.equal(now[:, [want[i][-1] for i in odd], 1], before[:, [want[i][-1] for i in odd], 1])
    # cut to an odd length inside shared pages, and others grown
    new = [x // 2 | 1 if i % 2 else x + 5 for i, x in enumerate(lens)]
    t2 = pool.resize(t1, i32(new), pool.table(n, sum(-(-x // page) for x in new)))
    assert pool.poll_error() == 0
    for i, (row, length) in enumerate(seqs_of(t2, page)):
        assert length == new[i] and len(row) == -(-new[i] // page)
        if i % 2:  # its last page is a copy of the shared one's first row
            j = len(row) - 1
            assert row[:j] == want[i][:j] and row[j] >= fresh
            assert torch.equal(bytes_row(pool, row[j], 0), before[:, pages[i][j], 0])
        else:
            assert row[:cnt[i]] == want[i]
    counts = torch.zeros(pool.num_pages, dtype=torch.int32)
    for t in (t0, t2):
        counts.index_add_(0, t[1][:int(t[0][-1])].long().cpu(), torch.ones(int(t[0][-1]), dtype=torch.int32))
    assert torch.equal(pool.refs.cpu(), counts)


@pytest.mark.parametrize("kv_dtype", DTYPES)
@pytest.mark.parametrize("page", [1, 16, 64])
def test_a_run_with_the_decode(orc, kv_dtype, page):  # noqa: F811
    """Prompts appended, forked, continued, parents ended, pages compacted: at
    each stage the decode of the paged cache agrees with the fp64 oracle on the
    rows that each sequence was given, and compaction changes no bit."""
    lens, extra = [70, 0, 131, 64], 3
    parents = [0, 2, 2, 3, 1]
    inp = synth.make_inputs(lens, kv_dtype, seed=page)
    g = gen(page)
    scale = float(inp.kv_scale[0]) if kv_dtype == "fp8" else 1.0
    pool = cache.MLACachePool.allocate(kv_dtype, 700 // page + 12, page, num_layers=1, device=DEV, kv_scale=scale)
    rows = inp.kv_bf16
    room = 900 // page + 20
    table = pool.resize(pool.table(4, 0), i32(lens), pool.table(4, room))
    slots, _ = pool.slots(table, inp.kv_indptr.to(DEV), sum(lens))
    pool.append(rows.to(DEV)[:, :512], rows.to(DEV)[:, 512:], slots)

    def decode(table, lens, q):
        counts = [-(-n // page) for n in lens]
        last = [n - (c - 1) * page if c else 0 for n, c in zip(lens, counts)]
        dec = binding.PagedMLADecoder([0] + np.cumsum(counts).tolist(), last, page, pool.num_pages, kv_dtype, device=DEV)
        out, lse = dec(q.to(DEV), pool.kv[0], table[0], table[1], table[2],
                       torch.arange(len(lens) + 1, dtype=torch.int32, device=DEV),
                       kv_scale=pool.kv_scale[0] if kv_dtype == "mxfp4" else pool.kv_scale)
        assert dec.poll_error() == 0 and pool.poll_error() == 0
        return out, lse

    def check(table, seqs, what):
        lens = [s.shape[0] for s in seqs]
        flat = torch.cat(seqs)
        ref_in = synth.make_inputs(lens, kv_dtype, seed=5)
        ref_in.kv_bf16 = flat
        if kv_dtype == "bf16":
            ref_in.kv = flat.contiguous()
        elif kv_dtype == "fp8":  # with the scale the cache was filled under
            ref_in.kv = (flat.float() / inp.kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            ref_in.kv_scale = inp.kv_scale
        else:
            ref_in.kv, ref_in.block_scales = synth.quantize_mxfp4(flat)
        out, lse = decode(table, lens, ref_in.q)
        ref, ref_lse = orc.decode(CODES[kv_dtype], ref_in.q, ref_in.kv, ref_in.kv_indptr, ref_in.qo_indptr,
                                  kv_scale=None if ref_in.kv_scale is None else ref_in.kv_scale.numpy(),
                                  block_scales=None if ref_in.block_scales is None else ref_in.block_scales.numpy())
        assert_parity(out.double().cpu().numpy(), ref, lse.double().cpu().numpy(), ref_lse, what,
                      gate_terms(ref_in, ref, ref_lse))
        return out, lse, ref_in.q

    seqs = list(rows.split(lens))
    check(table, seqs, "prompts")
    forks = pool.fork(table, i32(parents), pool.table(5, room))
    seqs = [seqs[p] for p in parents]
    check(forks, seqs, "forks")
    pool.free(table[1][:int(table[0][-1])].contiguous())  # the prompts end
    lens = [s.shape[0] + extra for s in seqs]
    forks = pool.resize(forks, i32(lens), pool.table(5, room))
    new = torch.randn(5 * extra, 576, generator=g).to(torch.bfloat16)
    slots, at = pool.slots(forks, i32([extra * b for b in range(6)]), 5 * extra,
                           rows=torch.empty(5 * extra, dtype=torch.int32, device=DEV))
    assert at.tolist() == [n - extra + i for n in lens for i in range(extra)]
    pool.append(new.to(DEV)[:, :512], new.to(DEV)[:, 512:], slots)
    seqs = [torch.cat([s, x]) for s, x in zip(seqs, new.split(extra))]
    out, lse, q = check(forks, seqs, "continued forks")
    held = sum(-(-n // page) for n in lens)
    idx, refs, live = pool.compact(forks[1][:held])
    assert pool.poll_error() == 0 and int(forks[0][-1]) == held
    assert int(idx.max()) < int(live) and int((refs > 0).sum()) == int(live)
    out2, lse2 = decode((forks[0], idx, forks[2]), lens, q)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # and every sequence reads back as it was stored
    slots, _ = pool.slots((forks[0], idx, forks[2]), i32(np.cumsum([0] + lens).tolist()), sum(lens))
    back = pool.gather(slots).cpu()
    if kv_dtype == "bf16":
        assert torch.equal(back, torch.cat(seqs))


def test_a_captured_decode_step():
    """Table growth, slots and append captured once and replayed: each replay
    appends another row (the table is grown by the replay itself)."""
    page, lens = 16, [15, 40]
    pool = cache.MLACachePool.allocate("bf16", 40, page, device=DEV)
    table = pool.resize(pool.table(2, 0), i32(lens), pool.table(2, 12))
    g = gen(1)
    x0 = torch.randn(sum(lens), 576, generator=g).to(torch.bfloat16).to(DEV)
    slots, _ = pool.slots(table, i32([0, 15, 55]), 55)
    pool.append(x0[:, :512], x0[:, 512:], slots)
    spare = pool.table(2, 12)
    length, x = i32(lens), torch.zeros(2, 576, dtype=torch.bfloat16, device=DEV)
    qo, slots, rows = i32([0, 1, 2]), i32([0, 0]), i32([0, 0])

    def step():
        length.add_(1)
        pool.resize(table, length, spare)
        for a, b in zip(table, spare):
            a.copy_(b)
        pool.slots(table, qo, 2, slots=slots, rows=rows)
        pool.append(x[:, :512], x[:, 512:], slots)

    step()  # once outside the capture
    graph = torch.cuda.CUDAGraph()
    saved = [t.clone() for t in (length, pool.refs, *table)]
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((length, pool.refs, *table), saved):
        t.copy_(s)
    want = [[x0[:15].cpu()], [x0[15:].cpu()]]
    for b in range(2):
        want[b].append(torch.zeros(1, 576, dtype=torch.bfloat16))
    for i in range(20):
        y = torch.randn(2, 576, generator=g).to(torch.bfloat16)
        x.copy_(y)
        graph.replay()
        for b in range(2):
            want[b].append(y[b:b + 1])
    torch.cuda.synchronize()
    assert pool.poll_error() == 0
    lens = [n + 21 for n in lens]
    assert length.tolist() == lens and rows.tolist() == [n - 1 for n in lens]
    slots, _ = pool.slots(table, i32([0, lens[0], sum(lens)]), sum(lens))
    assert torch.equal(pool.gather(slots).cpu(), torch.cat([torch.cat(w) for w in want]))


def test_two_graphs_share_a_pool():
    """Calls captured into two graphs and replayed in turn, the pool's workspace theirs both."""
    page = 8
    pool = new_pool("fp8", 200, page)
    t0 = pool.resize(pool.table(3, 0), i32([20, 0, 33]), pool.table(3, 30))
    t1, t2, parents = pool.table(5, 60), pool.table(5, 60), i32([0, 2, 2, 1, 0])
    longer = i32([29, 40, 33, 5, 20])
    held = pool.refs.clone()

    def one():
        pool.fork(t0, parents, t1)

    def two():
        pool.resize(t1, longer, t2)

    graphs = []
    for call in (one, two):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    want = None
    for _ in range(3):
        pool.refs.copy_(held)
        for t in (t1, t2):
            for x in t:
                x.fill_(-3)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = (pool.refs.tolist(), seqs_of(t1, page), seqs_of(t2, page))
        want = want or got
        assert got == want and pool.poll_error() == 0
    model = PoolModel(200, page)
    seqs = model.resize([([], 0)] * 3, [20, 0, 33])
    forks = model.fork(seqs, parents.tolist())
    assert want[1] == forks
    assert want[2] == model.resize(forks, longer.tolist()) and want[0] == model.refs


def test_pools_on_streams_of_their_own():
    """Two pools used at once from two streams, each as the model says."""
    rng = np.random.RandomState(3)
    pools = [new_pool("bf16", 300, 4), new_pool("mxfp4", 17000, 2)]
    streams = [torch.cuda.Stream() for _ in pools]
    models = [PoolModel(300, 4), PoolModel(17000, 2)]
    tables = [p.table(4, 0) for p in pools]
    seqs = [[([], 0)] * 4 for _ in pools]
    for _ in range(12):
        lengths = [[int(x) for x in rng.randint(0, 200, 4)] for _ in pools]
        dev = [i32(x) for x in lengths]
        outs = [p.table(4, 500) for p in pools]
        torch.cuda.synchronize()
        for p, s, t, n, o in zip(pools, streams, tables, dev, outs):
            p.resize(t, n, o, stream=s)
        torch.cuda.synchronize()
        for i in range(2):
            seqs[i] = models[i].resize(seqs[i], lengths[i])
            assert seqs_of(outs[i], pools[i].page_size) == seqs[i] and pools[i].refs.tolist() == models[i].refs
        tables = outs
    assert all(p.poll_error() == 0 for p in pools)


@pytest.mark.parametrize("first,width,wide", [(16, 18, 34), (32, 18, 64), (0, 18, 19), (0, 20, 24), (16, 32, 64)])
@pytest.mark.parametrize("page,layers,pages", [(1, 1, 60), (8, 1, 60), (4, 3, 60), (2, 2, 16500), (1, 1, 33000)])
def test_scales_in_columns_of_a_wider_tensor(first, width, wide, page, layers, pages):
    """Only the view's columns are the cache's: every page operator leaves the
    others, and what lies behind the last row, as they were, and does to the view
    what it does to scale rows of their own."""
    g = gen(wide + page)
    rows = pages * page
    kv = torch.randint(0, 256, (layers, rows, 288), generator=g, dtype=torch.uint8).to(DEV)
    # rows behind the last one of a layer: a guard
    store = torch.randint(0, 256, (layers, rows + 16, wide), generator=g, dtype=torch.uint8).to(DEV)
    view = store[:, :rows, first:first + width]
    kv1, own = kv.clone(), view.contiguous()
    before = store.clone()
    pools = [cache.MLACachePool(kv, "mxfp4", page, kv_scale=view), cache.MLACachePool(kv1, "mxfp4", page, kv_scale=own)]
    rng = np.random.RandomState(width)

    def same(what):
        rest = store.clone()
        rest[:, :rows, first:first + width] = before[:, :rows, first:first + width]
        assert torch.equal(rest, before), f"{what}: bytes that are not the cache's"
        assert torch.equal(view, own) and torch.equal(kv, kv1) and torch.equal(pools[0].refs, pools[1].refs), what
        assert all(p.poll_error() == 0 for p in pools), what

    perm = rng.permutation(pages)
    src, dst = i32(perm[:9].tolist() + [pages - 1]), i32(perm[9:18].tolist() + [pages - 1])
    for p in pools:
        p.copy_pages(src, dst)
    same("copy")
    some = i32([0, pages - 1, 3]), i32([pages - 1, 1, 5])
    for p in pools:
        p.copy_pages(*some)
    same("copy into the last page")
    # pages at random places, the last one among them
    lens = [5 * page + page // 2, 0, 3 * page, 6 * page + 1]
    held = [int(x) for x in perm[:20]]
    if pages - 1 not in held:
        held[7] = pages - 1
    seqs, at = [], 0
    for n in lens:
        k = -(-n // page)
        seqs.append((held[at:at + k], n))
        at += k
    tables = []
    for p in pools:
        p.refs[torch.tensor(held[:at], device=DEV)] = 1
        tables.append(table_of(seqs, page, device=DEV))
    parents, cut = i32([0, 3, 3, 2, 0]), i32([2 * page + page // 2, 6 * page + 3, 1, 3 * page, 5 * page])
    for k, p in enumerate(pools):
        tables[k] = p.fork(tables[k], parents, p.table(5, 60))
    same("fork")
    for k, p in enumerate(pools):
        tables[k] = p.resize(tables[k], cut, p.table(5, 60))
    same("resize")
    assert seqs_of(tables[0], page) == seqs_of(tables[1], page)
    idx = [p.compact(t[1][:int(t[0][-1])].contiguous())[0] for p, t in zip(pools, tables)]
    same("compact")
    assert torch.equal(*idx)


def test_two_pools_share_one_scale_tensor():
    """Two caches whose scales lie side by side in one tensor do not see each other."""
    g = gen(77)
    scales = torch.randint(0, 256, (64, 64), generator=g, dtype=torch.uint8).to(DEV)
    kv = [torch.randint(0, 256, (64, 288), generator=g, dtype=torch.uint8).to(DEV) for _ in range(2)]
    a, b = (cache.MLACachePool(x, "mxfp4", 8, kv_scale=scales[:, at:at + 18]) for x, at in zip(kv, (0, 32)))
    want = scales.clone()
    want[8:16, :18], want[56:, 32:50] = scales[:8, :18], scales[16:24, 32:50]
    a.copy_pages(i32([0]), i32([1]))
    b.copy_pages(i32([2]), i32([7]))
    assert a.poll_error() == 0 and b.poll_error() == 0
    assert torch.equal(scales, want)


@pytest.mark.parametrize("stride", [19, 24, 32])
@pytest.mark.parametrize("page,pages", [(8, 90), (4, 16500)])
def test_part_filled_pages_of_any_scale_stride(stride, page, pages):
    """Forks copy, and cuts inside a shared page copy, scale rows of odd and wide strides."""
    pool, model = new_pool("mxfp4", pages, page, 2, stride), PoolModel(pages, page)
    lens = [3 * page + 3, page + 1, 2 * page]
    t0 = pool.resize(pool.table(3, 0), i32(lens), pool.table(3, 20))
    s0 = model.resize([([], 0)] * 3, lens)
    before = bytes_of(pool)
    t1 = pool.fork(t0, i32([0, 1, 0, 2]), pool.table(4, 30))
    s1 = model.fork(s0, [0, 1, 0, 2])
    cut = [2 * page + 1, page + 2, 3 * page + 2, page // 2]
    t2 = pool.resize(t1, i32(cut), pool.table(4, 30))
    s2 = model.resize(s1, cut)
    assert pool.poll_error() == 0 and seqs_of(t1, page) == s1 and seqs_of(t2, page) == s2
    want = before.clone()
    for pages_of, source, n in ((s1[0][0], s0[0][0], 3), (s1[1][0], s0[1][0], 1), (s1[2][0], s0[0][0], 3)):
        want[:, pages_of[-1], :n] = before[:, source[-1], :n]
    assert s2[0][0][-1] != s1[0][0][2] and s2[3][0][-1] != s1[3][0][0]
    want[:, s2[0][0][-1], :1] = want[:, s1[0][0][2], :1]
    want[:, s2[3][0][-1], :page // 2] = want[:, s1[3][0][0], :page // 2]
    assert torch.equal(bytes_of(pool), want)


@pytest.mark.parametrize("pages", [12, 16500, 33000])
def test_tables_that_name_free_pages(pages):
    """A page that nobody holds is not shared, copied, kept or given back, whatever
    the table says, and the fresh page that it may become is the new owner's alone."""
    page, bad = 4, binding.MLA_ERR_DEVICE_INDEX
    held = [0, 2, 3]  # page 1 is the first that a call hands out

    def fresh_pool():
        pool = new_pool("fp8", pages, page)
        pool.refs[torch.tensor(held, device=DEV)] = 1
        return pool, bytes_of(pool)

    def refs(pool, want):
        assert pool.refs[:6].tolist() == want and int(pool.refs[6:].abs().sum()) == 0

    # grown: the free page within the table is dropped, the fresh one comes behind
    pool, before = fresh_pool()
    t = pool.resize((i32([0, 3]), i32([0, 1, 2]), i32([4])), i32([16]), pool.table(1, 9))
    assert pool.poll_error() == bad
    assert t[0].tolist() == [0, 4] and t[1][:4].tolist() == [0, -1, 2, 1] and t[2].tolist() == [4]
    refs(pool, [1, 1, 1, 1, 0, 0])
    # cut: it is not given back, and another sequence's fresh page stays that one's
    pool, before = fresh_pool()
    t = pool.resize((i32([0, 3, 4]), i32([0, 1, 2, 3]), i32([4, 4])), i32([0, 9]), pool.table(2, 9))
    assert pool.poll_error() == bad
    assert t[0].tolist() == [0, 0, 3] and t[1][:3].tolist() == [3, 1, 4]
    refs(pool, [0, 1, 0, 1, 1, 0])
    # forked as a full page
    pool, before = fresh_pool()
    t = pool.fork((i32([0, 3]), i32([0, 1, 2]), i32([4])), i32([0, 0]), pool.table(2, 9))
    assert pool.poll_error() == bad
    assert t[1][:6].tolist() == [0, -1, 2] * 2
    refs(pool, [3, 0, 3, 1, 0, 0])
    # forked as a part-filled last page, next to one whose copy goes into that page
    pool, before = fresh_pool()
    t = pool.fork((i32([0, 2, 4]), i32([0, 1, 2, 3]), i32([2, 3])), i32([0, 1]), pool.table(2, 9))
    assert pool.poll_error() == bad
    assert t[1][:4].tolist() == [0, -1, 2, 1] and t[2].tolist() == [2, 3]
    refs(pool, [2, 1, 2, 1, 0, 0])
    before[:, 1, :3] = before[:, 3, :3]
    assert torch.equal(bytes_of(pool), before)
    # cut inside it
    pool, before = fresh_pool()
    t = pool.resize((i32([0, 2]), i32([0, 1]), i32([4])), i32([6]), pool.table(1, 9))
    assert pool.poll_error() == bad
    assert t[1][:2].tolist() == [0, -1]
    refs(pool, [1, 0, 1, 1, 0, 0])
    assert torch.equal(bytes_of(pool), before) and pool.poll_error() == 0


@pytest.mark.parametrize("go_on", ["assign", "copy", "old", "in place"])
def test_counts_that_compact_wrote_elsewhere(go_on):
    """compact(out=...) leaves the pool's counts by the old numbers: calls that
    change counts refuse until it is said which counts go on, and then a grown
    sequence gets no page that holds live rows."""
    page = 4
    pool, model = new_pool("fp8", 12, page), PoolModel(12, page)
    lens = [8, 6, 9]
    t = pool.resize(pool.table(3, 0), i32(lens), pool.table(3, 12))
    seqs = model.resize([([], 0)] * 3, lens)
    t2 = pool.resize(t, i32([0, 6, 9]), pool.table(3, 12))  # pages 0 and 1 become holes
    seqs = model.resize(seqs, [0, 6, 9])
    entries = t2[1][:5].contiguous()
    out = (torch.empty_like(entries), torch.full_like(pool.refs, -1), i32([0]))
    old = pool.refs.clone()
    before = bytes_of(pool)
    got = pool.compact(entries, out=out)
    assert all(a is b for a, b in zip(got, out)) and torch.equal(pool.refs, old)
    pool.compact(entries, out=out)  # again, from the same counts: the same
    moved = (t2[0], out[0], t2[2])
    for call in (lambda: pool.resize(moved, i32([0, 9, 9]), pool.table(3, 12)),
                 lambda: pool.fork(moved, i32([1]), pool.table(1, 12)), lambda: pool.free(out[0])):
        with pytest.raises(ValueError, match="pool.refs"):
            call()
    assert torch.equal(pool.refs, old)
    if go_on == "old":
        pool.refs = pool.refs
        table = t2
    else:
        if go_on == "assign":
            pool.refs = out[1]
        elif go_on == "copy":
            pool.refs.copy_(out[1])
        else:
            moved = (t2[0], pool.compact(entries)[0], t2[2])
        place, _ = model.compact()
        seqs = [([place[g] for g in pages], n) for pages, n in seqs]
        table = moved
    grown = pool.resize(table, i32([5, 9, 9]), pool.table(3, 12))
    want = model.resize(seqs, [5, 9, 9])
    assert seqs_of(grown, page) == want and pool.refs.tolist() == model.refs
    now = bytes_of(pool)
    for (pages, n), (old_pages, m) in zip(want[1:], [([2, 3], 6), ([4, 5, 6], 9)]):
        for r in range(m):
            assert torch.equal(now[:, pages[r // page], r % page], before[:, old_pages[r // page], r % page])
    pool.compact(grown[1][:int(grown[0][-1])].contiguous())  # in place: nothing is refused after it
    pool.free(i32([0]))
    assert pool.poll_error() == 0


def test_compact_in_inference_mode():
    """Counts that are inference tensors: the new ones go on by assignment."""
    with torch.inference_mode():
        pool = cache.MLACachePool.allocate("bf16", 8, 4, device=DEV)
        t = pool.resize(pool.table(2, 0), i32([5, 7]), pool.table(2, 8))
        t = pool.resize(t, i32([0, 7]), pool.table(2, 8))
        idx, refs, live = pool.compact(t[1][:2].contiguous(), out=(i32([0, 0]), torch.empty_like(pool.refs), i32([0])))
        pool.refs = refs
        t = pool.resize((t[0], idx, t[2]), i32([3, 7]), pool.table(2, 8))
        assert seqs_of(t, 4) == [([2], 3), ([0, 1], 7)] and int(live) == 2 and pool.poll_error() == 0


def test_ending_a_batch():
    """A new table's buffer names no page, so that giving it back whole ends no
    hold; lengths of 0 end a batch whose length only the device knows."""
    page = 4
    pool = new_pool("bf16", 20, page)
    t = pool.resize(pool.table(2, 0), i32([9, 6]), pool.table(2, 16))
    assert t[1].tolist() == [0, 1, 2, 3, 4] + [-1] * 11
    forks = pool.fork(t, i32([0, 1]), pool.table(2, 16))
    assert pool.refs[:7].tolist() == [2, 2, 1, 2, 1, 1, 1]
    pool.free(forks[1])  # with its room to spare
    assert pool.poll_error() == 0 and pool.refs[:7].tolist() == [1, 1, 1, 1, 1, 0, 0]
    empty = pool.resize(t, i32([0, 0]), pool.table(2, 0))
    assert pool.poll_error() == 0 and int(pool.refs.sum()) == 0 and empty[0].tolist() == [0, 0, 0]


@pytest.mark.parametrize("pages", [16384, 16385, 32769, 262143, 262145, 300007])
def test_compaction_in_place_of_many_pages(pages):
    """Counts and table rewritten in place while rows move, on both sides of the
    sizes where other kernels take over, then fresh pages from the new counts."""
    rng = np.random.RandomState(pages)
    kv = torch.arange(pages, dtype=torch.int32, device=DEV).view(torch.uint8).view(pages, 4).repeat(1, 144)
    pool = cache.MLACachePool(kv, "fp8", 1, kv_scale=torch.ones(1, device=DEV))
    refs = (rng.rand(pages) < 0.4) * rng.randint(1, 4, pages)
    pool.refs.copy_(torch.from_numpy(refs.astype(np.int32)))
    alive = np.nonzero(refs)[0]
    live = alive.size
    holes, movers = np.nonzero(refs[:live] == 0)[0], alive[alive >= live]
    place = np.arange(pages)
    place[movers] = holes
    table = rng.permutation(np.concatenate([alive, alive[::3], np.full(50, -1)])).astype(np.int32)
    idx = torch.from_numpy(table).to(DEV)
    kv0 = kv.clone()
    got, counts, n = pool.compact(idx, out=(idx, pool.refs, i32([0])))
    assert pool.poll_error() == 0 and int(n) == live
    assert got.tolist() == np.where(table < 0, -1, place[table]).tolist()
    new = np.zeros(pages, dtype=np.int64)
    new[place[alive]] = refs[alive]
    assert pool.refs.tolist() == new.tolist()
    kv0[torch.from_numpy(holes).to(DEV)] = kv0[torch.from_numpy(movers).to(DEV)]
    assert torch.equal(kv, kv0)
    t = pool.resize(pool.table(1, 0), i32([100]), pool.table(1, 100))
    assert pool.poll_error() == 0 and t[1].tolist() == list(range(live, live + 100))
