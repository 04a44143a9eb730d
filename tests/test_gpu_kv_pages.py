"""awq_kv_keep, awq_kv_fork and awq_kv_copy on the GPU against their plain forms
(tests/draft_cases.py).  Codes, scales and whole numbers are equal."""
import math

import pytest
import torch

import draft_cases as dc
import kv_cases as kc
from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def keep(t, kept, counts, width=None, max_q=None):
    """awq_kv_keep, compared with the plain form; the cache's arrays after it."""
    cache, batch, *_ = t.device(max_q)
    width = max(1, max(len(x) for x in kept)) if width is None else width
    rows = torch.full((len(kept), width), 1 << 30, dtype=torch.int32)
    for b, x in enumerate(kept):
        rows[b, : len(x)] = torch.tensor(x, dtype=torch.int32)
    out = torch.full((len(kept),), 77, dtype=torch.int32, device=DEV)
    got = binding.kv_keep(rows.to(DEV), torch.tensor(counts, dtype=torch.int32, device=DEV), cache, batch, out=out)
    torch.cuda.synchronize()
    assert got is out
    padded = [x + [1 << 30] * (width - len(x)) for x in kept]
    K, V, ks, vs, lens, may = dc.keep(t, padded, counts)
    assert got.tolist() == lens
    k, v = cache.k.cpu(), cache.v.cpu()
    assert torch.equal(cache.k_scales.cpu().double(), ks) and torch.equal(cache.v_scales.cpu().double(), vs)
    nan = lambda x: torch.nan_to_num(x, 999.0)  # noqa: E731
    assert torch.equal(nan(k.double()), nan(K)) and torch.equal(nan(v.double()), nan(V))
    kb, vb = kc.bytes_of(k), kc.bytes_of(v)
    assert torch.equal(kb.transpose(1, 2)[~may], t.k.transpose(1, 2)[~may])
    assert torch.equal(vb.permute(0, 3, 1, 2)[~may], t.v.permute(0, 3, 1, 2)[~may])
    return cache


def subset(n, m, g):
    return torch.sort(torch.randperm(n, generator=g)[:m]).values.tolist()


@pytest.mark.parametrize("dim,page,heads", [(64, 16, (4, 4)), (128, 64, (8, 2)), (256, 32, (5, 1)), (128, 128, (14, 2)),
                                            (64, 256, (3, 3)), (256, 256, (1, 1)), (128, 16, (2, 2))])
def test_accepted_paths(dim, page, heads):
    """A few of a tree's rows, at any place of a page: none, one, all."""
    new = [1, 7, 64, 33, 12, 0, 20, 64, 5, 90]
    lens = [1, 7, 200, 100, 15, 9, page + 10, 3 * page + 64, 2 * page + 2, 400]
    t = kc.Batch(1, "fp16", new, lens, *heads, dim, page).fill()
    counts = [1, 3, 5, 0, 12, 0, 7, 9, 1, 40]
    kept = [subset(n, min(c, n), t.g) for n, c in zip(new, counts)]
    kept[4] = list(range(12))                          # all of them, in place
    kept[6] = list(range(7))                           # the first ones
    keep(t, kept, counts)
    keep(t, kept, [c + 3 for c in counts], width=100)  # the lists end before the counts
    keep(t, [x[::-1] for x in kept], counts)           # that do not ascend end at once


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 256), (256, 32)])
@pytest.mark.parametrize("share", [0.03, 0.5, 0.97])
def test_evictions(dim, page, share):
    """Whole sequences thinned out over many pages."""
    new = [700, 64, 1, 257]
    t = kc.Batch(2, "fp16", new, new, 2, 2, dim, page).fill()
    kept = [subset(n, max(1, int(n * share)), t.g) for n in new]
    keep(t, kept, [len(x) for x in kept], max_q=1)
    some = [x[: len(x) // 2] for x in kept]
    keep(t, some, [len(x) for x in some])


@pytest.mark.parametrize("dim,page,dead", [(64, 16, False), (128, 64, True), (256, 256, False), (64, 32, True), (128, 128, True)])
@pytest.mark.parametrize("new,counts", [([3000, 1500], [120, 70]), ([1100, 900, 40], [500, 899, 1]), ([2000], [300])])
def test_many_kept_rows(dim, page, dead, new, counts):
    """More rows than one workgroup takes, few and many of a stretch, after tokens that stay, with
    scales far apart and, among others, pages that are none and codes that are NaN."""
    lens = [n + 21 * b for b, n in enumerate(new)]
    t = kc.Batch(8, "fp16", new, lens, 2, 2, dim, page).fill()
    t.ks.copy_(torch.exp2(torch.randint(-12, 0, t.ks.shape, generator=t.g).float()))
    t.vs.copy_(torch.exp2(torch.randint(-12, 0, t.vs.shape, generator=t.g).float()))
    if dead:
        t.table[0, 3], t.table[0, 1] = -1, t.pages
        for j in range(0, lens[0], 7):
            id = int(t.table[0, j // page])
            if 0 <= id < t.pages:
                t.k[id, 1, j % page] = 0x7F
    keep(t, [subset(n, m, t.g) for n, m in zip(new, counts)], counts)


def test_cache_beyond_4_gib():
    """Pages whose codes lie past 2^32 bytes: copied, and compacted from one to another."""
    heads, page, dim, pages = 8, 256, 256, 8300
    cache = binding.new_kv_cache(pages, page, heads, dim, DEV)
    assert cache.k.numel() > 1 << 32
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    g = torch.Generator(device=DEV).manual_seed(1)
    rows = torch.randint(0, 0x7E, (3, heads, page, dim), generator=g, device=DEV, dtype=torch.uint8)
    last = [pages - 1, pages - 2, pages - 3]
    for i in range(3):
        k[i], v[i] = rows[i], rows[i].transpose(1, 2)
        k[last[i]], v[last[i]] = 0x7F, 0x7F
    cache.k_scales[:3], cache.v_scales[:3] = 0.5, 0.25
    cache.k_scales[pages - 3:], cache.v_scales[pages - 3:] = 7.0, 7.0
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    binding.kv_copy(ints([[i, last[i]] for i in range(3)]), cache)
    for i in range(3):
        assert torch.equal(k[last[i]], rows[i]) and torch.equal(v[last[i]], rows[i].transpose(1, 2))
    assert bool((cache.k_scales[pages - 3:] == 0.5).all()) and bool((cache.v_scales[pages - 3:] == 0.25).all())
    tokens = rows.transpose(0, 1).flatten(1, 2)                              # [heads][3 pages][dim]
    batch = binding.KvBatch(ints([last]), ints([3 * page]), ints([0, 3 * page]), 3 * page, 3 * page)
    for kept in (list(range(0, 3 * page, 3)), [1, 200]):                     # many; then few of those
        n = len(kept)
        lens = binding.kv_keep(ints([kept]), ints([n]), cache, batch)
        assert lens.tolist() == [n]
        tokens = torch.cat([tokens[:, kept], tokens[:, n:]], 1)
        for i in range(3):
            have = tokens[:, i * page: (i + 1) * page]
            assert torch.equal(k[last[i]], have) and torch.equal(v[last[i]], have.transpose(1, 2))
            assert torch.equal(k[i], rows[i]) and torch.equal(v[i], rows[i].transpose(1, 2))


@pytest.mark.parametrize("page", [16, 64])
def test_scales_far_apart(page):
    """Codes that become subnormal, or nothing, under the larger scale of a neighbour."""
    t = kc.Batch(3, "fp16", [100], [130], 2, 2, 64, page).fill()
    t.ks.copy_(torch.exp2(torch.randint(-20, 0, t.ks.shape, generator=t.g).float()))
    t.vs.copy_(torch.exp2(torch.randint(-126, 120, t.vs.shape, generator=t.g).float()))
    keep(t, [subset(100, 40, t.g)], [40])
    keep(t, [[0, 1, 2, 99]], [4])


def test_scales_that_are_no_powers_of_two():
    """The quotient is rounded to fp32, and its product with a code (4 bits) to fp32 before e4m3:
    half steps of e4m3 tie only where 2^-24 of the value does, so nearly all codes are equal."""
    t = kc.Batch(4, "fp16", [60], [100], 2, 2, 64, 16).fill()
    t.ks.copy_(torch.rand(t.ks.shape, generator=t.g) + 0.1)
    t.vs.copy_(torch.rand(t.vs.shape, generator=t.g) + 0.1)
    kept = [subset(60, 25, t.g)]
    cache, batch, *_ = t.device()
    lens = binding.kv_keep(torch.tensor(kept, dtype=torch.int32, device=DEV), torch.tensor([25], dtype=torch.int32, device=DEV), cache, batch)
    K, V, ks, vs, want, _ = dc.keep(t, kept, [25])
    assert lens.tolist() == want and torch.equal(cache.k_scales.cpu().double(), ks) and torch.equal(cache.v_scales.cpu().double(), vs)
    for a, b in ((cache.k, K), (cache.v, V)):
        a, b = torch.nan_to_num(a.cpu().double(), 0.0), torch.nan_to_num(b, 0.0)
        assert bool(((a - b).abs() <= torch.maximum(b.abs() * 2.0 ** -3, torch.tensor(2.0 ** -9, dtype=torch.float64))).all())
        assert float((a != b).double().mean()) < 1e-3


@pytest.mark.parametrize("page", [16, 32])
def test_pages_and_places_that_are_none(page):
    """Tokens from a page that is none come as NaN and zeros; a place without a page takes none;
    rows below position 0; a length behind the table."""
    new, lens = [60, 90, 9, 20], [100, 90, 4, 500]
    t = kc.Batch(5, "fp16", new, [n if n < 400 else 64 for n in lens], 2, 2, 64, page).fill()
    t.table[0, 64 // page] = -1
    t.table[1, 0] = t.pages
    t.table[1, 64 // page] = 1 << 30
    t.lens = lens
    t.width = t.table.shape[1]
    t.lens[3] = t.width * page + 300
    kept = [subset(60, 31, t.g), subset(90, 44, t.g), [0, 3], subset(20, 5, t.g)]
    keep(t, kept, [31, 44, 2, 5])


def test_not_finite_codes_move_as_they_are():
    t = kc.Batch(6, "fp16", [40], [70], 2, 2, 64, 16).fill()
    for j in (31, 40, 69):
        t.k[int(t.table[0, j // 16]), 1, j % 16] = 0x7F
    keep(t, [[1, 10, 20, 39]], [4])


def test_wrong_rows_and_a_side_stream():
    """Negative counts, a first row that is none, rows past the sequence's; on another stream."""
    t = kc.Batch(7, "fp16", [9, 9, 9, 9], [20, 30, 40, 50], 2, 2, 64, 16).fill()
    keep(t, [[0, 3], [-1, 3, 5], [2, 9, 10], [4, 4, 5]], [-2, 3, 3, 3])
    cache, batch, *_ = t.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = torch.tensor([[1, 5]] * 4, dtype=torch.int32, device=DEV)
    lens = binding.kv_keep(kept, torch.full((4,), 2, dtype=torch.int32, device=DEV), cache, batch, stream=side)
    side.synchronize()
    K, *_ = dc.keep(t, [[1, 5]] * 4, [2] * 4)
    assert lens.tolist() == [13, 23, 33, 43]
    assert torch.equal(torch.nan_to_num(cache.k.cpu().double(), 9e9), torch.nan_to_num(K, 9e9))


# ---- forks ----

class Pool:
    """A table over shared and own pages of a shuffled pool."""

    def __init__(self, seed, lens, page, width, spare, share=0):
        self.g = torch.Generator().manual_seed(seed)
        need = [-(-max(min(n, width * page), 0) // page) for n in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=self.g).tolist()
        self.table = [[order.pop() for _ in range(n)] + [-1] * (width - n) for n in need]
        for b in range(1, len(lens)):
            for j in range(min(share, need[b], need[0])):
                self.table[b][j] = self.table[0][j]
        self.lens, self.page, self.width = list(lens), page, width

    def device(self):
        d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        cache = binding.new_kv_cache(self.pages, self.page, 1, 64, DEV)
        table = d(self.table).view(len(self.lens), self.width)
        return cache, binding.KvBatch(table, d(self.lens), torch.zeros(len(self.lens) + 1, dtype=torch.int32, device=DEV), 1, 1)


def fork(p, from_, grow, held=None):
    cache, batch = p.device()
    d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    before = [x.clone() for x in (batch.page_table, batch.kv_lens)]
    need = binding.kv_fork_workspace_bytes(len(from_), cache, batch)
    work = torch.full((need + 16,), 0xA5, dtype=torch.uint8, device=DEV)
    hold = None if held is None else torch.tensor(held, dtype=torch.uint8, device=DEV)
    table, lens, copies, missing = binding.kv_fork(d(from_), d(grow), cache, batch, held=hold, workspace=work)
    torch.cuda.synchronize()
    assert bool((work[need:] == 0xA5).all())
    want = dc.fork(p.table, p.lens, from_, grow, p.page, p.pages, held)
    assert lens.tolist() == want[1]
    assert missing.tolist() == [want[3]]
    assert table.tolist() == want[0]
    assert [tuple(x) for x in copies.tolist()] == want[2]
    assert torch.equal(batch.page_table, before[0]) and torch.equal(batch.kv_lens, before[1])
    return want


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("seed", range(4))
def test_forks(page, seed):
    """Sequences that go on, split up, end and begin, with pages enough and too few."""
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi, n: torch.randint(lo, hi, (n,), generator=g).tolist()  # noqa: E731
    lens = r(0, 9 * page, 12) + [0, page, 2 * page]
    for spare in (300, 20, 0):
        p = Pool(seed, lens, page, 12, spare, share=3)
        for n in (1, 15, 70):
            fork(p, r(-2, 17, n), r(-3, 2 * page + 2, n))
            fork(p, r(0, 3, n), [1] * n)
            fork(p, r(0, 15, n), [5] * n, held=r(0, 2, p.pages))


@pytest.mark.parametrize("seqs,new,pages", [(40, 3000, 5000), (2, 70, 70000), (600, 1100, 40)])
def test_many_sequences_and_pages(seqs, new, pages):
    g = torch.Generator().manual_seed(seqs)
    lens = torch.randint(0, 60, (seqs,), generator=g).tolist()
    p = Pool(7, lens, 16, 5, pages)
    fork(p, torch.randint(-1, seqs, (new,), generator=g).tolist(), torch.randint(0, 30, (new,), generator=g).tolist())


def test_a_wide_table():
    """Rows of thousands of pages, growth over many of them."""
    p = Pool(8, [16 * 2500 + 3, 5, 16 * 3000], 16, 6000, 9000)
    fork(p, [0, 2, 1, 0, -1], [16 * 1000, 0, 16 * 2000, 1, 16 * 4000])
    fork(p, [2, -1, 0], [16 * 3001, 2 ** 31 - 1, 2 ** 31 - 1])                  # up to the table's width; too many


def test_lengths_and_pages_out_of_range():
    p = Pool(9, [40, 70, 30], 16, 5, 12)
    p.table[1][1], p.table[1][2], p.table[2][1] = -9, p.pages, 1 << 30
    p.lens = [-4, 500, 30]                              # counts as none; as the table's width
    fork(p, [0, 1, 2, 2, 1], [3, 3, 3, 20, 0])


def test_the_same_page_twice_and_no_sequences():
    p = Pool(10, [40, 40], 16, 4, 5)
    p.table[0][2] = p.table[0][1]                       # a row that has its own page twice
    fork(p, [0, 1], [1, 1])
    cache, _ = p.device()
    e = lambda *x: torch.empty(x, dtype=torch.int32, device=DEV)  # noqa: E731
    batch = binding.KvBatch(e(0, 4), e(0), torch.zeros(1, dtype=torch.int32, device=DEV), 0, 0)
    table, lens, copies, missing = binding.kv_fork(torch.zeros(2, dtype=torch.int32, device=DEV), torch.tensor([17, 16], dtype=torch.int32, device=DEV),
                                                   cache, batch)
    assert table.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]] and lens.tolist() == [0, 0] and missing.tolist() == [0]
    table, lens, copies, missing = binding.kv_fork(e(0), e(0), cache, batch)
    assert table.shape == (0, 4) and copies.shape == (0, 2) and missing.tolist() == [0]


@pytest.mark.parametrize("page,heads,dim", [(16, 1, 64), (64, 8, 128), (256, 3, 256)])
def test_copies(page, heads, dim):
    """Within a cache, and to another with a number of pages of its own; pairs that are none."""
    g = torch.Generator().manual_seed(1)
    new = lambda pages: [torch.randint(0, 256, (pages, heads, page, dim), generator=g, dtype=torch.uint8),  # noqa: E731
                         torch.randint(0, 256, (pages, heads, dim, page), generator=g, dtype=torch.uint8),
                         torch.rand((pages, heads), generator=g), torch.rand((pages, heads), generator=g)]
    a, b = new(9), new(5)
    view = lambda x: binding.KvCache(x[0].to(DEV).view(kc.F8), x[1].to(DEV).view(kc.F8), x[2].to(DEV), x[3].to(DEV))  # noqa: E731
    ca, cb = view(a), view(b)
    pairs = [(3, 0), (-1, -1), (3, 7), (8, 1), (5, -1), (9, 2), (-4, 4), (2, 9), (2, 1 << 30)]
    d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    binding.kv_copy(d(pairs), ca)
    for x in a:
        x[0], x[7], x[1] = x[3].clone(), x[3].clone(), x[8].clone()
    same = lambda c, x: all(torch.equal(p.view(torch.uint8).cpu() if p.dtype == kc.F8 else p.cpu(), y)  # noqa: E731
                            for p, y in zip((c.k, c.v, c.k_scales, c.v_scales), x))
    assert same(ca, a)
    binding.kv_copy(d([(6, 4), (6, 0), (1, 5), (9, 1)]), ca, cb)
    for x, y in zip(a, b):
        y[4], y[0] = x[6], x[6]
    assert same(ca, a) and same(cb, b)
    binding.kv_copy(d([(0, 1)])[:0], ca)
    assert same(ca, a)


def test_binding_refusals():
    t = kc.Batch(71, "fp16", [1, 3], [5, 40], 4, 2, 64, 16).fill()
    cache, batch, *_ = t.device()
    d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    two, kept = d([1, 1]), d([[0], [1]])
    with pytest.raises(ValueError, match="kept must be"):
        binding.kv_keep(kept[:1], two, cache, batch)
    with pytest.raises(TypeError, match="kept must be"):
        binding.kv_keep(kept.long(), two, cache, batch)
    with pytest.raises(ValueError, match="counts must be"):
        binding.kv_keep(kept, two[:1], cache, batch)
    with pytest.raises(ValueError, match="kept is on"):
        binding.kv_keep(kept.cpu(), two, cache, batch)
    with pytest.raises(binding.AwqError) as e:
        binding.kv_keep(kept, two, cache, batch, out=batch.kv_lens)
    assert e.value.status == binding.AWQ_ERROR_INVALID_VALUE
    with pytest.raises(ValueError, match="from_ and grow"):
        binding.kv_fork(two, two[:1], cache, batch)
    with pytest.raises(TypeError, match="grow must be"):
        binding.kv_fork(two, two.long(), cache, batch)
    with pytest.raises(ValueError, match="held must be"):
        binding.kv_fork(two, two, cache, batch, held=torch.zeros(3, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="table must be"):
        binding.kv_fork(two, two, cache, batch, out=(two, two, kept, two))
    many = torch.zeros(2000, dtype=torch.int32, device=DEV)
    with pytest.raises(binding.AwqError) as e:
        binding.kv_fork(many, many, cache, batch, workspace=torch.empty(4, dtype=torch.uint8, device=DEV))
    assert e.value.status == binding.AWQ_ERROR_WORKSPACE
    with pytest.raises(ValueError, match="pairs must be"):
        binding.kv_copy(two, cache)
    with pytest.raises(binding.AwqError) as e:
        binding.kv_copy(d([[0, 1]]), cache, binding.new_kv_cache(3, 32, 2, 64, DEV))
    assert e.value.status == binding.AWQ_ERROR_SHAPE
    assert math.isfinite(1.0) and torch.equal(kc.bytes_of(cache.k).cpu(), t.k)
