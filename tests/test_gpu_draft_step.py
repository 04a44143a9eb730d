"""Drafting as a decoder uses it: trees of drafted tokens through 4-bit projections and the
paged cache, their accepted paths kept, sequences forked; one graph captured once and replayed,
calls from two threads, and the sizes at which launches would be too large."""
import threading

import pytest
import torch

import draft_cases as dc
import kv_cases as kc
from test_gpu_kv_graph import attend, block, plain
from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def draft(x, qkv, out, cache, batch, parents, rope, heads, dim):
    """One block's attention for drafted rows."""
    linear = binding.gemv if x.shape[0] <= 16 else binding.gemm
    q_heads, kv_heads = heads
    mask, positions = binding.tree_rows(parents, batch)
    q, k, v = linear(x, qkv).split([q_heads * dim, kv_heads * dim, kv_heads * dim], 1)
    q = binding.kv_append_at(q.unflatten(1, (q_heads, dim)), k.unflatten(1, (kv_heads, dim)),
                             v.unflatten(1, (kv_heads, dim)), cache, batch, positions, rope)
    return linear(binding.tree_attention(q, cache, batch, mask).flatten(1), out)


def test_draft_accept_fork_through_quantized_layers():
    """Two prompts; twice a drafted tree for each, of which a path is accepted; then each sequence
    forked in two, which go on with tokens of their own.  Every row against the block in 64 bits
    without a cache, over the tokens that its path has.  The bound is that of a prompt and
    single tokens (keys and values in e4m3: 2^-4 in the 2-norm): moving codes rounds nothing, but
    for those that become subnormal, which are below 2^-9 of a page's largest."""
    hidden, heads, dim, page = 512, (8, 2), 64, 16
    qkv, out = block(1, hidden, *heads, dim)
    wq, wo = binding.dequant(qkv).cpu().double(), binding.dequant(out).cpu().double()
    g = torch.Generator().manual_seed(7)
    rope = kc.rope_table(80, dim)
    tokens = lambda n: torch.randn((n, hidden), generator=g).half()  # noqa: E731
    cache = binding.new_kv_cache(20, page, heads[1], dim, DEV)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7F)
    table = ints([[7, 2, 0, 9, -1], [5, 1, 3, 11, -1]])
    paths = [tokens(30), tokens(5)]
    lens = ints([30, 5])
    batch = binding.KvBatch(table, lens, ints([0, 30, 35]), 30, 30)
    attend(torch.cat(paths).to(DEV), qkv, out, cache, batch, rope.to(DEV), heads, dim)
    # row numbers accepted, of each of the steps' trees
    steps = [([[-1, 0, 0, 1, 1, 2, 5], [-1, 0, 1, 0, 3]], [[0, 2, 5, 6], [0, 3]]),
             ([[-1, -1, 0, 1, 3], [-1, 0, 0, 1, 2, 4, 3, 5, 7, 8, 9, 9, 2]], [[1, 3], [0, 2, 4, 5, 7, 8, 9, 11]])]
    for trees, accepted in steps:
        new = [len(t) for t in trees]
        xs = [tokens(n) for n in new]
        lens += ints(new)
        batch = binding.KvBatch(table, lens, ints([0, new[0], sum(new)]), max(new), 64)
        got = draft(torch.cat(xs).to(DEV), qkv, out, cache, batch, ints(sum(trees, [])), rope.to(DEV), heads, dim).cpu().double()
        for b in range(2):
            want = []
            for t in range(new[b]):
                path = [t]
                while trees[b][path[0]] >= 0:
                    path.insert(0, trees[b][path[0]])
                want.append(plain(torch.cat([paths[b], xs[b][path]]), wq, wo, rope, heads, dim)[-1])
            want, have = torch.stack(want), got[sum(new[:b]): sum(new[: b + 1])]
            assert float((have - want).norm() / want.norm()) <= 2.0 ** -4
            paths[b] = torch.cat([paths[b], xs[b][accepted[b]]])
        width = max(len(a) for a in accepted)
        kept = ints([a + [0] * (width - len(a)) for a in accepted])
        lens.copy_(binding.kv_keep(kept, ints([len(a) for a in accepted]), cache, batch))
        assert lens.tolist() == [p.shape[0] for p in paths]
    # each in two, and two tokens more, the second as a plain step
    from_ = [1, 0, 0, 1]
    fresh, lens, copies, missing = binding.kv_fork(ints(from_), ints([2] * 4), cache, batch)
    assert missing.item() == 0
    binding.kv_copy(copies, cache)
    paths = [paths[f] for f in from_]
    for i in range(2):
        lens += 1
        x = tokens(4)
        paths = [torch.cat([p, x[b: b + 1]]) for b, p in enumerate(paths)]
        batch = binding.KvBatch(fresh, lens, ints(range(5)), 1, 64)
        if i == 0:
            got = draft(x.to(DEV), qkv, out, cache, batch, ints([-1] * 4), rope.to(DEV), heads, dim)
        else:
            got = attend(x.to(DEV), qkv, out, cache, batch, rope.to(DEV), heads, dim)
        want = torch.stack([plain(p, wq, wo, rope, heads, dim)[-1] for p in paths])
        assert float((got.cpu().double() - want).norm() / want.norm()) <= 2.0 ** -4


class Step:
    """A step's buffers: three sequences that fork among each other, with trees of n rows each."""

    def __init__(self, seed, n, dtype, dim, page, ctx, heads=(6, 2)):
        self.n, self.heads, self.dim = n, heads, dim
        self.t = kc.Batch(seed, dtype, [n] * 3, [c + n for c in ctx], *heads, dim, page).fill(ctx)
        self.t.width += 12
        spare = 120
        t = self.t
        t.table = torch.cat([t.table, torch.full((3, t.width - t.table.shape[1]), -1, dtype=torch.int32)], 1)
        t.k, t.v = (torch.cat([x, torch.full((spare, *x.shape[1:]), 0x7F, dtype=torch.uint8)]) for x in (t.k, t.v))
        t.ks, t.vs = (torch.cat([x, torch.full((spare, x.shape[1]), float("nan"))]) for x in (t.ks, t.vs))
        self.cache, self.batch, *_ = t.device(max_kv=t.width * page)
        self.cache.k_scales.nan_to_num_(0.0)           # (pages that were never written)
        self.cache.v_scales.nan_to_num_(0.0)
        self.batch.kv_lens.copy_(ints(ctx))            # the tokens before a step's rows
        self.x = torch.zeros((3 * n, (heads[0] + 2 * heads[1]) * dim), dtype=t.dtype, device=DEV)
        self.parents, self.from_, self.rope = ints([-1] * 3 * n), ints([0, 1, 2]), kc.rope_table(700, dim).to(DEV)
        self.kept, self.counts = ints([[0] * n] * 3), ints([0] * 3)
        self.grow = ints([n] * 3)
        rows = 3 * n
        self.mask, self.positions = ints([[0] * -(-n // 32)] * rows), ints([0] * rows)
        self.turned, self.out = (torch.zeros((rows, heads[0], dim), dtype=t.dtype, device=DEV) for _ in range(2))
        self.lens = ints([0] * 3)
        self.table = torch.full_like(self.batch.page_table, -1)
        self.copies, self.missing = ints([[0, 0]] * 3), ints([0])
        need = binding.tree_attention_workspace_bytes(rows, heads[0], self.cache, self.batch)
        self.work = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
        need = binding.kv_fork_workspace_bytes(3, self.cache, self.batch)
        self.work2 = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
        self.next = binding.KvBatch(self.table, self.lens, self.batch.q_starts, n, t.width * page)

    def fresh(self, g):
        """Another step's inputs."""
        n, c = self.n, lambda t, x: t.copy_(torch.as_tensor(x).to(t.dtype))  # noqa: E731
        c(self.x, torch.randn(self.x.shape, generator=g))
        c(self.parents, sum((dc.random_tree(n, g, 0.5) for _ in range(3)), []))
        c(self.from_, torch.randint(0, 3, (3,), generator=g))
        for b in range(3):
            some = [i for i in range(n) if float(torch.rand((), generator=g)) < 0.3]
            c(self.kept[b, : len(some)], some)
            self.counts[b] = len(some)

    def same(self, other):
        """Another one with the same contents, in memory of its own."""
        for name in ("x", "parents", "from_", "kept", "counts"):
            getattr(other, name).copy_(getattr(self, name))

    def run(self):
        """Fork, copy, draft, attend, keep; then the forked table is the present one."""
        q, k, v = self.t.split(self.x)
        binding.kv_fork(self.from_, self.grow, self.cache, self.batch, out=(self.table, self.lens, self.copies, self.missing),
                        workspace=self.work2)
        binding.kv_copy(self.copies, self.cache)
        self.lens.add_(self.n)
        binding.tree_rows(self.parents, self.next, out=(self.mask, self.positions))
        binding.kv_append_at(q, k, v, self.cache, self.next, self.positions, self.rope, out=self.turned)
        binding.tree_attention(self.turned, self.cache, self.next, self.mask, out=self.out, workspace=self.work)
        binding.kv_keep(self.kept, self.counts, self.cache, self.next, out=self.batch.kv_lens)
        self.batch.page_table.copy_(self.table)

    def state(self):
        return [x.cpu() for x in (kc.bytes_of(self.cache.k), kc.bytes_of(self.cache.v), self.cache.k_scales, self.cache.v_scales,
                                  self.out.view(torch.int16), self.turned.view(torch.int16), self.mask, self.positions, self.table,
                                  self.lens, self.copies, self.missing, self.batch.kv_lens)]


SIZES = [(5, "fp16", 64, 16, [14, 200, 63]), (70, "bf16", 128, 64, [10, 130, 64]), (17, "fp16", 256, 32, [300, 1, 0])]


@pytest.mark.parametrize("n,dtype,dim,page,ctx", SIZES)
def test_one_graph_for_all_steps(n, dtype, dim, page, ctx):
    """A whole step captured once and replayed while everything changes in place, with other work
    and synchronizations between.  Every replay equals the eager calls bit for bit, and none
    runs out of pages."""
    one, two = Step(5, n, dtype, dim, page, ctx), Step(5, n, dtype, dim, page, ctx)
    g = torch.Generator().manual_seed(6)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one.run()
    for i in range(6):
        one.fresh(g)
        one.same(two)
        for s in (one, two):
            s.work.fill_(0xFF - i)
            s.work2.fill_(i)
        graph.replay()
        two.run()
        torch.cuda.synchronize()
        torch.mm(torch.ones((64, 64), device=DEV), torch.ones((64, 64), device=DEV))
        for j, (a, b) in enumerate(zip(one.state(), two.state())):
            assert torch.equal(a, b), (i, j)
        assert one.missing.item() == 0
        assert bool(torch.isfinite(one.out.float()).all())


def test_steps_on_two_streams_from_two_threads():
    """Steps of two batches from two host threads, each on a stream of its own: the bits of the
    same steps one after the other."""
    def steps(s, seed):
        g = torch.Generator().manual_seed(seed)
        for _ in range(4):
            s.fresh(g)
            s.run()
        torch.cuda.current_stream().synchronize()
        return s.state()

    want = [steps(Step(8 + i, *SIZES[i]), 20 + i) for i in range(2)]
    both, streams = [Step(8 + i, *SIZES[i]) for i in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                got[i] = steps(both[i], 20 + i)
        except Exception as e:          # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for i in range(2):
        for a, b in zip(want[i], got[i]):
            assert torch.equal(a, b)


def test_two_graphs_with_workspaces_of_their_own_at_once():
    """Two captured steps replayed on two streams at the same time."""
    steps = [Step(30 + i, *SIZES[i]) for i in range(2)]
    same = [Step(30 + i, *SIZES[i]) for i in range(2)]
    graphs, streams = [torch.cuda.CUDAGraph() for _ in steps], [torch.cuda.Stream() for _ in steps]
    g = torch.Generator().manual_seed(31)
    for s, o, graph in zip(steps, same, graphs):
        s.fresh(g)
        s.same(o)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            s.run()
    torch.cuda.synchronize()
    for i in range(4):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        for o in same:
            o.run()
        torch.cuda.synchronize()
        for s, o in zip(steps, same):
            for a, b in zip(s.state(), o.state()):
                assert torch.equal(a, b), i


def test_very_many_sequences():
    """Launches stay within 2^32 threads: compaction of 60000 sequences with 16 heads, and
    40000 rows of trees under a hint that any of 20000 may have them all."""
    seqs, heads = 60000, 16
    cache = binding.new_kv_cache(1, 16, heads, 256, DEV)
    cache.k.view(torch.uint8).fill_(0x31)
    cache.v.view(torch.uint8).fill_(0x32)
    cache.k_scales.fill_(0.25)
    cache.v_scales.fill_(0.25)
    table = torch.full((seqs, 6), -1, dtype=torch.int32, device=DEV)
    table[seqs - 1] = 0                                   # (one page at all places: all tokens have its scales)
    lens = torch.full((seqs,), 90, dtype=torch.int32, device=DEV)
    starts = torch.arange(seqs + 1, dtype=torch.int32, device=DEV) * 80
    batch = binding.KvBatch(table, lens, starts, 80, 90)
    kept = torch.arange(1, 71, dtype=torch.int32, device=DEV).repeat(seqs, 1)
    kept[5, 3] = 0                                        # (does not ascend)
    out = binding.kv_keep(kept, torch.full((seqs,), 70, dtype=torch.int32, device=DEV), cache, batch)
    want = torch.full((seqs,), 80, dtype=torch.int32)
    want[5] = 13
    assert torch.equal(out.cpu(), want)
    assert bool((cache.k.view(torch.uint8) == 0x31).all()) and bool((cache.v.view(torch.uint8) == 0x32).all())
    seqs = 20000
    parents = torch.tensor([-1, 0], dtype=torch.int32, device=DEV).repeat(seqs)
    lens = torch.full((seqs,), 7, dtype=torch.int32, device=DEV)
    batch = binding.KvBatch(torch.zeros((seqs, 1), dtype=torch.int32, device=DEV), lens,
                            torch.arange(seqs + 1, dtype=torch.int32, device=DEV) * 2, 2 * seqs, 7)
    mask, positions = binding.tree_rows(parents, batch, words=33)
    assert torch.equal(positions.cpu(), torch.tensor([5, 6], dtype=torch.int32).repeat(seqs))
    want = torch.zeros((2 * seqs, 33), dtype=torch.int32)
    want[0::2, 0], want[1::2, 0] = 1, 3
    assert torch.equal(mask.cpu(), want)
