"""The paged cache's calls as a decoder block uses them: the 4-bit projections before
and after, one graph captured once and replayed over growing sequences, and two calls
at once on streams of their own."""
import threading

import numpy as np
import pytest
import torch

import kv_cases as kc
from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def block(seed, hidden, q_heads, kv_heads, dim):
    """(fused q | k | v layer, output layer) of quantized weights, and their fp16 weights."""
    g = torch.Generator().manual_seed(seed)
    wide = (q_heads + 2 * kv_heads) * dim
    qkv = binding.quantize((torch.randn((hidden, wide), generator=g) * hidden ** -0.5).half().to(DEV), 128)
    out = binding.quantize((torch.randn((q_heads * dim, hidden), generator=g) * (q_heads * dim) ** -0.5).half().to(DEV), 128)
    return qkv, out


def attend(x, qkv, out, cache, batch, rope, heads, dim):
    """One block's attention for the rows x [rows][hidden]."""
    linear = binding.gemv if x.shape[0] <= 16 else binding.gemm
    q_heads, kv_heads = heads
    q, k, v = linear(x, qkv).split([q_heads * dim, kv_heads * dim, kv_heads * dim], 1)
    q = binding.kv_append(q.unflatten(1, (q_heads, dim)), k.unflatten(1, (kv_heads, dim)),
                          v.unflatten(1, (kv_heads, dim)), cache, batch, rope=rope)
    return linear(binding.attention(q, cache, batch).flatten(1), out)


def plain(x, wq, wo, rope, heads, dim):
    """The same for a whole sequence x [tokens][hidden] in 64 bits, with no cache: causal
    attention over all of it, keys and values as they are."""
    q_heads, kv_heads = heads
    y = x.double() @ wq
    q, k, v = y.split([q_heads * dim, kv_heads * dim, kv_heads * dim], 1)
    n = x.shape[0]
    turn = lambda z, h: torch.stack([kc.rotate(z[i].view(h, dim), rope[i], rope.shape[1], False) for i in range(n)])  # noqa: E731
    q, k, v = turn(q, q_heads), turn(k, kv_heads), v.view(n, kv_heads, dim)
    k, v = (z.repeat_interleave(q_heads // kv_heads, 1) for z in (k, v))
    s = torch.stack([q[:, h] @ k[:, h].t() for h in range(q_heads)]) * dim ** -0.5
    s.masked_fill_(torch.ones(n, n).triu(1).bool(), float("-inf"))
    p = torch.softmax(s, -1)
    o = torch.stack([p[h] @ v[:, h] for h in range(q_heads)], 1)
    return o.flatten(1) @ wo


def test_prompt_then_tokens_through_quantized_layers():
    """A prompt and then tokens one at a time, two sequences side by side, each with its own
    length.  Against the block in 64 bits without a cache: keys and values in e4m3 are off
    by 2^-4 of an element at most and about 2^-5.5 in the mean square, which reaches the
    output as that share of it (values), and of the scores' spread (keys); fp16 roundings
    are far smaller.  The bound is 2^-4 in the 2-norm."""
    hidden, heads, dim, page = 512, (8, 2), 64, 16
    qkv, out = block(1, hidden, *heads, dim)
    wq, wo = binding.dequant(qkv).cpu().double(), binding.dequant(out).cpu().double()
    g = torch.Generator().manual_seed(2)
    lens, steps = [37, 5], 9
    xs = [torch.randn((n + steps, hidden), generator=g).half() for n in lens]
    rope = kc.rope_table(64, dim)
    want = [plain(x, wq, wo, rope, heads, dim) for x in xs]
    cache = binding.new_kv_cache(9, page, heads[1], dim, DEV)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7F)
    table = torch.tensor([[7, 2, 0], [5, 1, -1]], dtype=torch.int32, device=DEV)
    kv = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rope = rope.to(DEV)
    batch = binding.KvBatch(table, kv, torch.tensor([0, 37, 42], dtype=torch.int32, device=DEV), 37, 37)
    got = attend(torch.cat([x[:n] for x, n in zip(xs, lens)]).to(DEV), qkv, out, cache, batch, rope, heads, dim)
    rows = [list(got[:37]), list(got[37:])]
    step = binding.KvBatch(table, kv, torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), 1, 64)
    for i in range(steps):
        kv += 1
        x = torch.stack([x[n + i] for x, n in zip(xs, lens)]).to(DEV)
        got = attend(x, qkv, out, cache, step, rope, heads, dim)
        for b in range(2):
            rows[b].append(got[b])
    for b in range(2):
        have = torch.stack(rows[b]).cpu().double()
        assert float((have - want[b]).norm() / want[b].norm()) <= 2.0 ** -4


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_one_graph_for_all_steps(window, sinks):
    """A step of append and attention captured once; replayed while lengths, pages and rows
    change in place, with other work and synchronizations between.  Every replay equals the
    eager calls bit for bit."""
    t = kc.Batch(31, "fp16", [1, 1, 1], [14, 200, 63], 8, 2, 64, 16).fill([13, 199, 62])
    t.width = 20
    t.pages = 60
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(60, generator=g).to(torch.int32).view(3, 20)
    fresh = kc.Batch(32, "fp16", [1] * 3, [320] * 3, 8, 2, 64, 16)
    t.table, t.k, t.v, t.ks, t.vs = table, *(x[:60].clone() for x in (fresh.k, fresh.v, fresh.ks, fresh.vs))
    t.fill([13, 199, 62])
    rope = kc.rope_table(320, 64).to(DEV)
    (c0, b0, q, k, v), (c1, b1, *_) = t.device(max_kv=320), t.device(max_kv=320)
    need = binding.attention_workspace_bytes(3, 8, c0, b0, window, sinks)
    work = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    out = torch.empty((3, 8, 64), dtype=torch.float16, device=DEV)
    turned = torch.empty_like(out)

    def step(cache, batch, out, turned, work):
        binding.kv_append(q, k, v, cache, batch, rope=rope, out=turned)
        binding.attention(turned, cache, batch, window=window, sinks=sinks, out=out, workspace=work)

    x = q._base if q._base is not None else q
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(c0, b0, out, turned, work)
    want, want_turned, other = torch.empty_like(out), torch.empty_like(out), torch.empty_like(work)
    for i in range(12):
        x.copy_(torch.randn(x.shape, generator=g).half() * (1 + i))
        out.fill_(7.0)
        work.fill_(0xFF)
        graph.replay()
        step(c1, b1, want, want_turned, other)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(turned, want_turned), i
        for a, b in ((c0.k, c1.k), (c0.v, c1.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
        assert torch.equal(c0.k_scales, c1.k_scales) and torch.equal(c0.v_scales, c1.v_scales)
        torch.mm(torch.ones((64, 64), device=DEV), torch.ones((64, 64), device=DEV))
        for b in (b0, b1):
            b.kv_lens.add_(1)


def test_two_graphs_with_workspaces_of_their_own_at_once():
    """Two captured calls replayed on two streams at the same time."""
    cases = [kc.Batch(s, "bf16", [1, 1], [4000, 900], 8, 2, 128, 64).fill() for s in (51, 52)]
    calls = []
    for t in cases:
        cache, batch, q, _, _ = t.device()
        want = binding.attention(q, cache, batch)
        need = binding.attention_workspace_bytes(2, 8, cache, batch)
        assert need > 0
        work = torch.empty(need, dtype=torch.uint8, device=DEV)
        out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            for _ in range(8):
                binding.attention(q, cache, batch, out=out, workspace=work)
        calls.append((graph, out, want, torch.cuda.Stream(), (cache, batch, q, work)))
    for _ in range(5):
        for graph, out, _, stream, _ in calls:
            with torch.cuda.stream(stream):
                out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _, _ in calls:
            assert torch.equal(out, want)


def test_calls_from_two_threads():
    """The binding and the library from two host threads, each on a stream of its own."""
    cases = [kc.Batch(s, "fp16", [1, 20], [1500, 300], 8, 2, 64, 32).fill([1499, 280]) for s in (61, 62)]
    ready = [(t.device(), torch.cuda.Stream()) for t in cases]
    want = []
    for t in cases:
        cache, batch, q, k, v = t.device()
        turned = binding.kv_append(q, k, v, cache, batch)
        want.append(binding.attention(turned, cache, batch).cpu())
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            (cache, batch, q, k, v), stream = ready[i]
            with torch.cuda.stream(stream):
                for _ in range(20):
                    turned = binding.kv_append(q, k, v, cache, batch)
                    out = binding.attention(turned, cache, batch)
                stream.synchronize()
                got[i] = out.cpu()
        except Exception as e:          # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for i in range(2):
        assert np.array_equal(got[i].numpy(), want[i].numpy())


def test_binding_refusals():
    t = kc.Batch(71, "fp16", [1, 3], [5, 40], 4, 2, 64, 16).fill()
    cache, batch, q, k, v = t.device()
    with pytest.raises(ValueError, match="multiple of"):
        binding.attention(q[:, :3], cache, batch)
    with pytest.raises(ValueError, match="q must be"):
        binding.attention(q[..., :32], cache, batch)
    with pytest.raises(TypeError, match="k must be fp16"):
        binding.kv_append(None, k[0], v, cache, batch)
    with pytest.raises(TypeError, match="fp16 or bf16"):
        binding.attention(q.float(), cache, batch)
    with pytest.raises(ValueError, match="contiguous"):
        binding.attention(q.contiguous().transpose(0, 1).contiguous().transpose(0, 1), cache, batch)
    with pytest.raises(ValueError, match="out must be"):
        binding.attention(q, cache, batch, out=torch.empty((4, 4, 32), dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError, match="window and sinks"):
        binding.attention(q, cache, batch, window=-1)
    with pytest.raises(binding.AwqError) as e:
        binding.attention(q, cache, batch, scale=float("nan"))
    assert e.value.status == binding.AWQ_ERROR_INVALID_VALUE
    with pytest.raises(TypeError, match="v must be"):
        binding.kv_append(q, k, v.bfloat16(), cache, batch)
    with pytest.raises(ValueError, match="k must be"):
        binding.kv_append(q, k[:, :1], v, cache, batch)
    with pytest.raises(ValueError, match="v must be"):
        binding.kv_append(q, k, v[:2], cache, batch)
    with pytest.raises(ValueError, match="rope must be"):
        binding.kv_append(q, k, v, cache, batch, rope=torch.zeros(64, device=DEV))
    with pytest.raises(binding.AwqError) as e:
        binding.kv_append(q, k, v, cache, batch, rope=torch.zeros((50, 24), device=DEV))
    assert e.value.status == binding.AWQ_ERROR_SHAPE
    with pytest.raises(binding.AwqError) as e:       # rows that begin off a 16-byte border
        binding.attention(torch.empty(4 * 4 * 64 + 1, dtype=torch.float16, device=DEV)[1:].view(4, 4, 64), cache, batch)
    assert e.value.status == binding.AWQ_ERROR_ALIGNMENT
    assert torch.equal(kc.bytes_of(cache.k).cpu(), t.k) and torch.equal(kc.bytes_of(cache.v).cpu(), t.v)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (128, 128), (256, 256)])
@pytest.mark.parametrize("new", [1, 9, 200])
def test_append_then_attend(dim, page, new):
    """The two together, from an empty cache, against both 64-bit forms: attention over the
    codes that the append left."""
    t = kc.Batch(81, "fp16", [new, 2], [new + page // 2, 2], 4, 2, dim, page).fill([page // 2, 0])
    cache, batch, q, k, v = t.device()
    rope = kc.rope_table(new + page, dim // 2)
    turned = binding.kv_append(q, k, v, cache, batch, rope=rope.to(DEV), interleaved=True)
    got = binding.attention(turned, cache, batch).cpu().double()
    t.k, t.v, t.ks, t.vs = kc.bytes_of(cache.k.cpu()), kc.bytes_of(cache.v.cpu()), cache.k_scales.cpu(), cache.v_scales.cpu()
    t.x[:, : 4 * dim] = turned.flatten(1).cpu()
    want, size, reach = kc.attention(t)
    assert bool(((got - want).abs() <= kc.attention_tolerance(t, want, size, reach)).all())


def test_tensors_that_get_other_memory():
    """A cache's or a batch's tensor whose storage is exchanged after construction: the calls
    follow it, and what no longer fits is refused.  (The old memory stays alive throughout.)"""
    t = kc.Batch(72, "fp16", [1, 3], [150, 40], 4, 2, 64, 16).fill()
    cache, batch, q, k, v = t.device()
    old = [x.clone() for x in (cache.k, cache.k_scales, batch.kv_lens, batch.page_table)]
    keep = [x.detach() for x in (cache.k, cache.k_scales, batch.kv_lens, batch.page_table)]
    shorter = torch.tensor([100, 30], dtype=torch.int32, device=DEV)
    want = binding.attention(q, cache, binding.KvBatch(batch.page_table, shorter, batch.q_starts, batch.max_q, batch.max_kv))
    batch.kv_lens.set_(shorter.clone())
    assert torch.equal(binding.attention(q, cache, batch), want)
    cache.k_scales.set_(old[1] * 4)
    again = binding.KvCache(cache.k, cache.v, old[1] * 4, cache.v_scales)
    assert torch.equal(binding.attention(q, cache, batch), binding.attention(q, again, batch))
    fresh = torch.zeros_like(old[0].view(torch.uint8)).view(kc.F8)
    cache.k.set_(fresh)
    turned = binding.kv_append(q, k, v, cache, batch)
    assert bool(fresh.view(torch.uint8).any()) and torch.equal(turned, q)
    assert torch.equal(keep[0].view(torch.uint8), old[0].view(torch.uint8))
    cache.k.set_(fresh[:2].clone())
    with pytest.raises(ValueError, match="v must be"):
        binding.attention(q, cache, batch)
    cache.k.set_(fresh)
    batch.page_table.set_(old[3].t().contiguous())
    with pytest.raises(ValueError, match="kv_lens must be"):
        binding.attention(q, cache, batch)
