"""awq_tree_rows and awq_tree_attention on the GPU against their plain forms
(tests/draft_cases.py): bits and positions are equal, outputs within the tolerance that
kv_cases.attention_tolerance derives from the kernels' arithmetic."""
import math

import pytest
import torch

import draft_cases as dc
import kv_cases as kc
from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def trees(t, reach=1.0):
    """Random trees for the batch's rows: (parents of all, bits of all)."""
    words = max(1, -(-max([0, *t.new]) // 32))
    parents, bits = [], []
    for n in t.new:
        one = dc.random_tree(n, t.g, reach)
        parents += one
        bits += dc.bits_of(one, words)[0]
    return parents, bits


def check(t, bits, words=None, scale=None, window=0, sinks=0, max_q=None, max_kv=None):
    cache, batch, q, _, _ = t.device(max_q, max_kv)
    words = max(1, -(-max([0, *t.new]) // 32)) if words is None else words
    mask = dc.mask_of(bits + [0] * (q.shape[0] - len(bits)), words).to(DEV)
    out = torch.full(q.shape, 7.0, dtype=t.dtype, device=DEV)
    need = binding.tree_attention_workspace_bytes(q.shape[0], t.q_heads, cache, batch, window, sinks)
    work = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device=DEV)           # NaN throughout
    got = binding.tree_attention(q, cache, batch, mask, scale=scale, window=window, sinks=sinks, out=out, workspace=work)
    torch.cuda.synchronize()
    assert bool((work[need:] == 0xFF).all())
    full = (1 << 32 * words) - 1
    want, size, reach = dc.tree_attention(t, [x & full for x in bits], scale, window, sinks)
    got = got.cpu()
    n = t.starts[-1]
    assert torch.equal(got[n:], torch.full_like(got[n:], 7.0))       # rows of no sequence
    have, want = got[:n].double(), want[:n]
    assert torch.equal(have.isnan(), want.isnan())
    tol = kc.attention_tolerance(t, want, size[:n], reach[:n])
    off = ((have - want).abs() - tol).nan_to_num(0.0)
    at = int(off.argmax()) if off.numel() else 0
    assert not off.numel() or float(off.max()) <= 0, (at, float(have.flatten()[at]), float(want.flatten()[at]))
    return got


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (4, 4)), (128, 64, (8, 2)), (256, 32, (5, 1)), (128, 128, (14, 2)),
                                            (64, 256, (36, 2)), (128, 16, (1, 1)), (256, 64, (3, 1))])
def test_trees(dtype, dim, page, heads):
    """Trees of one row to several words of them, behind prefixes that end anywhere in a tile."""
    new = [1, 7, 32, 33, 0, 2, 12]
    lens = [1, 64, 95, 300, 9, 66, 12]
    t = kc.Batch(1, dtype, new, lens, *heads, dim, page).fill()
    check(t, trees(t)[1])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 32, (6, 2)), (128, 64, (4, 1)), (256, 16, (4, 2)), (128, 256, (3, 3))])
@pytest.mark.parametrize("new,lens", [([200], [250]), ([100, 1, 64, 129], [130, 400, 500, 129]), ([65, 140], [1000, 147])])
def test_large_trees(dtype, dim, page, heads, new, lens):
    t = kc.Batch(2, dtype, new, lens, *heads, dim, page).fill()
    check(t, trees(t, 0.2)[1])


@pytest.mark.parametrize("dtype,dim,page,heads", [("fp16", 64, 16, (8, 1)), ("bf16", 128, 64, (8, 1)), ("fp16", 256, 32, (16, 1))])
@pytest.mark.parametrize("seqs", [64, 65, 150])
def test_many_large_trees(dtype, dim, page, heads, seqs):
    """More sequences than a wave has lanes, of many lengths, some without rows."""
    new = [0 if b % 7 == 3 else 20 + b * 5 % 24 for b in range(seqs)]
    t = kc.Batch(9, dtype, new, [n + b * 37 % 150 for b, n in enumerate(new)], *heads, dim, page).fill()
    check(t, trees(t, 0.3)[1])


@pytest.mark.parametrize("dim,page,heads", [(64, 16, (8, 2)), (128, 64, (8, 2)), (256, 128, (2, 1)), (128, 32, (5, 5))])
@pytest.mark.parametrize("new,lens", [([1, 5, 16], [300, 5, 777]), ([130, 70], [130, 500])])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_a_chain_is_causal_attention(dtype, dim, page, heads, new, lens):
    """The same outputs as awq_attention, each within its tolerance."""
    t = kc.Batch(3, dtype, new, lens, *heads, dim, page).fill()
    bits = [(2 << r) - 1 for n in new for r in range(n)]
    got = check(t, bits)
    cache, batch, q, _, _ = t.device()
    other = binding.attention(q, cache, batch).cpu().double()
    tol = kc.attention_tolerance(t, *kc.attention(t))
    assert bool(((got.double() - other).abs() <= 2 * tol).all())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (64, 0), (63, 1), (100, 16), (65, 64), (128, 65), (5000, 4),
                                          (200, 300), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("dim,new,lens", [(128, [1, 9, 1, 33], [700, 64, 3, 301]), (64, [5, 16, 1], [5, 800, 450]),
                                          (128, [100, 70], [600, 70]), (256, [130, 33], [400, 333])])
def test_window(dim, new, lens, window, sinks):
    t = kc.Batch(4, "fp16", new, lens, 4, 2, dim, 32).fill()
    check(t, trees(t, 0.3)[1], window=window, sinks=sinks)


@pytest.mark.parametrize("new,lens", [([4, 9], [4, 60]), ([70, 130], [70, 133])])
def test_any_bits(new, lens):
    """Bits that are no tree's: none, all, later rows, rows past the sequence's, a few words more
    than there are rows."""
    t = kc.Batch(5, "fp16", new, lens, 4, 2, 64, 16, extra_rows=2).fill()
    words = -(-max(new) // 32) + 2
    bits = []
    for b, n in enumerate(new):
        for r in range(n):
            some = int(torch.randint(0, 1 << 30, (), generator=t.g)) << (r % 90)
            bits.append((0, (1 << 32 * words) - 1, 1 << n, some, 1 << (n - 1))[r % 5])
    got = check(t, bits, words)
    assert bool((got[0] == 0).all()) and bool((got[2] == 0).all())       # no token before, no bit of a row
    check(t, bits, words, window=20, sinks=2)


def test_fewer_words_than_rows():
    t = kc.Batch(6, "bf16", [50, 3], [90, 20], 4, 2, 64, 16).fill()
    check(t, trees(t)[1], words=1)


@pytest.mark.parametrize("dtype,dim,page,heads", [("fp16", 128, 64, (8, 2)), ("bf16", 64, 16, (16, 2)), ("fp16", 256, 64, (4, 2))])
@pytest.mark.parametrize("new", [1, 7, 64])
def test_long_split(dtype, dim, page, heads, new):
    """A long axis in many chunks, joined; one sequence much shorter than the other."""
    t = kc.Batch(7, dtype, [new, new], [6001, 100], *heads, dim, page).fill()
    bits = trees(t, 0.5)[1]
    check(t, bits)
    check(t, bits, window=4000, sinks=70)


@pytest.mark.parametrize("new", [[1, 3, 1], [20, 3, 7], [80, 64, 90]])
@pytest.mark.parametrize("max_q,max_kv", [(1, 1), (0, 0), (3, 10), (10 ** 6, 10 ** 6)])
def test_wrong_hints(new, max_q, max_kv):
    t = kc.Batch(8, "fp16", new, [600, 205, 90], 4, 2, 64, 16).fill()
    check(t, trees(t)[1], max_q=max_q, max_kv=max_kv)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (8, 2)), (128, 64, (8, 2)), (256, 128, (3, 1))])
@pytest.mark.parametrize("window", [0, 500])
def test_large_trees_among_single_tokens(dtype, dim, page, heads, window):
    new = [200, 1, 3, 0, 60, 1, 1, 9, 31, 32, 33, 1]
    lens = [1501, 1500, 3, 7, 60, 1, 900, 400, 31, 700, 33, 64]
    t = kc.Batch(9, dtype, new, lens, *heads, dim, page, extra_rows=2).fill()
    check(t, trees(t, 0.1)[1], window=window, sinks=5)


@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1], [30, 6, 5, 9, 3], [100, 70, 65, 9, 130]])
def test_rows_that_see_little(new):
    """Rows without a place, sequences of no tokens, pages that are none."""
    t = kc.Batch(10, "fp16", new, [20, 0, 300, 5, 200], 4, 2, 128, 16, extra_rows=3).fill()
    t.table[2, 3] = -1
    t.table[2, 7] = t.pages
    t.table[4, :] = 1 << 30
    bits = trees(t)[1]
    check(t, bits)
    check(t, bits, window=40, sinks=3)


@pytest.mark.parametrize("new", [[2, 3], [9, 16], [140, 100]])
def test_not_finite(new):
    """Rows that see a NaN key come out NaN, its siblings and their children do not."""
    t = kc.Batch(11, "bf16", new, [200, 150], 4, 2, 64, 32).fill()
    pos = 200 - new[0] // 2
    t.k[int(t.table[0, pos // 32]), 0, pos % 32] = 0x7F
    bits = trees(t)[1]
    got = check(t, bits)
    nan = got.isnan().any(-1).any(-1)[: new[0]]
    assert nan.tolist() == [bool(x >> (new[0] - new[0] // 2) & 1) for x in bits[: new[0]]]
    check(t, bits, window=30, sinks=2)


def test_scale_argument_and_values_of_any_size():
    t = kc.Batch(12, "bf16", [9, 100], [300, 200], 4, 2, 128, 64).fill()
    bits = trees(t)[1]
    check(t, bits, scale=0.0)
    t.vs.copy_(torch.exp2(torch.randint(-30, 0, t.vs.shape, generator=t.g).float()))
    t.ks.copy_(torch.exp2(torch.randint(-30, -8, t.ks.shape, generator=t.g).float()))
    check(t, bits)
    t.x.mul_(2.0 ** 60)
    t.ks.mul_(2.0 ** -60)
    check(t, bits)


def test_same_bits_twice_and_on_a_side_stream():
    t = kc.Batch(14, "fp16", [1, 5, 90], [3000, 700, 90], 8, 2, 128, 64).fill()
    cache, batch, q, _, _ = t.device()
    mask = dc.mask_of(trees(t)[1], 3).to(DEV)
    a = binding.tree_attention(q, cache, batch, mask)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = binding.tree_attention(q, cache, batch, mask, stream=side)
    c = binding.tree_attention(q.contiguous(), cache, batch, mask)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_cache_beyond_4_gib():
    t = kc.Batch(16, "fp16", [9, 40], [70, 100], 4, 2, 128, 64).fill()
    pages = (9 << 29) // (2 * 64 * 128)               # 4.5 GiB of keys
    cache, batch, q, _, _ = t.device()
    big = binding.new_kv_cache(pages, 64, 2, 128, DEV)
    far = pages - t.pages
    for a, b in ((big.k, cache.k), (big.v, cache.v)):
        a.view(torch.uint8)[far:] = b.view(torch.uint8)
    big.k_scales[far:] = cache.k_scales
    big.v_scales[far:] = cache.v_scales
    moved = binding.KvBatch(torch.where(batch.page_table >= 0, batch.page_table + far, -1), batch.kv_lens,
                            batch.q_starts, batch.max_q, batch.max_kv)
    mask = dc.mask_of(trees(t)[1], 2).to(DEV)
    assert torch.equal(binding.tree_attention(q, big, moved, mask), binding.tree_attention(q, cache, batch, mask))
    # and a page copied there from the front, kept tokens moved there
    near = torch.tensor([[far + int(t.table[0, 0]), 5], [5, far - 3], [-1, 4], [3, -1], [pages, 1]], dtype=torch.int32, device=DEV)
    binding.kv_copy(near[:1], big)
    binding.kv_copy(near[1:].clone(), big)
    for p in (5, far - 3):
        assert torch.equal(kc.bytes_of(big.k[p]).cpu(), t.k[int(t.table[0, 0])]) and torch.equal(big.v_scales[p].cpu(), t.vs[int(t.table[0, 0])])
    kept = torch.tensor([[2, 3, 8], [0, 30, 39]], dtype=torch.int32, device=DEV)
    counts = torch.tensor([3, 3], dtype=torch.int32, device=DEV)
    lens = binding.kv_keep(kept, counts, big, moved)
    assert torch.equal(lens, binding.kv_keep(kept, counts, cache, batch)) and lens.tolist() == [64, 63]
    assert torch.equal(kc.bytes_of(big.k[far:]), kc.bytes_of(cache.k)) and torch.equal(kc.bytes_of(big.v[far:]), kc.bytes_of(cache.v))


def test_no_rows():
    t = kc.Batch(17, "fp16", [0, 0], [5, 0], 2, 2, 64, 16, extra_rows=2).fill()
    check(t, [])
    cache, batch, q, _, _ = t.device()
    assert binding.tree_attention(q[:0], cache, batch, torch.zeros((0, 1), dtype=torch.int32, device=DEV)).shape == (0, 2, 64)


# ---- rows ----

def rows_of(parents, new, lens, words, max_q=None, extra=0):
    """awq_tree_rows against the plain form."""
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    d = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    batch = binding.KvBatch(d([[0]] * len(new)), d(lens), d(starts), max(new) if max_q is None else max_q, 1)
    total = starts[-1] + extra
    out = (torch.full((total, words), 77, dtype=torch.int32, device=DEV), torch.full((total,), 77, dtype=torch.int32, device=DEV))
    mask, positions = binding.tree_rows(d(parents + [0] * extra), batch, words, out=out)
    mask, positions = mask.cpu(), positions.cpu()
    for b, n in enumerate(new):
        a = starts[b]
        bits, depth = dc.bits_of(parents[a: a + n], words)
        assert torch.equal(mask[a: a + n], dc.mask_of(bits, words)), b
        assert positions[a: a + n].tolist() == [max(lens[b], 0) - n + x for x in depth], b
    assert bool((mask[starts[-1]:] == 77).all()) and bool((positions[starts[-1]:] == 77).all())


@pytest.mark.parametrize("words", [1, 2, 3, 7])
@pytest.mark.parametrize("max_q", [None, 1, 10 ** 6])
def test_rows(words, max_q):
    """Random trees and chains, some of more rows than there are bits; parents that are none."""
    g = torch.Generator().manual_seed(1)
    new, lens = [1, 5, 31, 32, 0, 33, 64, 65, 100, 200], [1, 5, 1000, 40, 3, 2, 64, 2 ** 30, -5, 250]
    parents = []
    for b, n in enumerate(new):
        parents += [t - 1 for t in range(n)] if b % 3 == 2 else dc.random_tree(n, g, 0.4)
    for at in range(3, len(parents), 17):
        parents[at] = (1 << 30, -(1 << 31), 500, -2)[at % 4]
    rows_of(parents, new, lens, words, max_q, extra=3)


@pytest.mark.parametrize("chain", [False, True])
def test_rows_of_a_very_large_tree(chain):
    """More rows than a workgroup holds the parents of."""
    g = torch.Generator().manual_seed(2)
    n = 4500
    rows_of([t - 1 for t in range(n)] if chain else dc.random_tree(n, g, 0.01), [n], [9000], 20)


def test_rows_of_many_trees():
    g = torch.Generator().manual_seed(3)
    new = [(7 * b) % 23 for b in range(700)]
    rows_of([x for n in new for x in dc.random_tree(n, g)], new, [n + b for b, n in enumerate(new)], 1)


def test_binding_refusals():
    t = kc.Batch(71, "fp16", [1, 3], [5, 40], 4, 2, 64, 16).fill()
    cache, batch, q, _, _ = t.device()
    mask = torch.zeros((4, 1), dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="mask must be"):
        binding.tree_attention(q, cache, batch, mask[:3])
    with pytest.raises(ValueError, match="mask must be"):
        binding.tree_attention(q, cache, batch, mask[:, 0])
    with pytest.raises(TypeError, match="mask must be"):
        binding.tree_attention(q, cache, batch, mask.long())
    with pytest.raises(ValueError, match="mask is on"):
        binding.tree_attention(q, cache, batch, mask.cpu())
    with pytest.raises(ValueError, match="multiple of"):
        binding.tree_attention(q[:, :3], cache, batch, mask)
    with pytest.raises(binding.AwqError) as e:
        binding.tree_attention(q, cache, batch, mask[:, :0].contiguous())
    assert e.value.status == binding.AWQ_ERROR_INVALID_VALUE
    with pytest.raises(binding.AwqError) as e:
        binding.tree_attention(q, cache, batch, mask, scale=math.inf)
    assert e.value.status == binding.AWQ_ERROR_INVALID_VALUE
    up = torch.zeros(4, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="parents must be"):
        binding.tree_rows(mask, batch)
    with pytest.raises(TypeError, match="parents must be"):
        binding.tree_rows(up.long(), batch)
    with pytest.raises(ValueError, match="parents is on"):
        binding.tree_rows(up.cpu(), batch)
    with pytest.raises(ValueError, match="mask must be"):
        binding.tree_rows(up, batch, 2, out=(mask, up))
