"""awq_attention on the GPU against its 64-bit form (tests/kv_cases.py), within the
tolerance that kv_cases.attention_tolerance derives from the kernels' arithmetic."""
import math

import pytest
import torch

import kv_cases as kc
from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu


def check(t, scale=None, window=0, sinks=0, max_q=None, max_kv=None, exact_scores=False):
    cache, batch, q, _, _ = t.device(max_q, max_kv)
    out = torch.full(q.shape, 7.0, dtype=t.dtype, device="cuda:0")
    need = binding.attention_workspace_bytes(q.shape[0], t.q_heads, cache, batch, window, sinks)
    work = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda:0")      # NaN throughout
    got = binding.attention(q, cache, batch, scale=scale, window=window, sinks=sinks, out=out, workspace=work)
    torch.cuda.synchronize()
    assert bool((work[need:] == 0xFF).all())
    want, size, reach = kc.attention(t, scale, window, sinks)
    got = got.cpu()
    n = t.starts[-1]
    assert torch.equal(got[n:], torch.full_like(got[n:], 7.0))       # rows of no sequence
    have, want = got[:n].double(), want[:n]
    assert torch.equal(have.isnan(), want.isnan())
    tol = kc.attention_tolerance(t, want, size[:n], reach[:n] * (not exact_scores))
    off = ((have - want).abs() - tol).nan_to_num(0.0)
    at = int(off.argmax()) if off.numel() else 0
    assert not off.numel() or float(off.max()) <= 0, (at, float(have.flatten()[at]), float(want.flatten()[at]))
    return got


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (4, 4)), (128, 64, (32, 8)), (256, 32, (5, 1)),
                                            (128, 128, (14, 2)), (64, 256, (36, 2)), (128, 16, (1, 1))])
def test_single_tokens(dtype, dim, page, heads):
    """One row a sequence; lengths at the borders of tiles and pages, none among them."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 777, 0]
    new = [1] * 13 + [0]
    check(kc.Batch(1, dtype, new, lens, *heads, dim, page).fill())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 32, (6, 2)), (128, 64, (8, 2)), (256, 16, (7, 1)), (128, 256, (3, 3))])
def test_few_rows(dtype, dim, page, heads):
    new = [2, 5, 16, 3, 0, 8, 1, 11]
    lens = [2, 200, 16, 513, 90, 1000, 64, 70]
    check(kc.Batch(2, dtype, new, lens, *heads, dim, page).fill())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (4, 2)), (128, 64, (4, 1)), (256, 64, (2, 1)),
                                            (128, 32, (5, 1)), (64, 128, (2, 2)), (128, 16, (7, 7))])
@pytest.mark.parametrize("new,lens", [([257], [257]), ([130, 1, 64, 300], [130, 400, 500, 311]), ([65, 513], [1000, 520])])
def test_prompts(dtype, dim, page, heads, new, lens):
    check(kc.Batch(3, dtype, new, lens, *heads, dim, page).fill())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (64, 0), (63, 1), (100, 16), (65, 64), (128, 65), (5000, 4),
                                          (200, 300), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("dim,new,lens", [(128, [1, 1, 1, 1], [700, 64, 3, 301]), (64, [5, 16, 1], [5, 800, 450]),
                                          (128, [400, 70], [600, 70]), (256, [130, 33], [700, 333])])
def test_window(dim, new, lens, window, sinks):
    check(kc.Batch(4, "fp16", new, lens, 4, 2, dim, 32).fill(), window=window, sinks=sinks)


@pytest.mark.parametrize("new", [1, 7, 90])
def test_long_split(new):
    """A long axis in many chunks, joined; one sequence much shorter than the other."""
    check(kc.Batch(5, "fp16", [new, new], [9001, 100], 8, 2, 128, 64).fill())
    check(kc.Batch(5, "bf16", [new], [9001], 16, 2, 64, 16).fill(), window=8000, sinks=70)


@pytest.mark.parametrize("dim,page,heads", [(256, 64, (4, 2)), (128, 16, (5, 1)), (64, 256, (8, 1))])
@pytest.mark.parametrize("new", [1, 40, 130])
def test_long_split_of_other_shapes(dim, page, heads, new):
    check(kc.Batch(18, "bf16", [new, 3], [3001, 2500], *heads, dim, page).fill())
    check(kc.Batch(19, "fp16", [new], [3001], *heads, dim, page).fill(), window=2000, sinks=130)


@pytest.mark.parametrize("dim,heads", [(64, (10, 2)), (128, (4, 1)), (256, (6, 2))])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("window", [0, 100])
def test_few_rows_of_a_call_that_may_be_long(dim, heads, page, window):
    """A wide page table and a large max_kv choose the kernels of long calls, and most of
    their chunks turn out empty."""
    t = kc.Batch(22, "fp16", [9, 1, 0, 30], [900, 64, 5, 31], *heads, dim, page).fill()
    t.width = (1 << 20) // page
    t.table = torch.cat([t.table, torch.full((4, t.width - t.table.shape[1]), -1, dtype=torch.int32)], 1)
    check(t, max_kv=1 << 20, window=window, sinks=7)
    check(t, max_q=1, max_kv=1 << 20, window=window, sinks=7)


@pytest.mark.parametrize("new", [[1, 1, 1], [20, 3, 7], [150, 200, 90]])
@pytest.mark.parametrize("max_q,max_kv", [(1, 1), (0, 0), (3, 10), (10 ** 6, 10 ** 6)])
def test_wrong_hints(new, max_q, max_kv):
    """max_q and max_kv size grids: any values give the same outputs within the tolerance."""
    check(kc.Batch(6, "fp16", new, [600, 205, 90], 4, 2, 64, 16).fill(), max_q=max_q, max_kv=max_kv)


@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1], [30, 6, 5, 9, 3], [100, 170, 65, 9, 130]])
def test_rows_that_see_nothing(new):
    """Rows below position 0, sequences of no tokens, pages that are none: zeros, and the
    other rows as if those tokens were not there.  Rows behind the last sequence stay."""
    t = kc.Batch(7, "fp16", new, [20, 0, 300, 5, 200], 4, 2, 128, 16, extra_rows=3).fill()
    t.table[2, 3] = -1
    t.table[2, 7] = t.pages
    t.table[4, :] = 1 << 30
    check(t)
    check(t, window=40, sinks=3)


@pytest.mark.parametrize("new", [[1, 1], [4, 9], [140, 120]])
def test_not_finite(new):
    """Rows that see a NaN key come out NaN, rows that do not (causality, window, length)
    are not touched; a query's NaN or infinity stays in its row and head."""
    t = kc.Batch(8, "bf16", new, [200, 150], 4, 2, 64, 32).fill()
    for pos, h in ((199 - new[0] // 2, 0), (3, 1)):
        t.k[int(t.table[0, pos // 32]), h, pos % 32] = 0x7F
    check(t)
    check(t, window=30, sinks=2)
    q, _, _ = t.split()
    q[0, 1, 3] = math.nan
    check(t, window=30, sinks=2)


@pytest.mark.parametrize("new", [[1], [70]])
@pytest.mark.parametrize("spread", [1e-4, 30.0])
def test_flat_and_peaked(new, spread):
    """Weights that are all alike, and one that outweighs the rest."""
    check(kc.Batch(9, "fp16", new, [900], 4, 4, 128, 64, spread=spread).fill())


@pytest.mark.parametrize("new", [1, 70])
def test_small_weights_count(new):
    """One key at weight 1 and 4000 others at 2^-13 each, of far larger values: their sum
    is what the output is, and no weight is small enough to be lost."""
    t = kc.Batch(10, "fp16", [new], [4096], 1, 1, 64, 64).fill()
    t.k.zero_()
    t.ks.fill_(1.0)
    t.vs.fill_(1.0)
    t.x.zero_()
    t.x[:, 0] = 8.0                        # q: scale * q . k = k[0]
    first = torch.tensor(9.0).to(kc.F8).view(torch.uint8)          # e^9 = 2^13 times the others
    t.k[int(t.table[0, 0]), 0, 0, 0] = first
    t.v.copy_(torch.tensor(256.0).to(kc.F8).view(torch.uint8).expand_as(t.v))
    t.v[int(t.table[0, 0]), 0, :, 0] = 0
    check(t)


@pytest.mark.parametrize("new", [1, 70])
def test_scales_of_pages_far_apart(new):
    """Pages whose scales differ by 2^30, for keys and values."""
    t = kc.Batch(12, "fp16", [new], [500], 4, 2, 64, 16).fill()
    t.vs.copy_(torch.exp2(torch.randint(-30, 0, t.vs.shape, generator=t.g).float()))
    t.ks.copy_(torch.exp2(torch.randint(-30, -8, t.ks.shape, generator=t.g).float()))
    check(t)


def test_scale_argument_and_types_of_any_size():
    t = kc.Batch(13, "bf16", [1, 100], [300, 200], 4, 2, 128, 64).fill()
    check(t, scale=0.0)
    check(t, scale=-0.3)
    t.x.mul_(2.0 ** 60)                    # bf16 beyond fp16's range: peaked to one key
    t.ks.mul_(2.0 ** -60)
    check(t)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page,new,lens", [(64, [1, 1], [300, 40]), (16, [5, 2], [200, 70]), (64, [140], [300]),
                                           (16, [90, 40], [90, 150])])
def test_scores_of_any_size(dtype, page, new, lens):
    """Scores q k of one product, a power of two and its half: equal ones get equal weights
    whatever fp32 makes of them, and the others are 2^16 and more below: no weight.  So
    nothing of the scores' size comes into the tolerance."""
    t = kc.Batch(23, dtype, new, lens, 4, 2, 64, page).fill()
    code = lambda f: torch.tensor(f).to(kc.F8).view(torch.uint8)  # noqa: E731
    t.k.zero_()
    t.k[..., 0] = torch.where(torch.rand(t.k.shape[:3], generator=t.g) < 0.1, code(1.0), code(0.5))
    t.x.zero_()
    t.x.view(-1, t.dim)[:, 0] = 2.0 ** 10
    for level in [*range(17, 34), 60, 110]:
        t.ks.fill_(2.0 ** (level - 10))
        check(t, scale=1.0, exact_scores=True)
        check(t, scale=-1.0, exact_scores=True)


@pytest.mark.parametrize("new,lens", [([9], [4]), ([70], [20]), ([300], [130])])
@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 1])
def test_widest_window_over_rows_without_a_place(new, lens, window):
    check(kc.Batch(24, "fp16", new, lens, 4, 2, 64, 16).fill(), window=window)


def test_same_bits_twice_and_on_a_side_stream():
    t = kc.Batch(14, "fp16", [1, 5, 90], [3000, 700, 90], 8, 2, 128, 64).fill()
    cache, batch, q, _, _ = t.device()
    a = binding.attention(q, cache, batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = binding.attention(q, cache, batch, stream=side)
    c = binding.attention(q.contiguous(), cache, batch)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_shared_pages():
    """Two sequences over the same pages (a common prefix)."""
    t = kc.Batch(15, "fp16", [1, 1], [200, 200], 4, 2, 64, 16).fill()
    t.table[1] = t.table[0]
    check(t)


def test_cache_beyond_4_gib():
    """Pages past the 2^32nd byte of a cache."""
    t = kc.Batch(16, "fp16", [1, 40], [70, 100], 4, 2, 128, 64).fill()
    pages = (9 << 29) // (2 * 64 * 128)               # 4.5 GiB of keys
    cache, batch, q, k, v = t.device()
    big = binding.new_kv_cache(pages, 64, 2, 128, "cuda:0")
    far = pages - t.pages
    for a, b in ((big.k, cache.k), (big.v, cache.v)):
        a.view(torch.uint8)[far:] = b.view(torch.uint8)
    big.k_scales[far:] = cache.k_scales
    big.v_scales[far:] = cache.v_scales
    moved = binding.KvBatch(torch.where(batch.page_table >= 0, batch.page_table + far, -1), batch.kv_lens,
                            batch.q_starts, batch.max_q, batch.max_kv)
    assert torch.equal(binding.attention(q, big, moved), binding.attention(q, cache, batch))
    assert torch.equal(binding.kv_append(q, k, v, big, moved), binding.kv_append(q, k, v, cache, batch))
    for a, b in ((big.k, cache.k), (big.v, cache.v)):
        assert torch.equal(a[far:].view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(big.k_scales[far:], cache.k_scales) and torch.equal(big.v_scales[far:], cache.v_scales)


def test_no_rows():
    t = kc.Batch(17, "fp16", [0, 0], [5, 0], 2, 2, 64, 16, extra_rows=2).fill()
    check(t)
    cache, batch, q, _, _ = t.device()
    assert binding.attention(q[:0], cache, batch).shape == (0, 2, 64)


@pytest.mark.parametrize("seqs,max_kv", [(70, 1 << 15), (300, 1 << 15), (2100, 1 << 16)])
def test_many_sequences_of_a_call_that_may_be_long(seqs, max_kv):
    """Short sequences, some without tokens or rows, and a long one among them."""
    lens = [(7 * b) % 40 for b in range(seqs)]
    lens[seqs // 2] = 3300
    new = [min(1, n) * (b % 5 != 3) for b, n in enumerate(lens)]
    t = kc.Batch(25, "bf16", new, lens, 2, 1 if seqs < 1000 else 2, 64, 64).fill()
    check(t, max_kv=max_kv)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (8, 2)), (128, 64, (8, 2)), (256, 128, (3, 1))])
@pytest.mark.parametrize("window", [0, 500])
def test_prompts_among_single_tokens(dtype, dim, page, heads, window):
    """Each sequence by the kernel that its own rows call for, in one call; cut keys or not."""
    new = [200, 1, 3, 0, 60, 1, 1, 9, 31, 32, 33, 1]
    lens = [3001, 1500, 2, 7, 60, 1, 900, 400, 31, 700, 33, 64]
    check(kc.Batch(26, dtype, new, lens, *heads, dim, page, extra_rows=2).fill(), window=window, sinks=5)
    check(kc.Batch(27, dtype, [700] + [1, 0, 2] * 30, [900] + [80, 5, 2] * 30, *heads, dim, page).fill(), window=window)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("new", [1, 5])
def test_heads_of_64_over_some_tiles(dtype, page, new):
    """Eight waves to a workgroup: tiles fewer and more than they are."""
    lens = [1400, 1000, 700, new, 65 * 8, 64 * 8 + 1, 64 * 13]
    check(kc.Batch(28, dtype, [new] * 7, lens, 6, 2, 64, page).fill())
    check(kc.Batch(29, dtype, [new] * 7, lens, 6, 2, 64, page).fill(), window=900, sinks=70)
