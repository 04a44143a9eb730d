"""awq_kv_append on the GPU against its 64-bit form (tests/kv_cases.py).

Tolerances: fp32 products and sums of the rotation are each rounded once, so a
rotated element is off by at most 2^-22 (|a| + |b|); q is then rounded once to its
type, a key once to e4m3 (2^-4 of it, or half the least code step, 2^-10, times
the scale).  Without rotation nothing but the code's rounding happens, and codes,
scales and q are equal bit for bit.
"""
import math

import pytest
import torch

import kv_cases as kc
from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu


def run(t, rope=None, interleaved=False, **kw):
    cache, batch, q, k, v = t.device()
    out = torch.full(q.shape, 7.0, dtype=t.dtype, device="cuda:0")
    got = binding.kv_append(q, k, v, cache, batch, rope=None if rope is None else rope.to("cuda:0"),
                            interleaved=interleaved, out=out, **kw)
    torch.cuda.synchronize()
    assert got is out
    return got.cpu(), cache.k.cpu(), cache.v.cpu(), cache.k_scales.cpu(), cache.v_scales.cpu()


def compare(t, got, rope=None, interleaved=False):
    q, k, v, ks, vs = got
    wq, wk, wv, wks, wvs, done = kc.append(t, rope, interleaved)
    assert torch.equal(ks.double(), wks) and torch.equal(vs.double(), wvs)
    # rows without a place are left as they were
    gone = wq.isnan()
    assert torch.equal(q.double()[gone], torch.full_like(wq, 7.0)[gone])
    rq, rk, _ = t.split()
    if rope is None:
        assert torch.equal(q.double()[~gone], wq[~gone])
        assert torch.equal(torch.nan_to_num(k.double(), 999.0), torch.nan_to_num(wk, 999.0))
        assert torch.equal(torch.nan_to_num(v.double(), 999.0), torch.nan_to_num(wv, 999.0))
    else:
        near = 2.0 ** -22 * 2 * rq.double().abs().amax(-1, keepdim=True)
        off = (q.double() - wq).abs()
        ok = off <= near + kc.half_step(t.dtype) * (wq.abs() + near)
        assert bool(ok[~gone].all())
        # keys: half a code step and what the rotation may be off, as values
        s = wks[:, :, None, None]
        near = 2.0 ** -22 * 2 * rk.double().abs().max() / s
        want = torch.nan_to_num(wk, 0.0)
        have = torch.nan_to_num(k.double(), 0.0)
        assert torch.equal(k.double().isnan(), wk.isnan())
        # both are rounded: two half steps apart at most, where the rotation's error tips a tie
        step = torch.maximum(want.abs() * 2.0 ** -3, torch.tensor(2.0 ** -9, dtype=torch.float64))
        assert bool(((have - want).abs() <= step + near).all())
        assert float((have != want).double().mean()) < 1e-3
        assert torch.equal(torch.nan_to_num(v.double(), 999.0), torch.nan_to_num(wv, 999.0))
    # slots behind the last token, and other pages, are left as they were
    kb, vb = kc.bytes_of(k), kc.bytes_of(v)
    assert torch.equal(kb.transpose(1, 2)[~done], t.k.transpose(1, 2)[~done])
    assert torch.equal(vb.permute(0, 3, 1, 2)[~done], t.v.permute(0, 3, 1, 2)[~done])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (4, 4)), (128, 64, (8, 2)), (256, 32, (5, 1)),
                                            (128, 128, (14, 2)), (64, 256, (3, 3))])
def test_prompts_and_tokens(dtype, dim, page, heads):
    """Ragged rows from one to several pages, fresh and partly filled pages."""
    new = [1, 2 * page + 3, 5, 0, page, 1, page - 1]
    lens = [1, 2 * page + 3, page + 9, 7, 3 * page, 2 * page + 1, 2 * page - 1]
    t = kc.Batch(11, dtype, new, lens, *heads, dim, page).fill([n - m for n, m in zip(lens, new)])
    compare(t, run(t))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (32, True), (16, False),
                                             (112, False), (112, True)])
def test_rotation(dtype, rot, interleaved):
    new, lens = [3, 1, 70, 1], [3, 130, 95, 64]
    t = kc.Batch(5, dtype, new, lens, 6, 2, 128, 64).fill([n - m for n, m in zip(lens, new)])
    rope = kc.rope_table(160, rot)
    compare(t, run(t, rope, interleaved), rope, interleaved)


def test_far_positions():
    """A position past 2^17: the table's row is what counts."""
    far = 1 << 17
    t = kc.Batch(6, "fp16", [2], [far + 7], 2, 1, 64, 256).fill([0])
    rope = torch.zeros((far + 8, 64))
    rope[-8:] = kc.rope_table(8, 64)
    compare(t, run(t, rope), rope)


@pytest.mark.parametrize("steps", [40])
def test_token_by_token(steps):
    """One token a step over page borders; larger and larger ones move the scales, and the
    codes already there with them."""
    lens = [1, 14, 31]
    grow = torch.linspace(-6, 6, steps).exp2()
    t = kc.Batch(8, "fp16", [1] * 3, lens, 4, 2, 64, 16).fill([n - 1 for n in lens])
    wide = max(lens) + steps
    t.width = -(-wide // 16)
    t.pages = 3 * t.width
    t.table = torch.randperm(t.pages, generator=t.g).to(torch.int32).view(3, t.width)
    fresh = kc.Batch(9, "fp16", [1] * 3, [16 * t.width] * 3, 4, 2, 64, 16)
    t.k, t.v, t.ks, t.vs = (x[: t.pages].clone() for x in (fresh.k, fresh.v, fresh.ks, fresh.vs))
    t.fill([n - 1 for n in lens])
    for i in range(steps):
        t.x = (torch.randn(t.x.shape, generator=t.g) * grow[i]).half()
        got = run(t)
        compare(t, got)
        t.k, t.v, t.ks, t.vs = kc.bytes_of(got[1]), kc.bytes_of(got[2]), got[3], got[4]
        t.lens = [n + 1 for n in t.lens]


def test_places_that_are_none():
    """Rows below position 0, pages that are none, positions behind the rotation's table,
    lengths behind the page table, rows behind the last sequence."""
    new, lens = [9, 4, 40, 6, 3], [4, 60, 40, 34, 500]
    t = kc.Batch(21, "fp16", new, [n if n < 400 else 64 for n in lens], 4, 2, 64, 16, extra_rows=5)
    t.fill([max(0, n - m) for n, m in zip(t.lens, new)])
    t.table[2, 1] = t.pages
    t.table[2, 2] = -7
    t.lens = lens                                  # the last one counts as 64, the table's width
    rope = kc.rope_table(62, 32)
    compare(t, run(t, rope), rope)


def test_not_finite():
    """A token with a NaN or an infinity in a head: NaN key codes there, zeros among the
    values, and the page's scale from what is finite."""
    new, lens = [20, 3], [20, 30]
    t = kc.Batch(4, "bf16", new, lens, 2, 2, 64, 16).fill([0, 27])
    _, k, v = t.split()
    k[3, 1, 5] = math.nan
    k[4, 0, 63] = math.inf
    v[7, 1, 0] = -math.inf
    v[21, 0, 9] = math.nan
    k[22, 0] = -math.inf
    compare(t, run(t))


@pytest.mark.parametrize("value", [0.0, 1e-30, 448.0 * 2 ** -9, 449.0 * 2 ** -9, 65504.0])
def test_scale_borders(value):
    """The largest magnitude at the borders of a scale; zeros."""
    t = kc.Batch(3, "bf16" if value == 1e-30 else "fp16", [17], [17], 1, 1, 64, 32)
    t.x.copy_(torch.randint(-1, 2, t.x.shape, generator=t.g) * value)
    t.x[:, -1] = value
    compare(t, run(t))


def test_dense_rows_no_queries_and_a_side_stream():
    t = kc.Batch(2, "fp16", [30, 1], [30, 77], 4, 2, 128, 64).fill([0, 76])
    cache, batch, _, k, v = t.device(max_q=1, max_kv=1)          # understated: slower, not wrong
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert binding.kv_append(None, k.contiguous(), v.contiguous(), cache, batch, stream=side) is None
    side.synchronize()
    _, wk, wv, wks, wvs, _ = kc.append(t)
    assert torch.equal(torch.nan_to_num(cache.k.cpu().double(), 9e9), torch.nan_to_num(wk, 9e9))
    assert torch.equal(torch.nan_to_num(cache.v.cpu().double(), 9e9), torch.nan_to_num(wv, 9e9))
    assert torch.equal(cache.k_scales.cpu().double(), wks) and torch.equal(cache.v_scales.cpu().double(), wvs)


@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("held", [0, 1, 3, 6, 13])
@pytest.mark.parametrize("n", [2, 15, 16, 29, 30, 33, 64, 115])
def test_odd_places(max_q, held, n):
    """Rows that begin and end anywhere in a word, a store or a page, whatever the hint."""
    t = kc.Batch(40 + n, "fp16", [n], [held + n], 2, 1, 128, 128).fill([held])
    cache, batch, q, k, v = t.device(max_q=max_q)
    got = binding.kv_append(q, k, v, cache, batch)
    compare(t, (got.cpu(), cache.k.cpu(), cache.v.cpu(), cache.k_scales.cpu(), cache.v_scales.cpu()))


def test_empty_calls():
    t = kc.Batch(2, "fp16", [0, 0], [5, 0], 2, 2, 64, 16).fill()
    got = run(t)
    assert torch.equal(kc.bytes_of(got[1]), t.k) and torch.equal(kc.bytes_of(got[2]), t.v)


@pytest.mark.parametrize("dtype,dim,page", [("fp16", 128, 16), ("bf16", 64, 64)])
@pytest.mark.parametrize("rope", [None, 310])
def test_prompts_among_single_tokens(dtype, dim, page, rope):
    """So many sequences, of such different rows, that workgroups look for their work; some
    without rows, places, pages or rows of the table."""
    new, lens = [300, 2], [340, 1]
    for i in range(160):
        new.append((1, 0, 5, 1, 17)[i % 5])
        lens.append((1, 7, 3, 65 + i, 33)[i % 5])
    t = kc.Batch(31, dtype, new, lens, 4, 2, dim, page, extra_rows=1).fill([n - m for n, m in zip(lens, new)])
    t.table[6, :] = -1
    compare(t, run(t, None if rope is None else kc.rope_table(rope, dim // 2)), None if rope is None else kc.rope_table(rope, dim // 2))
    cache, batch, q, k, v = t.device()
    alone, _, _, _, _ = t.device()
    binding.kv_append(q, k, v, cache, batch)
    binding.kv_append(None, k, v, alone, batch)
    assert torch.equal(cache.k.view(torch.uint8), alone.k.view(torch.uint8))
    assert torch.equal(cache.v.view(torch.uint8), alone.v.view(torch.uint8))


@pytest.mark.parametrize("dtype,dim,page", [("fp16", 128, 64), ("bf16", 64, 16), ("fp16", 256, 32)])
@pytest.mark.parametrize("rot,interleaved", [(None, False), (48, False), (64, True)])
def test_queries_rotated_in_place(dtype, dim, page, rot, interleaved):
    """q_out the dense q itself: the same bits as apart from it."""
    new, lens = [150, 1, 3], [170, 33, 3]
    t = kc.Batch(33, dtype, new, lens, 6, 2, dim, page).fill([n - m for n, m in zip(lens, new)])
    rope = None if rot is None else kc.rope_table(180, rot).to("cuda:0")
    cache, batch, q, k, v = t.device()
    want = binding.kv_append(q, k, v, cache, batch, rope=rope, interleaved=interleaved)
    for max_q in (150, 1):
        cache, batch, q, k, v = t.device(max_q)
        dense = q.contiguous()
        assert binding.kv_append(dense, k, v, cache, batch, rope=rope, interleaved=interleaved, out=dense) is dense
        assert torch.equal(dense, want)
