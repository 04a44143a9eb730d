"""awq_attention on the GPU, as exact as fp32 weights make it, and at magnitudes where a
kernel's own numbers could leave their types."""
import math

import pytest
import torch

import kv_cases as kc
from w4a16_group_quantized_amd import binding

LOG2E = math.log2(math.e)


def run(t, **kw):
    cache, batch, q, _, _ = t.device(kw.pop("max_q", None), kw.pop("max_kv", None))
    out = binding.attention(q, cache, batch, **kw)
    torch.cuda.synchronize()
    return out.cpu()[: t.starts[-1]].double()


def code(x):
    return torch.tensor(float(x)).to(kc.F8).view(torch.uint8)


def within(have, want, tol):
    assert torch.equal(have.isnan(), want.isnan())
    off = ((have - want).abs() - tol).nan_to_num(0.0)
    at = int(off.argmax())
    assert float(off.max()) <= 0, (at, float(have.flatten()[at]), float(want.flatten()[at]), float(tol.flatten()[at]))


def one_hot(t):
    """Queries of one element each, 0.5 to 8 of either sign, so that a score is one product
    and nothing of a sum's roundings comes into it."""
    q = t.split()[0]
    at = torch.randint(0, t.dim, (*q.shape[:2], 1), generator=t.g)
    size = torch.exp2(torch.randint(-1, 4, at.shape, generator=t.g)) * (torch.randint(0, 2, at.shape, generator=t.g) * 2 - 1)
    q.zero_()
    q.scatter_(-1, at, size.to(q.dtype))
    return t


def fine_tolerance(t, out, size, reach, vmax, weight=2.0 ** -21):
    """Scores of one product each: with log2(e), the scale, the page's scale, the maximum and the
    exponential at most eight roundings of 2^-24 of numbers up to 2 * reach * log2(e) + 16.
    A weight as two halves: 2^-22 of it (twice that, for the output's two sums), and where it
    is so small that its remainder is a subnormal, 2^-25 where the row's largest is 2^5 or more:
    2^-30 of the largest for each key.  Sums over the keys as in kv_cases.attention_tolerance.
    Then the output's own rounding."""
    keys = max([1, *t.lens])
    each = 8 * 2.0 ** -24 * (2 * reach * LOG2E + 16) + weight + (keys / 8 + 64) * 2.0 ** -24
    near = 2 * each[..., None] * size + keys * 2.0 ** -30 * vmax
    return near + kc.half_step(t.dtype) * (out.abs() + near) + torch.finfo(t.dtype).smallest_normal * kc.half_step(t.dtype)


SHAPES = [(64, 16, (4, 2)), (128, 64, (8, 2)), (256, 64, (4, 2)), (256, 16, (2, 2)), (128, 128, (5, 1)), (64, 256, (6, 3))]
ROWS = [([1] * 9, [700, 90, 64, 33, 1000, 1, 500, 65, 300]), ([5, 3, 9], [1000, 64, 400]), ([270, 70], [300, 900])]


def signed_sums(dtype, dim, page, heads, new, lens):
    """Sums of values of either sign come out far below their terms, so weights rounded to one
    half (2^-12 of each term) show in them.  (inputs, the definition's outputs, tolerance)"""
    t = one_hot(kc.Batch(90, dtype, new, lens, *heads, dim, page)).fill()
    t.ks.fill_(2.0 ** -6)
    want, size, reach = kc.attention(t)
    return t, want, fine_tolerance(t, want, size, reach, 448 * float(t.vs.max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", SHAPES)
@pytest.mark.parametrize("new,lens", ROWS)
def test_weights_of_more_than_one_half(dtype, dim, page, heads, new, lens):
    t, want, tol = signed_sums(dtype, dim, page, heads, new, lens)
    within(run(t), want, tol)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("new,lens", ROWS)
def test_the_tolerance_tells_one_half_from_two(dtype, new, lens):
    """The same sums on the CPU with weights as halves: within the tolerance as two, not as one."""
    t, want, tol = signed_sums(dtype, 64, 16, (4, 2), new, lens)
    one, two = torch.zeros_like(want), torch.zeros_like(want)
    q = t.split()[0].double()
    for b, n in enumerate(new):
        rows = slice(t.starts[b], t.starts[b + 1])
        k, v, _ = t.held(b, lens[b])
        hidden = torch.arange(lens[b]) > (lens[b] - n + torch.arange(n))[:, None]
        for h in range(4):
            x = (q[rows, h] @ k[h // 2].t()).masked_fill(hidden, -math.inf) * t.dim ** -0.5
            w = torch.exp(x - x.amax(1, keepdim=True)) * 2.0 ** 11
            lead = w.half().double()
            one[rows, h] = lead @ v[h // 2] / w.sum(1, keepdim=True)
            two[rows, h] = (lead + (w - lead).half().double()) @ v[h // 2] / w.sum(1, keepdim=True)
    within(two.to(t.dtype).double(), want, tol)
    with pytest.raises(AssertionError):
        within(one.to(t.dtype).double(), want, tol)


def scale_of_one():
    """A scale whose product with log2(e) is 1 in fp32, so that scores are in the exponent's units."""
    e = torch.tensor(LOG2E, dtype=torch.float32)
    at = torch.tensor(1 / LOG2E, dtype=torch.float32)
    near = [at, torch.nextafter(at, at * 2), torch.nextafter(at, at * 0)]
    return float(next(s for s in near if float(s * e) == 1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 64), (128, 16), (128, 64), (256, 64), (256, 32)])
@pytest.mark.parametrize("new", [1, 6, 350])
@pytest.mark.parametrize("sign", [1, -1])
def test_maxima_one_step_of_fp32_apart(dtype, dim, page, new, sign):
    """Scores around 2^26, where fp32 has steps of 8: a maximum of 2^23 + 1 such steps (or
    -(2^23 + 3)) and, tiles later, one a step above it.  The weight of the first is 2^-8 of
    the second's; the other keys are far below both."""
    t = kc.Batch(91, dtype, [new], [600], 2, 1, dim, page).fill()
    t.ks.fill_(8.0)
    t.vs.fill_(1.0)
    q = t.split()[0]
    q.zero_()
    q[..., 0], q[..., 1] = 2.0 ** 15, 1.0
    t.k.zero_()
    if sign < 0:
        t.k[..., 0] = code(-288)
    first, later = (1, 2) if sign > 0 else (-3, -2)
    for pos, low, value in ((3, first, 1), (133, later, 2)):
        id, slot = int(t.table[0, pos // page]), pos % page
        t.k[id, 0, slot, 0], t.k[id, 0, slot, 1] = code(256 * sign), code(low)
        t.v[id, 0, :, slot] = code(value)
    want = torch.full((new, 2, dim), (2 + 2.0 ** -8) / (1 + 2.0 ** -8), dtype=torch.float64)
    # the exponential, a quotient and sums of two: a few of 2^-24; the output's rounding
    within(run(t, scale=scale_of_one()), want, want * (kc.half_step(t.dtype) + 2.0 ** -20))


def page_scales(t, level):
    """Values of one sequence: pages' scales 2^level(first token of the page, its number), and
    codes of zero where that is None (the append gives such pages 2^-64)."""
    for j in range(-(-t.lens[0] // t.page)):
        id, e = int(t.table[0, j]), level(j * t.page, j)
        t.vs[id] = 2.0 ** (-64 if e is None else e)
        if e is None:
            t.v[id] = 0
    return t


PATTERNS = {
    "zeros between large values": lambda pos, j: 50 if pos < 700 or pos > 1200 else None,
    "zeros before large values": lambda pos, j: None if pos < 700 else 50,
    "zeros beside large values": lambda pos, j: 60 if j % 3 else None,
    "one and the least normal number": lambda pos, j: 0 if pos < 700 else -126,
    "both in a tile": lambda pos, j: -126 if j % 2 else 0,
    "from end to end": lambda pos, j: 100 if j % 2 else -100,
    "large alone": lambda pos, j: 112,
    "small alone": lambda pos, j: -112,
    "the least normal number alone": lambda pos, j: -126,
}


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 64), (128, 32), (128, 128), (256, 16), (256, 64)])
@pytest.mark.parametrize("new", [1, 6, 270])
@pytest.mark.parametrize("pattern", PATTERNS)
def test_value_scales_from_end_to_end(dim, page, new, pattern):
    """Whatever a cache's scales are, from 2^-126 to values of 2^120 that bf16 holds, nothing on
    the way to an output leaves fp32, and the outputs are as exact as with scales alike."""
    t = one_hot(kc.Batch(92, "bf16", [new], [1500], 4, 2, dim, page)).fill()
    t.ks.fill_(2.0 ** -7)
    page_scales(t, PATTERNS[pattern])
    want, size, reach = kc.attention(t)
    within(run(t), want, fine_tolerance(t, want, size, reach, 448 * float(t.vs[t.table.long()].max())))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 64), (128, 32), (128, 64), (256, 16), (256, 128)])
@pytest.mark.parametrize("new", [1, 6, 350])
@pytest.mark.parametrize("far,small,large", [(64, -30, 5), (40, -20, 20), (64, -22, 8), (24, -16, 8)])
@pytest.mark.parametrize("place", ["in turn", "large first", "large last"])
def test_weights_and_scales_against_each_other(dtype, dim, page, new, far, small, large, place):
    """Keys with all the weight to speak of in pages of small values, and keys 2^-far of theirs in
    pages of large ones, which add less, as much or nothing to the outputs."""
    t = kc.Batch(93, dtype, [new], [1300], 2, 1, dim, page).fill()
    q = t.split()[0]
    q.zero_()
    q[..., 0] = 8.0
    t.k.zero_()
    t.ks.fill_(1.0)
    for j in range(-(-1300 // page)):
        id = int(t.table[0, j])
        big = {"in turn": j % 2, "large first": j * page < 600, "large last": j * page >= 600}[place]
        t.vs[id] = 2.0 ** (large if big else small)
        near = torch.randint(0, 8, t.k.shape[1:3], generator=t.g) / 64                # weights of 2^0 to 2^-0.875
        t.k[id, :, :, 0] = code(-far / 8) if big else (-near).to(kc.F8).view(torch.uint8)
    want, size, reach = kc.attention(t, scale_of_one())
    # the largest of weight times scale, as the sums count it
    most = 448 * max(2.0 ** small, 2.0 ** (large - far))
    within(run(t, scale=scale_of_one()), want, fine_tolerance(t, want, size, reach, most))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (16, 4)), (128, 64, (32, 8)), (256, 128, (8, 4))])
def test_long_single_tokens_beside_a_prompt(dim, page, heads):
    """A prompt that is not cut, and single tokens over keys that are."""
    t = one_hot(kc.Batch(94, "fp16", [2100, 1, 3, 1], [2100, 9000, 5003, 70], *heads, dim, page, extra_rows=2)).fill()
    t.ks.fill_(2.0 ** -7)
    cache, batch, q, _, _ = t.device()
    room = binding.attention_workspace_bytes(q.shape[0], heads[0], cache, batch)
    assert room > 0
    have = binding.attention(q, cache, batch, workspace=torch.full((room,), 0xFF, dtype=torch.uint8, device="cuda:0"))
    torch.cuda.synchronize()
    # (the definition of the prompt's last rows only: it is dear)
    cut, t.new, t.lens, t.table = 2080, [20, 1, 3, 1], t.lens, t.table
    t.x, t.starts = t.x[cut:], [0, 20, 21, 24, 25]
    want, size, reach = kc.attention(t)
    n = t.starts[-1]
    within(have.cpu()[cut: cut + n].double(), want[:n], fine_tolerance(t, want, size, reach, 448 * float(t.vs.max()))[:n])


def prompt(seed, dtype, dim, page):
    """More rows than any rule leaves to the kernel of few."""
    return kc.Batch(seed, dtype, [180, 240], [420, 240], 8, 2, dim, page).fill()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 64), (128, 64), (128, 32), (256, 16), (256, 128)])
def test_prompts_of_any_scale(dtype, dim, page):
    """Scores of one product each, a power of two and its half, from 2^17 to 2^110: equal ones get
    equal weights, the others none."""
    t = prompt(95, dtype, dim, page)
    t.k.zero_()
    t.k[..., 0] = torch.where(torch.rand(t.k.shape[:3], generator=t.g) < 0.1, code(1.0), code(0.5))
    t.x.zero_()
    t.split()[0][..., 0] = 2.0 ** 10
    for level in [17, 22, 23, 24, 26, 27, 30, 60, 110]:
        t.ks.fill_(2.0 ** (level - 10))
        for scale in (1.0, -1.0):
            want, size, reach = kc.attention(t, scale)
            within(run(t, scale=scale), want, fine_tolerance(t, want, size, reach * 0, 448 * float(t.vs.max())))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 64), (128, 16), (256, 64)])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
def test_prompts_with_a_scale_argument(dtype, dim, page, scale):
    t = one_hot(prompt(96, dtype, dim, page))
    want, size, reach = kc.attention(t, scale)
    within(run(t, scale=scale), want, fine_tolerance(t, want, size, reach, 448 * float(t.vs.max())))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (4, 2)), (128, 64, (8, 2)), (256, 64, (4, 2)), (256, 16, (4, 2))])
@pytest.mark.parametrize("new,lens,max_q", [([900, 700], [900, 3000], 300), ([1500, 2, 1, 1, 3], [1500, 900, 64, 2000, 3], 300)])
@pytest.mark.parametrize("window", [0, 300])
def test_prompts_past_their_hint(dim, page, heads, new, lens, max_q, window):
    """max_q understated, but not so far that the prompt kernel is not chosen: its workgroups take
    one row tile after the other.  The same bits as with the hint that holds, where the keys are
    cut the same, and within the tolerance."""
    t = one_hot(kc.Batch(97, "fp16", new, lens, *heads, dim, page, extra_rows=1)).fill()
    t.ks.fill_(2.0 ** -7)
    want, size, reach = kc.attention(t, window=window, sinks=5)
    tol = fine_tolerance(t, want, size, reach, 448 * float(t.vs.max()))
    n = t.starts[-1]
    for hint in (max_q, max(new)):
        within(run(t, max_q=hint, window=window, sinks=5), want[:n], tol[:n])


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 128), (128, 64), (128, 16), (256, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 2)])
def test_prompts_over_what_is_not_finite(dim, page, window, sinks):
    """Rows that see a NaN key come out NaN, the others not; codes of slots behind the last token,
    and pages that hold none, are NaN throughout."""
    t = one_hot(prompt(98, "bf16", dim, page))
    for b, pos, h in ((0, 300, 0), (0, 3, 1), (1, 100, 0)):
        t.k[int(t.table[b, pos // page]), h, pos % page] = 0x7F
    t.split()[0][5, 1, 3] = math.nan
    want, size, reach = kc.attention(t, window=window, sinks=sinks)
    within(run(t, window=window, sinks=sinks), want, fine_tolerance(t, want, size, reach.nan_to_num(0.0), 448 * float(t.vs.max())).nan_to_num(0.0))
