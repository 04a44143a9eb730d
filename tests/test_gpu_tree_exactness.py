"""awq_tree_attention as exact as awq_attention: weights go into the products as two halves in each
of its kernels, and nothing on the way to an output leaves fp32 at magnitudes from end to end."""
import pytest
import torch

import draft_cases as dc
import kv_cases as kc
from test_gpu_attention_exactness import PATTERNS, code, fine_tolerance, one_hot, page_scales, scale_of_one, within
from w4a16_group_quantized_amd import binding

DEV = "cuda:0"
E5 = torch.float8_e5m2


def run(t, bits, words, **kw):
    cache, batch, q, _, _ = t.device()
    mask = dc.mask_of(bits + [0] * (q.shape[0] - len(bits)), words).to(DEV)
    out = binding.tree_attention(q, cache, batch, mask, **kw)
    torch.cuda.synchronize()
    return out.cpu()[: t.starts[-1]].double()


def bits_of_trees(t):
    words = max(1, -(-max(t.new) // 32))
    return [b for n in t.new for b in dc.bits_of(dc.random_tree(n, t.g, 0.3), words)[0]], words


def bits_of_chains(t):
    return [(2 << r) - 1 for n in t.new for r in range(n)], max(1, -(-max(t.new) // 32))


# ---- weights of two halves ----

def half_and(w, rest):
    """w as a half and its remainder as `rest`, in 64 bits."""
    lead = w.half().double()
    return lead + (w - lead).to(rest).double()


def worst_weight(dtype):
    """Minus the score (in the exponent's units) whose weight loses most where its remainder is rounded
    to e5m2 in place of a half: among the type's numbers in [0.5, 1)."""
    steps = 2048 if dtype == torch.float16 else 256
    x = torch.arange(steps // 2, steps, dtype=torch.float64) / steps
    w = torch.exp2(-x) * 2.0 ** 11
    lost = (half_and(w, E5) / w - 1).abs()
    for near in (w * (1 + 2.0 ** -20), w * (1 - 2.0 ** -20)):      # (the same by an exponential off by a little)
        lost = torch.minimum(lost, (half_and(near, E5) / near - 1).abs())
    return float(x[int(lost.argmax())]), float(lost.max())


def as_codes(total, weights):
    """Values of e4m3, one for each weight, whose weighted sum is near the total (positive), from the
    heaviest on: first parts of equal size, then what is left."""
    out = []
    every = torch.arange(0, 0x7F, dtype=torch.uint8).view(kc.F8).double()
    for i, w in enumerate(weights):
        share = total / w / max(1, sum(1 for x in weights[i:] if x == w))
        out.append(float(every[int((every - share).abs().argmin())]) if share > 0 else 0.0)
        total -= w * out[-1]
    return out


def balanced(seed, dtype, dim, page, heads, new, first):
    """Sequences of first[b] tokens (a multiple of 16) before their rows, in which sixteen tokens at a time
    add next to nothing: eight with the worst weight, on even places, and on odd ones eight whose weights are
    powers of two (halves with no remainder), with values of the other sign.  The rows' own tokens add
    nothing but weight.  So all that rounding the weights loses adds up, and little hides it."""
    t = kc.Batch(seed, dtype, new, [f + n for f, n in zip(first, new)], *heads, dim, page).fill()
    at, _ = worst_weight(t.dtype)
    q = t.split()[0]
    q.zero_()
    q[..., 0], q[..., 1] = at, 1.0
    big = 224.0
    weights = [1.0] * 4 + [2.0 ** -4] * 2 + [2.0 ** -8] * 2
    other = as_codes(8 * big * 2.0 ** -at, weights)
    order = [0, 1, 4, 6, 2, 3, 5, 7]
    k, v = torch.zeros((16, 2)), torch.zeros(16)
    for i in range(8):
        k[2 * i, 0], v[2 * i] = -1.0, big
        k[2 * i + 1, 1] = {1.0: 0.0, 2.0 ** -4: -4.0, 2.0 ** -8: -8.0}[weights[order[i]]]
        v[2 * i + 1] = -other[order[i]]
    t.ks.fill_(1.0)
    t.vs.fill_(1.0)
    sign = torch.where(torch.arange(dim) % 3 == 1, -1.0, 1.0)
    for b, n in enumerate(t.lens):
        for j in range(-(-n // page)):
            id, pos = int(t.table[b, j]), torch.arange(j * page, min(n, (j + 1) * page))
            live = len(pos)
            some = (pos < first[b]).float()
            t.k[id, :, :live] = 0
            t.k[id, :, :live, :2] = kc.bytes_of((k[pos % 16] * some[:, None]).to(kc.F8))
            t.v[id, :, :, :live] = kc.bytes_of((v[pos % 16] * some * sign[:, None]).to(kc.F8))
    return t


def two_halves_tolerance(t, out, size):
    """Scores are exact.  The exponential: 2^-23 of a weight, and the scale's own rounding as much for
    scores up to 8; two halves: 2^-22.  Sums: each sixteen keys add next to nothing, so what an
    addition rounds is at most sixteen terms (of the 32 keys of a product), by 2^-24: for each term
    of the size, of which these are a half, 2^-21 for leading parts and as much for what is there when they
    are added to the sums.  In all 2^-19.4 of the size; the weights' sum touches the
    outputs alone, which are small, by (keys / 8 + 64) 2^-24.  Then the output's own rounding."""
    keys = max(t.lens)
    near = 2.0 ** -19 * size + (keys / 8 + 64) * 2.0 ** -24 * out.abs()
    return near + kc.half_step(t.dtype) * (out.abs() + near) + torch.finfo(t.dtype).smallest_normal * kc.half_step(t.dtype)


# few rows, with chunks and without, in workgroups of four and eight waves
FEW = [(64, 16, (4, 4), [1, 5, 16], [640, 64, 320]), (128, 64, (8, 2), [3], [6400]), (256, 32, (4, 2), [9], [1296]), (64, 64, (8, 8), [1, 1], [1008, 992]),
       (128, 16, (4, 2), [7, 2], [160, 3200])]
# many: four waves, cut and not; two waves, cut and not; heads of 256; among single tokens
MANY = [(128, 64, (8, 2), [270, 70], [304, 896]), (64, 16, (4, 2), [270, 70], [304, 896]), (128, 16, (8, 2), [200, 1, 3, 60], [1504, 1600, 16, 320]),
        (128, 64, (32, 8), [60 - b % 3 for b in range(16)], [16 * (5 + b) for b in range(16)]),
        (64, 32, (32, 8), [40], [3296]), (128, 128, (32, 8), [40], [3296]),
        (128, 16, (32, 8), [14] * 256, [368 - b % 3 * 16 for b in range(256)]),
        (256, 64, (4, 2), [270, 70], [304, 896]), (256, 16, (8, 2), [100], [1504])]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads,new,first", FEW + MANY)
def test_weights_of_two_halves(dtype, dim, page, heads, new, first):
    t = balanced(60, dtype, dim, page, heads, new, first)
    bits, words = bits_of_trees(t)
    want, size, _ = dc.tree_attention(t, bits, scale_of_one())
    within(run(t, bits, words, scale=scale_of_one()), want, two_halves_tolerance(t, want, size))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_the_tolerance_tells_two_halves_from_less(dtype):
    """The same sums on the CPU: within the tolerance with weights of two halves, and not with one, with
    remainders in e5m2, or with remainders that meet the values of other keys."""
    new, first = [5, 3], [640, 1296]
    t = balanced(60, dtype, 64, 16, (2, 1), new, first)
    bits, words = bits_of_trees(t)
    want, size, _ = dc.tree_attention(t, bits, scale_of_one())
    tol = two_halves_tolerance(t, want, size)
    q = t.split()[0].double()
    got = {name: torch.zeros_like(want) for name in ("two", "one", "e5m2", "shifted")}
    for b, n in enumerate(new):
        k, v, _ = t.held(b, t.lens[b])
        for r in range(n):
            row = t.starts[b] + r
            see = torch.tensor([j < first[b] or bits[row] >> (j - first[b]) & 1 for j in range(t.lens[b])], dtype=torch.bool)
            for h in range(2):
                w = torch.where(see, torch.exp2(q[row, h] @ k[0].t()), 0) * 2.0 ** 11
                lead = w.half().double()
                rest = (w - lead).half().double()
                for name, x in (("two", lead + rest), ("one", lead), ("e5m2", half_and(w, E5)), ("shifted", lead + rest.roll(1))):
                    got[name][row, h] = x @ v[0] / w.sum()
    within(got["two"].to(t.dtype).double(), want, tol)
    for name in ("one", "e5m2", "shifted"):
        with pytest.raises(AssertionError):
            within(got[name].to(t.dtype).double(), want, tol)


# ---- magnitudes from end to end ----

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 64), (128, 16), (128, 64), (256, 64), (256, 32)])
@pytest.mark.parametrize("new", [6, 350])
@pytest.mark.parametrize("sign", [1, -1])
def test_maxima_one_step_of_fp32_apart(dtype, dim, page, new, sign):
    """Scores around 2^26, where fp32 has steps of 8: a maximum, and tiles later one a step above it, whose
    weight the first has 2^-8 of; the other keys are far below both.  (The rows' own tokens among these.)"""
    t = kc.Batch(61, dtype, [new], [600], 2, 1, dim, page).fill()
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
    bits, words = bits_of_trees(t)
    want = torch.full((new, 2, dim), (2 + 2.0 ** -8) / (1 + 2.0 ** -8), dtype=torch.float64)
    # the exponential, a quotient and sums of two: a few of 2^-24; the output's rounding
    within(run(t, bits, words, scale=scale_of_one()), want, want * (kc.half_step(t.dtype) + 2.0 ** -20))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 64), (128, 32), (128, 128), (256, 16), (256, 64)])
@pytest.mark.parametrize("new", [6, 270])
@pytest.mark.parametrize("pattern", PATTERNS)
def test_value_scales_from_end_to_end(dim, page, new, pattern):
    """Chains, whose definition is causal attention's."""
    t = one_hot(kc.Batch(62, "bf16", [new], [1500], 4, 2, dim, page)).fill()
    t.ks.fill_(2.0 ** -7)
    page_scales(t, PATTERNS[pattern])
    want, size, reach = kc.attention(t)
    within(run(t, *bits_of_chains(t)), want, fine_tolerance(t, want, size, reach, 448 * float(t.vs[t.table.long()].max())))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 64), (128, 32), (128, 64), (256, 16), (256, 128)])
@pytest.mark.parametrize("new", [6, 350])
@pytest.mark.parametrize("far,small,large", [(64, -30, 5), (40, -20, 20), (24, -16, 8)])
@pytest.mark.parametrize("place", ["in turn", "large first", "large last"])
def test_weights_and_scales_against_each_other(dtype, dim, page, new, far, small, large, place):
    """Keys with all the weight to speak of in pages of small values, and keys 2^-far of theirs in
    pages of large ones, which add less, as much or nothing to the outputs."""
    t = kc.Batch(63, dtype, [new], [1300], 2, 1, dim, page).fill()
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
    most = 448 * max(2.0 ** small, 2.0 ** (large - far))                              # of weight times scale
    within(run(t, *bits_of_chains(t), scale=scale_of_one()), want, fine_tolerance(t, want, size, reach, most))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (4, 2)), (128, 64, (8, 2)), (256, 64, (4, 2)), (128, 128, (5, 1))])
@pytest.mark.parametrize("new,lens", [([5, 3, 9], [1000, 64, 400]), ([270, 70], [300, 900])])
def test_signed_sums(dtype, dim, page, heads, new, lens):
    """Weights of any size under scales of any, values of either sign."""
    t = one_hot(kc.Batch(64, dtype, new, lens, *heads, dim, page)).fill()
    t.ks.fill_(2.0 ** -6)
    bits, words = bits_of_trees(t)
    want, size, reach = dc.tree_attention(t, bits)
    within(run(t, bits, words), want, fine_tolerance(t, want, size, reach, 448 * float(t.vs.max())))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 64), (128, 16), (256, 64)])
@pytest.mark.parametrize("new,lens", [([6, 2], [420, 240]), ([180, 240], [420, 240])])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30])
def test_a_scale_argument(dtype, dim, page, new, lens, scale):
    t = one_hot(kc.Batch(65, dtype, new, lens, 8, 2, dim, page)).fill()
    bits, words = bits_of_trees(t)
    want, size, reach = dc.tree_attention(t, bits, scale)
    within(run(t, bits, words, scale=scale), want, fine_tolerance(t, want, size, reach, 448 * float(t.vs.max())))
