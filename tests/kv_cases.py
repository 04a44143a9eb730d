"""Plain 64-bit forms of the paged key/value cache's calls, and seeded inputs.

Everything here is torch on the CPU in float64, written from the formulas of
include/awq.h: one sequence, one head and one page after the other.
"""
from __future__ import annotations

import math

import torch

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


def half_step(dtype) -> float:
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


def bytes_of(t):
    return t.contiguous().view(torch.uint8)


def e4m3(x):
    """Nearest e4m3 value of doubles up to 448 in magnitude, ties to the even code."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step          # torch.round: half to even


def scale_for(most: float) -> float:
    """2^e with the least e >= -64 such that most <= 448 * 2^e."""
    e = -64
    while most > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Batch:
    """Sequences with `new[b]` rows and `lens[b]` tokens after them, in pages of a
    shuffled pool.  Unused slots and pages hold NaN codes, unused table entries
    no page."""

    def __init__(self, seed, dtype, new, lens, q_heads, kv_heads, dim, page, extra_rows=0, spread=1.0):
        self.g = torch.Generator().manual_seed(seed)
        self.dtype, self.new, self.lens = TYPES[dtype], list(new), list(lens)
        self.q_heads, self.kv_heads, self.dim, self.page = q_heads, kv_heads, dim, page
        need = [-(-max(n, 0) // page) for n in lens]
        self.width = max(1, max(need))
        self.pages = sum(need) + 2
        order = torch.randperm(self.pages, generator=self.g).tolist()
        self.table = torch.full((len(new), self.width), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for j in range(n):
                self.table[b, j] = order.pop()
        self.starts = [0]
        for n in new:
            self.starts.append(self.starts[-1] + n)
        rows = self.starts[-1] + extra_rows
        wide = (q_heads + 2 * kv_heads) * dim
        x = (torch.randn((rows, wide), generator=self.g, dtype=torch.float64) * spread).to(self.dtype)
        self.x = x                                               # a fused projection's output
        self.k = torch.full((self.pages, kv_heads, page, dim), 0x7F, dtype=torch.uint8)
        self.v = torch.full((self.pages, kv_heads, dim, page), 0xFF, dtype=torch.uint8)
        self.ks = torch.exp2(torch.randint(-9, -5, (self.pages, kv_heads), generator=self.g).float())
        self.vs = torch.exp2(torch.randint(-9, -5, (self.pages, kv_heads), generator=self.g).float())

    def fill(self, upto=None):
        """Codes for the tokens [0, upto[b]) of each sequence (all, unless given)."""
        for b, n in enumerate(self.lens if upto is None else upto):
            for j in range(-(-max(n, 0) // self.page)):
                live = min(self.page, n - j * self.page)
                shape = (self.kv_heads, live, self.dim)
                code = lambda: (torch.randn(shape, generator=self.g) * 90).clamp(-448, 448).to(F8)  # noqa: E731
                id = int(self.table[b, j])
                self.k[id, :, :live] = bytes_of(code())
                self.v[id, :, :, :live] = bytes_of(code()).transpose(1, 2)
        return self

    def split(self, x=None):
        x = self.x if x is None else x
        q, k, v = x.split([self.q_heads * self.dim, self.kv_heads * self.dim, self.kv_heads * self.dim], 1)
        return (q.unflatten(1, (self.q_heads, self.dim)), k.unflatten(1, (self.kv_heads, self.dim)),
                v.unflatten(1, (self.kv_heads, self.dim)))

    def device(self, max_q=None, max_kv=None):
        """(cache, batch, q, k, v) on the GPU."""
        from w4a16_group_quantized_amd import binding
        d = lambda t: t.to("cuda:0")  # noqa: E731
        cache = binding.KvCache(d(self.k).view(F8), d(self.v).view(F8), d(self.ks), d(self.vs))
        batch = binding.KvBatch(d(self.table), d(torch.tensor(self.lens, dtype=torch.int32)),
                                d(torch.tensor(self.starts, dtype=torch.int32)),
                                max([0, *self.new]) if max_q is None else max_q,
                                max([0, *self.lens]) if max_kv is None else max_kv)
        return (cache, batch, *self.split(d(self.x)))

    def held(self, b, n):
        """Keys and values [kv_heads][n][dim] of sequence b in 64 bits, and which of the
        tokens have a page."""
        k = torch.zeros((self.kv_heads, n, self.dim), dtype=torch.float64)
        v, has = torch.zeros_like(k), torch.zeros(n, dtype=torch.bool)
        for j in range(-(-n // self.page)):
            id, live = int(self.table[b, j]), min(self.page, n - j * self.page)
            if not 0 <= id < self.pages:
                continue
            at = slice(j * self.page, j * self.page + live)
            has[at] = True
            k[:, at] = self.k[id, :, :live].contiguous().view(F8).double() * self.ks[id].double()[:, None, None]
            v[:, at] = (self.v[id, :, :, :live].contiguous().view(F8).double()
                        * self.vs[id].double()[:, None, None]).transpose(1, 2)
        return k, v, has


def rope_table(positions, rot, base=10000.0):
    a = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (
        -torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, row, rot, interleaved):
    """One token's heads [heads][dim] in 64 bits, turned by a row of the table."""
    x = x.double().clone()
    for i in range(rot // 2):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = float(row[i]), float(row[i + rot // 2])
        a, b = x[:, p].clone(), x[:, q].clone()
        x[:, p], x[:, q] = a * c - b * s, b * c + a * s
    return x


def append(t: Batch, rope=None, interleaved=False):
    """(q [rows] or NaN where nothing is written, k codes, v codes, k scales, v scales,
    where codes are written, sizes of the fp32 terms): awq_kv_append in 64 bits."""
    q, k, v = t.split()
    rot = 0 if rope is None else rope.shape[1]
    qo = torch.full(q.shape, math.nan, dtype=torch.float64)
    K, V = t.k.view(F8).double(), t.v.view(F8).double()
    ks, vs = t.ks.double().clone(), t.vs.double().clone()
    done = torch.zeros((t.pages, t.page), dtype=torch.bool)
    for b, n in enumerate(t.new):
        length = min(max(t.lens[b], 0), t.width * t.page)
        first = length - n
        by_page = {}
        for i in range(n):
            pos, r = first + i, t.starts[b] + i
            if pos < 0 or (rot and pos >= rope.shape[0]):
                continue
            turn = lambda z: rotate(z, rope[pos], rot, interleaved) if rot else z.double()  # noqa: E731
            qo[r] = turn(q[r])
            by_page.setdefault(pos // t.page, []).append((pos % t.page, turn(k[r]), v[r].double()))
        for j, tokens in by_page.items():
            id = int(t.table[b, j])
            if not 0 <= id < t.pages:
                continue
            held = tokens[0][0]
            for h in range(t.kv_heads):
                for which, codes, scales in ((1, K, ks), (2, V, vs)):
                    new = torch.stack([tok[which][h] for tok in tokens])            # [tokens][dim]
                    fine = torch.isfinite(new)
                    s = scale_for(float(torch.where(fine, new, 0).abs().max()))
                    old = float(scales[id, h])
                    s = max(s, old) if held else s
                    slab = codes[id, h] if which == 1 else codes[id, h].t()
                    if held and s != old:
                        slab[:held] = e4m3(slab[:held] * (old / s))
                    slab[held: held + len(tokens)] = torch.where(fine, e4m3(torch.where(fine, new, 0) / s), 0)
                    scales[id, h] = s
                bad = torch.stack([~(torch.isfinite(tok[1][h]) & torch.isfinite(tok[2][h])).all() for tok in tokens])
                K[id, h, held: held + len(tokens)][bad] = math.nan
            done[id, : held + len(tokens)] = True
    return qo, K, V, ks, vs, done


def attention(t: Batch, scale=None, window=0, sinks=0):
    """(out [rows][q_heads][dim] (NaN for rows of no sequence), sum p|v| / sum p, the
    largest scale * sum |q k| of each row and head): awq_attention in 64 bits."""
    q, _, _ = t.split()
    scale = t.dim ** -0.5 if scale is None else scale
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    size, reach = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    group = t.q_heads // t.kv_heads
    for b, n in enumerate(t.new):
        length = min(max(t.lens[b], 0), t.width * t.page)
        k, v, has = t.held(b, length)
        j = torch.arange(length)
        i = (length - n + torch.arange(n))[:, None]
        see = (j <= i) & has
        if window:
            see &= (j > i - window) | (j < sinks)
        rows = slice(t.starts[b], t.starts[b + 1])
        for h in range(t.q_heads):
            kh, vh = k[h // group], v[h // group]
            x = (q[rows, h].double() @ kh.t()) * scale
            x = x.masked_fill(~see, -math.inf)
            top = x.amax(1, keepdim=True) if length else torch.zeros((n, 1), dtype=torch.float64)
            p = torch.where(see, torch.exp(x - torch.where(top.isinf(), 0, top)), 0)
            total = p.sum(1, keepdim=True)
            some = total != 0
            out[rows, h] = torch.where(some, (p @ vh.nan_to_num(0.0)) / torch.where(some, total, 1), 0)
            size[rows, h] = torch.where(some, (p @ vh.nan_to_num(0.0).abs()) / torch.where(some, total, 1), 0)
            far = (q[rows, h].double().abs() @ kh.abs().t()) * scale
            reach[rows, h] = torch.where(see, far, 0).amax(1) if length else 0
    return out, size, reach


def attention_tolerance(t: Batch, out, size, reach):
    """What the kernels may be off, by their own arithmetic.

    Scores: products of fp16 and e4m3 numbers are exact in fp32; a sum of dim of
    them, then scaling and exponent, are off by at most (dim + 16) 2^-24 of
    scale * sum |q k| (in units of the exponent).  Weights: rounded to fp16 once,
    2^-11 of each (kernels that keep a remainder are far below).  Sums over the
    keys in fp32: at most 2^-24 of the total for each addition, (keys / 8 + 64) in
    a row.  All of this reaches the output in proportion to sum p|v| / sum p,
    twice for the quotient's two sums.  Then one rounding to the type, or a half
    of its least subnormal."""
    keys = max([1, *t.lens])
    each = (t.dim + 16) * 2.0 ** -24 * reach + 2.0 ** -11 + (keys / 8 + 64) * 2.0 ** -24
    return 2 * each[..., None] * size + half_step(t.dtype) * (out.abs() + 2 * each[..., None] * size) + \
        torch.finfo(t.dtype).smallest_normal * half_step(t.dtype)
