"""Plain 64-bit forms of what drafting does over the paged cache: appending at given
positions, drafted trees and their attention, compaction, and forks of the page table.

Torch on the CPU and Python integers, written from the formulas of include/awq.h, on the
batches of kv_cases.py.
"""
from __future__ import annotations

import copy
import math

import torch

import kv_cases as kc


def turned(t: kc.Batch, positions, rope, axis_of, interleaved):
    """The batch with its rows' queries and keys turned, in 64 bits (no rounding)."""
    rot = rope.shape[1]
    q, k, v = t.split()
    qo, ko = torch.empty(q.shape, dtype=torch.float64), torch.empty(k.shape, dtype=torch.float64)
    for r in range(q.shape[0]):
        row = [0.0] * rot
        for f in range(rot // 2):
            at = int(positions[r][axis_of[f]])
            inside = 0 <= at < rope.shape[0]
            row[f] = float(rope[at][f]) if inside else math.nan
            row[f + rot // 2] = float(rope[at][f + rot // 2]) if inside else math.nan
        qo[r], ko[r] = (kc.rotate(x[r], row, rot, interleaved) for x in (q, k))
    out = copy.copy(t)
    out.x = torch.cat([qo.flatten(1), ko.flatten(1), v.double().flatten(1)], 1)
    return out


def append_at(t: kc.Batch, positions, rope, axis_of, interleaved=False):
    """kv_cases.append's results for rows at given positions [rows][axes]."""
    return kc.append(turned(t, positions, rope, axis_of, interleaved))


def bits_of(parents, words):
    """(the rows that each row of one tree sees, as an integer's bits cut to 32 * words; depths)."""
    seen, depth = [], []
    for t, up in enumerate(parents):
        some = 0 <= up < t
        seen.append((seen[up] if some else 0) | 1 << t)
        depth.append(depth[up] + 1 if some else 0)
    return [s & ((1 << 32 * words) - 1) for s in seen], depth


def mask_of(bits, words):
    """Integers to int32 words [rows][words]."""
    out = torch.zeros((len(bits), words), dtype=torch.int64)
    for r, s in enumerate(bits):
        for w in range(words):
            out[r, w] = s >> 32 * w & 0xFFFFFFFF
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def random_tree(n, g, reach=1.0):
    """Parents of n rows: any row before, near ones for a small reach; some none."""
    return [t - 1 - int(float(torch.rand((), generator=g)) * max(1, reach * t)) for t in range(n)]


def tree_attention(t: kc.Batch, bits, scale=None, window=0, sinks=0):
    """kv_cases.attention's results for rows that see the tokens before their sequence's rows
    and those of the rows whose bits (an integer for each row) are set."""
    q, _, _ = t.split()
    scale = t.dim ** -0.5 if scale is None else scale
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    size, reach = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    group = t.q_heads // t.kv_heads
    for b, n in enumerate(t.new):
        length = min(max(t.lens[b], 0), t.width * t.page)
        first = length - n
        k, v, has = t.held(b, length)
        see = torch.zeros((n, length), dtype=torch.bool)
        for r in range(n):
            mine = bits[t.starts[b] + r]
            place = first + bin(mine).count("1") - 1
            for j in range(length):
                if j < first:
                    see[r, j] = not window or j > place - window or j < sinks
                else:
                    see[r, j] = bool(mine >> (j - first) & 1)
        see &= has
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
            far = (q[rows, h].double().abs() @ kh.abs().t()) * abs(scale)
            reach[rows, h] = torch.where(see, far, 0).amax(1) if length else 0
    return out, size, reach


def keep(t: kc.Batch, kept, counts):
    """(k codes, v codes, k scales, v scales as doubles, lengths, the places [pages][page] that
    may change, and those of them that tokens come to): awq_kv_keep."""
    K, V = t.k.view(kc.F8).double(), t.v.view(kc.F8).double()
    ks, vs = t.ks.double().clone(), t.vs.double().clone()
    lens, may = [], torch.zeros((t.pages, t.page), dtype=torch.bool)
    for b, n in enumerate(t.new):
        length = min(max(t.lens[b], 0), t.width * t.page)
        first = length - n
        rows = []
        for i in range(min(max(counts[b], 0), n, len(kept[b]))):
            if kept[b][i] <= (rows[-1] if rows else -1) or kept[b][i] >= n:
                break
            rows.append(kept[b][i])
        if first < 0:
            lens.append(length)
            continue
        lens.append(first + len(rows))
        come = list(range(first)) + [first + r for r in rows]
        number = lambda j: int(t.table[b, j]) if 0 <= int(t.table[b, j]) < t.pages else -1  # noqa: E731
        for j in range(first // t.page, -(-len(come) // t.page)):
            here = come[j * t.page: (j + 1) * t.page]
            page = number(j)
            if page < 0 or here == list(range(j * t.page, j * t.page + len(here))):
                continue
            at = [(number(x // t.page), x % t.page) for x in here]
            may[page, : len(here)] = True
            for h in range(t.kv_heads):
                for codes, old, scales, dead in ((K, t.ks, ks, math.nan), (V, t.vs, vs, 0.0)):
                    from_page = [float(old[p, h]) for p, _ in at if p >= 0]
                    if not from_page:
                        scale = float(old[page, h])
                    else:
                        scale = max(from_page)
                    scales[page, h] = scale
                    src = t.k.view(kc.F8) if codes is K else t.v.view(kc.F8)
                    for slot, (p, s) in enumerate(at):
                        if p < 0:
                            x = torch.full((t.dim,), dead, dtype=torch.float64)
                        else:
                            x = (src[p, h, s] if codes is K else src[p, h, :, s]).double()
                            if float(old[p, h]) != scale:
                                x = torch.where(x.isnan(), x, kc.e4m3(x.nan_to_num(0.0) * (float(old[p, h]) / scale)))
                        if codes is K:
                            K[page, h, slot] = x
                        else:
                            V[page, h, :, slot] = x
    return K, V, ks, vs, lens, may


def fork(table, lens, from_, grow, page, pages, held=None):
    """(table, lens, copies, missing) as lists: awq_kv_fork."""
    width = len(table[0]) if table else 0
    cap = width * page
    lens_out, rows = [], []
    for f in from_:
        some = 0 <= f < len(lens)
        lens_out.append(min(max(lens[f], 0), cap) if some else 0)
        n = -(-lens_out[-1] // page)
        rows.append([x if 0 <= x < pages else -1 for x in table[f][:n]] + [-1] * (width - n) if some else [-1] * width)
    refs = [2 * bool(held is not None and held[p]) for p in range(pages)]
    for r in rows:
        for x in r:
            if x >= 0:
                refs[x] += 1
    free = [p for p in range(pages) if refs[p] == 0]
    asked = missing = 0
    copies = []
    for b, row in enumerate(rows):
        want = min(lens_out[b] + max(grow[b], 0), cap)
        places = list(range(-(-lens_out[b] // page), -(-want // page)))
        at, pair = lens_out[b] // page, (-1, -1)
        copy_ = want > lens_out[b] and lens_out[b] % page and row[at] >= 0 and refs[row[at]] > 1
        if copy_:
            places.insert(0, at)
        asked += len(places)
        if asked <= len(free):
            given = free[asked - len(places): asked]
            if copy_:
                pair = (row[at], given[0])
        else:
            given = [-1] * len(places)
            missing += len(places)
        for i, x in zip(places, given):
            row[i] = x
        copies.append(pair)
    return rows, lens_out, copies, missing
