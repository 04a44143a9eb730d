"""Measured cases of drafting over the 8-bit paged key/value cache: trees of tokens that are
checked in one step, positions with several axes, and the cache's pages.

* ``append``: append rows whose rotary positions are given, one for each axis (time,
  height, width of images and video; the depth of a drafted token), while their places
  in the cache follow from the sequence's length.
* ``rows``: the rows of drafted trees: which rows each sees (itself and its ancestors, as
  bits), and its position, from the parents.
* ``tree``: attention of drafted trees over the cache: a row sees all tokens before the
  tree (under a window the last ones, and the first few), and of the tree the rows that
  its bits name.
* ``keep``: compaction: of a sequence's rows the kept ones move together, the others
  are dropped (an accepted path of a tree; tokens that survive an eviction).
* ``fork``: the next step's page table: sequences that go on, split up, end or begin; pages
  for what they are to grow by, and copies of pages that they share and would write.

``own`` false computes each in its plain form (elementary torch operations in 32 bits);
true calls the framework.  ``exact`` is the definition in 64 bits.

The cache: k e4m3 [pages][kv_heads][page][dim], v e4m3 [pages][kv_heads][dim][page],
scales fp32 [pages][kv_heads]; a key or value is its code times its page's scale.  A
sequence b has ``kv_lens[b]`` tokens in the cache, the last ones of them its rows
(rows ``q_starts[b]`` to ``q_starts[b + 1] - 1``).
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, **kw):
    return {"name": name, "op": op, **kw}


def _append(name, dtype, seqs, rows, ctx, q_heads, kv_heads, dim, page, rot, pairs, axes, mixed):
    """``axes``: positions of a row; ``mixed``: whether the axes take frequencies in turn, or in sections."""
    return _case(name, "append", dtype=dtype, seqs=seqs, rows=rows, ctx=ctx, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                 page=page, rot=rot, pairs=pairs, axes=axes, mixed=mixed)


def _tree(name, dtype, seqs, rows, ctx, q_heads, kv_heads, dim, page, window=0, sinks=0):
    return _case(name, "tree", dtype=dtype, seqs=seqs, rows=rows, ctx=ctx, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                 page=page, window=window, sinks=sinks)


def _keep(name, seqs, rows, ctx, kept, kv_heads, dim, page):
    return _case(name, "keep", seqs=seqs, rows=rows, ctx=ctx, kept=kept, kv_heads=kv_heads, dim=dim, page=page)


def _fork(name, seqs, new_seqs, beams, ctx, grow, kv_heads, dim, page):
    """``beams``: old sequences that share the first half of their pages."""
    return _case(name, "fork", seqs=seqs, new_seqs=new_seqs, beams=beams, ctx=ctx, grow=grow, kv_heads=kv_heads, dim=dim, page=page)


def listed():
    """``rows``: the most rows of a sequence; ``ctx``: the most tokens that a sequence has before them."""
    return [
        # one step's drafted trees: positions are depths, places are not
        _append("append_tree", "fp16", 32, 32, 4000, 32, 8, 128, 64, 128, "half", 1, False),
        # a video as a prompt: time, height and width, each with its section of the frequencies
        _append("append_video", "bf16", 1, 16000, 500, 64, 8, 128, 128, 128, "half", 3, False),
        # the trees of a step's batch
        _case("rows_batch", "rows", seqs=16, rows=64, ctx=4000),
        # many wide trees
        _case("rows_wide", "rows", seqs=256, rows=512, ctx=30000),
        # one user's tree over a short conversation: latency
        _tree("tree_one", "fp16", 1, 24, 1000, 32, 8, 128, 64),
        # a serving batch of trees over ragged contexts
        _tree("tree_batch", "fp16", 16, 64, 8191, 32, 8, 128, 64),
        # a tree over one very long context: the split over the key axis carries it
        _tree("tree_long", "bf16", 1, 48, 131000, 64, 8, 128, 128),
        # small trees of many sequences under a window, small heads, small pages
        _tree("tree_window", "bf16", 24, 16, 16000, 28, 4, 64, 32, window=2048, sinks=4),
        # a step's accepted paths: a few rows each, a matter of latency
        _keep("keep_accepted", 16, 64, 4000, 6, 8, 128, 64),
        # half the tokens of long sequences are dropped
        _keep("keep_evicted", 8, 8192, 0, 4096, 8, 128, 64),
        # a step of beam search: beams go on from others, and copy the page that they write next
        _fork("fork_beams", 64, 64, 8, 1000, 1, 8, 128, 64),
        # prompts split up into samples, large pages
        _fork("fork_samples", 32, 256, 1, 4000, 100, 4, 256, 128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges, of no more work than the largest of the listed ones."""
    while True:
        op = rng.choice(["append", "append", "rows", "tree", "tree", "tree", "keep", "fork"])
        kv = rng.choice([1, 2, 4, 8, 16])
        heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        dim = rng.choice([64, 128, 128, 256])
        page = rng.choice([16, 32, 64, 128])
        seqs = _spread(rng, 1, 64)
        ctx = _spread(rng, 1, 131000) - 1
        dtype = rng.choice(["fp16", "bf16"])
        if op == "append":
            axes = rng.choice([1, 2, 3, 3, 4])
            rows = _spread(rng, 1, 256) if axes == 1 else rng.choice([1, _spread(rng, 2, 4096)])
            if seqs * rows * heads * dim > 1 << 27 or seqs * (rows + ctx) * kv * dim > 1 << 28:
                continue
            c = _append("", dtype, seqs, rows, ctx, heads, kv, dim, page, rng.choice([dim, dim, dim // 2]),
                        rng.choice(["half", "adjacent"]), axes, rng.choice([False, True]))
        elif op == "rows":
            seqs = _spread(rng, 1, 256)
            c = _case("", op, seqs=seqs, rows=_spread(rng, 12, 512), ctx=ctx)
        elif op == "tree":
            rows = _spread(rng, 1, 256)
            if heads > 64 or seqs * rows * (rows + ctx) * heads > 3 << 27 or seqs * (rows + ctx) * kv * dim > 1 << 28:
                continue
            windowed = rng.random() < 0.35
            c = _tree("", dtype, seqs, rows, ctx, heads, kv, dim, page, _spread(rng, 16, 8192) if windowed else 0,
                      rng.choice([0, 1, 4, 16, 100]) if windowed else 0)
        elif op == "keep":
            rows = rng.choice([_spread(rng, 1, 128), _spread(rng, 64, 8192)])
            ctx = min(ctx, 32000)
            if seqs * (rows + ctx) * kv * dim > 1 << 26:
                continue
            c = _keep("", seqs, rows, ctx, rng.randint(0, rows), kv, dim, page)
        else:
            new = _spread(rng, 1, 256)
            ctx = min(ctx, 16000)
            if seqs * ctx * kv * dim > 1 << 27 or new * kv * dim * (page + 512) > 1 << 27:
                continue
            c = _fork("", seqs, new, rng.choice([1, 1, 4, 8]), ctx, rng.choice([1, 1, _spread(rng, 1, 512)]), kv, dim, page)
        del c["name"]
        return c


def _lengths(c):
    """(rows, tokens with them) of each sequence: ragged, the first sequence the longest."""
    new, kv = [], []
    for b in range(c["seqs"]):
        n = c.get("rows", 0) - (b * 397) % max(1, c.get("rows", 0) // 2)
        before = c["ctx"] - (b // c.get("beams", 1) * 7919) % max(1, c["ctx"] // 2 + 1)
        new.append(n)
        kv.append(before + n)
    return new, kv


def _kept(c, b, n):
    """How many of its n rows sequence b keeps."""
    return min(n, max(0, c["kept"] - (b * 5) % max(1, c["kept"] // 2 + 1)))


def work(case):
    c, (new, kv) = case, _lengths(case)
    rows = sum(new)
    if c["op"] == "append":
        width = c["dim"]
        codes = 2 * rows * c["kv_heads"] * width
        table = 4 * rows * c["rot"] if c["axes"] > 1 else sum(4 * c["rot"] * n for n in new)
        return {"bytes": 2 * rows * (2 * c["q_heads"] + 2 * c["kv_heads"]) * width + codes + table + 4 * rows * c["axes"],
                "flops": 3 * rows * (c["q_heads"] + c["kv_heads"]) * c["rot"] + 4 * rows * c["kv_heads"] * width}
    if c["op"] == "rows":
        return {"bytes": rows * (8 + 4 * -(-c["rows"] // 32)), "flops": 0}
    if c["op"] == "tree":
        held = pairs = 0
        for n, total in zip(new, kv):
            first = total - n
            low = max(0, first + 1 - c["window"]) if c["window"] else 0
            seen = first - low + min(c["sinks"], low)
            held += seen + n
            pairs += n * seen + 4 * n                 # (of the tree a few ancestors each)
        return {"bytes": 2 * held * c["kv_heads"] * c["dim"] + 4 * rows * c["q_heads"] * c["dim"]
                + 8 * (held // c["page"] + 1) * c["kv_heads"],
                "flops": 4 * pairs * c["q_heads"] * c["dim"]}
    if c["op"] == "keep":
        moved = sum(_kept(c, b, n) for b, n in enumerate(new))
        return {"bytes": 4 * moved * c["kv_heads"] * c["dim"] + 4 * moved + 16 * c["seqs"], "flops": 2 * moved * c["kv_heads"] * c["dim"]}
    size = 2 * c["page"] * c["kv_heads"] * c["dim"]
    width = max(-(-n // c["page"]) for n in kv) + c["grow"] // c["page"] + 2
    return {"bytes": 8 * c["new_seqs"] * width + size * (c["new_seqs"] + min(c["seqs"], c["new_seqs"])), "flops": 0}


def _axis_of(c):
    """The axis of each frequency."""
    half, axes = c["rot"] // 2, c["axes"]
    if c["mixed"]:
        return [i % axes for i in range(half)]
    return [min(axes - 1, (i * axes + axes // 2) // half) for i in range(half)]


def _parents(new, g):
    """Random trees: a row's parent is any row before it, and some of the first rows hang on the last token before the tree."""
    n = torch.tensor(new)
    t = torch.arange(int(n.sum())) - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    up = torch.floor(torch.rand(len(t), generator=g, dtype=torch.float64) ** 0.7 * (t + 0.15)).long() - (t == 0).long()
    return torch.minimum(up, t - 1).to(torch.int32)


def _bits(parents, starts, n, words):
    """The rows' bits and depths, from the parents: all on their device."""
    B, dev = len(starts) - 1, parents.device
    counts = starts[1:] - starts[:-1]
    t = torch.arange(n, device=dev)
    at = (starts[:-1, None] + t).clamp(max=max(0, len(parents) - 1)).long()
    up = torch.where(t < counts[:, None], parents[at].long(), -1)                 # [B][n]
    step = ((up[:, :, None] == t) & (t < t[:, None])).float()                     # row t's parent is row u < t
    reach = torch.eye(n, device=dev) + step
    k = 1
    while k < n:
        reach = (torch.bmm(reach, reach) > 0).float()
        k *= 2
    depth = reach.sum(-1).long() - 1
    bits = torch.zeros((B, n, words * 32), dtype=torch.int64, device=dev)
    bits[:, :, :n] = reach.long()
    word = (bits.unflatten(2, (words, 32)) << torch.arange(32, device=dev)).sum(-1)
    word = torch.where(word >= 1 << 31, word - (1 << 32), word)
    return word.to(torch.int32), depth


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)
    new, kv = _lengths(c)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    rows = starts[-1]
    s = {"case": dict(c), "max_q": max(new), "max_kv": max(kv), "rows": rows}
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    s["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    # where each row stands, as a serving program's scheduler knows it
    n, first = torch.tensor(new), torch.tensor(kv) - torch.tensor(new)
    seq = torch.repeat_interleave(torch.arange(c["seqs"]), n)
    t = torch.arange(rows) - torch.tensor(starts)[:-1][seq]
    pos = first[seq] + t
    s["row_seq"], s["row_t"], s["row_pos"] = seq.to(dev), t.to(dev), pos.to(dev)
    if c["op"] in ("rows", "tree") or (c["op"] == "append" and c["axes"] == 1):
        s["parents"] = _parents(new, h).to(dev)
        s["words"] = -(-s["max_q"] // 32)
    if c["op"] == "rows":
        if own:
            from w4a16_group_quantized_amd import binding
            table = torch.zeros((c["seqs"], 1), dtype=torch.int32, device=dev)
            s["batch"] = binding.KvBatch(table, s["kv_lens"], s["q_starts"], s["max_q"], s["max_kv"])
        return s
    P, Hk, D = c["page"], c["kv_heads"], c["dim"]
    need = [-(-x // P) for x in kv]
    width = max(need)
    if c["op"] == "fork":
        width += c["grow"] // P + 2
    if c["op"] == "fork" and c["beams"] > 1:           # beams of one prompt share the first half of its pages
        shared = [x // 2 for x in need]
        table = torch.full((c["seqs"], width), -1, dtype=torch.int32)
        used = 0
        lead = {}
        for b, x in enumerate(need):
            k = shared[b]
            if b // c["beams"] not in lead:
                lead[b // c["beams"]] = torch.arange(used, used + k, dtype=torch.int32)
                used += k
            table[b, :k] = lead[b // c["beams"]]
            table[b, k:x] = torch.arange(used, used + x - k, dtype=torch.int32)
            used += x - k
    else:
        used = sum(need)
        at = torch.arange(width) < torch.tensor(need)[:, None]
        table = torch.full((c["seqs"], width), -1, dtype=torch.int32)
        table[at] = torch.arange(used, dtype=torch.int32)
    pages = used + 1
    if c["op"] == "fork":
        pages += c["new_seqs"] * (c["grow"] // P + 2) + used // 8
    # each sequence's pages anywhere in the pool; entries behind its last one name no page
    order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
    table = table.to(dev)
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], -1).to(torch.int32)
    s["table"] = table

    # codes of normal values under a scale that leaves the largest near 448; a scale of its own for each page and head
    def codes(shape):
        out = torch.empty(shape, dtype=torch.uint8, device=dev)
        flat, step = out.view(-1), 1 << 27
        for a in range(0, flat.numel(), step):
            m = min(step, flat.numel() - a)
            flat[a: a + m] = (torch.randn(m, device=dev, generator=g) * 90).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return out.view(torch.float8_e4m3fn)

    def scales():
        return torch.exp2(torch.randint(-9, -6, (pages, Hk), device=dev, generator=g).float())

    s["k"], s["v"], s["k_scales"], s["v_scales"] = codes((pages, Hk, P, D)), codes((pages, Hk, D, P)), scales(), scales()
    if own:
        from w4a16_group_quantized_amd import binding
        s["cache"] = binding.KvCache(s["k"], s["v"], s["k_scales"], s["v_scales"])
        s["batch"] = binding.KvBatch(s["table"], s["kv_lens"], s["q_starts"], s["max_q"], s["max_kv"])
    if c["op"] == "fork":
        # a child's sequence goes on from one of its prompt's; some end, and some begin with nothing
        b = torch.arange(c["new_seqs"])
        old = b * c["seqs"] // c["new_seqs"]
        group = old // c["beams"] * c["beams"]
        pick = group + torch.floor(torch.rand(len(b), generator=h) * (torch.clamp(group + c["beams"], max=c["seqs"]) - group)).long()
        fresh = torch.rand(len(b), generator=h) < 1 / 16
        s["from"] = torch.where(fresh, -1, pick).to(torch.int32).to(dev)
        s["grow"] = (c["grow"] - (b * 3) % max(1, c["grow"] // 2)).to(torch.int32).to(dev)
        return s
    if c["op"] == "keep":
        kept = torch.full((c["seqs"], max(1, max(_kept(c, i, x) for i, x in enumerate(new)))), -1, dtype=torch.int32)
        counts = []
        for i, x in enumerate(new):
            m = _kept(c, i, x)
            kept[i, :m] = torch.sort(torch.randperm(x, generator=h)[:m]).values.to(torch.int32)
            counts.append(m)
        s["kept"], s["counts"] = kept.to(dev), torch.tensor(counts, dtype=torch.int32, device=dev)
        # for the plain form: of each page that changes, the place that each of its tokens comes from
        ids, src_id, src_slot, live = [], [], [], []
        host = table.cpu().long()
        for i, m in enumerate(counts):
            if not m:
                continue
            f = int(first[i])
            a, e = f // P, (f + m - 1) // P
            j = torch.arange(a * P, (e + 1) * P)
            come = torch.where(j < f, j, f + kept[i].long()[(j - f).clamp(0, m - 1)])
            ids.append(host[i, a: e + 1])
            src_id.append(host[i][come // P])
            src_slot.append(come % P)
            live.append(j < f + m)
        if ids:
            s["to_page"] = torch.cat(ids).to(dev)
            s["come_page"], s["come_slot"], s["come_live"] = (torch.cat(x).view(-1, P).to(dev) for x in (src_id, src_slot, live))
        return s
    # the rows as a fused projection leaves them: queries, keys and values of a token side by side
    Hq, dtype = c["q_heads"], DTYPES[c["dtype"]]
    x = (torch.randn((rows, (Hq + 2 * Hk) * D), device=dev, generator=g) * 1.2).to(dtype)
    s["q"] = x[:, : Hq * D].unflatten(1, (Hq, D))
    if c["op"] == "tree":
        word, depth = _bits(s["parents"], s["q_starts"], s["max_q"], s["words"])
        s["mask"] = word[s["row_seq"], s["row_t"]].contiguous()
        s["depth"] = depth[s["row_seq"], s["row_t"]]
        return s
    s["new_k"] = x[:, Hq * D: (Hq + Hk) * D].unflatten(1, (Hk, D))
    s["new_v"] = x[:, (Hq + Hk) * D:].unflatten(1, (Hk, D))
    f = first[seq]
    if c["axes"] == 1:
        depth = _bits(s["parents"], s["q_starts"], s["max_q"], s["words"])[1][s["row_seq"], s["row_t"]]
        s["positions"] = (f.to(dev) + depth).to(torch.int32)[:, None].contiguous()
    else:                                              # some text, then frames of a grid of patches
        text, high, wide = 20, 12, 18
        u = (t - text).clamp(min=0)
        grid = torch.stack([u // (high * wide), u // wide % high, u % wide, u % 7], 1)[:, (1 if c["axes"] == 2 else 0):][:, : c["axes"]]
        s["positions"] = (f[:, None] + torch.where((t < text)[:, None], t[:, None], text + grid)).to(torch.int32).to(dev).contiguous()
    touched, where = torch.unique(seq * width + pos // P, return_inverse=True)
    tseq, tpage = touched // width, touched % width
    s["touch_pages"] = table.cpu()[tseq, tpage].long().to(dev)
    s["touch_old"] = (first[tseq] - tpage * P).clamp(0, P).to(dev)              # slots that hold tokens before the call
    s["row_touch"], s["row_slot"] = where.to(dev), (pos % P).to(dev)
    # cosines and sines of every position, from 64-bit angles
    freq = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
    a = torch.arange(int(s["positions"].max()) + 1, dtype=torch.float64, device=dev)[:, None] * freq
    s["rope"] = torch.cat([a.cos(), a.sin()], 1).float()
    s["axis_of"] = bytes(_axis_of(c))
    s["axis_at"] = torch.tensor(_axis_of(c), device=dev)
    return s


def run(state):
    s, c = state, state["case"]
    if own:
        from w4a16_group_quantized_amd import binding
        if c["op"] == "append":
            q = binding.kv_append_at(s["q"], s["new_k"], s["new_v"], s["cache"], s["batch"], s["positions"], s["rope"],
                                     axis_of=s["axis_of"], interleaved=c["pairs"] == "adjacent")
            return {"q": q, "k": s["k"], "v": s["v"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
        if c["op"] == "rows":
            mask, positions = binding.tree_rows(s["parents"], s["batch"])
            return {"mask": mask, "positions": positions}
        if c["op"] == "tree":
            return binding.tree_attention(s["q"], s["cache"], s["batch"], s["mask"], window=c["window"], sinks=c["sinks"])
        if c["op"] == "keep":
            lens = binding.kv_keep(s["kept"], s["counts"], s["cache"], s["batch"])
            return {"lens": lens, "k": s["k"], "v": s["v"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
        table, lens, copies, missing = binding.kv_fork(s["from"], s["grow"], s["cache"], s["batch"])
        binding.kv_copy(copies, s["cache"])
        return {"table": table, "lens": lens, "copies": copies, "missing": missing, "k": s["k"], "v": s["v"],
                "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    return {"append": _plain_append, "rows": _plain_rows, "tree": _plain_tree, "keep": _plain_keep, "fork": _plain_fork}[c["op"]](s, c)


# ---- plain forms: 32 bits, elementary operations ----

def _rotate(x, s, c):
    x, R = x.float(), c["rot"]
    i = torch.arange(R // 2, device=x.device)
    at = s["positions"].long()[:, s["axis_at"]]                                   # [rows][rot / 2]
    cos, sin = s["rope"][at, i][:, None, :], s["rope"][at, i + R // 2][:, None, :]
    if c["pairs"] == "half":
        a, b, rest = x[..., : R // 2], x[..., R // 2: R], x[..., R:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b, rest = x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _scale_for(amax):
    """The least power of two, from 2^-64 on, under which amax is at most 448."""
    m, x = torch.frexp(amax)
    e = torch.where(amax > 0, x - 9 + (m > 0.875).int(), -64).clamp(min=-64)
    return torch.ldexp(torch.ones_like(amax), e)


def _write(cache, scales, new, s, c, transposed):
    """The touched pages of one cache array with `new` [rows][heads][dim] in them."""
    pages, P = s["touch_pages"], c["page"]
    got = cache.view(torch.uint8)[pages].view(torch.float8_e4m3fn)
    held = got.float().transpose(2, 3) if transposed else got.float()           # [touched][heads][page][dim]
    put = torch.zeros_like(held)
    put.transpose(1, 2)[s["row_touch"], s["row_slot"]] = new
    fresh = torch.zeros((len(pages), P), dtype=torch.bool, device=held.device)
    fresh[s["row_touch"], s["row_slot"]] = True
    before = torch.arange(P, device=held.device) < s["touch_old"][:, None]
    want = _scale_for(put.abs().amax((2, 3)))
    old = scales[pages]
    scale = torch.where((s["touch_old"] == 0)[:, None], want, torch.maximum(old, want))
    moved = held * (old / scale)[..., None, None]
    out = torch.where(before[:, None, :, None], moved, held)
    out = torch.where(fresh[:, None, :, None], put / scale[..., None, None], out)
    if transposed:
        out = out.transpose(2, 3)
    cache.view(torch.uint8)[pages] = out.contiguous().to(torch.float8_e4m3fn).view(torch.uint8)
    scales[pages] = scale


def _plain_append(s, c):
    q = _rotate(s["q"], s, c).to(DTYPES[c["dtype"]])
    _write(s["k"], s["k_scales"], _rotate(s["new_k"], s, c), s, c, False)
    _write(s["v"], s["v_scales"], s["new_v"].float(), s, c, True)
    return {"q": q, "k": s["k"], "v": s["v"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _plain_rows(s, c):
    word, depth = _bits(s["parents"], s["q_starts"], s["max_q"], s["words"])
    first = s["kv_lens"] - (s["q_starts"][1:] - s["q_starts"][:-1])
    return {"mask": word[s["row_seq"], s["row_t"]], "positions": (first[s["row_seq"]] + depth[s["row_seq"], s["row_t"]]).to(torch.int32)}


def _plain_tree(s, c):
    B, n, L = c["seqs"], s["max_q"], s["max_kv"]
    Hk, D, G = c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    at = s["table"].clamp(min=0).long()
    k = s["k"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["k_scales"][at][..., None, None]
    v = s["v"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["v_scales"][at][..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(B * Hk, D, -1)[:, :, :L].contiguous()
    v = v.permute(0, 2, 1, 4, 3).reshape(B * Hk, -1, D)[:, :L].contiguous()
    q = torch.zeros((B, n, Hk, G, D), device=k.device)
    q[s["row_seq"], s["row_t"]] = s["q"].float().unflatten(1, (Hk, G))
    q = q.permute(0, 2, 3, 1, 4).reshape(B * Hk, G * n, D)
    score = torch.bmm(q * (1 / math.sqrt(D)), k).view(B, Hk, G, n, L)
    first = (s["kv_lens"] - (s["q_starts"][1:] - s["q_starts"][:-1])).long()[:, None, None]
    j = torch.arange(L, device=k.device)
    word = torch.zeros((B, n, s["words"]), dtype=torch.int32, device=k.device)
    word[s["row_seq"], s["row_t"]] = s["mask"]
    u = (j - first).clamp(0, s["words"] * 32 - 1)                                 # [B][1][L]
    bit = (word.gather(2, (u // 32).expand(B, n, L)) >> (u % 32)) & 1
    seen = torch.where(j < first, torch.ones_like(bit), bit) > 0
    seen &= j < s["kv_lens"][:, None, None]
    if c["window"]:
        depth = torch.zeros((B, n), dtype=torch.int64, device=k.device)
        depth[s["row_seq"], s["row_t"]] = s["depth"]
        seen &= (j >= first) | (j > first + depth[..., None] - c["window"]) | (j < c["sinks"])
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p.view(B * Hk, G * n, L), v).view(B, Hk, G, n, D) / total.clamp(min=1e-30)
    return out.permute(0, 3, 1, 2, 4)[s["row_seq"], s["row_t"]].flatten(1, 2).to(DTYPES[c["dtype"]])


def _plain_keep(s, c):
    lens = s["kv_lens"] - (s["q_starts"][1:] - s["q_starts"][:-1]) + s["counts"]
    if "to_page" in s:
        live = s["come_live"]
        for name in ("k", "v"):
            cache, scales = s[name], s[name + "_scales"]
            value = cache.view(torch.uint8)
            if name == "v":
                value = value.transpose(2, 3)
            come = value[s["come_page"], :, s["come_slot"]].view(torch.float8_e4m3fn).float()          # [touched][page][heads][dim]
            old = scales[s["come_page"]]                                                             # [touched][page][heads]
            scale = torch.where(live[..., None], old, torch.zeros_like(old)).amax(1)
            now = come * (old / scale[:, None])[..., None]
            was = value[s["to_page"]].view(torch.float8_e4m3fn).float()                              # [touched][heads][page][dim]
            out = torch.where(live[:, None, :, None], now.transpose(1, 2), was)
            if name == "v":
                out = out.transpose(2, 3)
            cache.view(torch.uint8)[s["to_page"]] = out.contiguous().to(torch.float8_e4m3fn).view(torch.uint8)
            scales[s["to_page"]] = scale
    return {"lens": lens.to(torch.int32), "k": s["k"], "v": s["v"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _plain_fork(s, c):
    P, width, pages = c["page"], s["table"].shape[1], s["k"].shape[0]
    come = s["from"].long()
    some = come >= 0
    lens = torch.where(some, s["kv_lens"].long()[come.clamp(min=0)], 0)
    have = (lens + P - 1) // P
    j = torch.arange(width, device=come.device)
    table = torch.where(some[:, None] & (j < have[:, None]), s["table"].long()[come.clamp(min=0)], -1)
    refs = torch.zeros(pages + 1, dtype=torch.int64, device=come.device)
    refs.index_add_(0, torch.where(table >= 0, table, pages).flatten(), torch.ones(table.numel(), dtype=torch.int64, device=come.device))
    refs = refs[:pages]
    want = torch.minimum(lens + s["grow"].clamp(min=0), torch.full_like(lens, width * P))
    last = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    copy = (lens % P != 0) & (want > lens) & (last >= 0) & (refs[last.clamp(min=0)] > 1)
    get = (j >= (have - copy.long())[:, None]) & (j < ((want + P - 1) // P)[:, None])
    upto = torch.cumsum(get.sum(1), 0)
    granted = upto <= (refs == 0).sum()
    order = torch.sort((refs > 0).to(torch.int32), stable=True).indices          # the free pages first, ascending
    rank = (torch.cumsum(get.flatten(), 0) - 1).view(get.shape).clamp(max=pages - 1)
    table = torch.where(get, torch.where(granted[:, None], order[rank], -1), table)
    moved = copy & granted
    pairs = torch.stack([torch.where(moved, last, -1), torch.where(moved, table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0], -1)], 1)
    missing = torch.where(granted, 0, get.sum(1)).sum().to(torch.int32).view(1)
    # the copies: those that are none copy a page to itself, one in use if there is any
    src, dst = torch.where(moved, last, order[-1]), torch.where(moved, pairs[:, 1], order[-1])
    for name in ("k", "v"):
        codes = s[name].view(torch.uint8)
        codes[dst] = codes[src]
        s[name + "_scales"][dst] = s[name + "_scales"][src]
    return {"table": table.to(torch.int32), "lens": lens.to(torch.int32), "copies": pairs.to(torch.int32), "missing": missing, "k": s["k"],
            "v": s["v"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


# ---- the definitions in 64 bits, one sequence after the other ----

def _e4m3(x):
    """Nearest e4m3 value of each double, ties to the even code (none is beyond 448)."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    new, kv = _lengths(c)
    if c["op"] == "rows":
        parents = s["parents"].tolist()
        mask, positions, at = [], [], 0
        for b, n in enumerate(new):
            seen = []
            for t in range(n):
                up = parents[at + t]
                seen.append((seen[up] if 0 <= up < t else 0) | 1 << t)
                word = [seen[t] >> 32 * w & 0xFFFFFFFF for w in range(s["words"])]
                mask.append([x - (1 << 32) if x >> 31 else x for x in word])
                positions.append(kv[b] - n + bin(seen[t]).count("1") - 1)
            at += n
        return {"mask": torch.tensor(mask, dtype=torch.int32), "positions": torch.tensor(positions, dtype=torch.int32)}
    P, D, Hk = c["page"], c["dim"], c["kv_heads"]
    host = s["table"].cpu()
    if c["op"] == "tree":
        G = c["q_heads"] // Hk
        if sum(n * t for n, t in zip(new, kv)) * c["q_heads"] > 3 << 30:
            return None
        outs, at = [], 0
        word = s["mask"].cpu()
        for b in range(c["seqs"]):
            n, L = new[b], kv[b]
            ids = host[b, : -(-L // P)].long().to(s["k"].device)
            first = L - n
            drafted = torch.stack([(word[at: at + n, u // 32] >> (u % 32)) & 1 for u in range(n)], 1).bool().to(ids.device)
            j = torch.arange(first, device=ids.device)[None, :]
            hidden = torch.zeros((n, first), dtype=torch.bool, device=ids.device)
            if c["window"]:
                place = first + drafted.sum(1, keepdim=True) - 1
                hidden = (place - j >= c["window"]) & (j >= c["sinks"])
            hidden = torch.cat([hidden, ~drafted], 1)
            rows = s["q"][at: at + n].double()
            one = torch.empty((n, c["q_heads"], D), dtype=torch.float64, device=ids.device)
            for h in range(Hk):
                kh = (s["k"][:, h].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * s["k_scales"][ids, h].double()[:, None, None]).reshape(-1, D)[:L]
                vh = (s["v"][:, h].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * s["v_scales"][ids, h].double()[:, None, None]).transpose(1, 2).reshape(-1, D)[:L]
                for x in range(h * G, (h + 1) * G):
                    w = torch.softmax((rows[:, x] @ kh.t().contiguous() / math.sqrt(D)).masked_fill_(hidden, -math.inf), -1)
                    one[:, x] = w @ vh
            outs.append(one)
            at += n
        return torch.cat(outs)
    if c["op"] == "fork":
        width, pages = host.shape[1], s["k"].shape[0]
        lens, rows = [], []
        for b, f in enumerate(s["from"].tolist()):
            lens.append(kv[f] if f >= 0 else 0)
            held = -(-lens[-1] // P)
            rows.append(host[f, :held].tolist() + [-1] * (width - held) if f >= 0 else [-1] * width)
        refs = [0] * pages
        for r in rows:
            for p in r:
                if p >= 0:
                    refs[p] += 1
        free = [p for p in range(pages) if not refs[p]]
        taken = asked = missing = 0
        pairs = []
        for b, more in enumerate(s["grow"].tolist()):
            want = min(lens[b] + max(more, 0), width * P)
            places = list(range(-(-lens[b] // P), -(-want // P)))
            pair = [-1, -1]
            at = lens[b] // P
            if want > lens[b] and lens[b] % P and rows[b][at] >= 0 and refs[rows[b][at]] > 1:
                places.insert(0, at)
                pair[0] = rows[b][at]
            asked += len(places)
            if asked > len(free):
                missing += len(places)
                for i in places:
                    rows[b][i] = -1
                pair = [-1, -1]
            else:
                for i in places:
                    rows[b][i] = free[taken]
                    taken += 1
                if pair[0] >= 0:
                    pair[1] = rows[b][at]
            pairs.append(pair)
        out = {"table": torch.tensor(rows, dtype=torch.int32), "lens": torch.tensor(lens, dtype=torch.int32),
               "copies": torch.tensor(pairs, dtype=torch.int32), "missing": torch.tensor([missing], dtype=torch.int32)}
        for name in ("k", "v", "k_scales", "v_scales"):
            x = s[name].double()
            for a, b in pairs:
                if a >= 0:
                    x[b] = s[name][a].double()
            out[name] = x
        return out
    if c["op"] == "keep":
        if sum(m // P + 1 for m in s["counts"].tolist()) > 20000:
            return None
        kept, counts = s["kept"].tolist(), s["counts"].tolist()
        out = {"lens": torch.tensor([kv[b] - new[b] + counts[b] for b in range(c["seqs"])], dtype=torch.int32)}
        for name in ("k", "v"):
            codes, scales = s[name].double(), s[name + "_scales"].double()
            old = (codes.transpose(2, 3) if name == "v" else codes).clone()
            now, then = old.clone(), scales.clone()
            for b, m in enumerate(counts):
                first = kv[b] - new[b]
                come = torch.cat([torch.arange(first), first + torch.tensor(kept[b][:m], dtype=torch.int64)])
                for j in range(first // P, -(-(first + m) // P)):
                    src = come[j * P: (j + 1) * P].to(old.device)
                    if not m:
                        continue
                    id = host[b].long().to(old.device)[src // P]
                    most = then[id].amax(0)                                       # [heads]
                    x = old[id, :, src % P] * (then[id] / most)[..., None]          # [tokens][heads][dim]
                    page = int(host[b, j])
                    now[page, :, : len(src)] = _e4m3(x).transpose(0, 1)
                    scales[page] = most
            out[name] = now.transpose(2, 3).contiguous() if name == "v" else now
            out[name + "_scales"] = scales
        return out
    R, half = c["rot"], c["pairs"] == "half"
    axis = torch.tensor(_axis_of(c), device=s["rope"].device)

    def turned(x):
        x = x.double().clone()
        f = torch.arange(R // 2, device=x.device)
        lo, hi = (f, f + R // 2) if half else (2 * f, 2 * f + 1)
        place = s["positions"].long().index_select(1, axis)
        cos = torch.stack([s["rope"][place[:, i], i] for i in range(R // 2)], 1).double()[:, None]
        sin = torch.stack([s["rope"][place[:, i], R // 2 + i] for i in range(R // 2)], 1).double()[:, None]
        a, b = x[..., lo].clone(), x[..., hi].clone()
        x[..., lo] = a * cos - b * sin
        x[..., hi] = a * sin + b * cos
        return x

    out = {"q": turned(s["q"])}
    for name, fresh in (("k", turned(s["new_k"])), ("v", s["new_v"].double())):
        codes, scales = s[name].double(), s[name + "_scales"].double()
        if name == "v":
            codes = codes.transpose(2, 3)
        at = 0
        for b in range(c["seqs"]):
            n, first = new[b], kv[b] - new[b]
            for j in range(first // P, (kv[b] - 1) // P + 1):
                page, lo, hi = int(host[b, j]), max(first, j * P), min(kv[b], (j + 1) * P)
                x = fresh[at + lo - first: at + hi - first].transpose(0, 1)                     # [heads][tokens][dim]
                most = x.abs().amax((1, 2))
                need = torch.exp2(torch.ceil(torch.log2((most / 448).clamp(min=2.0 ** -64))))
                held = lo - j * P
                scale = torch.maximum(need, scales[page]) if held else need
                codes[page, :, :held] = _e4m3(codes[page, :, :held] * (scales[page] / scale)[:, None, None])
                codes[page, :, held: held + hi - lo] = _e4m3(x / scale[:, None, None])
                scales[page] = scale
            at += n
        out[name] = codes.transpose(2, 3).contiguous() if name == "v" else codes
        out[name + "_scales"] = scales
    return out
