"""Measured cases of the 8-bit paged key/value cache: appending to it, and attention over it.

Three operators of a decoder block's attention, beside its 4-bit linear layers:

* ``append``: rotate the new queries and keys by their positions, and write the
  keys and values into a paged cache of e4m3 codes, with one power-of-two scale
  for each page and kv head.
* ``attention``: causal attention of a ragged batch over such a cache, from one
  row per sequence (decode) to thousands (prefill).
* ``window``: the same with a sliding window and a few first tokens that stay
  visible.

``own`` false computes each in its plain form (elementary torch operations in
32 bits); true calls the framework.  ``exact`` is the definition in 64 bits.

The cache: k e4m3 [pages][kv_heads][page][dim], v e4m3 [pages][kv_heads][dim][page],
scales fp32 [pages][kv_heads]; a key or value is its code times its page's scale.
A sequence b has ``kv_lens[b]`` tokens in the cache, the last ones of them its
rows of this call (rows ``q_starts[b]`` to ``q_starts[b + 1] - 1``).
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, dtype, seqs, rows, ctx, q_heads, kv_heads, dim, page, rot=0, pairs="half", window=0, sinks=0):
    return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "rows": rows, "ctx": ctx, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "rot": rot, "pairs": pairs, "window": window, "sinks": sinks}


def listed():
    """``rows``: the most new tokens of a sequence; ``ctx``: the most tokens that a sequence has before them."""
    return [
        # one decode step of a small batch: the smallest append, a matter of latency
        _case("append_decode", "append", "fp16", 16, 1, 4000, 32, 8, 128, 64, rot=128),
        # prompts of several lengths arrive behind what their sequences hold already
        _case("append_prompts", "append", "fp16", 5, 2048, 1000, 32, 8, 128, 64, rot=128),
        # one long prompt, half of each head rotated, in adjacent pairs
        _case("append_long", "append", "bf16", 1, 16384, 0, 64, 8, 128, 128, rot=64, pairs="adjacent"),
        # one user, a short conversation: latency
        _case("decode_one", "attention", "fp16", 1, 1, 1000, 32, 8, 128, 64),
        # a serving batch of ragged lengths
        _case("decode_batch", "attention", "fp16", 32, 1, 8191, 32, 8, 128, 64),
        # two very long contexts: the split over the key axis carries it
        _case("decode_long", "attention", "bf16", 2, 1, 131000, 64, 8, 128, 128),
        # a few drafted tokens of each sequence verified at once, small heads, small pages
        _case("verify", "attention", "bf16", 16, 5, 2000, 32, 4, 64, 16),
        # a prompt from its first token
        _case("prefill", "attention", "fp16", 1, 4096, 0, 32, 8, 128, 64),
        # chunks of prompts over long contexts
        _case("prefill_chunks", "attention", "bf16", 4, 512, 16000, 64, 8, 128, 64),
        # a serving batch of long contexts where each row sees its last 4096 tokens and the first four
        _case("window_decode", "window", "fp16", 48, 1, 32000, 32, 8, 128, 64, window=4096, sinks=4),
        # a prompt under a window, wide heads
        _case("window_prefill", "window", "bf16", 1, 8192, 0, 16, 8, 256, 64, window=1024, sinks=4),
        # a few rows over a short window, no group of heads
        _case("window_verify", "window", "fp16", 8, 7, 5000, 12, 12, 64, 32, window=500, sinks=16),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges, of no more work than the largest of the listed ones."""
    while True:
        op = rng.choice(["append", "attention", "attention", "window"])
        kv = rng.choice([1, 2, 4, 8, 16])
        heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        dim = rng.choice([64, 128, 128, 256])
        page = rng.choice([16, 32, 64, 128])
        rows = rng.choice([1, _spread(rng, 2, 16), _spread(rng, 17, 4096)])
        seqs = _spread(rng, 1, 64)
        ctx = _spread(rng, 1, 131000) - 1
        if op == "append":
            if seqs * rows * heads * dim > 1 << 27 or seqs * (rows + ctx) * kv * dim > 1 << 28:
                continue
            rot = rng.choice([0, dim, dim, dim // 2])
            c = _case("", op, rng.choice(["fp16", "bf16"]), seqs, rows, ctx, heads, kv, dim, page, rot,
                      rng.choice(["half", "adjacent"]))
            break
        if heads > 64 or seqs * rows * (rows + ctx) * heads > 1 << 29 or seqs * (rows + ctx) * kv * dim > 1 << 28:
            continue
        window = _spread(rng, 16, 8192) if op == "window" else 0
        sinks = rng.choice([0, 1, 4, 16, 100]) if op == "window" else 0
        c = _case("", op, rng.choice(["fp16", "bf16"]), seqs, rows, ctx, heads, kv, dim, page,
                  window=window, sinks=sinks)
        break
    del c["name"]
    return c


def _lengths(c):
    """(new tokens, tokens after them) of each sequence: ragged, the first sequence the longest."""
    new, kv = [], []
    for b in range(c["seqs"]):
        n = c["rows"] - (b * 397) % max(1, c["rows"] // 2)
        before = c["ctx"] - (b * 7919) % max(1, c["ctx"] // 2 + 1)
        new.append(n)
        kv.append(before + n)
    return new, kv


def _sees(c, i):
    """How many keys a row at position i sees."""
    if not c["window"] or i + 1 <= c["window"]:
        return i + 1
    return c["window"] + min(c["sinks"], i + 1 - c["window"])


def work(case):
    c, (new, kv) = case, _lengths(case)
    rows, width = sum(new), c["dim"]
    if c["op"] == "append":
        codes = 2 * rows * c["kv_heads"] * width
        table = sum(4 * c["rot"] * n for n in new)
        return {"bytes": 2 * rows * (2 * c["q_heads"] + 2 * c["kv_heads"]) * width + codes + table,
                "flops": 3 * rows * (c["q_heads"] + c["kv_heads"]) * c["rot"] + 4 * rows * c["kv_heads"] * width}
    held = pairs = 0
    for n, total in zip(new, kv):
        first = total - n
        low = max(0, first + 1 - c["window"]) if c["window"] else 0
        held += total - low + min(c["sinks"], low)
        if c["window"]:
            pairs += sum(_sees(c, first + t) for t in range(n))
        else:
            pairs += n * first + n * (n + 1) // 2
    return {"bytes": 2 * held * c["kv_heads"] * width + 4 * rows * c["q_heads"] * width
            + 8 * (held // c["page"] + 1) * c["kv_heads"],
            "flops": 4 * pairs * c["q_heads"] * width}


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    new, kv = _lengths(c)
    P, Hk, D, Hq = c["page"], c["kv_heads"], c["dim"], c["q_heads"]
    dtype = DTYPES[c["dtype"]]
    need = [-(-n // P) for n in kv]
    width = max(need)
    pages = sum(need) + 1
    order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
    # page table: each sequence's pages anywhere in the pool; entries behind its last one name no page
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32, device=dev)
    at = torch.zeros((c["seqs"], width), dtype=torch.bool)
    for b, n in enumerate(need):
        at[b, :n] = True
    table[at.to(dev)] = order[: sum(need)]

    # codes of normal values under a scale that leaves the largest near 448; a scale of its own for each page and head
    def codes(shape):
        out = torch.empty(shape, dtype=torch.uint8, device=dev)
        flat, step = out.view(-1), 1 << 27
        for a in range(0, flat.numel(), step):
            n = min(step, flat.numel() - a)
            flat[a: a + n] = (torch.randn(n, device=dev, generator=g) * 90).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return out.view(torch.float8_e4m3fn)

    def scales():
        e = torch.randint(-9, -6, (pages, Hk), device=dev, generator=g)
        return torch.exp2(e.float())

    s = {"case": dict(c), "k": codes((pages, Hk, P, D)), "v": codes((pages, Hk, D, P)), "k_scales": scales(), "v_scales": scales(),
         "table": table, "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev)}
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    rows = starts[-1]
    s["max_q"], s["max_kv"] = max(new), max(kv)
    # the rows as a fused projection leaves them: queries, keys and values of a token side by side
    wide = torch.randn((rows, (Hq + 2 * Hk) * D), device=dev, generator=g) * 1.2
    x = wide.to(dtype)
    s["q"] = x[:, : Hq * D].unflatten(1, (Hq, D))
    s["new_k"] = x[:, Hq * D: (Hq + Hk) * D].unflatten(1, (Hk, D))
    s["new_v"] = x[:, (Hq + Hk) * D:].unflatten(1, (Hk, D))
    # where each row stands, as a serving program's scheduler knows it
    n, first = torch.tensor(new), torch.tensor(kv) - torch.tensor(new)
    seq = torch.repeat_interleave(torch.arange(c["seqs"]), n)
    t = torch.arange(rows) - torch.tensor(starts)[:-1][seq]
    pos = first[seq] + t
    s["row_seq"], s["row_t"], s["row_pos"] = seq.to(dev), t.to(dev), pos.to(dev)
    if c["op"] == "append":
        touched, where = torch.unique(seq * width + pos // P, return_inverse=True)
        tseq, tpage = touched // width, touched % width
        s["touch_pages"] = table.cpu()[tseq, tpage].long().to(dev)
        s["touch_old"] = (first[tseq] - tpage * P).clamp(0, P).to(dev)          # slots that hold tokens before the call
        s["row_touch"], s["row_slot"] = where.to(dev), (pos % P).to(dev)
        if c["rot"]:  # cosines and sines of every position, from 64-bit angles
            freq = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
            a = torch.arange(max(kv), dtype=torch.float64, device=dev)[:, None] * freq
            s["rope"] = torch.cat([a.cos(), a.sin()], 1).float()
        else:
            s["rope"] = None
    if own:
        from w4a16_group_quantized_amd import binding
        s["cache"] = binding.KvCache(s["k"], s["v"], s["k_scales"], s["v_scales"])
        s["batch"] = binding.KvBatch(s["table"], s["kv_lens"], s["q_starts"], s["max_q"], s["max_kv"])
    return s


def run(state):
    s, c = state, state["case"]
    if own:
        from w4a16_group_quantized_amd import binding
        if c["op"] == "append":
            q = binding.kv_append(s["q"], s["new_k"], s["new_v"], s["cache"], s["batch"], rope=s["rope"],
                                  interleaved=c["pairs"] == "adjacent")
            return {"q": q, "k": s["k"], "v": s["v"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}
        return binding.attention(s["q"], s["cache"], s["batch"], window=c["window"], sinks=c["sinks"])
    return _append(s, c) if c["op"] == "append" else _attention(s, c)


# ---- plain forms: 32 bits, elementary operations ----

def _rotate(x, s, c):
    x, R = x.float(), c["rot"]
    if not R:
        return x
    cos, sin = s["rope"][s["row_pos"]][:, None, :].split(R // 2, -1)
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


def _append(s, c):
    q = _rotate(s["q"], s, c).to(DTYPES[c["dtype"]])
    _write(s["k"], s["k_scales"], _rotate(s["new_k"], s, c), s, c, False)
    _write(s["v"], s["v_scales"], s["new_v"].float(), s, c, True)
    return {"q": q, "k": s["k"], "v": s["v"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _attention(s, c):
    B, n, L = c["seqs"], s["max_q"], s["max_kv"]
    P, Hk, D, G = c["page"], c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    at = s["table"].clamp(min=0).long()
    k = s["k"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["k_scales"][at][..., None, None]
    v = s["v"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["v_scales"][at][..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(B * Hk, D, -1)[:, :, :L].contiguous()
    v = v.permute(0, 2, 1, 4, 3).reshape(B * Hk, -1, D)[:, :L].contiguous()
    q = torch.zeros((B, n, Hk, G, D), device=k.device)
    q[s["row_seq"], s["row_t"]] = s["q"].float().unflatten(1, (Hk, G))
    q = q.permute(0, 2, 3, 1, 4).reshape(B * Hk, G * n, D)
    score = torch.bmm(q * (1 / math.sqrt(D)), k).view(B, Hk, G, n, L)
    counts = (s["q_starts"][1:] - s["q_starts"][:-1])[:, None]
    i = (s["kv_lens"][:, None] - counts + torch.arange(n, device=k.device))[..., None]      # positions of the rows
    j = torch.arange(L, device=k.device)
    seen = (j <= i) & (j < s["kv_lens"][:, None, None])
    if c["window"]:
        seen &= (j > i - c["window"]) | (j < c["sinks"])
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p.view(B * Hk, G * n, L), v).view(B, Hk, G, n, D) / total.clamp(min=1e-30)
    return out.permute(0, 3, 1, 2, 4)[s["row_seq"], s["row_t"]].flatten(1, 2).to(DTYPES[c["dtype"]])


# ---- the definition in 64 bits, one sequence after the other ----

def _e4m3(x):
    """Nearest e4m3 value of each double, ties to the even code (none is beyond 448)."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    new, kv = _lengths(c)
    P, D, Hk, G = c["page"], c["dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    table = s["table"].cpu()
    if c["op"] != "append":
        if sum(n * t for n, t in zip(new, kv)) * c["q_heads"] > 3 << 30:
            return None
        outs, at = [], 0
        for b in range(c["seqs"]):
            n, L = new[b], kv[b]
            ids = table[b, : -(-L // P)].long().to(s["k"].device)
            pos = torch.arange(L - n, L, device=ids.device)[:, None]
            j = torch.arange(L, device=ids.device)[None, :]
            hidden = j > pos
            if c["window"]:
                hidden |= (pos - j >= c["window"]) & (j >= c["sinks"])
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
    R, half = c["rot"], c["pairs"] == "half"

    def turned(x):
        x = x.double().clone()
        if R:
            f = torch.arange(R // 2, device=x.device)
            lo, hi = (f, f + R // 2) if half else (2 * f, 2 * f + 1)
            row = s["rope"].double()[s["row_pos"]]
            cos, sin = row[:, None, : R // 2], row[:, None, R // 2:]
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
                page, lo, hi = int(table[b, j]), max(first, j * P), min(kv[b], (j + 1) * P)
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
