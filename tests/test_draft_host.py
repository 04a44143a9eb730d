"""What the calls of drafting refuse, on the CPU: nothing here launches a kernel, and the
made-up device addresses are never read."""
import pytest
import torch

from test_kv_host import ALIGN, FAKE, INVALID, MISALIGNED, SHAPE, UNSUPPORTED, WS, arrays, batch, cache
from w4a16_group_quantized_amd import binding

OTHER = FAKE + 0x1000


def append_at(c=None, b=None, q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, out=FAKE, heads=4, type=0, rope=FAKE,
              table=100, rot=128, adjacent=0, positions=FAKE, axes=3, axis_of=bytes([0, 1, 2, 2] * 16)):
    return binding.load().awq_kv_append_at(q, qs, k, ks, v, vs, out, heads, type, rope, table, rot, adjacent, positions,
                                           axes, axis_of, cache() if c is None else c, batch() if b is None else b, None)


def tree_attention(c=None, b=None, q=FAKE, qs=512, out=FAKE, heads=4, type=0, scale=0.1, window=0, sinks=0, mask=FAKE, words=1,
                   ws=FAKE, nbytes=1 << 40):
    return binding.load().awq_tree_attention(q, qs, out, heads, type, scale, window, sinks, mask, words,
                                             cache() if c is None else c, batch() if b is None else b, ws, nbytes, None)


def keep(c=None, b=None, kept=FAKE, width=4, counts=FAKE, lens=OTHER):
    return binding.load().awq_kv_keep(kept, width, counts, lens, cache() if c is None else c, batch() if b is None else b, None)


def fork(c=None, b=None, from_=FAKE, grow=FAKE, n=3, held=None, table=OTHER, lens=OTHER, copies=FAKE, missing=FAKE, ws=FAKE,
         nbytes=1 << 40):
    return binding.load().awq_kv_fork(from_, grow, n, held, cache() if c is None else c, batch() if b is None else b, table, lens,
                                      copies, missing, ws, nbytes, None)


def copy(c=None, to=None, pairs=FAKE, n=2):
    c = cache() if c is None else c
    return binding.load().awq_kv_copy(pairs, n, c, c if to is None else to, None)


@pytest.mark.parametrize("call", [append_at, tree_attention, keep, fork, copy])
@pytest.mark.parametrize("c,want", [
    (dict(k=None), INVALID), (dict(vs=None), INVALID), (dict(pages=0), INVALID), (dict(dim=-64), INVALID), (dict(page=48), SHAPE),
    (dict(heads=65536), SHAPE), (dict(pages=1 << 30), SHAPE), (dict(k=MISALIGNED), ALIGN), (dict(vs=MISALIGNED), ALIGN),
    (dict(dim=32), UNSUPPORTED),
])
def test_cache_refusals(call, c, want):
    assert call(c=cache(**c)) == want


@pytest.mark.parametrize("call", [append_at, tree_attention, keep, fork])
@pytest.mark.parametrize("b,want", [
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(starts=None), INVALID), (dict(seqs=-1), INVALID),
    (dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(max_q=-1), INVALID), (dict(seqs=65536), SHAPE),
    (dict(width=(1 << 24) + 1), SHAPE), (dict(table=MISALIGNED), ALIGN), (dict(lens=MISALIGNED), ALIGN),
])
def test_batch_refusals(call, b, want):
    assert call(b=batch(**b)) == want


def test_null_views_and_nothing_to_do():
    lib, c, b = binding.load(), cache(), batch()
    assert lib.awq_kv_keep(FAKE, 4, FAKE, OTHER, None, b, None) == INVALID
    assert lib.awq_kv_keep(FAKE, 4, FAKE, OTHER, c, None, None) == INVALID
    assert lib.awq_kv_copy(FAKE, 2, c, None, None) == INVALID and lib.awq_kv_copy(FAKE, 2, None, c, None) == INVALID
    assert lib.awq_tree_rows(FAKE, FAKE, 1, FAKE, None, None) == INVALID
    for call in (append_at, tree_attention):
        assert call(b=batch(rows=0)) == 0
    for call in (append_at, tree_attention, keep):
        assert call(b=batch(seqs=0, table=None, lens=None, starts=None)) == 0
    assert append_at(b=batch(rows=0), positions=None) == 0
    assert fork(n=0, from_=None) == 0 and copy(n=0, pairs=None) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(type=2), INVALID), (dict(heads=3), SHAPE), (dict(rot=8), SHAPE), (dict(qs=504), SHAPE),
    (dict(rope=None), INVALID), (dict(table=0), INVALID), (dict(out=None), INVALID), (dict(k=MISALIGNED), ALIGN),
    (dict(positions=None), INVALID), (dict(positions=MISALIGNED), ALIGN), (dict(axes=0), INVALID), (dict(axes=5), INVALID),
    (dict(axes=2), INVALID),                                          # the map names axis 2
    (dict(axis_of=bytes(63) + b"\x03"), INVALID), (dict(axis_of=bytes(63) + b"\xff"), INVALID),
])
def test_append_at_refusals(kw, want):
    assert append_at(**kw) == want


def test_the_map_is_checked_without_rows_too():
    assert append_at(b=batch(rows=0), axes=2) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(mask=None), INVALID), (dict(words=0), INVALID),
    (dict(words=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(heads=5), SHAPE), (dict(words=1 << 30), SHAPE), (dict(mask=MISALIGNED), ALIGN), (dict(q=MISALIGNED), ALIGN),
])
def test_tree_attention_refusals(kw, want):
    assert tree_attention(**kw) == want


def test_tree_attention_workspace():
    lib, c = binding.load(), cache()
    b = batch(seqs=1, width=1000, rows=8, max_q=8, max_kv=60000)
    need = lib.awq_tree_attention_workspace_bytes(4, 0, 0, c, b)
    assert need > 0 and tree_attention(b=b, ws=None) == WS and tree_attention(b=b, nbytes=need - 1) == WS
    assert tree_attention(b=b, ws=MISALIGNED) == WS
    assert lib.awq_tree_attention_workspace_bytes(3, 0, 0, c, b) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(parents=None), INVALID), (dict(mask=None), INVALID), (dict(words=0), INVALID), (dict(b=dict(lens=None)), INVALID),
    (dict(b=dict(starts=None)), INVALID), (dict(b=dict(seqs=-1)), INVALID), (dict(b=dict(rows=-1)), INVALID),
    (dict(b=dict(seqs=65536)), SHAPE), (dict(words=1 << 30), SHAPE), (dict(parents=MISALIGNED), ALIGN),
    (dict(mask=MISALIGNED), ALIGN), (dict(positions=MISALIGNED), ALIGN), (dict(b=dict(lens=MISALIGNED)), ALIGN),
    (dict(b=dict(rows=0)), 0), (dict(b=dict(seqs=0)), 0),
])
def test_tree_rows_refusals(kw, want):
    a = dict(parents=FAKE, mask=FAKE, words=1, positions=FAKE, b={}) | kw
    assert binding.load().awq_tree_rows(a["parents"], a["mask"], a["words"], a["positions"], batch(**a["b"]), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(kept=None), INVALID), (dict(counts=None), INVALID), (dict(lens=None), INVALID), (dict(lens=FAKE), INVALID),
    (dict(width=0), INVALID), (dict(width=1 << 30), SHAPE), (dict(kept=MISALIGNED), ALIGN), (dict(counts=MISALIGNED), ALIGN),
    (dict(lens=MISALIGNED), ALIGN),
])
def test_keep_refusals(kw, want):
    assert keep(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(from_=None), INVALID), (dict(grow=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(copies=None), INVALID), (dict(missing=None), INVALID), (dict(table=FAKE), INVALID), (dict(lens=FAKE), INVALID),
    (dict(n=-1), INVALID), (dict(n=65536), SHAPE), (dict(n=65535, b=dict(width=1 << 16)), SHAPE), (dict(from_=MISALIGNED), ALIGN),
    (dict(held=MISALIGNED), ALIGN), (dict(copies=MISALIGNED), ALIGN),
])
def test_fork_refusals(kw, want):
    assert fork(**{k: batch(**v) if k == "b" else v for k, v in kw.items()}) == want


def test_fork_workspace():
    """A small table takes none, a large one a few words for each entry and bits for each page."""
    lib, c, b = binding.load(), cache(), batch(width=1 << 15)
    need = lib.awq_kv_fork_workspace_bytes(3, c, b)
    assert need > 0 and fork(b=b, nbytes=need - 1) == WS
    assert fork(b=b, ws=None) == WS and fork(b=b, ws=MISALIGNED) == WS
    assert lib.awq_kv_fork_workspace_bytes(3, c, batch()) == 0
    assert lib.awq_kv_fork_workspace_bytes(3, cache(pages=1 << 20), batch()) > 0 < lib.awq_kv_fork_workspace_bytes(2000, c, batch())
    assert lib.awq_kv_fork_workspace_bytes(0, c, b) == 0 and lib.awq_kv_fork_workspace_bytes(3, None, b) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(pairs=None), INVALID), (dict(n=-1), INVALID), (dict(n=(1 << 22) + 1), SHAPE), (dict(pairs=MISALIGNED), ALIGN),
    (dict(to=dict(page=32)), SHAPE), (dict(to=dict(heads=1)), SHAPE), (dict(to=dict(dim=64)), SHAPE), (dict(to=dict(k=None)), INVALID),
])
def test_copy_refusals(kw, want):
    assert copy(**{k: cache(**v) if k == "to" else v for k, v in kw.items()}) == want


def test_axis_map():
    assert binding.axis_map([2, 0, 3]) == bytes([0, 0, 2, 2, 2])
    assert binding.axis_map([2, 1, 3], in_turn=True) == bytes([0, 1, 2, 0, 2, 2])
    assert binding.axis_map([]) == b""
    with pytest.raises(ValueError, match="sections"):
        binding.axis_map([3, -1])


def test_the_most_axes_are_the_headers():
    text = open(binding.os.path.join(binding.os.path.dirname(binding.HERE), "include", "awq.h")).read()
    assert "#define AWQ_MAX_AXES 4\n" in text
    assert append_at(axes=4, positions=None) == INVALID and arrays()["k"].dtype == torch.float8_e4m3fn
