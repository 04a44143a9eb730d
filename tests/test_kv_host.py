"""What the paged cache's calls refuse, on the CPU: nothing here launches a kernel, and
the made-up device addresses are never read."""
import ctypes

import pytest
import torch

from w4a16_group_quantized_amd import binding

FAKE, MISALIGNED = 0x10000000, 0x10000008
INVALID, SHAPE, ALIGN, UNSUPPORTED, WS = 1, 2, 3, 4, 5


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=8, page=64, heads=2, dim=128) | kw
    return binding.CKvCache(*a.values())


def batch(**kw):
    a = dict(table=FAKE, lens=FAKE, starts=FAKE, seqs=2, width=4, rows=3, max_q=2, max_kv=200) | kw
    return binding.CKvBatch(*a.values())


def append(c=None, b=None, q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, out=FAKE, heads=4, type=0, rope=FAKE,
           positions=100, rot=128, adjacent=0):
    return binding.load().awq_kv_append(q, qs, k, ks, v, vs, out, heads, type, rope, positions, rot, adjacent,
                                        cache() if c is None else c, batch() if b is None else b, None)


def attention(c=None, b=None, q=FAKE, qs=512, out=FAKE, heads=4, type=0, scale=0.1, window=0, sinks=0, ws=FAKE,
              nbytes=1 << 40):
    return binding.load().awq_attention(q, qs, out, heads, type, scale, window, sinks, cache() if c is None else c,
                                        batch() if b is None else b, ws, nbytes, None)


@pytest.mark.parametrize("call", [append, attention])
@pytest.mark.parametrize("c,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(heads=0), INVALID), (dict(dim=-64), INVALID),
    (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE), (dict(heads=65536), SHAPE),
    (dict(pages=1 << 30), SHAPE),
    (dict(k=MISALIGNED), ALIGN), (dict(v=MISALIGNED), ALIGN), (dict(ks=MISALIGNED), ALIGN), (dict(vs=MISALIGNED), ALIGN),
    (dict(dim=32), UNSUPPORTED), (dict(dim=512), UNSUPPORTED),
])
def test_cache_refusals(call, c, want):
    assert call(c=cache(**c)) == want


@pytest.mark.parametrize("call", [append, attention])
@pytest.mark.parametrize("b,want", [
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(starts=None), INVALID),
    (dict(seqs=-1), INVALID), (dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(max_q=-1), INVALID),
    (dict(max_kv=-1), INVALID), (dict(seqs=65536), SHAPE), (dict(seqs=65535, width=(1 << 15) + 1), SHAPE),
(dict(width=(1 << 24) + 1), SHAPE), (dict(rows=1 << 23), SHAPE),
    (dict(table=MISALIGNED), ALIGN), (dict(lens=MISALIGNED), ALIGN), (dict(starts=MISALIGNED), ALIGN),
    (dict(seqs=0, table=None, lens=None, starts=None), 0), (dict(rows=0), 0),        # nothing to do
])
def test_batch_refusals(call, b, want):
    assert call(b=batch(**b)) == want


@pytest.mark.parametrize("call", [append, attention])
def test_too_many_sequences_and_heads(call):
    wide = dict(qs=512 * 128, ks=512 * 128, vs=512 * 128) if call is append else dict(qs=512 * 128)
    assert call(c=cache(heads=512), b=batch(seqs=1 << 15), heads=512, **wide) == SHAPE


def test_null_views():
    lib, c, b = binding.load(), cache(), batch()
    args = (FAKE, 512, FAKE, 256, FAKE, 256, FAKE, 4, 0, FAKE, 100, 128, 0)
    assert lib.awq_kv_append(*args, None, b, None) == INVALID
    assert lib.awq_kv_append(*args, c, None, None) == INVALID
    assert lib.awq_attention(FAKE, 512, FAKE, 4, 0, 0.1, 0, 0, None, b, FAKE, 1 << 40, None) == INVALID
    assert lib.awq_attention(FAKE, 512, FAKE, 4, 0, 0.1, 0, 0, c, None, FAKE, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(type=2), INVALID), (dict(heads=0), INVALID), (dict(rot=-16), INVALID), (dict(rope=None), INVALID),
    (dict(positions=0), INVALID),
    (dict(heads=3), SHAPE), (dict(rot=8), SHAPE), (dict(rot=144), SHAPE), (dict(qs=504), SHAPE), (dict(qs=516), SHAPE),
    (dict(ks=248), SHAPE), (dict(vs=257), SHAPE),
    (dict(q=MISALIGNED), ALIGN), (dict(k=MISALIGNED), ALIGN), (dict(v=MISALIGNED), ALIGN), (dict(out=MISALIGNED), ALIGN),
    (dict(rope=MISALIGNED), ALIGN),
])
def test_append_refusals(kw, want):
    assert append(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(type=-1), INVALID), (dict(heads=-2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(heads=5), SHAPE), (dict(qs=500), SHAPE), (dict(qs=511), SHAPE),
    (dict(q=MISALIGNED), ALIGN), (dict(out=MISALIGNED), ALIGN),
])
def test_attention_refusals(kw, want):
    assert attention(**kw) == want


def test_workspace():
    lib, c = binding.load(), cache()
    b = batch(seqs=1, width=1000, rows=1, max_q=1, max_kv=60000)
    need = lib.awq_attention_workspace_bytes(4, 0, 0, c, b)
    assert need > 0 and need % 4 == 0
    assert attention(b=b, ws=None) == WS and attention(b=b, ws=MISALIGNED) == WS and attention(b=b, nbytes=need - 1) == WS
    # a short axis is not cut; what is refused, or empty, needs nothing
    assert lib.awq_attention_workspace_bytes(4, 0, 0, c, batch(max_kv=64)) == 0
    assert lib.awq_attention_workspace_bytes(4, 64, 0, c, b) < need
    assert lib.awq_attention_workspace_bytes(3, 0, 0, c, b) == 0
    assert lib.awq_attention_workspace_bytes(4, -1, 0, c, b) == 0
    assert lib.awq_attention_workspace_bytes(4, 0, 0, None, b) == 0
    assert lib.awq_attention_workspace_bytes(4, 0, 0, c, batch(rows=0)) == 0


def test_views_match_the_header():
    assert ctypes.sizeof(binding.CKvCache) == 48 and binding.CKvCache.pages.offset == 32
    assert ctypes.sizeof(binding.CKvBatch) == 48 and binding.CKvBatch.seqs.offset == 24
    text = open(binding.os.path.join(binding.os.path.dirname(binding.HERE), "include", "awq.h")).read()
    for name, value in (("FP16", binding.ROW_TYPES[torch.float16]), ("BF16", binding.ROW_TYPES[torch.bfloat16])):
        assert f"#define AWQ_TYPE_{name} {value}\n" in text


F8 = torch.float8_e4m3fn


def arrays(pages=3, heads=2, page=16, dim=64, **kw):
    a = dict(k=torch.empty((pages, heads, page, dim), dtype=F8), v=torch.empty((pages, heads, dim, page), dtype=F8),
             k_scales=torch.empty((pages, heads)), v_scales=torch.empty((pages, heads)))
    return a | kw


@pytest.mark.parametrize("kw,error,what", [
    (dict(k=torch.empty((3, 2, 16, 64))), TypeError, "k must be"),
    (dict(k=torch.empty((3, 2, 16), dtype=F8)), ValueError, "k must be"),
    (dict(v=torch.empty((3, 2, 16, 64), dtype=F8)), ValueError, "v must be"),
    (dict(v_scales=torch.empty((2, 3))), ValueError, "v_scales"),
    (dict(k_scales=torch.empty((3, 2), dtype=torch.float16)), TypeError, "k_scales"),
    (dict(v=torch.empty((3, 2, 64, 16), dtype=F8, device="meta")), ValueError, "v is on"),
    ({}, TypeError, "CUDA"),
])
def test_binding_cache(kw, error, what):
    with pytest.raises(error, match=what):
        binding.KvCache(**arrays(**kw))


@pytest.mark.parametrize("kw,error,what", [
    (dict(page_table=torch.zeros(4, dtype=torch.int32)), ValueError, "page_table"),
    (dict(kv_lens=torch.zeros(3, dtype=torch.int32)), ValueError, "kv_lens"),
    (dict(kv_lens=torch.zeros(2, dtype=torch.int64)), TypeError, "kv_lens"),
    (dict(q_starts=torch.zeros(2, dtype=torch.int32)), ValueError, "q_starts"),
    (dict(max_q=-1), ValueError, "max_q"), (dict(max_kv=1 << 31), ValueError, "max_kv"),
    ({}, TypeError, "CUDA"),
])
def test_binding_batch(kw, error, what):
    a = dict(page_table=torch.zeros((2, 4), dtype=torch.int32), kv_lens=torch.zeros(2, dtype=torch.int32),
             q_starts=torch.zeros(3, dtype=torch.int32), max_q=1, max_kv=1) | kw
    with pytest.raises(error, match=what):
        binding.KvBatch(**a)


def test_long_single_tokens_beside_a_prompt_are_cut():
    """The prompt's row tiles fill the GPU, so the prompt kernel cuts nothing; the kernel of the
    two single tokens, which may be long, cuts by its own count, within 256 MiB of room."""
    lib, c = binding.load(), cache(heads=8)
    need = lambda rows, kv: lib.awq_attention_workspace_bytes(  # noqa: E731
        32, 0, 0, c, batch(seqs=3, width=4096, rows=rows + 2, max_q=rows, max_kv=kv))
    one = lambda rows: (rows + 2) * 32 * (128 + 4) * 4  # noqa: E731
    assert need(2048, 131000) == 7 * one(2048) <= 1 << 28
    assert need(4096, 131000) == 3 * one(4096)
    assert need(16384, 131000) == 0                  # no room for two chunks
    assert need(2048, 500) == 0                      # too short to cut
