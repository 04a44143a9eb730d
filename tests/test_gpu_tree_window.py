"""awq_tree_attention under a window: where the border of what a row sees lies, by the bits set in
its mask, bits past the sequence's rows among them, and what chains have in common with causal
attention."""
import pytest
import torch

import kv_cases as kc
from test_gpu_tree_attention import check, trees
from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu

# few rows; many of heads of 64 and 128, in workgroups of four waves and of two; many of 256
FEW = [("fp16", 64, 16, (4, 2), [4, 8], [1004, 648]), ("bf16", 128, 64, (8, 2), [4], [1004]), ("fp16", 256, 128, (2, 1), [9, 1], [649, 1001])]
MANY = [("fp16", 64, 16, (8, 2), [100], [1100]), ("bf16", 128, 64, (8, 2), [100, 65], [900, 1065]), ("fp16", 256, 64, (4, 2), [100], [1003]),
        ("bf16", 64, 64, (32, 8), [40], [3400])]


def bits_for(t, words, kind):
    """All bits of the words for each row ("sees all rows"), a tree's for every other row beside that, or bits past
    the rows beside a tree's, more of them from row to row."""
    own = trees(t)[1]
    full = (1 << 32 * words) - 1
    out, at = [], 0
    for n in t.new:
        for r in range(n):
            past = ((1 << r % (32 * words - n + 1)) - 1) << n
            out.append({"all": full, "every other": full if r % 2 else own[at], "past": own[at] | past}[kind])
            at += 1
    return out


@pytest.mark.parametrize("kind", ["all", "every other", "past"])
@pytest.mark.parametrize("window,sinks", [(120, 0), (80, 0), (333, 70), (1, 0), (2000, 4)])
@pytest.mark.parametrize("dtype,dim,page,heads,new,lens", FEW + MANY)
def test_bits_past_the_rows_count(dtype, dim, page, heads, new, lens, window, sinks, kind):
    """Behind prefixes of many tiles: a row of a sequence of n stands at first + (bits set) - 1, which
    may be behind the last token, and keys up to that less the window are hidden in whichever tile they are."""
    t = kc.Batch(40, dtype, new, lens, *heads, dim, page).fill()
    for words in (-(-max(new) // 32), -(-max(new) // 32) + 2):
        check(t, bits_for(t, words, kind), words, window=window, sinks=sinks)


@pytest.mark.parametrize("window", [100, 101, 128, 300, 5000])
@pytest.mark.parametrize("dim,page,heads", [(64, 16, (8, 2)), (128, 64, (8, 2)), (256, 128, (2, 1))])
@pytest.mark.parametrize("new,lens", [([3, 16], [700, 300]), ([100, 64], [600, 700])])
def test_a_chain_under_a_window_of_its_rows_and_more(dim, page, heads, new, lens, window):
    """Then it sees what causal attention does: the same outputs, each within its tolerance."""
    t = kc.Batch(41, "fp16", new, lens, *heads, dim, page).fill()
    bits = [(2 << r) - 1 for n in new for r in range(n)]
    got = check(t, bits, window=window, sinks=3)
    cache, batch, q, _, _ = t.device()
    other = binding.attention(q, cache, batch, window=window, sinks=3).cpu().double()
    tol = kc.attention_tolerance(t, *kc.attention(t, window=window, sinks=3))
    assert bool(((got.double() - other).abs() <= 2 * tol).all())


@pytest.mark.parametrize("dim,page,heads", [(64, 16, (8, 2)), (128, 64, (8, 2)), (256, 128, (2, 1))])
@pytest.mark.parametrize("new,lens,window", [([20], [300], 7), ([100, 70], [600, 70], 64)])
def test_a_chain_longer_than_the_window(dim, page, heads, new, lens, window):
    """The rows' own tokens are not subject to the window, so rows from the window's on see more than
    causal attention shows them: equal up to there, and to a window for the prefix alone behind."""
    t = kc.Batch(42, "fp16", new, lens, *heads, dim, page).fill()
    bits = [(2 << r) - 1 for n in new for r in range(n)]
    got = check(t, bits, window=window).double()
    cache, batch, q, _, _ = t.device()
    other = binding.attention(q, cache, batch, window=window).cpu().double()
    tol = 2 * kc.attention_tolerance(t, *kc.attention(t, window=window))
    same = ((got - other).abs() <= tol).flatten(1).all(1)
    for b, n in enumerate(new):
        rows = same[t.starts[b]: t.starts[b + 1]].tolist()
        assert rows[: window] == [True] * min(n, window) and not any(rows[window + 1:])
