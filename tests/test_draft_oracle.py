"""The plain forms of tests/draft_cases.py, pinned to hand-worked values (CPU)."""
import math

import torch

import draft_cases as dc
import kv_cases as kc


def test_bits_by_hand():
    #      0 - 1 - 3        2 and 5 hang on nothing (5's parent is behind it), 4 on 2
    bits, depth = dc.bits_of([-1, 0, -7, 1, 2, 6, 0], 1)
    assert bits == [0b1, 0b11, 0b100, 0b1011, 0b10100, 0b100000, 0b1000001]
    assert depth == [0, 1, 0, 2, 1, 0, 1]
    long = dc.bits_of([t - 1 for t in range(40)], 1)
    assert long[0][39] == 0xFFFFFFFF and long[1][39] == 39
    assert dc.mask_of(dc.bits_of([t - 1 for t in range(40)], 2)[0], 2)[39].tolist() == [-1, 0xFF]


def test_turns_by_hand():
    t = kc.Batch(1, "fp16", [1], [1], 1, 1, 64, 16)
    # position 1 turns every pair by a quarter, position 0 by nothing
    rope = torch.tensor([[1.0] * 8 + [0.0] * 8, [0.0] * 8 + [1.0] * 8])
    x = t.x[0, :64].double()
    q = dc.turned(t, [[1, 0]], rope, [0, 1] * 4, False).x[0, :64]
    even = torch.arange(8) % 2 == 0
    assert torch.equal(q[:8], torch.where(even, -x[8:16], x[:8])) and torch.equal(q[8:16], torch.where(even, x[:8], x[8:16]))
    assert torch.equal(q[16:], x[16:])
    q = dc.turned(t, [[1, 2]], rope, [0] * 7 + [1], True).x[0, :64]
    assert torch.equal(q[0:14:2], -x[1:14:2]) and torch.equal(q[1:14:2], x[0:14:2]) and bool(q[14:16].isnan().all())


def test_tree_attention_by_hand():
    t = kc.Batch(1, "fp16", [3], [5], 1, 1, 64, 16).fill()
    id = int(t.table[0, 0])
    t.k[id, 0, :5] = 0                                          # equal weights
    t.vs[id] = 1.0
    for j, x in enumerate((2, 4, 8, 16, 32)):
        t.v[id, 0, :, j] = torch.full((64,), float(x)).to(kc.F8).view(torch.uint8)
    out, *_ = dc.tree_attention(t, [0b001, 0b010, 0b101])
    want = [(2 + 4 + 8) / 3, (2 + 4 + 16) / 3, (2 + 4 + 8 + 32) / 4]
    assert torch.allclose(out[:, 0, 0], torch.tensor(want, dtype=torch.float64), rtol=1e-15)
    # places 2, 2 and 3; under a window of 2 the tokens from 1, 1 and 2 on
    out, *_ = dc.tree_attention(t, [0b001, 0b010, 0b101], window=2)
    assert torch.allclose(out[:, 0, 0], torch.tensor([6.0, 10.0, 20.0], dtype=torch.float64), rtol=1e-15)
    out, *_ = dc.tree_attention(t, [0b001, 0b010, 0b101], window=1, sinks=1)
    assert torch.allclose(out[:, 0, 0], torch.tensor([5.0, 9.0, 14.0], dtype=torch.float64), rtol=1e-15)
    t.lens, t.new = [3], [3]
    out, *_ = dc.tree_attention(t, [0, 0b111, 0b100])
    assert out[:, 0, 0].tolist()[0::2] == [0.0, 8.0] and math.isclose(float(out[1, 0, 0]), 14 / 3)


def test_a_chain_is_causal_attention():
    t = kc.Batch(2, "fp16", [5, 2], [40, 2], 2, 1, 64, 16).fill()
    bits = [(2 << r) - 1 for n in t.new for r in range(n)]
    for a, b in zip(dc.tree_attention(t, bits), kc.attention(t)):
        assert torch.equal(a, b)


def test_keep_by_hand():
    t = kc.Batch(3, "fp16", [4], [18], 1, 1, 64, 16).fill()      # rows at places 14, 15 | 16, 17
    a, b = int(t.table[0, 0]), int(t.table[0, 1])
    t.ks[a], t.ks[b], t.vs[a], t.vs[b] = 0.25, 0.5, 1.0, 0.25
    old = t.k.view(kc.F8).double()
    K, V, ks, vs, lens, may = dc.keep(t, [[0, 2, 3]], [3])
    assert lens == [17] and float(ks[a, 0]) == 0.5 and float(vs[a, 0]) == 1.0 and float(ks[b, 0]) == 0.5
    assert torch.equal(K[a, 0, 15], old[b, 0, 0]) and torch.equal(K[b, 0, 0], old[b, 0, 1])
    assert torch.equal(K[a, 0, :15], kc.e4m3(old[a, 0, :15] / 2))
    was = t.v.view(kc.F8).double()
    assert torch.equal(V[a, 0, :, 15], kc.e4m3(was[b, 0, :, 0] / 4)) and torch.equal(V[a, 0, :, :15], was[a, 0, :, :15])
    assert may[a].all() and may[b].tolist() == [True] + [False] * 15
    assert dc.keep(t, [[0, 1, 5]], [3])[4] == [16]               # 5 names no row
    assert dc.keep(t, [[1, 1]], [2])[4] == [15]
    K, V, ks, *_ = dc.keep(t, [[0, 1]], [2])                     # all in place
    assert torch.equal(K.nan_to_num(9e9), old.nan_to_num(9e9)) and float(ks[a, 0]) == 0.25


def test_fork_by_hand():
    table, lens = [[5, 7, -1, -1], [2, 9, 4, -1]], [20, 48]
    # two go on from the first: both write its shared page 7; one is new, one ends
    rows, out, copies, missing = dc.fork(table, lens, [0, 0, -1], [1, 13, 17], 16, 12)
    assert out == [20, 20, 0] and missing == 0
    assert rows == [[5, 0, -1, -1], [5, 1, 2, -1], [3, 4, -1, -1]]
    assert copies == [(7, 0), (7, 1), (-1, -1)]
    # alone, a page is not copied; a full page is not written
    rows, _, copies, _ = dc.fork(table, lens, [1, 0], [16, 12], 16, 12)
    assert rows == [[2, 9, 4, 0], [5, 7, -1, -1]] and copies == [(-1, -1)] * 2
    # held pages are copied, and not given
    rows, _, copies, missing = dc.fork(table, lens, [0], [1], 16, 12, [1, 1] + [0] * 5 + [1] + [0] * 4)
    assert rows == [[5, 2, -1, -1]] and copies == [(7, 2)] and missing == 0
    # three free pages (0, 1, 3) for 2 + 2 + 1: the second gets none, and none behind it
    rows, _, copies, missing = dc.fork([[5, 7, 6, 8], [2, 9, 4, 10]], [64, 64], [0, 1, -1, -1, -1, -1], [9, 0, 20, 30, 0, 1], 16, 11)
    assert rows == [[5, 7, 6, 8], [2, 9, 4, 10], [0, 1, -1, -1]] + [[-1] * 4] * 3 and missing == 3 and copies == [(-1, -1)] * 6
