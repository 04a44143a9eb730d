"""The plain forms that the GPU tests compare with, pinned to hand-worked values (CPU)."""
import math

import pytest
import torch

import kv_cases as kc


def test_e4m3_rounding_is_the_types():
    """Every half-way point and its neighbours, against torch's own conversion."""
    codes = torch.arange(0, 0x7F, dtype=torch.uint8).view(kc.F8).double()
    mid = (codes[1:] + codes[:-1]) / 2
    for x in (codes, mid, mid * (1 + 1e-6), mid * (1 - 1e-6)):
        for y in (x, -x):
            assert torch.equal(kc.e4m3(y), y.float().to(kc.F8).double())


@pytest.mark.parametrize("most,want", [(0.0, -64), (448.0, 0), (448.1, 1), (224.0, -1), (1.0, -8), (0.875, -9),
                                       (2.0 ** -80, -64)])
def test_scale(most, want):
    assert kc.scale_for(most) == 2.0 ** want


def test_append_by_hand():
    t = kc.Batch(1, "fp16", [1], [2], 1, 1, 64, 16)
    id = int(t.table[0, 0])
    t.k[id, 0, 0] = torch.full((64,), 100.0).to(kc.F8).view(torch.uint8)       # rounds to 96 or 104: 96
    t.ks[id] = t.vs[id] = 0.25
    t.v[id, 0, :, 0] = torch.full((64,), 3.0).to(kc.F8).view(torch.uint8)
    t.x[0, 64:128] = 448.0                                                     # key: raises the scale to 1
    t.x[0, 128:] = 0.25                                                        # value: does not
    q, k, v, ks, vs, done = kc.append(t)
    assert float(ks[id, 0]) == 1.0 and float(vs[id, 0]) == 0.25
    assert k[id, 0, 0].tolist() == [24.0] * 64 and k[id, 0, 1].tolist() == [448.0] * 64
    assert v[id, 0, :, 0].tolist() == [3.0] * 64 and v[id, 0, :, 1].tolist() == [1.0] * 64
    assert done[id].tolist() == [True] * 2 + [False] * 14
    # a quarter turn: (a, b) -> (-b, a)
    rope = torch.tensor([[0.0] * 16 + [1.0] * 16] * 2)
    q, *_ = kc.append(t, rope)
    x = t.x[0, :64].double()
    assert torch.equal(q[0, 0], torch.cat([-x[16:32], x[:16], x[32:]]))
    q, *_ = kc.append(t, rope, True)
    assert torch.equal(q[0, 0, :32], torch.stack([-x[1:32:2], x[0:32:2]], 1).flatten())


def test_attention_by_hand():
    t = kc.Batch(1, "fp16", [2], [3], 1, 1, 64, 16).fill()
    id = int(t.table[0, 0])
    t.k[id, 0, :3] = 0                                          # equal weights
    t.vs[id] = 0.5
    one = lambda x: torch.full((64,), float(x)).to(kc.F8).view(torch.uint8)  # noqa: E731
    for j, x in enumerate((2, 4, 12)):
        t.v[id, 0, :, j] = one(x)
    out, size, reach = kc.attention(t)
    assert torch.allclose(out[0], torch.full((1, 64), 1.5, dtype=torch.float64), rtol=1e-15)       # (2 + 4) / 4
    assert torch.allclose(out[1], torch.full((1, 64), 3.0, dtype=torch.float64), rtol=1e-15)       # 18 / 6
    out, *_ = kc.attention(t, window=1)
    assert out[:, 0, 0].tolist() == [2.0, 6.0]
    out, *_ = kc.attention(t, window=1, sinks=1)
    assert out[:, 0, 0].tolist() == [1.5, 3.5]
    t.lens = [1]                                                # the first row is below position 0
    out, *_ = kc.attention(t)
    assert out[:, 0, 0].tolist() == [0.0, 1.0]
    assert float(reach.max()) == 0.0 and math.isclose(float(size[1, 0, 0]), 3.0)
