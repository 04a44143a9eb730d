"""awq_kv_append_at on the GPU against its 64-bit form (tests/draft_cases.py), with the
tolerances of test_gpu_kv_append.py, which follow from the same arithmetic."""
import math

import pytest
import torch

import draft_cases as dc
import kv_cases as kc
from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def run(t, positions, rope, axis_of, interleaved=False, max_q=None):
    cache, batch, q, k, v = t.device(max_q)
    out = torch.full(q.shape, 7.0, dtype=t.dtype, device=DEV)
    got = binding.kv_append_at(q, k, v, cache, batch, positions.to(DEV), rope.to(DEV), axis_of=axis_of,
                               interleaved=interleaved, out=out)
    torch.cuda.synchronize()
    assert got is out
    return got.cpu(), cache.k.cpu(), cache.v.cpu(), cache.k_scales.cpu(), cache.v_scales.cpu()


def compare(t, got, positions, rope, axis_of, interleaved=False):
    q, k, v, ks, vs = got
    at = positions if positions.dim() == 2 else positions[:, None]
    full = dc.turned(t, at, rope, axis_of or bytes(rope.shape[1] // 2), interleaved)
    wq, wk, wv, wks, wvs, done = kc.append(full)
    assert torch.equal(vs.double(), wvs)
    # the key scale is decided by the largest turned magnitude, of which fp32 has 2^-22: powers of two apart only at a border
    assert torch.equal(ks.double(), wks)
    placed = torch.zeros(q.shape[0], dtype=torch.bool)
    for b, n in enumerate(t.new):
        length = min(max(t.lens[b], 0), t.width * t.page)
        for i in range(n):
            placed[t.starts[b] + i] = length - n + i >= 0
    assert torch.equal(q[~placed], torch.full_like(q, 7.0)[~placed])
    rq, rk, _ = t.split()
    near = 2.0 ** -22 * 2 * rq.double().abs().amax(-1, keepdim=True)
    assert torch.equal(q[placed].isnan(), wq[placed].isnan())
    off = (q.double() - wq).abs().nan_to_num(0.0)
    assert bool((off <= near + kc.half_step(t.dtype) * (wq.abs().nan_to_num(0.0) + near))[placed].all())
    s = wks[:, :, None, None]
    near = 2.0 ** -22 * 2 * rk.double().abs().max() / s
    assert torch.equal(k.double().isnan(), wk.isnan())
    want, have = torch.nan_to_num(wk, 0.0), torch.nan_to_num(k.double(), 0.0)
    step = torch.maximum(want.abs() * 2.0 ** -3, torch.tensor(2.0 ** -9, dtype=torch.float64))
    assert bool(((have - want).abs() <= step + near).all())
    assert float((have != want).double().mean()) < 1e-3
    assert torch.equal(torch.nan_to_num(v.double(), 999.0), torch.nan_to_num(wv, 999.0))
    kb, vb = kc.bytes_of(k), kc.bytes_of(v)
    assert torch.equal(kb.transpose(1, 2)[~done], t.k.transpose(1, 2)[~done])
    assert torch.equal(vb.permute(0, 3, 1, 2)[~done], t.v.permute(0, 3, 1, 2)[~done])


def places(t):
    """Where each row stands."""
    return torch.tensor([t.lens[b] - n + i for b, n in enumerate(t.new) for i in range(n)], dtype=torch.int32)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,page,heads,rot,interleaved", [(64, 16, (4, 4), 64, False), (128, 64, (8, 2), 128, True),
                                                            (256, 32, (5, 1), 96, False), (128, 128, (14, 2), 16, True),
                                                            (64, 256, (3, 3), 48, True), (256, 64, (2, 2), 256, False)])
@pytest.mark.parametrize("axes,in_turn", [(1, False), (2, True), (3, False), (4, True)])
def test_axes(dtype, dim, page, heads, rot, interleaved, axes, in_turn):
    """Positions anywhere in the table, in ragged rows from one to several pages."""
    new = [1, page + 3, 5, 0, 1, page - 1]
    lens = [1, page + 3, page + 9, 7, 2 * page + 1, 2 * page - 1]
    t = kc.Batch(11 + axes, dtype, new, lens, *heads, dim, page).fill([n - m for n, m in zip(lens, new)])
    positions = torch.randint(0, 300, (sum(new), axes), generator=t.g, dtype=torch.int32)
    half, rope = rot // 2, kc.rope_table(300, rot)
    sections = [half // axes + (a < half % axes) for a in range(axes)]
    axis_of = binding.axis_map(sections, in_turn)
    compare(t, run(t, positions, rope, axis_of, interleaved), positions, rope, axis_of, interleaved)


@pytest.mark.parametrize("dim,page,rot,interleaved", [(128, 64, 128, False), (64, 16, 32, True), (256, 128, 256, False)])
@pytest.mark.parametrize("axes", [0, 1, 3])
def test_positions_that_are_places(dim, page, rot, interleaved, axes):
    """The same bits as awq_kv_append, however many axes say the same; prompts and tokens."""
    new, lens = [300, 1, 7], [333, 65, 7]
    t = kc.Batch(20, "fp16", new, lens, 6, 2, dim, page).fill([n - m for n, m in zip(lens, new)])
    rope = kc.rope_table(400, rot)
    at = places(t) if axes == 0 else places(t)[:, None].repeat(1, axes)
    axis_of = None if axes == 0 else bytes(f * 7 % axes for f in range(rot // 2))
    cache, batch, q, k, v = t.device()
    want = binding.kv_append(q, k, v, cache, batch, rope=rope.to(DEV), interleaved=interleaved)
    got = run(t, at, rope, axis_of, interleaved)
    assert torch.equal(got[0], want.cpu())
    for a, b in zip(got[1:3], (cache.k, cache.v)):
        assert torch.equal(kc.bytes_of(a), kc.bytes_of(b).cpu())
    assert torch.equal(got[3], cache.k_scales.cpu()) and torch.equal(got[4], cache.v_scales.cpu())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_turn", [False, True])
def test_positions_behind_the_table(interleaved, in_turn):
    """They turn by NaN: the query's pairs on that axis, the key's codes; no other row is touched,
    and an axis that no frequency takes does not count."""
    new, lens = [20, 3, 40], [20, 30, 75]
    t = kc.Batch(21, "bf16", new, lens, 4, 2, 64, 16).fill([0, 27, 35])
    positions = torch.randint(0, 50, (63, 4), generator=t.g, dtype=torch.int32)
    positions[:, 3] = -1
    for row, axis, at in ((3, 0, 50), (17, 1, -1), (22, 2, 2 ** 31 - 1), (40, 0, -2 ** 31), (41, 1, 1 << 30)):
        positions[row, axis] = at
    axis_of = binding.axis_map([6, 5, 5], in_turn)
    rope = kc.rope_table(50, 32)
    got = run(t, positions, rope, axis_of, interleaved)
    assert int(got[0].isnan().any(-1).all(-1).sum()) == 5
    compare(t, got, positions, rope, axis_of, interleaved)


def test_places_that_are_none():
    """Rows below position 0 and pages that are none; a position has no say in that."""
    new, lens = [9, 4, 40, 6, 3], [4, 60, 40, 34, 500]
    t = kc.Batch(22, "fp16", new, [n if n < 400 else 64 for n in lens], 4, 2, 64, 16, extra_rows=5)
    t.fill([max(0, n - m) for n, m in zip(t.lens, new)])
    t.table[2, 1] = t.pages
    t.table[2, 2] = -7
    t.lens = lens
    positions = torch.randint(0, 30, (t.x.shape[0], 2), generator=t.g, dtype=torch.int32)
    rope, axis_of = kc.rope_table(30, 32), binding.axis_map([3, 13])
    compare(t, run(t, positions, rope, axis_of), positions, rope, axis_of)


@pytest.mark.parametrize("max_q", [1, 1000])
@pytest.mark.parametrize("held,n", [(0, 2), (3, 29), (6, 64), (13, 115)])
def test_odd_places(max_q, held, n):
    t = kc.Batch(40 + n, "fp16", [n], [held + n], 2, 1, 128, 128).fill([held])
    positions = torch.randint(0, 90, (n, 3), generator=t.g, dtype=torch.int32)
    rope, axis_of = kc.rope_table(90, 128), binding.axis_map([16, 24, 24], True)
    compare(t, run(t, positions, rope, axis_of, max_q=max_q), positions, rope, axis_of)


@pytest.mark.parametrize("dtype,dim,page", [("fp16", 128, 16), ("bf16", 64, 64)])
def test_prompts_among_single_tokens(dtype, dim, page):
    """So many sequences, of such different rows, that workgroups look for their work."""
    new, lens = [300, 2], [340, 1]
    for i in range(160):
        new.append((1, 0, 5, 1, 17)[i % 5])
        lens.append((1, 7, 3, 65 + i, 33)[i % 5])
    t = kc.Batch(31, dtype, new, lens, 4, 2, dim, page, extra_rows=1).fill([n - m for n, m in zip(lens, new)])
    positions = torch.randint(0, 400, (t.x.shape[0], 3), generator=t.g, dtype=torch.int32)
    rope, axis_of = kc.rope_table(400, dim // 2), bytes(f % 3 for f in range(dim // 4))
    compare(t, run(t, positions, rope, axis_of), positions, rope, axis_of)


def test_not_finite_rows():
    new, lens = [20, 3], [20, 30]
    t = kc.Batch(4, "bf16", new, lens, 2, 2, 64, 16).fill([0, 27])
    _, k, v = t.split()
    k[3, 1, 5] = math.nan
    k[4, 0, 63] = math.inf
    v[7, 1, 0] = -math.inf
    positions = torch.randint(0, 30, (23, 2), generator=t.g, dtype=torch.int32)
    rope, axis_of = kc.rope_table(30, 32), binding.axis_map([8, 8])
    got = run(t, positions, rope, axis_of)
    full = dc.append_at(t, positions, rope, axis_of)
    assert torch.equal(got[1].double().isnan(), full[1].isnan()) and torch.equal(got[3].double(), full[3])


def test_in_place_without_queries_and_on_a_side_stream():
    new, lens = [150, 1, 3], [170, 33, 3]
    t = kc.Batch(33, "fp16", new, lens, 6, 2, 128, 64).fill([n - m for n, m in zip(lens, new)])
    positions = torch.randint(0, 180, (154, 3), generator=t.g, dtype=torch.int32).to(DEV)
    rope, axis_of = kc.rope_table(180, 128).to(DEV), binding.axis_map([16, 24, 24])
    cache, batch, q, k, v = t.device()
    want = binding.kv_append_at(q, k, v, cache, batch, positions, rope, axis_of)
    again, batch, q, k, v = t.device(max_q=1)
    dense = q.contiguous()
    assert binding.kv_append_at(dense, k, v, again, batch, positions, rope, list(axis_of), out=dense) is dense
    assert torch.equal(dense, want) and torch.equal(kc.bytes_of(again.k), kc.bytes_of(cache.k))
    alone, batch, _, k, v = t.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert binding.kv_append_at(None, k.contiguous(), v.contiguous(), alone, batch, positions, rope, axis_of, stream=side) is None
    side.synchronize()
    assert torch.equal(kc.bytes_of(alone.k), kc.bytes_of(cache.k)) and torch.equal(kc.bytes_of(alone.v), kc.bytes_of(cache.v))


def test_binding_refusals():
    t = kc.Batch(71, "fp16", [1, 3], [5, 40], 4, 2, 64, 16).fill()
    cache, batch, q, k, v = t.device()
    rope, at = torch.zeros((50, 32), device=DEV), torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    call = lambda at, axis_of=None: binding.kv_append_at(q, k, v, cache, batch, at, rope, axis_of)  # noqa: E731
    with pytest.raises(ValueError, match="positions must be"):
        call(at[:3])
    with pytest.raises(ValueError, match="positions must be"):
        call(at[None])
    with pytest.raises(TypeError, match="positions must be"):
        call(at.long())
    with pytest.raises(ValueError, match="contiguous"):
        call(at.t().contiguous().t())
    with pytest.raises(ValueError, match="positions is on"):
        call(at.cpu())
    with pytest.raises(ValueError, match="axis_of"):
        call(at, bytes(15))
    with pytest.raises(binding.AwqError) as e:
        call(at, bytes([2] * 16))
    assert e.value.status == binding.AWQ_ERROR_INVALID_VALUE
    with pytest.raises(binding.AwqError) as e:
        call(torch.zeros((4, 5), dtype=torch.int32, device=DEV))
    assert e.value.status == binding.AWQ_ERROR_INVALID_VALUE
    assert torch.equal(kc.bytes_of(cache.k).cpu(), t.k) and torch.equal(kc.bytes_of(cache.v).cpu(), t.v)
