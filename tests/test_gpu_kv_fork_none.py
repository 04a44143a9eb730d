"""awq_kv_fork through the binding where there are no new sequences: nothing is missing, on the
stream of the call, whether or not the outputs are there already."""
import pytest
import torch

from w4a16_group_quantized_amd import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def parts():
    ints = lambda *shape: torch.empty(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    cache = binding.new_kv_cache(4, 16, 1, 64, DEV)
    batch = binding.KvBatch(torch.zeros((1, 3), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV),
                            torch.zeros(2, dtype=torch.int32, device=DEV), 0, 1)
    return cache, batch, ints


def test_nothing_is_missing_in_given_outputs():
    cache, batch, ints = parts()
    missing = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    out = (ints(0, 3), ints(0), ints(0, 2), missing)
    assert binding.kv_fork(ints(0), ints(0), cache, batch, out=out) is out and missing.tolist() == [0]


def test_behind_what_the_stream_of_the_call_has():
    """Another value that the stream is still to write comes first, whatever the current stream is at."""
    cache, batch, ints = parts()
    out = (ints(0, 3), ints(0), ints(0, 2), torch.zeros(1, dtype=torch.int32, device=DEV))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                # (a bounded wait on the GPU)
        out[3].fill_(9)
    binding.kv_fork(ints(0), ints(0), cache, batch, out=out, stream=side)
    torch.cuda.synchronize()
    assert out[3].tolist() == [0]


def test_before_what_comes_on_the_stream_of_the_call():
    """A new output is there for that stream, while the current one is busy."""
    cache, batch, ints = parts()
    side, busy = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(100_000_000)
        missing = binding.kv_fork(ints(0), ints(0), cache, batch, stream=side)[3]
    with torch.cuda.stream(side):
        got = missing.clone()
    side.synchronize()
    assert got.tolist() == [0]
    torch.cuda.synchronize()


def test_captured():
    cache, batch, ints = parts()
    out = (ints(0, 3), ints(0), ints(0, 2), torch.full((1,), 9, dtype=torch.int32, device=DEV))
    none = ints(0)
    binding.kv_fork(none, none, cache, batch, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.kv_fork(none, none, cache, batch, out=out)
    for _ in range(3):
        out[3].fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert out[3].tolist() == [0]
