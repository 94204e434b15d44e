"""The decoder example after a shared system prompt, from a pool that runs dry."""
import pytest
import torch

from examples import decoder
from tests.test_decoder_example import SHAPE

pytestmark = pytest.mark.gpu


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("replayed", [False, True])
def test_a_pool_that_runs_dry_is_noticed(replayed):
    """4 pages of 16: two for 20 shared tokens, one for each of two sequences, which both need another
    after 12 tokens. Noticed also once pages are free again."""
    model = decoder.Decoder(SHAPE, seed=4)
    cache = decoder.SharedCache(SHAPE, 2, 4, 64, "cuda")

    def tokens(n):
        return 0.05 * torch.randn(n, SHAPE.hidden, device="cuda").bfloat16()
    model.shared_pass(tokens(20), ints(0, 0, 20), cache)
    for b in range(2):
        cache.share(b)
    x, one = tokens(2), ints(1, 1, 0)

    def step():
        return model.shared_pass(x, one, cache)
    steps = 0
    if replayed:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            step()
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        torch.cuda.default_stream().wait_stream(side)
        steps, step = 1, graph.replay
    for _ in range(12 - steps):  # up to the end of the page that each has: 20 + 12 = 32
        step()
        cache.check()
    step()
    with pytest.raises(RuntimeError, match="too small"):
        cache.check()
    cache.advance(ints(-1, 0, 0), 0)
    assert cache.state.tolist()[1:] == [1, 1]
    one.copy_(ints(0, 1, 0))
    cache.advance(one, 1)
    assert cache.state.tolist()[1:] == [0, 0]
    with pytest.raises(RuntimeError, match="too small"):
        cache.check()
