"""The decoder example after a shared system prompt: pages given out on the GPU, attention over the shared
keys, sequences that end and begin; against a plain implementation in 64 bits of each whole sequence."""
import numpy as np
import pytest
import torch

from examples import decoder
from tests import layer_reference as ref
from tests.test_decoder_example import SHAPE, f64, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_sequences_after_a_system_prompt(window, sinks):
    """Prompts and single tokens after 37 shared ones (two pages of 16 and 5 tokens of a third); the
    first sequence ends and another takes its place and its pages. The bound is that of
    test_prompts_then_steps, plus one rounding a layer: partial results of shared and own keys."""
    shape = decoder.Shape(**{**SHAPE.__dict__, "window": window, "sinks": sinks})
    model = decoder.Decoder(shape, seed=3)
    rng = np.random.default_rng(6)

    def tokens(n):
        return torch.from_numpy(0.05 * rng.standard_normal((n, shape.hidden))).float().bfloat16().cuda()

    P, plans = 37, [[30, 1, 1], [1, 1, 1, 1, 1], [70, 1, 1, 1, 1]]
    late = [[12, 1]]  # after the first has ended
    system, seqs = tokens(P), [tokens(sum(p)) for p in plans + late]
    pages = 3 + 3 + 1 + 6
    cache = decoder.SharedCache(shape, 3, pages, P + 80, "cuda")

    def run(counts, rows):
        n_new = torch.tensor(counts, dtype=torch.int32, device="cuda")
        return f64(model.shared_pass(torch.cat(rows), n_new, cache))

    run([0, 0, 0, P], [system])
    for b in range(3):
        cache.share(b)
    got, at = [[] for _ in seqs], [0] * len(seqs)
    owner = [0, 1, 2]
    for i in range(5):
        if i == 3:  # the first ends
            cache.advance(torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device="cuda"), 0)
            cache.share(0)
            owner[0] = 3
        counts = [(plans + late)[s][i if s < 3 else i - 3] for s in owner]
        y = run(counts + [0], [seqs[s][at[s]:at[s] + n] for s, n in zip(owner, counts)])
        for s, part in zip(owner, np.split(y, np.cumsum(counts)[:-1])):
            got[s] += list(part)
            at[s] += len(part)
    used = -(-(37 % 16 + 13) // 16) + -(-(37 % 16 + 5) // 16) + -(-(37 % 16 + 74) // 16) + 3
    assert cache.state.tolist()[1:] == [pages - used, 0]
    bound = (15 * shape.layers + 1) * ref.BF16
    for x, rows in zip(seqs, got):
        want = plain(model, torch.cat([system, x]))[P:]
        err = np.linalg.norm(np.array(rows) - want, axis=1) / np.linalg.norm(want, axis=1)
        assert err.max() <= bound, (err.max(), bound, int(err.argmax()))


def test_command(capsys):
    decoder.main(["--layers", "1", "--prompts", "5,130", "--steps", "4", "--system", "100"])
    out = capsys.readouterr().out
    assert "135 prompt tokens" in out and "2 sequences, 4 steps" in out
