"""The decoder example: prompts and single tokens through int4 linears, the cache and the norms,
against a plain implementation in 64 bits on the dequantized weights."""
import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from examples import decoder
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

SHAPE = decoder.Shape(layers=2, hidden=256, heads=6, kv_heads=2, head_dim=64, inter=320,
                      group_size=128, page_size=16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def dequantized(linear):
    qweight, scales, _, _, d_in, group = linear
    b = qweight.cpu().numpy()
    code = np.stack([b & 15, b >> 4], axis=2).reshape(b.shape[0], -1)[:, :d_in]
    return (code.astype(np.float64) - 8) * np.repeat(f64(scales), group, axis=1)[:, :d_in]


def plain(model, x):
    """The whole of one sequence, x [n][hidden], every token over the tokens before it."""
    s = model.shape
    h, n = f64(x), x.shape[0]
    freq = f64(model.inv_freq)
    table = np.arange(n)[None]
    for layer in model.layers:
        y = ref.rms(h, f64(layer["norm_in"]), 1e-6, 0.0)
        qkv = (y @ dequantized(layer["qkv"]).T).reshape(n, -1, s.head_dim)
        c, sn = np.cos(np.outer(np.arange(n), freq)), np.sin(np.outer(np.arange(n), freq))
        c, sn = c[:, None], sn[:, None]
        qk, v = qkv[:, :s.heads + s.kv_heads], qkv[:, s.heads + s.kv_heads:]
        a, b = np.split(qk, 2, axis=2)
        qk = np.concatenate([a * c - b * sn, a * sn + b * c], axis=2)
        q, k = qk[:, :s.heads].reshape(n, -1), qk[:, s.heads:]
        att = ref.attention(q, k[:, None], v[:, None], table, [n], [0, n], s.heads,
                            s.head_dim ** -0.5, s.window, s.sinks)[0]
        h = h + att.reshape(n, -1) @ dequantized(layer["o"]).T
        y = ref.rms(h, f64(layer["norm_mlp"]), 1e-6, 0.0)
        gate, up = np.split(y @ dequantized(layer["gate_up"]).T, 2, axis=1)
        h = h + (gate / (1 + np.exp(-gate)) * up) @ dequantized(layer["down"]).T
    return ref.rms(h, f64(model.norm_out), 1e-6, 0.0)


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_prompts_then_steps(window, sinks):
    """A batch of prompts in one pass, then three tokens each, equals each whole sequence's pass.

    The bound is on the norm of a row's error over the norm of the row: 14 roundings to bf16 a layer
    (input norm, qkv, rope, weights, attention, o, norm, gate, up, silu, product, down, and the
    residual's two inputs again in the next norm), each at most 2^-8 of what it rounds, and one more
    at the end; worst cases added up."""
    shape = decoder.Shape(**{**SHAPE.__dict__, "window": window, "sinks": sinks})
    model = decoder.Decoder(shape, seed=3)
    lens, steps = [1, 70, 33], 3
    rng = np.random.default_rng(5)
    # small inputs: the blocks' outputs, not the input, make up most of the residual
    seqs = [torch.from_numpy(0.05 * rng.standard_normal((n + steps, shape.hidden))).float()
            .bfloat16().cuda() for n in lens]
    cache = decoder.Cache(shape, [n + steps for n in lens], "cuda")
    y = model.prompts(torch.cat([x[:n] for x, n in zip(seqs, lens)]), lens, cache)
    got = [list(f64(part)) for part in y.split(lens)]
    for i in range(steps):
        y = model.step(torch.stack([x[n + i] for x, n in zip(seqs, lens)]), cache)
        for rows, row in zip(got, f64(y)):
            rows.append(row)
    bound = (14 * shape.layers + 1) * ref.BF16
    for x, rows in zip(seqs, got):
        want = plain(model, x)
        err = np.linalg.norm(np.array(rows) - want, axis=1) / np.linalg.norm(want, axis=1)
        assert err.max() <= bound, (err.max(), bound, int(err.argmax()))


def test_command(capsys):
    decoder.main(["--layers", "1", "--prompts", "5,130", "--steps", "4", "--window", "64"])
    out = capsys.readouterr().out
    assert "135 prompt tokens" in out and "2 sequences, 4 steps" in out
