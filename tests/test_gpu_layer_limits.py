"""The operators between a decoder layer's linears at the limits of their arguments, on the GPU."""
import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from tests.test_gpu_layer import bf16

pytestmark = pytest.mark.gpu


def test_rope_output_beside_its_input():
    """q may take columns of the same buffer beside qkv, not columns of qkv."""
    rng = np.random.default_rng(80)
    T, H, n_kv, D = 5, 4, 2, 64
    width = (H + 2 * n_kv) * D
    buf = bf16(rng.normal(size=(T, width + H * D + 16))).cuda()
    qkv = buf[:, 8:8 + width]
    table = torch.arange(T, dtype=torch.int32, device="cuda")[:, None]
    n = torch.full((T,), 7, dtype=torch.int32, device="cuda")
    f = w4.w4_rope_frequencies(D)[0].cuda()

    def run(out):
        k, v = (torch.zeros(T, 16, n_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return w4.w4_rope_append(qkv, H, k, v, table, n, f, out=out)
    want = run(None)
    out = buf[:, 8 + width:8 + width + H * D]
    assert torch.equal(run(out), want) and torch.equal(out, want)
    before = buf.clone()
    for bad in (qkv[:, :H * D], buf[:, 8 + width - 8:][:, :H * D], buf[:, :H * D]):
        with pytest.raises(w4.W4Error, match="status 2"):
            run(bad)
    assert torch.equal(buf, before)


def test_norm_of_more_rows_than_a_launch_has():
    """2^23 rows of 2049 (512 threads each) pass 2^32 threads: rows on both sides of where the
    launches part, as they come out of a small call."""
    T, d = (1 << 23) + 5, 2049
    rng = np.random.default_rng(81)
    at = torch.tensor([0, 1, (1 << 23) - 3, (1 << 23) - 2, (1 << 23) - 1, 1 << 23, T - 1])
    x, r, gate, y = (torch.empty((T, d), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    small = [bf16(rng.normal(size=(len(at), d))).cuda() for _ in range(3)]
    for big, rows in zip((x, r, gate), small):
        big[at.cuda()] = rows
    w = bf16(1 + 0.2 * rng.normal(size=d)).cuda()
    want = w4.w4_residual_norm(small[0], small[1], w, w_post=w, gate=small[2])
    w4.w4_residual_norm(x, r, w, w_post=w, gate=gate, out=y, residual_out=r)
    assert torch.equal(y[at.cuda()], want[0]) and torch.equal(r[at.cuda()], want[1])
    del x, r, gate, y
    torch.cuda.empty_cache()


def test_rope_of_the_most_rows():
    """T = 2^24 with heads wide enough for 256 threads a token."""
    T, H, n_kv, D, page = 1 << 24, 6, 1, 256, 32768
    rng = np.random.default_rng(82)
    width = (H + 2 * n_kv) * D
    qkv = torch.empty((T, width), dtype=torch.bfloat16, device="cuda")
    rows = bf16(rng.normal(size=(2, width))).cuda()
    qkv[0], qkv[-1] = rows[0], rows[1]
    table = torch.full((1, T // page), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, -1] = 1, 0
    f = w4.w4_rope_frequencies(D)[0].cuda()

    def run(x, n, starts):
        k, v = (torch.zeros(2, page, n_kv, D, dtype=torch.bfloat16, device="cuda")
                for _ in range(2))
        n, starts = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in (n, starts))
        return w4.w4_rope_append(x, H, k, v, table, n, f, q_start=starts), k, v
    q, k, v = run(qkv, [T], [0, T])
    for i, (row, n, page_at, slot) in enumerate(((0, 1, 1, 0), (-1, T, 0, page - 1))):
        q1, k1, v1 = run(rows[i:i + 1], [n], [0, 1])
        assert torch.equal(q[row], q1[0])
        assert torch.equal(k[page_at, slot], k1[page_at, slot])
        assert torch.equal(v[page_at, slot], v1[page_at, slot])
    del qkv, q
    torch.cuda.empty_cache()
