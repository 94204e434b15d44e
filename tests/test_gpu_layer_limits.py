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
