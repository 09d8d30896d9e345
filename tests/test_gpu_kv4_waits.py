"""The waits of the attention kernels over the 4-bit cache: behind other kernels."""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl

from heads_helpers import Batch, draw, sharded

pytestmark = pytest.mark.gpu
MESH1 = tsl.DeviceMesh((1,), ("tp",))


def test_prompts_behind_kernels_that_hold_tensor_memory(lib):
    """Linears, library products and prompts in turn, nothing synchronised between them: the results of each alone."""
    rng = np.random.default_rng(90)
    b = Batch(rng, MESH1, [300, 80], [300, 900], 2, 128, 64, 16)
    q = sharded(draw(rng, (380, 8 * 128), "bf16"), MESH1, "bf16")
    x = tsl.DTensor(q.slots, MESH1, [tsl.Replicate()], (380, 1024), torch.bfloat16)
    w = sharded(draw(rng, (1024, 1024), "bf16", 1 / 32), MESH1, "bf16")
    cache, (pt, kl, qs) = b.cache(), b.operands()
    want = tsl.tp_kv4_attention(q, cache, pt, kl, qs, head_dim=128).slots[0]
    torch.cuda.synchronize()
    y = tsl.column_parallel_linear(x, w)
    z = q.slots[0] @ w.slots[0]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append(tsl.column_parallel_linear(x, w).slots[0])
        got.append(tsl.tp_kv4_attention(q, cache, pt, kl, qs, head_dim=128).slots[0])
        got.append(q.slots[0] @ w.slots[0])
        got.append(tsl.tp_kv4_attention(q, cache, pt, kl, qs, head_dim=128).slots[0])
    torch.cuda.synchronize()
    assert tsl.read_device_status() == 0
    for i, r in enumerate(got):
        assert torch.equal(r, (y.slots[0], want, z, want)[i % 4]), i
