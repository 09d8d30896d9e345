"""The attention over the 4-bit cache against the error of its own arithmetic: the bound shrinks with the result, so
long sequences, their split and their join are held as closely as short ones."""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl

from attention_close import check
from heads_helpers import Batch, draw, full, sharded

pytestmark = pytest.mark.gpu


def run(seed, q_lens, kv_lens, hq, hk, d, group, dtype, causal=True, window=0, many=False, page=16, p=1, scale=None):
    rng, mesh = np.random.default_rng(seed), tsl.DeviceMesh((p,), ("tp",))
    b = Batch(rng, mesh, q_lens, kv_lens, hk, d, group, page)
    q = draw(rng, (b.tokens, hq * d), dtype)
    lse = tsl.DTensor.empty(mesh, [tsl.Shard(1)], (b.tokens, hq), torch.float32)
    pt, kl, qs = b.operands()
    y = full(tsl.tp_kv4_attention(sharded(q, mesh, dtype), b.cache(), pt, kl, qs, head_dim=d, group=group, causal=causal,
                                  window=window, lse=lse, scale=scale)).reshape(b.tokens, hq, d)
    assert tsl.read_device_status() == 0
    at, logs = 0, full(lse)
    for s, n in enumerate(q_lens):
        check(y[at:at + n], logs[at:at + n], q[at:at + n].reshape(n, hq, d), b.kv[s], d, group, hq,
              d ** -0.5 if scale is None else scale, dtype, causal, window, many)
        at += n


FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,group", FORMATS)
def test_few_rows(lib, d, group, dtype):
    run(100, [1, 1, 3, 2, 1], [1, 37, 1000, 130, 5000], 4, 2, d, group, dtype, p=2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_long_sequence(lib, d, dtype):
    """Split over all CTAs and joined from tens of pieces."""
    run(101, [1, 2], [40000, 3], 2, 1, d, 64, dtype)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_drafts(lib, d):
    run(102, [11, 16], [9000, 20], 2, 1, d, 64, "bf16")


@pytest.mark.parametrize("d,group", FORMATS)
def test_prompts(lib, d, group):
    run(103, [70, 64, 65], [400, 64, 300], 2, 1, d, group, "bf16", many=True)


@pytest.mark.parametrize("d,group", [(64, 64), (128, 64), (256, 64)])
def test_prompts_split_over_ctas(lib, d, group):
    """One row block on a long context: every CTA holds a piece, and joins of two and of many."""
    run(104, [64], [12000], 1, 1, d, group, "bf16", many=True)
    run(105, [200, 64, 64], [1500, 2500, 700], 1, 1, d, group, "bf16", many=True)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 700), (True, 64)])
def test_masks(lib, causal, window):
    run(106, [1, 3], [3000, 900], 4, 2, 128, 64, "bf16", causal, window, p=2)
    run(107, [80], [2000], 1, 1, 128, 64, "bf16", causal, window, many=True)


@pytest.mark.parametrize("scale", [0.01, 0.5])
def test_scales(lib, scale):
    """All but equal weights, and a few keys that take most."""
    run(108, [1, 2], [3000, 900], 2, 1, 128, 64, "bf16", scale=scale)
    run(109, [70], [1500], 1, 1, 128, 64, "bf16", many=True, scale=scale)
