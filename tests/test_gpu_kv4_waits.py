"""The waits of the attention kernels over the 4-bit cache: behind other kernels, and for copies that do not come.

The second kind makes the waits run out without a fault: DT_KV4_STARVE=n lets the barriers of each CTA's n-th step
(each warp's n-th tile, with few rows) and of those after it await more bytes than are copied (the copies themselves are those of any call), and
DT_KV4_WAIT_LIMIT_MS shortens the limit.  The kernel has to report DT_DEV_ERR_TIMEOUT and to end, and the context has
to be usable after it.  A process each, since the hooks are read once."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl

from heads_helpers import Batch, draw, sharded

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


CHILD = r"""
import sys, numpy as np, torch
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import tensor_sharded_linear_gb300 as tsl
from tensor_sharded_linear_gb300 import _lib as L
from oracle import heads
from heads_helpers import Batch, cache_bits, draw, full, ints, sharded
mesh = tsl.DeviceMesh((1,), ("tp",))
for d, group, n, kv in {cases!r}:
    rng = np.random.default_rng(91)
    b = Batch(rng, mesh, [n, n], [kv, kv // 2], 2, d, group, 16)
    q = sharded(draw(rng, (2 * n, 4 * d), {dtype!r}), mesh, {dtype!r})
    cache, (pt, kl, qs) = b.cache(), b.operands()
    for _ in range(3):
        tsl.read_device_status(clear=True)
        tsl.tp_kv4_attention(q, cache, pt, kl, qs, head_dim=d, group=group)
        status = tsl.read_device_status(clear=True)
        assert status == L.DEV_ERR_TIMEOUT, (d, status)
    # the context still works: an append, bit for bit, and a library product
    k = draw(rng, (2, 2 * d), "bf16")
    tsl.tp_kv4_append(sharded(k, mesh, "bf16"), sharded(k, mesh, "bf16"), cache, pt, kl, ints([0, 1, 2], mesh), head_dim=d,
                      group=group)
    assert tsl.read_device_status(clear=True) == 0
    bits = cache_bits(cache)
    want = heads.pack(np.float32(k.reshape(2, 2, d)), np.float32(k.reshape(2, 2, d)), group)
    for s, m in enumerate(b.kv_lens):
        assert (bits[b.table[s, (m - 1) // 16], :, (m - 1) % 16] == want[s]).all()
    x = torch.ones(256, 256, device="cuda", dtype=torch.bfloat16)
    assert ((x @ x) == 256).all()
print("OK")
"""


def starved(cases, dtype, step):
    env = dict(os.environ, DT_KV4_STARVE=str(step), DT_KV4_WAIT_LIMIT_MS="30")
    code = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), cases=cases, dtype=dtype)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("step", [1, 2, 5])
def test_prompt_waits_run_out_and_report(lib, step):
    starved([(64, 32, 300, 6000), (128, 64, 300, 6000), (256, 64, 200, 6000)], "bf16", step)


@pytest.mark.parametrize("step,dtype", [(1, "bf16"), (2, "bf16"), (3, "fp32")])
def test_waits_of_few_rows_run_out_and_report(lib, step, dtype):
    starved([(64, 32, 1, 90000), (128, 64, 7, 60000), (256, 64, 2, 60000)], dtype, step)
