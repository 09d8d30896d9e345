"""First calls of the attention over the 4-bit cache from many host threads at once."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys, threading, numpy as np, torch
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import tensor_sharded_linear_gb300 as tsl
from heads_helpers import Batch, draw, sharded
mesh = tsl.DeviceMesh((1,), ("tp",))
cases = []
for d, group, n, dtype in ((64, 32, 1, "bf16"), (64, 64, 80, "bf16"), (128, 64, 1, "bf16"), (128, 32, 12, "bf16"),
                           (128, 64, 90, "bf16"), (256, 64, 70, "bf16"), (256, 32, 1, "fp32"), (128, 64, 3, "fp32")):
    rng = np.random.default_rng(92)
    b = Batch(rng, mesh, [n, n], [200, 90], 1, d, group, 16)
    cases.append((d, group, sharded(draw(rng, (2 * n, 2 * d), dtype), mesh, dtype), b.cache(), b.operands()))
torch.cuda.synchronize()
got, start = [[None] * len(cases) for _ in range(8)], threading.Barrier(8)

def work(me):
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        for i in range(len(cases)):
            j = (i + me) % len(cases)
            d, group, q, cache, (pt, kl, qs) = cases[j]
            got[me][j] = tsl.tp_kv4_attention(q, cache, pt, kl, qs, head_dim=d, group=group)

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert tsl.read_device_status() == 0
for j, (d, group, q, cache, (pt, kl, qs)) in enumerate(cases):
    want = tsl.tp_kv4_attention(q, cache, pt, kl, qs, head_dim=d, group=group).slots[0]
    assert torch.isfinite(want).all()
    for me in range(8):
        assert torch.equal(got[me][j].slots[0], want), (me, j)
print("OK")
"""


@pytest.mark.gpu
def test_first_calls_from_many_threads(lib):
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))],
                       capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout + r.stderr


def test_what_calls_keep_by_device_is_atomic():
    """Per-device tables in the library's host code are read and written by whichever thread calls."""
    csrc = os.path.join(ROOT, "tensor_sharded_linear_gb300", "csrc")
    seen = 0
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            for kind in re.findall(r"^\s*static ([\w:<>* ]+?) ?\w+\[64\]", f.read(), re.M):
                seen += 1
                assert kind.startswith("std::atomic<"), (name, kind)
    assert seen >= 4
