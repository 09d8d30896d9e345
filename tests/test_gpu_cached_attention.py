"""The attention block over the paged 4-bit cache: a prompt of ragged sequences, then decode steps, against the
whole chain in fp64.

Tolerance.  The chain rounds to bf16 after each operator, which is 2^-9 of a value at most.  What that moves most
are the codes: a key or value that moves by d changes its code with a probability of d over the step, and then by
a step.  A step is about a third of the values' deviation (5 deviations over 15), d about 2^-9 of it, twice
rounded: 2 / 512 / 0.33 = 1.2% of the codes, so sqrt(0.012) * 0.33 = 3.6% of the values' deviation in the mean
square.  Keys reach the result through logits of norm sqrt(d) * deviation / sqrt(d) ~ 1, values directly, and both
average over the same keys as the result does: sqrt(2) * 3.6% = 5% of the result's norm.  The bound is twice that;
a wrong head, position, page or sequence is off by the norm itself."""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from oracle import heads

from heads_helpers import draw, full, ints, sharded, table, whole

pytestmark = pytest.mark.gpu
RELATIVE = 0.10


class Block:
    """Weights, cache and page table of one layer, and the same in fp64."""

    def __init__(self, rng, p, hidden, hq, hk, d, page, batch, longest, norm):
        self.mesh = tsl.DeviceMesh((p,), ("tp",))
        self.hq, self.hk, self.d, self.norm = hq, hk, d, norm
        self.w = {n: draw(rng, (hidden, h * d), "bf16", hidden ** -0.5) for n, h in (("q", hq), ("k", hk), ("v", hk))}
        self.wo = draw(rng, (hq * d, hidden), "bf16", (hq * d) ** -0.5)
        self.qw, self.kw = (draw(rng, (d,), "bf16", 0.2) + 1 for _ in "qk") if norm else (None, None)
        self.cs = table(longest, d)
        width = -(-longest // page)
        self.pt = rng.permutation(batch * width).reshape(batch, width)
        self.cache = tsl.kv4_cache(self.mesh, batch * width, hk, page, head_dim=d, device="cuda")
        for s in self.cache.slots:
            s.fill_(-1)  # NaN parameters
        c = hq * d // p
        self.args = [sharded(self.w[n], self.mesh, "bf16") for n in "qkv"] + [
            tsl.DTensor([torch.from_numpy(self.wo[i * c:(i + 1) * c]).cuda().bfloat16() for i in range(p)], self.mesh,
                        [tsl.Shard(0)], self.wo.shape, torch.bfloat16), self.cache, ints(self.pt, self.mesh)]
        self.kwargs = dict(head_dim=d, cos_sin=whole(self.cs, self.mesh), out_dtype=torch.float32)
        if norm:
            self.kwargs.update(q_weight=whole(self.qw, self.mesh, torch.bfloat16),
                               k_weight=whole(self.kw, self.mesh, torch.bfloat16))
        self.k = [np.zeros((0, hk, d)) for _ in range(batch)]  # what the cache holds
        self.v = [np.zeros((0, hk, d)) for _ in range(batch)]

    def step(self, x, lens, in_norm, ragged):
        """Device result and fp64 result for the new tokens x of the sequences."""
        kv = [len(k) + n for k, n in zip(self.k, lens)]
        pos = np.concatenate([np.arange(t - n, t) for t, n in zip(kv, lens)])
        starts = np.concatenate([[0], np.cumsum(lens)])
        y = tsl.tp_cached_attention(whole(x, self.mesh, torch.bfloat16), *self.args, ints(kv, self.mesh),
                                    ints(starts, self.mesh) if ragged else None,
                                    positions=ints(pos, self.mesh) if in_norm else None, **self.kwargs)
        q, k, v = ((x @ self.w[n]).reshape(len(x), -1, self.d) for n in "qkv")
        q, k = heads.norm_rope(q, self.qw, self.cs, pos, False, 1e-6), heads.norm_rope(k, self.kw, self.cs, pos, False,
                                                                                      1e-6)
        ks, vs, _, _ = heads.unpack(heads.pack(k.astype(np.float32), v.astype(np.float32), 64), self.d, 64)
        a, g = np.zeros_like(q), self.hq // self.hk
        for b, n in enumerate(lens):
            rows = slice(starts[b], starts[b + 1])
            self.k[b], self.v[b] = np.concatenate([self.k[b], ks[rows]]), np.concatenate([self.v[b], vs[rows]])
            for h in range(self.hq):
                a[rows, h] = heads.attention(q[rows, h], self.k[b][:, h // g], self.v[b][:, h // g], self.d ** -0.5,
                                             True, 0)[0]
        return full(y), a.reshape(len(x), -1) @ self.wo


@pytest.mark.parametrize("p,hq,hk,d,norm,in_norm", [(4, 8, 4, 64, True, True), (2, 8, 2, 128, True, False),
                                                    (1, 4, 4, 64, False, False), (2, 4, 2, 256, False, True)])
def test_prompt_then_decode(p, hq, hk, d, norm, in_norm):
    rng = np.random.default_rng(100 + d + p)
    blk = Block(rng, p, 256, hq, hk, d, 16, 3, 96, norm)
    for lens in ([70, 1, 33], [1, 1, 1], [1, 1, 1], [2, 0, 5]):
        x = draw(rng, (sum(lens), 256), "bf16")
        got, want = blk.step(x, lens, in_norm, ragged=len(set(lens)) > 1)
        assert np.linalg.norm(got - want) <= RELATIVE * np.linalg.norm(want), lens
        for b in range(3):  # each sequence by itself
            r = slice(sum(lens[:b]), sum(lens[:b + 1]))
            assert np.linalg.norm(got[r] - want[r]) <= 2 * RELATIVE * np.linalg.norm(want[r]), (lens, b)
    assert tsl.read_device_status() == 0


def test_a_captured_step_replays_with_new_tokens():
    """One decode step as a graph: x, lengths and positions are written in place between replays; the results are
    those of plain calls on a second cache, bit for bit."""
    rng = np.random.default_rng(5)
    a = Block(rng, 2, 256, 8, 2, 64, 16, 2, 64, True)
    b = Block(np.random.default_rng(5), 2, 256, 8, 2, 64, 16, 2, 64, True)
    x = whole(np.zeros((2, 256)), a.mesh, torch.bfloat16)
    lens, pos = ints([1, 1], a.mesh), ints([0, 0], a.mesh)
    out = whole(np.zeros((2, 256), dtype=np.float32), a.mesh)

    def step(blk, x, lens, pos, out):
        return tsl.tp_cached_attention(x, *blk.args, lens, positions=pos, out=out, **blk.kwargs)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # (its record is overwritten by the first replay)
        step(a, x, lens, pos, out)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(a, x, lens, pos, out)
    for n in range(1, 20):
        xs = torch.from_numpy(draw(rng, (2, 256), "bf16")).cuda().bfloat16()
        x.slots[0].copy_(xs)
        lens.slots[0].fill_(n)
        pos.slots[0].fill_(n - 1)
        graph.replay()
        want = step(b, whole(xs, b.mesh), ints([n, n], b.mesh), ints([n - 1, n - 1], b.mesh), None)
        torch.cuda.synchronize()
        assert torch.equal(out.slots[0], want.slots[0]), n
        for s, t in zip(a.cache.slots, b.cache.slots):
            assert torch.equal(s, t), n
    assert tsl.read_device_status() == 0
