"""Embedding, block norms, MLP, head and log probabilities as a training step runs them, with the way back.

Each stage's result is compared with the 64-bit formula of what that stage was
given, so a stage's bound is that of its own roundings: an output in bf16 is off
by half a step (2^-8 of its value, 2^-9 of the norm of many values on average, so
2^-8 bounds the norm), and what precedes it by fp32 sums (2^-24 times a few
hundred).
"""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from heads_helpers import draw, ints, whole
from oracle import decoder

pytestmark = pytest.mark.gpu
R, S0, S1, PART = tsl.Replicate(), tsl.Shard(0), tsl.Shard(1), tsl.Partial()
T, N, F, V, P = 96, 256, 512, 1000, 4
BF = torch.bfloat16


def dist(a, mesh, pl, dtype=BF):
    return tsl.DTensor.distribute_tensor(torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype), mesh, [pl])


def host(d, dim):
    return np.concatenate([s.double().cpu().numpy() for s in d.slots], dim)


def near(got, want, tol=2.0 ** -8):
    assert np.linalg.norm(got - want) <= tol * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)


class Step:
    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.mesh = mesh = tsl.DeviceMesh((P,), ("tp",))
        d = lambda *s, scale=1.0: draw(rng, s, "bf16", scale)  # noqa: E731
        self.table, self.w = d(V, N), [d(N, F, scale=N ** -0.5), d(N, F, scale=N ** -0.5), d(F, N, scale=F ** -0.5)]
        self.head = d(N, V, scale=2 * N ** -0.5)
        self.g1, self.post, self.g2 = (1 + draw(rng, (N,), "fp32", 0.1) for _ in range(3))
        self.g1, self.post, self.g2 = (v.astype(np.float32).astype(np.float64) for v in (self.g1, self.post, self.g2))
        self.ids, self.next = rng.integers(0, V, (T,)), rng.integers(0, V, (T,))
        self.next[5] = -100
        self.seed = rng.integers(-2 ** 31, 2 ** 31, 4)
        self.d_table = dist(self.table, mesh, S1)
        self.d_w = [dist(self.w[0], mesh, S1), dist(self.w[1], mesh, S1), dist(self.w[2], mesh, S0)]
        self.d_head = dist(self.head, mesh, S1)
        self.d_g = [whole(v, mesh, torch.float32) for v in (self.g1, self.post, self.g2)]
        self.d_ids, self.d_next, self.d_seed = ints(self.ids, mesh), ints(self.next, mesh), ints(self.seed, mesh)
        self.d_dlp = whole(np.full((T,), -1.0 / T), mesh, torch.float32)

    def run(self):
        g1, post, g2 = self.d_g
        x0 = tsl.tp_embedding(self.d_ids, self.d_table)
        _, y0 = tsl.tp_block_norm(x0, pre_weight=g1, out=(None, tsl.DTensor.empty(self.mesh, [R], (T, N), BF)))
        m = tsl.tp_mlp(y0, *self.d_w, mode=tsl.PARTIAL)
        kw = dict(dropout=0.25, rng=self.d_seed, residual_scale=0.5)
        res = x0.redistribute([S0])
        h, y1 = tsl.tp_block_norm(m, res, post, None, g2, **kw)
        z = tsl.column_parallel_linear(y1, self.d_head, out_dtype=torch.float32)
        r = tsl.tp_log_probs(z, self.d_next, top=3, entropy=True)
        dz = tsl.tp_log_probs_backward(self.d_dlp, None, z, self.d_next, r.lse)
        dzb = tsl.DTensor([s.to(BF) for s in dz.slots], self.mesh, [S1], (T, V), BF)
        back = tsl.DTensor([s.t() for s in self.d_head.slots], self.mesh, [S0], (V, N), BF)
        dy1 = tsl.row_parallel_linear(dzb, back, mode=tsl.REDUCE_SCATTER)
        grads = tsl.tp_block_norm_backward(None, dy1, m, res, post, None, g2, **kw)
        return x0, y0, m, h, y1, z, r, dz, dzb, dy1, grads


def check(s, out):
    x0, y0, m, h, y1, z, r, dz, dzb, dy1, (dx, dr, dpost, dgate, dpre) = out
    hx0, parts = host(x0, 0), [t.double().cpu().numpy() for t in m.slots]
    assert np.array_equal(hx0, s.table[s.ids])
    near(host(y0, 0), decoder.Block([hx0], pre=s.g1).y)
    b = decoder.Block(parts, hx0, s.post, None, s.g2, scale=0.5, keep=decoder.keep_mask(s.seed, T, N, 0.25), p=0.25)
    near(host(h, 0), b.h)
    near(host(y1, 0), b.y)
    near(host(z, 1), host(y1, 0) @ s.head, 2.0 ** -16)
    hz, there = host(z, 1), s.next >= 0
    logp, lse, ent = decoder.log_probs(hz)
    want = np.where(there, logp[np.arange(T), np.maximum(s.next, 0)], 0.0)
    for got, e in ((r.logprobs, want), (r.lse, lse), (r.entropy, ent)):
        near(host(got, 0), e, 2.0 ** -18)
    assert np.array_equal(r.top_ids.slots[0].cpu().numpy(), decoder.top(hz, 3))
    near(host(dz, 1), decoder.log_probs_backward(hz, s.next[:, None], np.full((T, 1), -1.0 / T), lse)[0], 2.0 ** -16)
    near(host(dy1, 0), host(dzb, 1) @ s.head.T)
    e = b.backward(None, host(dy1, 0))
    near(host(dx, 0), e["dx"][0])
    near(host(dr, 0), e["dr"][0])
    near(host(dpost, 0), e["dpost"][0], 2.0 ** -16)
    near(host(dpre, 0), e["dpre"][0], 2.0 ** -16)
    assert dgate is None and h.placements == (S0,) and dx.placements == (R,) and dr.placements == (S0,)


def test_training_step():
    s = Step(1)
    out = s.run()
    check(s, out)
    assert tsl.read_device_status() == 0


def test_training_step_captured():
    s = Step(2)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = s.run()
    new = Step(3)
    for name in ("d_table", "d_head"):
        for a, b in zip(getattr(s, name).slots, getattr(new, name).slots):
            a.copy_(b)
    for name in ("d_ids", "d_next", "d_seed"):
        getattr(s, name).slots[0].copy_(getattr(new, name).slots[0])
    s.table, s.head, s.ids, s.next, s.seed = new.table, new.head, new.ids, new.next, new.seed
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    check(s, out)


@pytest.mark.parametrize("place", [R, S0, PART])
def test_head_log_probs_is_its_parts(place):
    s = Step(4)
    rng = np.random.default_rng(5)
    x = [draw(rng, (T, N), "bf16") for _ in range(P)]
    xd = tsl.DTensor([torch.from_numpy(v).cuda().to(BF) for v in x], s.mesh, [PART], (T, N), BF)
    if place != PART:
        xd = xd.redistribute([place])
    res = dist(draw(rng, (T, N), "bf16"), s.mesh, S0)
    kw = dict(top=4, entropy=True, logits_dtype=torch.float32)
    r = tsl.tp_head_log_probs(xd, s.d_head, s.d_next, residual=res, post_weight=s.d_g[1], pre_weight=s.d_g[2], scale=0.8,
                              **kw)
    _, y = tsl.tp_block_norm(xd, res, s.d_g[1], None, s.d_g[2])
    z = tsl.column_parallel_linear(y, s.d_head, out_dtype=torch.float32)
    want = tsl.tp_log_probs(z, s.d_next, scale=0.8, top=4, entropy=True)
    assert all(torch.equal(a.slots[0], b.slots[0]) for a, b in zip(r, want))
    if place == R:
        r = tsl.tp_head_log_probs(xd, s.d_head, **kw)
        want = tsl.tp_log_probs(tsl.column_parallel_linear(xd, s.d_head, out_dtype=torch.float32), top=4, entropy=True)
        assert r.logprobs is None and all(torch.equal(a.slots[0], b.slots[0]) for a, b in zip(r[1:], want[1:]))
