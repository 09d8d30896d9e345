"""Distributed tensors and batches for the tests of the operators on attention heads."""
import numpy as np
import torch

import tensor_sharded_linear_gb300 as tsl
from oracle import bf16, heads

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def table(rows, rotary, theta=10000.0):
    a = np.arange(rows)[:, None] * theta ** (-np.arange(0, rotary, 2) / rotary)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def draw(rng, shape, dtype, scale=1.0):
    """fp64 values that are exact in dtype."""
    x = rng.standard_normal(shape) * scale
    return bf16.widen64(bf16.round_rne(x)) if dtype == "bf16" else x.astype(np.float32).astype(np.float64)


def strided(t, extra, offset):
    """The values of 2-D t in a view with `extra` more columns of pitch, `offset` elements in."""
    if not extra and not offset:
        return t.contiguous()
    buf = torch.full((t.shape[0] * (t.shape[1] + extra) + offset,), 7, dtype=t.dtype, device=t.device)
    v = buf[offset:].as_strided(t.shape, (t.shape[1] + extra, 1))
    v.copy_(t)
    return v


def sharded(x, mesh, dtype, extra=0, offset=0, replicate=False, device="cuda"):
    """[tokens, width] values as a DTensor, Shard(1) over the mesh (or one Replicate slot)."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(device).to(DT[dtype])
    p = 1 if replicate else mesh.shape[0]
    c = -(-t.shape[1] // p)
    slots = [strided(t[:, min(i * c, t.shape[1]):min((i + 1) * c, t.shape[1])], extra, offset) for i in range(p)]
    return tsl.DTensor(slots, mesh, [tsl.Replicate() if replicate else tsl.Shard(1)], tuple(t.shape), DT[dtype])


def whole(x, mesh, dtype=None, device="cuda"):
    t = x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))
    t = t.to(device)
    if dtype is not None:
        t = t.to(dtype)
    return tsl.DTensor([t], mesh, [tsl.Replicate()], tuple(t.shape), t.dtype)


def ints(x, mesh, device="cuda"):
    return whole(torch.tensor(np.asarray(x), dtype=torch.int32), mesh, device=device)


def full(dt):
    """All slots side by side, fp64 (with the dtype's values)."""
    return np.concatenate([s.detach().double().cpu().numpy() for s in dt.slots], -1)


class Batch:
    """Sequences in a paged cache: pages in a random order, the rest of the cache poisoned with NaN parameters."""

    def __init__(self, rng, mesh, q_lens, kv_lens, hk, d, group, page, dtype="bf16", replicate=False, spare=2,
                 kv_scale=1.0, poison=0xFFFFFFFF):
        self.mesh, self.q_lens, self.kv_lens = mesh, list(q_lens), list(kv_lens)
        self.hk, self.d, self.group, self.page = hk, d, group, page
        need = [-(-n // page) for n in self.kv_lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.width = max(need + [1]) + 1
        self.table = np.zeros((len(self.kv_lens), self.width), dtype=np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.words = heads.record_words(d, group)
        self.records = np.full((self.pages, hk, page, self.words), poison, dtype=np.uint32)
        ks = np.exp(0.4 * rng.standard_normal((hk, d))) * kv_scale
        ko = 0.5 * rng.standard_normal((hk, d)) * kv_scale
        self.kv = []
        for b, n in enumerate(self.kv_lens):
            k = (rng.standard_normal((n, hk, d)) * ks + ko).astype(np.float32)
            v = (rng.standard_normal((n, hk, d)) * kv_scale).astype(np.float32)
            rec = heads.pack(k, v, group)
            for j in range(n):
                self.records[self.table[b, j // page], :, j % page] = rec[j]
            self.kv.append(rec)
        self.replicate = replicate

    def cache(self):
        t = torch.from_numpy(self.records.view(np.int32)).cuda()
        p = 1 if self.replicate else self.mesh.shape[0]
        c = max(1, -(-self.hk // p))
        slots = [t[:, min(i * c, self.hk):min((i + 1) * c, self.hk)].contiguous() for i in range(p)]
        pl = [tsl.Replicate() if self.replicate else tsl.Shard(1)]
        return tsl.DTensor(slots, self.mesh, pl, tuple(t.shape), torch.int32)

    def operands(self):
        starts = np.concatenate([[0], np.cumsum(self.q_lens)])
        return (ints(self.table, self.mesh), ints(self.kv_lens, self.mesh), ints(starts, self.mesh))

    @property
    def tokens(self):
        return int(sum(self.q_lens))


def cache_bits(cache):
    return np.concatenate([s.cpu().numpy().view(np.uint32) for s in cache.slots], 1)
