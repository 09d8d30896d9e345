"""Log probabilities of logits of every finite size, masks of finite numbers among them, against 64 bits.

Bounds.  With d = scale (z - max), S the sum of exp(d), in half steps of fp32
(2^-24).  Where the kernel takes differences, they and their product with the
scale are rounded: 2 of |d|.  Where it takes one multiply-add, c z - fl(c m), that
is rounded once, and the scale's product with log2 e: 2 of |d| again; what fl(c m)
leaves out is at most 2^-3 and the same for all of a row.  A maximum that moves
on multiplies the sums by a factor whose exponent is a difference, a product and
two sums: 4 of |d|, for the terms that came before.  Terms below d = -40 are less
than 2^-57 of S.  So a term is off by at most 6 x 40, and 4 for the exponentials;
a sum by as many additions as a thread makes in a row (v / 128 at most) and 40.
ln S is off by as much absolutely, and by 2 of itself and of the 2^-3; a log
probability by 4 of its own size on top, lse by 4 of the largest |scale z|.  The
entropy's sum is weighted by d: 4 times (1 + H) covers it.
"""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from heads_helpers import DT, ints, whole
from oracle import decoder

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
MAX32 = float(torch.finfo(torch.float32).max)


def terms(v):
    return (6 * 40 + 4 + v / 128 + 40 + 2 * 24) * E24  # (ln S at most 24)


def host(d):
    return d.slots[0].double().cpu().numpy()


def in_fp32(e):
    """What is beyond fp32's range is an infinity in it."""
    return np.where(np.abs(e) > MAX32, np.copysign(np.inf, e), e)


def close(a, e, tol):
    with np.errstate(invalid="ignore"):
        ok = (a == e) | (np.abs(a - e) <= tol)
    assert ok.all(), [(i.tolist(), a[tuple(i)], e[tuple(i)]) for i in np.argwhere(~ok)[:5]]


def finite(e):
    return np.where(np.isfinite(e), np.abs(e), 0.0)


class Logits:
    """Logits on the device, and what is read off them in 64 bits."""

    def __init__(self, z, mesh, dtype, scale):
        t = torch.from_numpy(z).cuda().to(DT[dtype])
        c = -(-t.shape[1] // mesh.shape[0])
        slots = [t[:, i * c:(i + 1) * c].contiguous() for i in range(mesh.shape[0])]
        self.d = tsl.DTensor(slots, mesh, [tsl.Shard(1)], tuple(t.shape), t.dtype)
        self.mesh, self.scale, self.z = mesh, scale, t.double().cpu().numpy()
        s = float(np.float32(scale))
        self.logp, self.lse, self.ent = decoder.log_probs(self.z, s)
        self.size = finite(self.z).max(1) * s
        self.order = np.argsort(-self.z, axis=1, kind="stable")

    def check(self, ids, k, entropy):
        """One call, its results against 64 bits; the results."""
        r = tsl.tp_log_probs(self.d, ints(ids, self.mesh), scale=self.scale, top=k, entropy=entropy)
        tol = terms(self.z.shape[1])
        close(host(r.lse), in_fp32(self.lse), tol + 4 * E24 * self.size)
        e = in_fp32(np.take_along_axis(self.logp, ids, 1))
        close(host(r.logprobs), e, tol + 4 * E24 * finite(e))
        if entropy:
            close(host(r.entropy), self.ent, 4 * (1 + self.ent) * tol)
        if k:
            best = self.order[:, :k]
            assert np.array_equal(r.top_ids.slots[0].cpu().numpy(), best)
            e = in_fp32(np.take_along_axis(self.logp, best, 1))
            close(host(r.top_logprobs), e, tol + 4 * E24 * finite(e))
        return r


def rows_of(rng, size, v):
    """Rows about one number: alike, beside ordinary ones, hiding ordinary ones, ordinary ones times it."""
    z = rng.standard_normal((9, v)) * 2
    z[0] = size
    z[1, : v // 2] = size
    z[2, v // 2:] = size
    z[3, rng.random(v) < 0.9] = size
    z[4, : v - 2] = size
    z[5] = 0
    z[5, v // 3] = size
    z[6] *= size
    z[7] = size
    z[7, v - 1] = -size
    z[8, :] = np.where(np.arange(v) % 3 == 0, size, -np.inf)
    return z


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [2.0 ** -20, 0.7, 1.0, 2.0 ** 20])
@pytest.mark.parametrize("v,p", [(37, 1), (12000, 2)])
def test_logits_of_every_size(v, p, scale, dtype):
    """About 10^k for k from 3 to 37 (as far as scale times them is a number of fp32), several units a warp."""
    rng = np.random.default_rng(v)
    mesh = tsl.DeviceMesh((p,), ("tp",))
    sizes = [sign * 10.0 ** k for k in range(3, 38) for sign in (1, -1) if scale * 10.0 ** k < 1e38]
    z = np.concatenate([rows_of(rng, s, v) for s in sizes])
    z = np.clip(z, -1e38 / max(scale, 1), 1e38 / max(scale, 1), where=np.isfinite(z), out=z)
    x = Logits(z, mesh, dtype, scale)
    ids = rng.integers(0, v, (len(z), 2))
    for k, entropy in ((5, True), (0, False), (0, True), (32, False)):
        x.check(ids, k, entropy)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [2.0 ** -20, 0.7, 1.0, 2.0 ** 20])
def test_logits_about_a_border(scale, dtype):
    """Rows whose maxima lie on both sides of the sizes at which one way of rounding may end: 2^k for scale log2(e) z."""
    rng = np.random.default_rng(3)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    v = 12000
    spread = np.array([[1], [8], [40]]) / scale
    z = np.concatenate([sign * 2.0 ** k / (scale * np.log2(np.e)) + rng.standard_normal((3, v)) * spread
                        for k in range(17, 34) for sign in (1, -1)])
    z[:, ::7] = z[:, :1]  # (many alike)
    x = Logits(z, mesh, dtype, scale)
    ids = rng.integers(0, v, (len(z), 2))
    for k, entropy in ((5, True), (0, False)):
        x.check(ids, k, entropy)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,v,p,k", [(1, 128256, 4, 20), (320, 16000, 1, 0), (320, 16000, 2, 5)])
def test_masks_of_finite_numbers(t, v, p, k, dtype):
    """Ordinary rows under masks of -10^k that fill whole units: the results are those of the rest, and so are the gradients."""
    rng = np.random.default_rng(t)
    mesh = tsl.DeviceMesh((p,), ("tp",))
    for size in (-1e4, -1e10, -1e11, -1e20, -1e30):
        z = rng.standard_normal((t, v)) * 2
        left = rng.integers(v // 2, v - 40, t)
        columns = np.arange(v)[None]
        z[(columns < left[:, None]) | (columns >= (left + rng.integers(1, 40, t))[:, None])] = size
        x = Logits(z, mesh, dtype, 1.0)
        ids = left[:, None].repeat(2, 1)
        r = x.check(ids, k, True)
        dlp, dent = (torch.from_numpy(rng.standard_normal(s)).float() for s in ((t, 2), (t,)))
        d = tsl.tp_log_probs_backward(whole(dlp, mesh), whole(dent, mesh), x.d, ints(ids, mesh), r.lse, r.entropy)
        d = np.concatenate([s.double().cpu().numpy() for s in d.slots], 1)
        e, mag = decoder.log_probs_backward(x.z, ids, dlp.double().numpy(), host(r.lse), 1.0, dent.double().numpy(),
                                            host(r.entropy))
        seen = x.z > size / 2
        assert (d[~seen] == 0).all()
        # z - lse is rounded at the size of z and lse, and so is p's exponent; two ids' gradients are added
        rel = (18 + 2 * (np.abs(x.z) + np.abs(host(r.lse))[:, None])) * E24
        assert (np.abs(d - e) <= HALF[dtype] * np.abs(e) + 2 * rel * mag + 2.0 ** -130)[seen].all()
    assert tsl.read_device_status() == 0
