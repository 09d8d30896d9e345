"""Log probabilities over a sharded vocabulary and their gradient against the 64-bit restatement.

Bounds.  With d = scale (z - max): fp32 rounds the difference and the product,
so d is off by 2 half steps (2^-24) of |d|, and an exponential of it by that much
of itself and 4 half steps more (the exponential's own error).  Terms with d
below -40 are less than 2^-57 of the sum and count by no more than that, so
|d| <= 40 where it matters: a term is off by 84 half steps at most, the sum by
that and by the additions: as many as a thread adds in a row (v / 128 at most)
and 40.  ln S is off by the same amount absolutely, a log probability by twice
2^-24 of |d| and |l| on top, lse by as much of |max scale|.  The entropy's sum is
weighted by d, at most max(1, H) + ln terms on average: 4 times (1 + H) covers it.
"""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from heads_helpers import DT, draw, ints, strided, whole
from oracle import decoder

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
R = tsl.Replicate()
E24 = 2.0 ** -24


def vocab(z, mesh, dtype, replicate=False, extra=0, offset=0):
    t = torch.from_numpy(np.ascontiguousarray(z)).cuda().to(DT[dtype])
    p = 1 if replicate else mesh.shape[0]
    c = max(1, -(-t.shape[1] // p))
    slots = [strided(t[:, min(i * c, t.shape[1]):min((i + 1) * c, t.shape[1])], extra, offset) for i in range(p)]
    return tsl.DTensor(slots, mesh, [R if replicate else tsl.Shard(1)], tuple(t.shape), DT[dtype])


def host(d):
    return d.slots[0].double().cpu().numpy()


def side(d):
    return np.concatenate([s.double().cpu().numpy() for s in d.slots], 1)


def terms(v):
    return (84 + v / 128 + 40) * E24


def check_forward(r, z, ids, scale, k, ignore=-100, nan=False):
    """The five results against the restatement of fp64 logits z (given their dtype's values)."""
    t, v = z.shape
    scale = float(np.float32(scale))
    logp, lse, ent = decoder.log_probs(z, scale)
    with np.errstate(invalid="ignore"):
        size = np.abs(np.where(np.isfinite(z), z, 0).max(1)) * scale

    def close(a, e, tol):
        same = (a == e) | (np.isnan(a) & np.isnan(e))
        with np.errstate(invalid="ignore"):
            assert (same | (np.abs(a - e) <= tol)).all(), np.nanmax(np.abs(a - e) - tol)

    close(host(r.lse), lse, terms(v) + 4 * E24 * size)
    if ids is not None:
        there = (ids >= 0) & (ids < v)
        e = np.where(there, np.take_along_axis(logp, np.clip(ids, 0, v - 1), 1), 0.0)
        a = host(r.logprobs).reshape(ids.shape)
        close(a, e, terms(v) + 4 * E24 * np.abs(np.where(np.isfinite(e), e, 0)))
    if r.entropy is not None:
        close(host(r.entropy), ent, 4 * (1 + np.abs(ent)) * terms(v))
    if k:
        best = decoder.top(z, k)
        assert np.array_equal(r.top_ids.slots[0].cpu().numpy(), best)
        e = np.take_along_axis(logp, best, 1)
        close(host(r.top_logprobs), e, terms(v) + 4 * E24 * np.abs(np.where(np.isfinite(e), e, 0)))


def logits(rng, t, v, dtype, hot=3):
    z = draw(rng, (t, v), dtype, 2.0)
    for i in range(t):
        z[i, rng.integers(0, v, hot)] = draw(rng, (hot,), dtype, 3.0) + 8 if dtype == "fp32" else 8.0
    return z.astype(np.float32).astype(np.float64) if dtype == "fp32" else z


CASES = [  # tokens, vocabulary, parts, dtype, ids per token, top, scale, layout
    (1, 128256, 4, "bf16", 1, 20, 1.0, {}), (3, 1, 1, "bf16", 1, 1, 1.0, {}), (2, 2, 2, "fp32", 2, 2, 0.5, {}),
    (5, 7, 4, "bf16", 3, 7, 1.0, {}), (4, 31, 8, "fp32", 1, 5, 2.0, {}), (9, 1000, 3, "bf16", 1, 32, 1.0, {}),
    (33, 50257, 1, "bf16", 5, 10, 1.0, {}), (17, 50257, 2, "fp32", 1, 3, 0.7, {}), (400, 4099, 4, "bf16", 1, 1, 1.3, {}),
    (700, 2048, 2, "fp32", 64, 0, 1.0, {}), (64, 32000, 8, "bf16", 1, 0, 1.0, {}),
    (12, 9000, 2, "bf16", 1, 8, 1.0, dict(extra=3, offset=1)), (12, 9000, 2, "fp32", 1, 8, 1.0, dict(extra=5, offset=3)),
    (20, 8191, 4, "bf16", 2, 4, 1.0, dict(replicate=True)), (3, 262144, 8, "fp32", 1, 32, 1.0, {}),
    (2, 700001, 8, "bf16", 2, 20, 1.0, {}),
]


@pytest.mark.parametrize("t,v,p,dtype,c,k,scale,lay", CASES)
def test_log_probs(t, v, p, dtype, c, k, scale, lay):
    rng = np.random.default_rng(v + t)
    mesh = tsl.DeviceMesh((p,), ("tp",))
    z = logits(rng, t, v, dtype)
    ids = rng.integers(0, v, (t, c))
    ids[rng.random(t) < 0.2] = -100
    zd = vocab(z, mesh, dtype, **lay)
    r = tsl.tp_log_probs(zd, ints(ids, mesh), scale=scale, top=k, entropy=True)
    check_forward(r, z, ids, scale, k)
    # the gradient, with the library's own lse and entropy
    dlp, dent = draw(rng, (t, c), "fp32"), draw(rng, (t,), "fp32")
    args = [whole(dlp, mesh, torch.float32), whole(dent, mesh, torch.float32)]
    s32 = float(np.float32(scale))
    lse, ent = host(r.lse), host(r.entropy)
    for given, de in ((ids, dent), (ids, None), (None, dent)):
        out = vocab(np.zeros((t, v)), mesh, dtype, **lay)
        d = tsl.tp_log_probs_backward(args[0] if given is not None else None, args[1] if de is not None else None, zd,
                                      ints(ids, mesh) if given is not None else None, r.lse, r.entropy, scale=scale, out=out)
        e, mag = decoder.log_probs_backward(z, given, dlp, lse, s32, de, ent)
        # z scale - lse is rounded at the size of z scale and lse, and so is p's exponent
        rel = (12 + 2 * (np.abs(z * s32) + np.abs(lse)[:, None])) * E24 + (3 * c) * E24
        # logp + H: two numbers that may cancel, each off by its own rounding
        err = np.abs(side(d) - e)
        assert (err <= HALF[dtype] * np.abs(e) + rel * (mag + np.abs(mag)) + 2.0 ** -130).all(), \
            (err / (mag + 1e-30)).max()
    assert tsl.read_device_status() == 0


def test_backward_in_place_of_the_logits():
    rng = np.random.default_rng(5)
    for dtype, p, v in (("bf16", 4, 5000), ("fp32", 2, 4001)):
        mesh = tsl.DeviceMesh((p,), ("tp",))
        z, ids = logits(rng, 30, v, dtype), rng.integers(0, v, (30, 3))
        ids[:, 1] = ids[:, 0]
        zd, idd = vocab(z, mesh, dtype), ints(ids, mesh)
        r = tsl.tp_log_probs(zd, idd)
        g = whole(draw(rng, (30, 3), "fp32"), mesh, torch.float32)
        want = tsl.tp_log_probs_backward(g, None, zd, idd, r.lse)
        d = tsl.tp_log_probs_backward(g, None, zd, idd, r.lse, out=zd)
        assert all(torch.equal(a, b) for a, b in zip(d.slots, want.slots))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("v,p", [(64, 1), (5003, 4), (40000, 2)])
def test_masked_and_unusual_rows(dtype, v, p):
    """Masks of -inf and of the type's lowest value, rows of nothing else, infinities, NaN, equal logits, zeros of both
    signs."""
    rng = np.random.default_rng(v)
    mesh = tsl.DeviceMesh((p,), ("tp",))
    low = float(torch.finfo(DT[dtype]).min)
    z = draw(rng, (12, v), dtype, 2.0)
    z[0] = -np.inf
    z[1, : v - 3] = -np.inf
    z[2] = low
    z[3, : v - 2] = low
    z[4, v // 3] = np.nan
    z[5, v // 2] = np.inf
    z[6] = 1.5
    z[7] = np.where(np.arange(v) % 2, 0.0, -0.0)
    z[8] = -low
    z[9, 0] = -low
    z[10, rng.random(v) < 0.7] = -np.inf
    z[11] = np.where(np.arange(v) == v - 1, -np.inf, low)
    ids = rng.integers(0, v, (12, 2))
    ids[:, 1] = v - 1
    zd, idd = vocab(z, mesh, dtype), ints(ids, mesh)
    k = min(v, 32)
    with np.errstate(over="ignore", invalid="ignore"):
        for scale in (1.0, 0.25):
            r = tsl.tp_log_probs(zd, idd, scale=scale, top=k, entropy=True)
            check_forward(r, z, ids, scale, k)
    r = tsl.tp_log_probs(zd, idd, entropy=True)
    dlp, dent = draw(rng, (12, 2), "fp32"), draw(rng, (12,), "fp32")
    d = side(tsl.tp_log_probs_backward(whole(dlp, mesh, torch.float32), whole(dent, mesh, torch.float32), zd, idd, r.lse,
                                       r.entropy))
    with np.errstate(over="ignore", invalid="ignore"):
        e, mag = decoder.log_probs_backward(z, ids, dlp, host(r.lse), 1.0, dent, host(r.entropy))
    assert (d[0] == 0).all() and np.isnan(d[4]).all() and np.isnan(d[5]).all()
    for i in (1, 2, 3, 6, 7, 9, 10, 11):
        # where lse is of the size of the type's range, exp(z - lse) is 1 or 0 and not 1 / n
        if np.abs(host(r.lse)[i]) > 1e30:
            assert np.isfinite(d[i]).all()
        else:
            assert (np.abs(d[i] - e[i]) <= HALF[dtype] * np.abs(e[i]) + 400 * E24 * mag[i] + 2.0 ** -120).all(), i


def test_rows_without_gradients_are_zero_whatever_they_hold():
    rng = np.random.default_rng(6)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    z = draw(rng, (6, 300), "bf16")
    z[2] = np.nan
    ids = rng.integers(0, 300, (6, 1))
    ids[2] = -100
    zd, idd = vocab(z, mesh, "bf16"), ints(ids, mesh)
    r = tsl.tp_log_probs(zd, idd)
    assert host(r.logprobs)[2] == 0
    dlp = draw(rng, (6, 1), "fp32")
    dlp[4] = 0
    d = side(tsl.tp_log_probs_backward(whole(dlp, mesh, torch.float32), None, zd, idd, r.lse))
    assert (d[[2, 4]] == 0).all() and (d[[0, 1, 3, 5]] != 0).any(1).all()
    assert tsl.read_device_status() == 0


def test_ids_outside_the_vocabulary():
    rng = np.random.default_rng(7)
    mesh = tsl.DeviceMesh((4,), ("tp",))
    z, ids = draw(rng, (5, 90), "fp32"), np.array([[0], [90], [-1], [89], [2 ** 31 - 1]])
    zd, idd = vocab(z, mesh, "fp32"), ints(ids, mesh)
    tsl.read_device_status()
    r = tsl.tp_log_probs(zd, idd)
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX
    check_forward(r, z, ids, 1.0, 0)
    r = tsl.tp_log_probs(zd, idd, ignore_index=-1)
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX
    d = side(tsl.tp_log_probs_backward(whole(np.ones((5, 1)), mesh, torch.float32), None, zd, idd, r.lse))
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX
    assert (d[[1, 2, 4]] == 0).all() and (d[[0, 3]] != 0).all()


@pytest.mark.parametrize("ignore", [0, 999, -1])
def test_an_ignored_id_may_be_a_column(ignore):
    rng = np.random.default_rng(5)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    t, v = 12, 1000
    z = logits(rng, t, v, "fp32")
    given = rng.integers(1, v - 1, (t, 3))
    given[::2, 1] = ignore
    given[3] = ignore  # a token of nothing else
    zd = vocab(z, mesh, "fp32")
    r = tsl.tp_log_probs(zd, ints(given, mesh), ignore_index=ignore)
    seen = np.where(given == ignore, -100, given)
    check_forward(r, z, seen, 1.0, 0)
    g = draw(rng, (t, 3), "fp32")
    d = tsl.tp_log_probs_backward(whole(g, mesh, torch.float32), None, zd, ints(given, mesh), r.lse, ignore_index=ignore)
    e, mag = decoder.log_probs_backward(z, seen, g, host(r.lse))
    rel = (12 + 2 * (np.abs(z) + np.abs(host(r.lse))[:, None]) + 3 * 3) * E24  # as above
    assert (np.abs(side(d) - e) <= HALF["fp32"] * np.abs(e) + rel * mag + 2.0 ** -130).all()
    assert not side(d)[3].any()
    torch.cuda.synchronize()
    assert tsl.read_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_hidden_columns_under_large_entropy_gradients(dtype):
    """-inf and the lowest value have no gradient, however large scale and the entropy's gradient are."""
    mesh = tsl.DeviceMesh((1,), ("tp",))
    z = np.zeros((3, 40))
    z[:, 20:30], z[:, 30:] = -np.inf, torch.finfo(DT[dtype]).min
    zd = vocab(z, mesh, dtype)
    r = tsl.tp_log_probs(zd, scale=2.0 ** 20, entropy=True)
    g = whole(torch.full((3,), 1e9), mesh)
    d = side(tsl.tp_log_probs_backward(None, g, zd, None, r.lse, r.entropy, scale=2.0 ** 20))
    # the others are alike, each at the mean of log p: what is left is a rounding of ln 20 times scale g / 20
    assert (d[:, 20:] == 0).all() and (np.abs(d[:, :20]) <= 2.0 ** 20 * 1e9 / 20 * 16 * E24).all()


def test_the_same_id_given_twice():
    rng = np.random.default_rng(8)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    z, ids = draw(rng, (4, 1000), "fp32"), rng.integers(0, 1000, (4, 3))
    ids[:, 2] = ids[:, 0]
    zd = vocab(z, mesh, "fp32")
    r = tsl.tp_log_probs(zd, ints(ids, mesh))
    g = draw(rng, (4, 3), "fp32")
    d = side(tsl.tp_log_probs_backward(whole(g, mesh, torch.float32), None, zd, ints(ids, mesh), r.lse))
    e, mag = decoder.log_probs_backward(z, ids, g, host(r.lse))
    assert (np.abs(d - e) <= E24 * np.abs(e) + 64 * E24 * mag).all()


def test_leading_dims_and_partial_requests():
    rng = np.random.default_rng(9)
    mesh = tsl.DeviceMesh((2, 2), ("dp", "tp"))
    z = draw(rng, (3, 4, 700), "bf16")
    t = torch.from_numpy(z).cuda().to(torch.bfloat16)
    zd = tsl.DTensor([t[..., :350].contiguous(), t[..., 350:].contiguous()], mesh, [R, tsl.Shard(-1)], z.shape, t.dtype)
    ids = rng.integers(0, 700, (3, 4))
    idd = tsl.DTensor([torch.from_numpy(ids).int().cuda()], mesh, [R, R], ids.shape, torch.int32)
    r = tsl.tp_log_probs(zd, idd, top=5)
    assert r.logprobs.shape == r.lse.shape == (3, 4) and r.top_ids.shape == (3, 4, 5) and r.entropy is None
    logp, lse, _ = decoder.log_probs(z.reshape(12, 700))
    assert np.abs(host(r.lse).ravel() - lse).max() <= 1e-5
    assert np.array_equal(r.top_ids.slots[0].cpu().numpy().reshape(12, 5), decoder.top(z.reshape(12, 700), 5))
    assert np.abs(host(r.logprobs).ravel() - logp[np.arange(12), ids.ravel()]).max() <= 1e-5
    only = tsl.tp_log_probs(zd, top=5)
    assert only.logprobs is None and torch.equal(only.top_ids.slots[0], r.top_ids.slots[0])
    g = tsl.DTensor([torch.ones(3, 4, device="cuda")], mesh, [R, R], (3, 4), torch.float32)
    d = tsl.tp_log_probs_backward(g, None, zd, idd, r.lse)
    assert d.placements == zd.placements and d.shape == zd.shape


def test_captured_with_new_logits():
    rng = np.random.default_rng(10)
    mesh = tsl.DeviceMesh((4,), ("tp",))
    zs = [logits(rng, 8, 6001, "bf16") for _ in range(2)]
    idss = [rng.integers(0, 6001, (8, 1)) for _ in range(2)]
    zd, idd, g = vocab(zs[0], mesh, "bf16"), ints(idss[0], mesh), whole(np.ones((8, 1)), mesh, torch.float32)
    r = tsl.tp_log_probs(zd, idd, top=4, entropy=True)
    d = tsl.tp_log_probs_backward(g, None, zd, idd, r.lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tsl.tp_log_probs(zd, idd, top=4, entropy=True, out=r)
        tsl.tp_log_probs_backward(g, None, zd, idd, r.lse, out=d)
    new = vocab(zs[1], mesh, "bf16")
    for a, b in zip(zd.slots, new.slots):
        a.copy_(b)
    idd.slots[0].copy_(ints(idss[1], mesh).slots[0])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check_forward(r, zs[1], idss[1], 1.0, 4)
    e, mag = decoder.log_probs_backward(zs[1], idss[1], np.ones((8, 1)), host(r.lse))
    assert (np.abs(side(d) - e) <= 2.0 ** -8 * np.abs(e) + 128 * E24 * mag).all()


def test_gradient_against_differences():
    rng = np.random.default_rng(11)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    z, ids = draw(rng, (6, 200), "fp32"), rng.integers(0, 200, (6, 2))
    dlp, dent = draw(rng, (6, 2), "fp32"), draw(rng, (6,), "fp32")
    idd = ints(ids, mesh)

    def loss(x):
        r = tsl.tp_log_probs(vocab(x, mesh, "fp32"), idd, entropy=True, scale=1.5)
        return (host(r.logprobs) * dlp).sum() + (host(r.entropy) * dent).sum()

    r = tsl.tp_log_probs(vocab(z, mesh, "fp32"), idd, entropy=True, scale=1.5)
    g = side(tsl.tp_log_probs_backward(whole(dlp, mesh, torch.float32), whole(dent, mesh, torch.float32),
                                       vocab(z, mesh, "fp32"), idd, r.lse, r.entropy, scale=1.5))
    step = 2.0 ** -7
    for i in range(5):
        v = draw(rng, z.shape, "fp32")
        diff = (loss(z + step * v) - loss(z - step * v)) / (2 * step)
        assert abs(diff - (g * v).sum()) <= 2.0 ** -10 * np.abs(g * v).sum() + 2.0 ** -18 / step


def test_what_lies_beside_the_gradient_stays():
    rng = np.random.default_rng(12)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    for dtype, v in (("bf16", 2002), ("fp32", 1001)):
        z, ids = draw(rng, (9, v), dtype), rng.integers(0, v, (9, 1))
        zd = vocab(z, mesh, dtype)
        r = tsl.tp_log_probs(zd, ints(ids, mesh))
        out = vocab(np.zeros((9, v)), mesh, dtype, extra=5, offset=3)
        tsl.tp_log_probs_backward(whole(np.ones((9, 1)), mesh, torch.float32), None, zd, ints(ids, mesh), r.lse, out=out)
        want = tsl.tp_log_probs_backward(whole(np.ones((9, 1)), mesh, torch.float32), None, zd, ints(ids, mesh), r.lse)
        for s, w in zip(out.slots, want.slots):
            n = s.shape[1]
            assert torch.equal(s, w) and (torch.as_strided(s, (8, 5), (n + 5, 1), s.storage_offset() + n) == 7).all()


def test_offsets_past_32_bits():
    v, t = 128256, (1 << 32) // 128256 + 3
    mesh = tsl.DeviceMesh((1,), ("tp",))
    z = torch.empty(t, v, dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.randint(0, v, (t,), dtype=torch.int32, device="cuda")
    zd, idd = tsl.DTensor([z], mesh, [tsl.Shard(1)], z.shape, z.dtype), whole(ids, mesh)
    r = tsl.tp_log_probs(zd, idd, top=3)
    last = z[-2:].double().cpu().numpy()
    logp, lse, _ = decoder.log_probs(last)
    assert np.abs(host(r.lse)[-2:] - lse).max() <= terms(v) + 4 * E24 * 8
    assert np.array_equal(r.top_ids.slots[0][-2:].cpu().numpy(), decoder.top(last, 3))
    g = whole(torch.ones(t), mesh)
    tsl.tp_log_probs_backward(g, None, zd, idd, r.lse, out=zd)
    e, mag = decoder.log_probs_backward(last, ids[-2:].long().cpu().numpy()[:, None], np.ones((2, 1)), host(r.lse)[-2:])
    assert (np.abs(z[-2:].double().cpu().numpy() - e) <= 2.0 ** -8 * np.abs(e) + 64 * E24 * mag + 2.0 ** -130).all()
