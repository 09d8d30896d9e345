"""GPU parity of dt_tp_kv4_append against the oracle: the whole cache bit for bit.

The records are functions of fp32 operations that each round once, so the
oracle's fp32 arithmetic gives the same bits; so do the rotated queries and
the stored values (one rounding of an fp32 value to the output's type)."""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from oracle import bf16, heads

from heads_helpers import Batch, cache_bits, draw, full, ints, sharded, table, whole

pytestmark = pytest.mark.gpu


def rounded(x, dtype):
    return bf16.widen64(bf16.round_rne(x)) if dtype == "bf16" else np.float32(x).astype(np.float64)


def expect(batch, rec0, k, v, q, cs, inter, dtype):
    """The cache after the append, q_out, stored k and v, and the rows that are written."""
    t, d = batch.tokens, batch.d
    pos, seq = np.zeros(t, int), np.zeros(t, int)
    at = 0
    for b, (n, kv) in enumerate(zip(batch.q_lens, batch.kv_lens)):
        pos[at:at + n], seq[at:at + n] = np.arange(kv - n, kv), b
        at += n
    rot = lambda x: heads.rotate(x.reshape(t, -1, d), cs, pos, inter, dtype=np.float32)  # noqa: E731
    k2, v2 = rot(k), np.float32(v.reshape(t, -1, d))
    rec = heads.pack(k2, v2, batch.group)
    cache = rec0.copy()
    for i in range(t):
        cache[batch.table[seq[i], pos[i] // batch.page], :, pos[i] % batch.page] = rec[i]
    ks, vs = [], []
    for x, out in ((k2, ks), (v2, vs)):
        c, sb, mb = heads.quantise(x, batch.group)
        s, m = (np.repeat(bf16.widen(z), batch.group, -1) for z in (sb, mb))
        out.append(rounded(np.float32(c) * s + m, dtype).reshape(t, -1))
    return cache, (None if q is None else rounded(rot(q), dtype).reshape(t, -1)), ks[0], vs[0]


# q_lens, kv_lens, q heads, kv heads, d, group, page, parts, dtype, rotary, interleaved
CASES = [
    ([1], [1], 4, 1, 128, 64, 16, 1, "bf16", 128, False),
    ([1] * 5, [7, 16, 17, 32, 300], 8, 2, 128, 64, 16, 2, "bf16", 128, False),
    ([3, 0, 17, 1], [40, 0, 17, 33], 8, 4, 128, 64, 16, 4, "bf16", 128, True),
    ([3, 9, 17, 1], [40, 9, 65, 33], 4, 4, 64, 64, 24, 2, "fp32", 64, False),
    ([5, 40], [5, 90], 6, 2, 64, 32, 8, 2, "bf16", 32, False),
    ([5, 40], [5, 90], 6, 2, 64, 32, 7, 1, "bf16", 32, True),
    ([2, 30], [77, 30], 4, 2, 256, 64, 32, 2, "bf16", 256, False),
    ([2, 30], [77, 30], 7, 1, 256, 32, 64, 1, "fp32", 64, False),
    ([70, 33, 1], [100, 33, 900], 14, 2, 128, 32, 1, 1, "bf16", 96, False),
]


@pytest.mark.parametrize("stored", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_append(lib, case, stored):
    q_lens, kv_lens, hq, hk, d, group, page, p, dtype, rot, inter = case
    rng = np.random.default_rng(21)
    mesh = tsl.DeviceMesh((p,), ("tp",))
    b = Batch(rng, mesh, q_lens, kv_lens, hk, d, group, page)
    cache = b.cache()
    q, k, v = (draw(rng, (b.tokens, h * d), dtype, np.exp(rng.standard_normal((1, h * d)))) for h in (hq, hk, hk))
    if dtype == "bf16":
        q, k, v = (rounded(x, "bf16") for x in (q, k, v))
    else:
        q, k, v = (np.float32(x).astype(np.float64) for x in (q, k, v))
    cs = table(max(kv_lens), rot)
    st = tuple(sharded(np.zeros_like(k), mesh, dtype) for _ in range(2)) if stored else None
    qo = tsl.tp_kv4_append(sharded(k, mesh, dtype), sharded(v, mesh, dtype), cache, *b.operands(),
                           q=sharded(q, mesh, dtype), cos_sin=whole(cs, mesh), head_dim=d, group=group,
                           interleaved=inter, stored=st)
    assert tsl.read_device_status() == 0
    ec, eq, ek, ev = expect(b, b.records, k, v, q, cs, inter, dtype)
    np.testing.assert_array_equal(cache_bits(cache), ec)
    np.testing.assert_array_equal(full(qo), eq)
    if stored:
        np.testing.assert_array_equal(full(st[0]), ek)
        np.testing.assert_array_equal(full(st[1]), ev)


@pytest.mark.parametrize("case", [
    ([5000, 1, 0, 4100], [5003, 200, 9, 4100], 4, 2, 64, 64, 64, 1, "bf16", 64, False),
    ([5000, 1, 0, 4100], [5003, 200, 9, 4100], 3, 1, 64, 32, 24, 1, "fp32", 32, True),
    ([3001, 1200], [3001, 1300], 16, 3, 128, 64, 16, 1, "bf16", 128, False),
])
def test_long_prompts(lib, case):
    """More units than warps: every warp takes several, of several blocks each."""
    test_append(lib, case, True)


def test_without_rotation_queries_or_starts(lib):
    rng = np.random.default_rng(22)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    b = Batch(rng, mesh, [4] * 3, [4, 20, 64], 2, 128, 64, 16)
    cache = b.cache()
    k, v = (draw(rng, (12, 256), "bf16") for _ in range(2))
    pt, kl, _ = b.operands()
    assert tsl.tp_kv4_append(sharded(k, mesh, "bf16"), sharded(v, mesh, "bf16"), cache, pt, kl, head_dim=128) is None
    np.testing.assert_array_equal(cache_bits(cache), expect(b, b.records, k, v, None, None, False, "bf16")[0])


def test_many_sequences(lib):
    """More than 32 and more than 1024 sequences: the token's sequence is found in several steps."""
    rng = np.random.default_rng(23)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    for n in (33, 1100):
        q_lens = rng.integers(0, 4, n)
        kv_lens = q_lens + rng.integers(0, 9, n)
        b = Batch(rng, mesh, q_lens, kv_lens, 1, 64, 64, 8)
        cache = b.cache()
        k, v = (draw(rng, (b.tokens, 64), "bf16") for _ in range(2))
        cs = table(20, 64)
        tsl.tp_kv4_append(sharded(k, mesh, "bf16"), sharded(v, mesh, "bf16"), cache, *b.operands(),
                          cos_sin=whole(cs, mesh), head_dim=64)
        np.testing.assert_array_equal(cache_bits(cache), expect(b, b.records, k, v, None, cs, False, "bf16")[0])


def test_special_values(lib):
    """Constant groups, NaN, infinities, ranges that overflow, steps below the normal numbers, -0."""
    rng = np.random.default_rng(24)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    b = Batch(rng, mesh, [9], [9], 1, 128, 64, 16)
    cache = b.cache()
    k = draw(rng, (9, 128), "fp32")
    k[0], k[1, 3], k[2, 70], k[3, 0] = 2.5, np.nan, np.inf, -np.inf
    k[4, 1], k[4, 2] = 3.3e38, -3.3e38
    k[5] = k[5] * 1e-39
    k[6] = -0.0
    k[7, :64] = np.linspace(0, 15, 64)
    k = np.float32(k).astype(np.float64)
    v = k[::-1].copy()
    tsl.tp_kv4_append(sharded(k, mesh, "fp32"), sharded(v, mesh, "fp32"), cache, *b.operands(), head_dim=128)
    got, want = cache_bits(cache), expect(b, b.records, k, v, None, None, False, "fp32")[0]
    rec = b.table[0, 0]
    # a NaN parameter may carry any sign and payload
    isnan = lambda w: ((w & 0x7F80) == 0x7F80) & ((w & 0x7F) != 0)  # noqa: E731
    g, w = got[rec, 0, :9], want[rec, 0, :9]
    np.testing.assert_array_equal(g[:, :32], w[:, :32])
    for sh in (0, 16):
        gp, wp = (g[:, 32:] >> sh) & 0xFFFF, (w[:, 32:] >> sh) & 0xFFFF
        np.testing.assert_array_equal(isnan(gp), isnan(wp))
        np.testing.assert_array_equal(np.where(isnan(gp), 0, gp), np.where(isnan(wp), 0, wp))
    assert isnan(w[1:5, 32:] & 0xFFFF).any(1).all()


def test_bad_pages_lengths_and_positions(lib):
    """Entries that are no page are skipped, lengths are clamped to the page table, positions beyond the
    rotation table store nothing; each sets the status bit, and nothing else of the cache changes."""
    rng = np.random.default_rng(25)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    for what in ("page", "negative page", "length", "negative length", "position", "starts"):
        b = Batch(rng, mesh, [2, 2], [20, 20], 1, 64, 64, 16)
        cache = b.cache()
        k, v, q = (draw(rng, (4, 64), "bf16") for _ in range(3))
        tab, lens, starts, rows = b.table.copy(), [20, 20], [0, 2, 4], 64
        if what == "page":
            tab[0, 1] = b.pages
        elif what == "negative page":
            tab[0, 1] = -3
        elif what == "length":
            lens[0] = 10 ** 6
        elif what == "negative length":
            lens[0] = -5
        elif what == "position":
            rows = 18
        else:
            starts = [0, -7, 900]
        cs = table(rows, 64)
        qo = tsl.tp_kv4_append(sharded(k, mesh, "bf16"), sharded(v, mesh, "bf16"), cache, ints(tab, mesh),
                               ints(lens, mesh), ints(starts, mesh), q=sharded(q, mesh, "bf16"),
                               cos_sin=whole(cs, mesh), head_dim=64)
        status = tsl.read_device_status()
        got = cache_bits(cache)
        changed = {tuple(x) for x in np.argwhere((got != b.records).any((1, 3)))}
        mine = {(int(b.table[s, p // 16]), p % 16) for s in range(2) for p in (18, 19)}
        if what != "starts":
            assert status == tsl._lib.DEV_ERR_INDEX, what
            second = {(int(b.table[1, 1]), 2), (int(b.table[1, 1]), 3)}
            if what == "position":
                assert not changed and (full(qo) == 0).all()
            elif what == "length":  # clamped to 3 pages of 16: positions 46 and 47
                assert second <= changed and changed <= second | {(int(tab[0, 2]), 14), (int(tab[0, 2]), 15)}
            else:
                assert changed == second, what
        else:
            assert changed <= mine | {(int(t), o) for t in tab.reshape(-1) for o in range(16)}


def test_pitched_views_and_strided_cache(lib):
    rng = np.random.default_rng(26)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    b = Batch(rng, mesh, [3, 5], [30, 5], 4, 64, 32, 16)
    k, v, q = (draw(rng, (8, h * 64), "bf16") for h in (4, 4, 8))
    base = b.cache()
    slots = []
    for s in base.slots:  # heads outside, pages inside, and room between them
        n, h, ps, w = s.shape
        buf = torch.full((h, n, ps * w + 8), 3, dtype=torch.int32, device="cuda")
        view = buf.as_strided((n, h, ps, w), (ps * w + 8, n * (ps * w + 8), w, 1))
        view.copy_(s)
        slots.append(view)
    cache = tsl.DTensor(slots, mesh, base.placements, base.gshape, torch.int32)
    cs = table(40, 64)
    qo = sharded(np.zeros_like(q), mesh, "bf16", 16, 8)
    tsl.tp_kv4_append(sharded(k, mesh, "bf16", 8, 8), sharded(v, mesh, "bf16", 24), cache, *b.operands(),
                      q=sharded(q, mesh, "bf16", 8), cos_sin=whole(cs, mesh), head_dim=64, group=32, q_out=qo)
    ec, eq, _, _ = expect(b, b.records, k, v, q, cs, False, "bf16")
    np.testing.assert_array_equal(cache_bits(cache), ec)
    np.testing.assert_array_equal(full(qo), eq)
    for s in slots:
        gap = s.as_strided((s.shape[1] * s.shape[0], 8), (16 * b.words + 8, 1), 16 * b.words)
        assert (gap == 3).all()


def test_replays_with_new_lengths(lib):
    """One captured step appends at the lengths found on the device when it runs."""
    rng = np.random.default_rng(27)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    b = Batch(rng, mesh, [1, 1], [20, 33], 2, 128, 64, 16)
    cache, (pt, kl, qs) = b.cache(), b.operands()
    k, v, q = (draw(rng, (2, h * 128), "bf16") for h in (2, 2, 4))
    kd, vd, qd = (sharded(x, mesh, "bf16") for x in (k, v, q))
    cs = table(60, 128)
    csd, qo = whole(cs, mesh), sharded(np.zeros_like(q), mesh, "bf16")
    step = lambda: tsl.tp_kv4_append(kd, vd, cache, pt, kl, q=qd, cos_sin=csd, head_dim=128, q_out=qo)  # noqa: E731
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    kl.slots[0] += 1
    b.kv_lens = [21, 34]
    before = cache_bits(cache)
    g.replay()
    torch.cuda.synchronize()
    ec, eq, _, _ = expect(b, before, k, v, q, cs, False, "bf16")
    np.testing.assert_array_equal(cache_bits(cache), ec)
    np.testing.assert_array_equal(full(qo), eq)
