"""GPU parity of dt_tp_kv4_attention against the fp64 oracle, whose bounds (per query, from the inputs'
magnitudes) are the tolerances: fp32 sums, codes offset by 128, and for bf16 activations the rounding of
probability times step, plus half an ulp of the output's type."""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from oracle import bf16, heads

from heads_helpers import Batch, draw, full, ints, sharded

pytestmark = pytest.mark.gpu
HALF_ULP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -23}


def check(b, q, hq, dtype, out, lse, scale, causal, window, prompt=False):
    """Every query of every sequence; returns the largest error over its bound.
    ``prompt``: the tensor-core kernel's fp16 operands add theirs."""
    t, d, g = b.tokens, b.d, hq // b.hk
    got = full(out).reshape(t, hq, d)
    got_lse = full(lse) if lse is not None else None
    at, worst = 0, 0.0
    for s, (n, kv) in enumerate(zip(b.q_lens, b.kv_lens)):
        k, v, ks, vs = heads.unpack(b.kv[s], d, b.group)
        for h in range(hq):
            kh = h // g
            e, el, b32, b16 = heads.attention(q[at:at + n].reshape(n, hq, d)[:, h], k[:, kh], v[:, kh], scale, causal,
                                              window, ks[:, kh], vs[:, kh])
            tol = b32 + (b16 if dtype == "bf16" else 0)
            if prompt:
                tol = tol + heads.prompt_bound(q[at:at + n].reshape(n, hq, d)[:, h], k[:, kh], v[:, kh], scale, causal,
                                               window)
            y = got[at:at + n, h]
            np.testing.assert_array_equal(np.isnan(y), np.isnan(e))
            err = np.abs(y - e)
            bound = tol[:, None] + HALF_ULP[dtype] * np.abs(e)
            ok = (err <= bound) | np.isnan(e)
            assert ok.all(), (s, h, np.argwhere(~ok)[:4], err[~ok][:4], bound[~ok][:4])
            with np.errstate(all="ignore"):
                worst = max(worst, float(np.nanmax(np.where(bound > 0, err / bound, 0), initial=0)))
            if got_lse is not None:
                gl = got_lse[at:at + n, h]
                np.testing.assert_array_equal(np.isneginf(gl), np.isneginf(el))
                f = np.isfinite(el)
                vmax = np.maximum(np.abs(v[:, kh]).max(initial=0), 1e-30)
                assert (np.abs(gl[f] - el[f]) <= 1e-5 + tol[f] / vmax * 4 + 2.0 ** -20 * np.abs(el[f])).all()
        at += n
    return worst


def run(rng, q_lens, kv_lens, hq, hk, d, group, page, p, dtype, causal=True, window=0, scale=None, with_lse=True,
        starts=True, replicate=False, q_scale=1.0, prompt=False, **kw):
    mesh = tsl.DeviceMesh((p,), ("tp",))
    b = Batch(rng, mesh, q_lens, kv_lens, hk, d, group, page, replicate=replicate, **kw)
    q = draw(rng, (b.tokens, hq * d), dtype, q_scale)
    qd = sharded(q, mesh, dtype)
    pt, kl, qs = b.operands()
    lse = tsl.DTensor.empty(mesh, [tsl.Shard(1)], (b.tokens, hq), torch.float32) if with_lse else None
    out = sharded(np.full_like(q, 9), mesh, dtype)
    y = tsl.tp_kv4_attention(qd, b.cache(), pt, kl, qs if starts else None, head_dim=d, group=group, scale=scale,
                             causal=causal, window=window, lse=lse, out=out)
    assert tsl.read_device_status() == 0
    return check(b, q, hq, dtype, y, lse, d ** -0.5 if scale is None else scale, causal, window, prompt)


FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,group", FORMATS)
def test_single_tokens(lib, d, group, dtype):
    """One query per sequence; lengths of zero and one, at and around the tiles' and pages' ends."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300, 1000]
    run(np.random.default_rng(31), [1] * len(lens), lens, 8, 2, d, group, 16, 2, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,group", FORMATS)
def test_drafts(lib, d, group, dtype):
    """A few queries per sequence, none for one of them, more than there are keys for another."""
    run(np.random.default_rng(32), [3, 5, 0, 4, 1, 9], [40, 5, 33, 2, 200, 77], 6, 2, d, group, 24, 2, dtype)


@pytest.mark.parametrize("hq,hk,p", [(1, 1, 1), (5, 5, 5), (7, 1, 1), (8, 8, 4), (16, 1, 1), (40, 8, 8), (24, 2, 2)])
def test_head_groups(lib, hq, hk, p):
    run(np.random.default_rng(33), [1, 2, 1], [50, 130, 257], hq, hk, 128, 64, 16, p, "bf16")


@pytest.mark.parametrize("page", [1, 3, 8, 16, 32, 33, 64, 128, 500])
def test_page_sizes(lib, page):
    run(np.random.default_rng(34), [1, 1, 2], [400, 129, 64], 4, 1, 128, 64, page, 1, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 5), (True, 32), (True, 100), (True, 10 ** 6)])
def test_masks(lib, causal, window, dtype):
    run(np.random.default_rng(35), [1, 4, 40, 2], [300, 150, 90, 2], 4, 2, 64, 64, 16, 2, dtype, causal, window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_chunks(lib, d):
    """Many queries per sequence: whole prompts, and a chunk behind a context."""
    run(np.random.default_rng(36), [130, 64, 1], [130, 200, 70], 4, 1, d, 64, 16, 1, "bf16", prompt=d <= 128)


# What follows has 64 (query, head) rows per sequence and kv head or more: the tensor-core kernel.

@pytest.mark.parametrize("d,group", FORMATS[:4])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hk", [
    ([64], [64], 1, 1),                               # one tile, one step
    ([65, 64, 63], [65, 300, 129], 2, 1),             # at and around the tiles' ends
    ([256, 300], [256, 1000], 1, 1),                  # two tiles, several row blocks
    ([100, 1, 0, 37, 200], [100, 500, 0, 37, 900], 6, 2),  # prompts, a decode step, no queries, odd group of 3
    ([90, 40], [60, 40], 2, 2),                       # more queries than keys
])
def test_prompt_lengths(lib, d, group, q_lens, kv_lens, hq, hk):
    run(np.random.default_rng(50), q_lens, kv_lens, hq, hk, d, group, 16, hk, "bf16", prompt=True)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 60), (True, 128), (True, 250), (True, 10 ** 6)])
def test_prompt_masks(lib, causal, window):
    run(np.random.default_rng(51), [150, 70], [400, 70], 4, 2, 64, 64, 16, 2, "bf16", causal, window, prompt=True)


@pytest.mark.parametrize("page", [1, 7, 8, 33, 64, 128, 500])
def test_prompt_page_sizes(lib, page):
    run(np.random.default_rng(52), [80, 90], [300, 129], 2, 1, 128, 64, page, 1, "bf16", prompt=True)


def test_prompt_split_over_ctas(lib):
    """One row block on a long context: every CTA holds a piece of it."""
    run(np.random.default_rng(53), [70, 64], [9000, 64], 4, 2, 128, 64, 64, 2, "bf16", prompt=True)


@pytest.mark.parametrize("kv_scale,q_scale", [(1e5, 1e-4), (1e-5, 1.0), (1.0, 30.0), (1e-30, 1e20)])
def test_prompt_magnitudes(lib, kv_scale, q_scale):
    """Keys and values beyond and far below fp16's range; large logits."""
    run(np.random.default_rng(54), [70, 80], [300, 200], 2, 1, 64, 64, 16, 1, "bf16", kv_scale=kv_scale,
        q_scale=q_scale, prompt=True)


def test_prompt_values_that_grow(lib):
    """Steps of 128 keys whose values grow by powers of two, and shrink again: what O is scaled by follows."""
    rng = np.random.default_rng(55)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    b = Batch(rng, mesh, [70], [900], 1, 64, 64, 16)
    k, _, _, _ = heads.unpack(b.kv[0], 64, 64)
    v = rng.standard_normal((900, 1, 64)) * 2.0 ** np.array([0, 9, -5, 20, 30, 3, -20, 0])[np.arange(900) // 128][:, None, None]
    b.kv[0] = heads.pack(np.float32(k), np.float32(v), 64)
    for j in range(900):
        b.records[b.table[0, j // 16], :, j % 16] = b.kv[0][j]
    q = draw(rng, (70, 64), "bf16")
    pt, kl, qs = b.operands()
    y = tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), pt, kl, qs, head_dim=64)
    check(b, q, 1, "bf16", y, None, 0.125, True, 0, True)


@pytest.mark.parametrize("poison", [0x7F807F80, 0xFF80FF80, 0x7FC07FC0, 0xFFFFFFFF])
def test_prompt_hidden_keys(lib, poison):
    """NaN and infinities in hidden keys and beyond the lengths; a visible one reaches the queries that see it."""
    rng = np.random.default_rng(56)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    b = Batch(rng, mesh, [100], [300], 1, 128, 64, 16, poison=poison)
    q = draw(rng, (100, 2 * 128), "bf16")
    rec = b.kv[0][250].copy()
    rec[..., 32:] = poison  # key 250: seen by queries at positions 250 to 289 of 200 to 299
    b.records[b.table[0, 250 // 16], :, 250 % 16] = rec
    pt, kl, qs = b.operands()
    y = full(tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), pt, kl, qs, head_dim=128, window=40))
    bad = np.zeros(100, bool)
    bad[50:90] = True
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()
    k, v, ks, vs = heads.unpack(b.kv[0], 128, 64)
    for h in range(2):
        qh = q.reshape(100, 2, 128)[:, h]
        e, _, b32, b16 = heads.attention(qh, k[:, 0], v[:, 0], 128 ** -0.5, True, 40, ks[:, 0], vs[:, 0])
        tol = b32 + b16 + heads.prompt_bound(qh, k[:, 0], v[:, 0], 128 ** -0.5, True, 40)
        err = np.abs(y.reshape(100, 2, 128)[:, h] - e)
        assert (err <= tol[:, None] + 2.0 ** -8 * np.abs(e))[~bad].all()


def test_prompt_bad_pages(lib):
    rng = np.random.default_rng(57)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    q = draw(rng, (80, 2 * 64), "bf16")
    b = Batch(rng, mesh, [80], [240], 1, 64, 64, 16)
    tab = b.table.copy()
    tab[0, 1], tab[0, 8] = -1, 10 ** 6
    y = tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), ints(tab, mesh), b.operands()[1], head_dim=64,
                             causal=False)
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX
    b.kv[0] = np.concatenate([b.kv[0][:16], b.kv[0][32:128], b.kv[0][144:]])
    b.kv_lens = [208]
    check(b, q, 2, "bf16", y, None, 0.125, False, 0, True)


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hk,causal,window", [
    ([64], [64], 1, 1, True, 0),
    ([65, 64, 63], [65, 300, 129], 2, 1, True, 0),
    ([300], [1000], 1, 1, True, 0),                              # several row blocks of 128
    ([100, 1, 0, 37, 200], [100, 500, 0, 37, 700], 6, 2, True, 0),
    ([90, 40], [60, 40], 2, 2, True, 60),
    ([80], [400], 4, 2, False, 0),
    ([70, 64], [5000, 64], 4, 2, True, 0),                       # split over CTAs
])
def test_prompt_wide_heads(lib, group, q_lens, kv_lens, hq, hk, causal, window):
    run(np.random.default_rng(59), q_lens, kv_lens, hq, hk, 256, group, 24, hk, "bf16", causal, window, prompt=True)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("rise", [0.02, 0.2, 3.0, -0.2])
def test_prompt_rising_logits(lib, d, rise):
    """Logits that rise (fall) by `rise` (log2 units, about) from key to key: references that follow late or each
    step."""
    rng = np.random.default_rng(60)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    b = Batch(rng, mesh, [96], [500], 1, d, 64, 16)
    _, v, _, _ = heads.unpack(b.kv[0], d, 64)
    k = np.ones((500, 1, d)) * (rise * np.log(2) * (np.arange(500) - 250)[:, None, None] / d ** 0.5) \
        + 0.1 * rng.standard_normal((500, 1, d))
    b.kv[0] = heads.pack(np.float32(k), np.float32(v), 64)
    for j in range(500):
        b.records[b.table[0, j // 16], :, j % 16] = b.kv[0][j]
    q = draw(rng, (96, d), "bf16", 0.05) + 1
    q = bf16.widen64(bf16.round_rne(q))
    pt, kl, qs = b.operands()
    y = tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), pt, kl, qs, head_dim=d)
    check(b, q, 1, "bf16", y, None, d ** -0.5, True, 0, True)


def test_prompt_repeats_and_graph(lib):
    rng = np.random.default_rng(58)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    b = Batch(rng, mesh, [100, 64], [700, 64], 2, 128, 64, 16)
    q = draw(rng, (164, 8 * 128), "bf16")
    qd, cache, (pt, kl, qs) = sharded(q, mesh, "bf16"), b.cache(), b.operands()
    n = tsl.tp_kv4_attention_workspace_bytes(qd, cache, pt, head_dim=128)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    a = tsl.tp_kv4_attention(qd, cache, pt, kl, qs, head_dim=128, workspace=buf[:n])
    assert (buf[n:] == 0xA5).all()
    check(b, q, 8, "bf16", a, None, 128 ** -0.5, True, 0, True)
    out = sharded(np.zeros_like(q), mesh, "bf16")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsl.tp_kv4_attention(qd, cache, pt, kl, qs, head_dim=128, workspace=buf[:n], out=out)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, u) for s, u in zip(a.slots, out.slots))


def test_long_sequence_is_split(lib):
    """A sequence far longer than the others, and than one CTA's share."""
    run(np.random.default_rng(37), [1, 1, 2], [20000, 3, 700], 8, 2, 128, 64, 16, 2, "bf16")


def test_long_sequence_fp32(lib):
    run(np.random.default_rng(38), [2], [9000], 2, 1, 64, 32, 64, 1, "fp32")


def test_many_sequences(lib):
    rng = np.random.default_rng(39)
    run(rng, [1] * 300, rng.integers(0, 60, 300), 2, 1, 64, 64, 8, 1, "bf16")


def test_same_number_of_queries_needs_no_starts(lib):
    run(np.random.default_rng(40), [3] * 4, [3, 60, 35, 9], 4, 2, 128, 64, 16, 2, "bf16", starts=False)


def test_scale_and_no_lse(lib):
    run(np.random.default_rng(41), [1, 2], [100, 40], 4, 2, 128, 64, 16, 2, "bf16", scale=0.5, with_lse=False)


def test_one_key_takes_all(lib):
    """Large logits: the softmax's maximum grows along the sequence."""
    run(np.random.default_rng(42), [1, 1], [500, 130], 4, 2, 64, 64, 16, 2, "fp32", q_scale=20.0)


def test_replicated_cache_beside_sharded_queries(lib):
    run(np.random.default_rng(43), [1, 3], [90, 33], 8, 1, 128, 64, 16, 4, "bf16", replicate=True)


@pytest.mark.parametrize("poison", [0x7F807F80, 0xFF80FF80, 0x7FC07FC0, 0x00000000])
def test_what_is_hidden_does_not_reach_the_result(lib, poison):
    """Places beyond the lengths, spare pages and hidden keys hold infinities or NaN."""
    rng = np.random.default_rng(44)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    b = Batch(rng, mesh, [2, 1], [45, 70], 1, 128, 64, 16, poison=poison)
    q = draw(rng, (3, 4 * 128), "bf16")
    # the first query of sequence 0 does not see its last key, the window hides the first keys
    for s, j in ((0, 44), (1, 0), (1, 5)):
        rec = b.kv[s][j].copy()
        rec[..., 32:] = poison if poison else 0x7F807F80
        b.kv[s][j] = rec
        b.records[b.table[s, j // 16], :, j % 16] = rec
    pt, kl, qs = b.operands()
    y = tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), pt, kl, qs, head_dim=128, window=40)
    got = full(y)
    assert np.isfinite(got[0]).all() and np.isfinite(got[2]).all() and np.isnan(got[1]).all()
    for row, s, n in ((0, 0, 44), (2, 1, 70)):
        k, v, ks, vs = heads.unpack(b.kv[s][:n], 128, 64)
        for h in range(4):
            e, _, b32, b16 = heads.attention(q[row].reshape(4, 128)[h:h + 1], k[:, 0], v[:, 0], 128 ** -0.5, True, 40,
                                             ks[:, 0], vs[:, 0])
            assert (np.abs(got[row].reshape(4, 128)[h] - e[0]) <= b32 + b16 + 2.0 ** -8 * np.abs(e[0])).all()


def test_bad_pages_and_lengths(lib):
    """An entry that is no page hides its keys, a length beyond the table is cut; both set the status bit."""
    rng = np.random.default_rng(45)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    q = draw(rng, (2, 2 * 64), "bf16")
    for bad in (-1, 10 ** 6):
        b = Batch(rng, mesh, [1, 1], [40, 40], 1, 64, 64, 16)
        tab = b.table.copy()
        tab[0, 1] = bad
        y = tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), ints(tab, mesh), b.operands()[1], head_dim=64)
        assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX
        b.kv[0] = np.concatenate([b.kv[0][:16], b.kv[0][32:]])
        b.kv_lens = [24, 40]
        check(b, q, 2, "bf16", y, None, 0.125, False, 0)
    b = Batch(rng, mesh, [1, 1], [48, 40], 1, 64, 64, 16)
    b.table, keep = b.table[:, :3], b.kv_lens
    y = tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), ints(b.table, mesh), ints([10 ** 9, 40], mesh),
                             head_dim=64)
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX and keep == [48, 40]
    check(b, q, 2, "bf16", y, None, 0.125, True, 0)
    y = tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), ints(b.table, mesh), ints([-4, 40], mesh), head_dim=64)
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX and (full(y)[0] == 0).all()


def test_rows_of_no_sequence_and_odd_starts_stay_in_bounds(lib):
    """Rows outside every sequence keep what they held; starts out of order are clamped."""
    rng = np.random.default_rng(46)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    b = Batch(rng, mesh, [1, 1], [40, 33], 1, 64, 64, 16)
    q = draw(rng, (6, 128), "bf16")
    out = sharded(np.full((6, 128), 9.0), mesh, "bf16")
    tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), b.operands()[0], b.operands()[1], ints([2, 3, 4], mesh),
                         head_dim=64, out=out)
    y = full(out)
    assert (y[[0, 1, 4, 5]] == 9).all() and (y[2:4] != 9).any()
    tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), b.cache(), b.operands()[0], b.operands()[1], ints([5, -2, 99], mesh),
                         head_dim=64, out=out)
    torch.cuda.synchronize()


def test_workspace(lib):
    """Exactly the queried bytes, any contents, guarded; one byte less is refused."""
    rng = np.random.default_rng(47)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    b = Batch(rng, mesh, [1] * 3, [3000, 5, 700], 2, 128, 64, 16)
    q = draw(rng, (3, 8 * 128), "bf16")
    qd, cache, (pt, kl, qs) = sharded(q, mesh, "bf16"), b.cache(), b.operands()
    n = tsl.tp_kv4_attention_workspace_bytes(qd, cache, pt, head_dim=128)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    first = None
    for fill in (0xA5, 0xFF, 0x00):
        buf[:n] = fill
        y = tsl.tp_kv4_attention(qd, cache, pt, kl, qs, head_dim=128, workspace=buf[:n])
        check(b, q, 8, "bf16", y, None, 128 ** -0.5, True, 0)
        assert (buf[n:] == 0xA5).all()
        if first is not None:
            assert all(torch.equal(s, u) for s, u in zip(first.slots, y.slots))
        first = y
    with pytest.raises(tsl.DtError) as e:
        tsl.tp_kv4_attention(qd, cache, pt, kl, qs, head_dim=128, workspace=buf[:n - 1])
    assert e.value.status == tsl._lib.ERR_INVALID_ARG
    with pytest.raises(tsl.DtError) as e:
        tsl.tp_kv4_attention(qd, cache, pt, kl, qs, head_dim=128, workspace=buf[1:])
    assert e.value.status == tsl._lib.ERR_ALIGNMENT


def test_two_streams_and_a_graph(lib):
    rng = np.random.default_rng(48)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    b = Batch(rng, mesh, [1] * 4, [900, 40, 333, 64], 2, 128, 64, 16)
    q = draw(rng, (4, 8 * 128), "bf16")
    qd, cache, (pt, kl, qs) = sharded(q, mesh, "bf16"), b.cache(), b.operands()
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s in streams * 3:
        with torch.cuda.stream(s):
            outs.append(tsl.tp_kv4_attention(qd, cache, pt, kl, qs, head_dim=128))
    torch.cuda.synchronize()
    for y in outs:
        check(b, q, 8, "bf16", y, None, 128 ** -0.5, True, 0)
    n = tsl.tp_kv4_attention_workspace_bytes(qd, cache, pt, head_dim=128)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), outs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsl.tp_kv4_attention(qd, cache, pt, kl, qs, head_dim=128, out=out, workspace=ws)
    kl.slots[0].copy_(torch.tensor([500, 40, 300, 1], dtype=torch.int32))
    for s, n in enumerate([500, 40, 300, 1]):
        b.kv[s], b.kv_lens[s] = b.kv[s][:n], n
    g.replay()
    torch.cuda.synchronize()
    check(b, q, 8, "bf16", out, None, 128 ** -0.5, True, 0)


def test_offsets_beyond_32_bits(lib):
    """A cache of more than 2^31 words, its used pages at the far end."""
    rng = np.random.default_rng(49)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    b = Batch(rng, mesh, [1], [200], 1, 128, 64, 16)
    q = draw(rng, (1, 4 * 128), "bf16")
    pages = (2 ** 31 + 2 ** 20) // (16 * 36)
    big = torch.zeros(pages, 1, 16, 36, dtype=torch.int32, device="cuda")
    small = torch.from_numpy(b.records.view(np.int32)).cuda()
    big[pages - b.pages:] = small
    cache = tsl.DTensor([big], mesh, [tsl.Shard(1)], tuple(big.shape), torch.int32)
    tab = ints(b.table + (pages - b.pages), mesh)
    y = tsl.tp_kv4_attention(sharded(q, mesh, "bf16"), cache, tab, b.operands()[1], head_dim=128)
    check(b, q, 4, "bf16", y, None, 128 ** -0.5, True, 0)
    k = draw(rng, (1, 128), "bf16")
    tsl.tp_kv4_append(sharded(k, mesh, "bf16"), sharded(k, mesh, "bf16"), cache, tab, b.operands()[1], head_dim=128)
    at = pages - b.pages + int(b.table[0, 199 // 16])
    want = heads.pack(np.float32(k), np.float32(k), 64)[0]
    np.testing.assert_array_equal(big[at, 0, 199 % 16].cpu().numpy().view(np.uint32), want)
