"""Attention over the 4-bit cache at the edges of its range, against the fp64 oracle.

Tolerance: relative to the norm of each (sequence, head)'s result.  Rounding to bf16 is at most 2^-8 of an element.
Operands in fp16 add 2^-11 of a probability and of a value, and 2^-11 of a key through a logit: with logits whose
terms sum to less than 3 in magnitude on average that is under 2^-9 of the result, altogether less than 2^-7.
"""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from oracle import bf16, heads

from heads_helpers import Batch, draw, full, ints, sharded

pytestmark = pytest.mark.gpu
CLOSE = 2.0 ** -7


def put(b, s, j, rec):
    """Record `rec` [kv heads, words] as key j of sequence s, in the pages and for the oracle."""
    b.kv[s][j] = rec
    b.records[b.table[s, j // b.page], :, j % b.page] = rec


def put_all(b, s, k, v):
    """fp32 keys and values [n, kv heads, d] as sequence s's."""
    rec = heads.pack(np.float32(k), np.float32(v), b.group)
    for j in range(len(rec)):
        put(b, s, j, rec[j])


def expected(b, q, hq, scale, causal=True, window=0):
    """fp64 results [tokens, hq, d] and logs [tokens, hq]."""
    out, logs, at, g = [], [], 0, hq // b.hk
    for s, n in enumerate(b.q_lens):
        k, v, _, _ = heads.unpack(b.kv[s][:b.kv_lens[s]], b.d, b.group)
        qs = q[at:at + n].reshape(n, hq, b.d)
        r = [heads.attention(qs[:, h], k[:, h // g], v[:, h // g], scale, causal, window) for h in range(hq)]
        out.append(np.stack([x[0] for x in r], 1))
        logs.append(np.stack([x[1] for x in r], 1))
        at += n
    return np.concatenate(out), np.concatenate(logs)


def call(b, q, hq, dtype="bf16", table=None, kv_lens=None, status=0, **kw):
    """Results [tokens, hq, d] and logs [tokens, hq] of one call."""
    pt, kl, qs = b.operands()
    if table is not None:
        pt = ints(table, b.mesh)
    if kv_lens is not None:
        kl = ints(kv_lens, b.mesh)
    tsl.read_device_status(clear=True)
    lse = tsl.DTensor.empty(b.mesh, [tsl.Shard(1)], (b.tokens, hq), torch.float32)
    y = tsl.tp_kv4_attention(sharded(q, b.mesh, dtype), b.cache(), pt, kl, qs, head_dim=b.d, group=b.group, lse=lse, **kw)
    assert tsl.read_device_status() == status
    return full(y).reshape(b.tokens, hq, b.d), full(lse)


def assert_close(got, want, b, limit=CLOSE):
    at = 0
    for s, n in enumerate(b.q_lens):
        for h in range(want.shape[1]):
            y, e = got[at:at + n, h], want[at:at + n, h]
            assert np.isfinite(y).all(), (s, h)
            err = np.linalg.norm(y - e)
            assert err <= limit * np.linalg.norm(e), (s, h, err / np.linalg.norm(e))
        at += n


MESH1 = tsl.DeviceMesh((1,), ("tp",))


@pytest.mark.parametrize("n", [4, 80])
@pytest.mark.parametrize("scale", [1e-9, 1e-20, 1e-37])
def test_tiny_scales_and_queries_of_zero(lib, n, scale):
    """A row of zeros, or logits that are all but zero, weigh all visible keys alike; the hidden ones stay hidden."""
    rng = np.random.default_rng(70)
    b = Batch(rng, MESH1, [n, n], [n, 150], 1, 64, 64, 16)
    q = draw(rng, (2 * n, 2 * 64), "bf16")
    q[1::2] = 0
    q[2::4] *= 2.0 ** -100
    got, logs = call(b, q, 2, scale=scale)
    want, want_logs = expected(b, q, 2, scale)
    assert_close(got, want, b)
    assert (np.abs(logs - want_logs) <= 1e-4).all()


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 64), (256, 32)])
@pytest.mark.parametrize("n", [6, 90])
@pytest.mark.parametrize("small", [1e-4, 1e-6, 1e-8, 1e-20, 1e-30])
def test_small_keys_and_large_queries(lib, n, small, d, group):
    """Keys far below fp16's range with queries as far above it: ordinary logits."""
    rng = np.random.default_rng(71)
    b = Batch(rng, MESH1, [n, n], [300, n], 1, d, group, 16)
    for s, m in enumerate(b.kv_lens):
        put_all(b, s, rng.standard_normal((m, 1, d)) * small, rng.standard_normal((m, 1, d)))
    q = draw(rng, (2 * n, 2 * d), "bf16", 1 / small)
    got, _ = call(b, q, 2)
    assert_close(got, expected(b, q, 2, d ** -0.5)[0], b)


@pytest.mark.parametrize("n", [6, 90])
@pytest.mark.parametrize("small,large", [(1e-6, 10.0), (1e-3, 1e4), (1e-12, 1e-6)])
def test_small_group_of_channels_beside_a_large_one(lib, n, small, large):
    """Both halves of the channels make up half of each logit, their keys 10^6 and more apart."""
    rng = np.random.default_rng(72)
    b = Batch(rng, MESH1, [n], [300], 1, 128, 64, 16)
    size = np.repeat([small, large], 64)
    put_all(b, 0, rng.standard_normal((300, 1, 128)) * size, rng.standard_normal((300, 1, 128)))
    q = draw(rng, (n, 128), "bf16") / size
    q = bf16.widen64(bf16.round_rne(q))
    got, _ = call(b, q, 1)
    assert_close(got, expected(b, q, 1, 128 ** -0.5)[0], b)


@pytest.mark.parametrize("n", [6, 90])
def test_steps_of_keys_of_very_different_size(lib, n):
    """Each 64 keys have a scale of their own, from 1e-12 to 1e3; the logits stay ordinary."""
    rng = np.random.default_rng(73)
    b = Batch(rng, MESH1, [n], [512], 1, 64, 64, 16)
    size = 10.0 ** np.array([3, -12, 0, -6, 2, -9, -3, 1])[np.arange(512) // 64]
    put_all(b, 0, rng.standard_normal((512, 1, 64)) * size[:, None, None], rng.standard_normal((512, 1, 64)))
    q = draw(rng, (n, 64), "bf16", 1e-3)
    got, _ = call(b, q, 1)
    assert_close(got, expected(b, q, 1, 0.125)[0], b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,window", [
    ([1, 1], [1000, 500], 128), ([1, 1], [1000, 333], 1), ([3, 5], [700, 200], 37), ([40, 1], [700, 1000], 200),
    ([90, 70], [700, 1000], 100)])
def test_pages_behind_the_window_need_not_exist(lib, q_lens, kv_lens, window, d, dtype):
    """Entries of pages that lie wholly before the first query's window are no pages: nothing is reported, and the
    results are those of the whole table."""
    rng = np.random.default_rng(74)
    b = Batch(rng, MESH1, q_lens, kv_lens, 1, d, 64, 16)
    q = draw(rng, (b.tokens, 2 * d), dtype)
    table = b.table.copy()
    for s, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        first = max(0, kv - n - window + 1)
        table[s, :first // 16] = -1
    got, logs = call(b, q, 2, dtype, table=table, window=window)
    whole, whole_logs = call(b, q, 2, dtype, window=window)
    np.testing.assert_array_equal(got, whole)
    np.testing.assert_array_equal(logs, whole_logs)
    assert_close(got, expected(b, q, 2, d ** -0.5, True, window)[0], b)


def test_pages_of_the_window_are_still_looked_at(lib):
    """The page with the window's first key is used: an entry that is none is reported."""
    rng = np.random.default_rng(75)
    for n in (1, 70):
        b = Batch(rng, MESH1, [n], [500], 1, 64, 64, 16)
        q = draw(rng, (n, 64), "bf16")
        table = b.table.copy()
        table[0, (500 - n - 100 + 1) // 16] = -1
        call(b, q, 1, table=table, window=100, status=tsl._lib.DEV_ERR_INDEX)


@pytest.mark.parametrize("n", [1, 4, 80])
@pytest.mark.parametrize("e", [40, 100, 120])
def test_finite_numbers_in_hidden_keys(lib, n, e):
    """Steps and minima of 2^e in places that no query sees: before the window, beyond the length, in spare pages."""
    rng = np.random.default_rng(76)
    word = int((127 + e) << 7) * 0x10001  # step and minimum 2^e
    b = Batch(rng, MESH1, [n, n], [400, 333], 1, 128, 64, 16, poison=word)
    q = draw(rng, (2 * n, 2 * 128), "bf16")
    for s, kv in enumerate(b.kv_lens):
        for j in range(max(0, kv - n - 100 - 70), kv - n - 100 + 1):  # the first query sees keys from kv - n - 99
            rec = b.kv[s][j].copy()
            rec[..., 32:36] = word
            put(b, s, j, rec)
    got, _ = call(b, q, 2, window=100)
    assert_close(got, expected(b, q, 2, 128 ** -0.5, True, 100)[0], b)


@pytest.mark.parametrize("n,hq,e", [(5, 1, 10), (5, 1, 16), (5, 2, 16), (12, 4, 16), (80, 4, 16)])
def test_finite_numbers_in_keys_that_some_queries_see(lib, n, hq, e):
    """The last key holds steps and minima of 2^e and only the last query sees it: the others, which share a power of
    two with it, resolve their values to 2^-36 of the largest and do not notice."""
    rng = np.random.default_rng(79)
    b = Batch(rng, MESH1, [n, n], [n, 200], 1, 128, 64, 16)
    q = draw(rng, (2 * n, hq * 128), "bf16")
    want = expected(b, q, hq, 128 ** -0.5)[0]
    for s, kv in enumerate(b.kv_lens):
        rec = b.kv[s][kv - 1].copy()
        rec[..., 32:36] = ((127 + e) << 7) * 0x10001
        put(b, s, kv - 1, rec)
    got, _ = call(b, q, hq)
    keep = np.arange(2 * n) % n < n - 1
    b.q_lens = [n - 1, n - 1]
    assert_close(got[keep], want[keep], b)


@pytest.mark.parametrize("d,value_words", [(64, slice(17, 18)), (256, slice(68, 72))])
@pytest.mark.parametrize("word", [0x7F007F00, 0x00007F00, 0x7F803F80, 0x3F807F80])
def test_values_whose_sum_is_infinite_stay_with_their_key(lib, word, d, value_words):
    """The last key's value steps and minima are finite, minimum + 15 steps is not (or one of them is not): queries
    that do not see it do not notice."""
    rng = np.random.default_rng(77)
    for n in (5, 80):
        if n == 5 and word & 0x7F80 == 0x7F00:
            continue  # few rows share the scale of all finite steps, however large
        b = Batch(rng, MESH1, [n], [200], 1, d, 64, 16)
        q = draw(rng, (n, 2 * d), "bf16")
        want = expected(b, q, 2, d ** -0.5)[0]
        rec = b.kv[0][199].copy()
        rec[..., value_words] = word
        put(b, 0, 199, rec)
        got, _ = call(b, q, 2)
        b.q_lens = [n - 1]
        assert_close(got[:-1], want[:-1], b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,kv", [(10, 5), (90, 40), (70, 0), (3, 1)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, 2 ** 31, 2 ** 40 + 5])
def test_windows_beyond_every_key(lib, window, n, kv, dtype):
    """More queries than keys, so the first positions are negative, and windows near the end of 32 bits or beyond it:
    the results without a window."""
    rng = np.random.default_rng(85)
    b = Batch(rng, MESH1, [n, 2], [kv, 300], 1, 64, 64, 16)
    q = draw(rng, (n + 2, 2 * 64), dtype)
    got, logs = call(b, q, 2, dtype, window=window)
    whole, whole_logs = call(b, q, 2, dtype)
    np.testing.assert_array_equal(got, whole)
    np.testing.assert_array_equal(logs, whole_logs)
    if kv:
        assert_close(got, expected(b, q, 2, 0.125)[0], b)


@pytest.mark.parametrize("n,kv", [(10, 5), (90, 40)])
@pytest.mark.parametrize("window", [1, 3, 2 ** 20])
def test_windows_with_more_queries_than_keys(lib, window, n, kv):
    rng = np.random.default_rng(86)
    b = Batch(rng, MESH1, [n, 2], [kv, 300], 1, 64, 64, 16)
    q = draw(rng, (n + 2, 2 * 64), "bf16")
    got, _ = call(b, q, 2, window=window)
    assert_close(got, expected(b, q, 2, 0.125, True, window)[0], b)


@pytest.mark.parametrize("n", [1, 80])
def test_a_window_without_the_causal_mask(lib, n):
    """The window belongs to the causal mask: without that every key is seen."""
    rng = np.random.default_rng(78)
    b = Batch(rng, MESH1, [n], [200], 1, 64, 64, 16)
    q = draw(rng, (n, 64), "bf16")
    a = call(b, q, 1, causal=False, window=64)
    c = call(b, q, 1, causal=False)
    np.testing.assert_array_equal(a[0], c[0])
    assert_close(a[0], expected(b, q, 1, 0.125, False)[0], b)
