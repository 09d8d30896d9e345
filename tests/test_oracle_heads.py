"""Pins of the oracle for the operators on attention heads."""
import numpy as np
import pytest
import torch

from oracle import bf16, heads


def table(rows, rotary, theta=10000.0):
    a = np.arange(rows)[:, None] * theta ** (-np.arange(0, rotary, 2) / rotary)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [4, 12, 16])
def test_rotation_is_a_complex_product(rotary, interleaved):
    rng = np.random.default_rng(1)
    x, pos, cs = rng.standard_normal((5, 3, 16)), rng.integers(0, 40, 5), table(40, rotary)
    y = heads.rotate(x, cs, pos, interleaved)
    for t in range(5):
        for i in range(rotary // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
            z = (x[t, :, a] + 1j * x[t, :, b]) * complex(cs[pos[t], i], cs[pos[t], rotary // 2 + i])
            np.testing.assert_allclose(y[t, :, a], z.real, atol=1e-14)
            np.testing.assert_allclose(y[t, :, b], z.imag, atol=1e-14)
    np.testing.assert_array_equal(y[..., rotary:], x[..., rotary:])
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-6)
    np.testing.assert_allclose(heads.rotate(y, cs, pos, interleaved, back=True), x, atol=1e-6)


def test_positions_outside_the_table_give_zero_rows():
    y = heads.rotate(np.ones((3, 2, 8)), table(4, 8), np.array([4, -1, 3]), False)
    assert (y[:2] == 0).all() and (y[2] != 0).any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_backward_against_differences(interleaved):
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 2, 8)), 1 + 0.3 * rng.standard_normal(8)
    dy, pos, cs = rng.standard_normal((3, 2, 8)), np.array([0, 5, 2]), table(6, 4)
    dx, dw, _, _ = heads.norm_rope_backward(dy, x, w, cs, pos, interleaved, 1e-3)
    f = lambda x_, w_: (heads.norm_rope(x_, w_, cs, pos, interleaved, 1e-3) * dy).sum()  # noqa: E731
    h = 1e-6
    for idx in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[idx] = h
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - dx[idx]) < 1e-7
    for c in range(8):
        d = np.zeros_like(w)
        d[c] = h
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * h) - dw[c]) < 1e-7


def test_norm_is_torchs_rms_norm():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((4, 3, 32)), rng.standard_normal(32)
    y = torch.nn.functional.rms_norm(torch.from_numpy(x), (32,), torch.from_numpy(w), 1e-5).numpy()
    np.testing.assert_allclose(heads.norm_rope(x, w, None, None, False, 1e-5), y, atol=1e-13)


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (256, 32), (256, 64)])
def test_record_round_trip(d, group):
    rng = np.random.default_rng(d + group)
    k, v = (rng.standard_normal((7, 3, d)).astype(np.float32) * 10.0 ** rng.integers(-3, 4, (7, 3, 1)) for _ in range(2))
    k, v = k.astype(np.float32), v.astype(np.float32)
    rec = heads.pack(k, v, group)
    assert rec.shape == (7, 3, heads.record_words(d, group)) and rec.shape[-1] % 4 == 0
    k2, v2, ks, vs = heads.unpack(rec, d, group)
    for x, y, s in ((k, k2, ks), (v, v2, vs)):
        # half a step, the bf16 rounding of the minimum, and the step's at the top code
        rng_ = np.repeat(np.abs(x).reshape(7, 3, -1, group).max(-1), group, -1)
        assert (np.abs(x - y) <= s / 2 * 1.0001 + rng_ * 2.0 ** -8 + 15 * s * 2.0 ** -8).all()


def test_record_layout_by_hand():
    x = np.arange(64, dtype=np.float32) % 16  # minimum 0, step 1: the codes are the values
    rec = heads.pack(x[None], x[None] * 2 + 1, 64)[0]
    assert [int(w) for w in rec[:2]] == [0x76543210, 0xFEDCBA98]
    assert [int(w) for w in rec[8:10]] == [0x76543210, 0xFEDCBA98]
    assert int(rec[16]) == 0x00003F80 and int(rec[17]) == 0x3F804000  # (step 1, min 0), (step 2, min 1)
    assert (rec[18:] == 0).all()


def test_special_groups():
    x = np.zeros((6, 64), dtype=np.float32)
    x[0] = 3.0                       # constant
    x[1, 5] = np.nan
    x[2, 7] = np.inf
    x[3, 1], x[3, 2] = 3e38, -3e38   # the range overflows
    x[4, 1] = 1e-40                  # a step below the normal numbers
    x[5] = np.linspace(-1, 1, 64)
    rec = heads.pack(x, x, 64)
    k, _, s, _ = heads.unpack(rec, 64, 64)
    assert (k[0] == 3.0).all() and np.isnan(k[1:4]).all() and (k[4] == 0).all()
    assert (rec[:5, :8] == 0).all() and np.abs(k[5] - x[5]).max() < 0.08


def test_attention_against_torch():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((5, 16)), rng.standard_normal((23, 16)), rng.standard_normal((23, 16))
    for causal, window in ((False, 0), (True, 0), (True, 4)):
        out, lse, _, _ = heads.attention(q, k, v, 0.3, causal, window)
        s = torch.from_numpy(0.3 * q @ k.T)
        mask = torch.ones(5, 23, dtype=torch.bool)
        if causal:
            mask = mask.tril(18)
            if window:
                mask &= ~torch.ones(5, 23, dtype=torch.bool).tril(18 - window)
        s = s.masked_fill(~mask, float("-inf"))
        np.testing.assert_allclose(out, torch.softmax(s, -1).numpy() @ v, atol=1e-12)
        np.testing.assert_allclose(lse, torch.logsumexp(s, -1).numpy(), atol=1e-12)


def test_attention_rows_that_see_nothing():
    q, k = np.ones((4, 8)), np.ones((2, 8))  # 4 queries, 2 keys: the first two sit before the first key
    out, lse, _, _ = heads.attention(q, k, k, 1.0, True, 0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and (out[2:] == 1).all()
    out, lse, _, _ = heads.attention(q, k[:0], k[:0], 1.0, False, 0)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_planted_mistakes_show():
    rng = np.random.default_rng(6)
    x, pos, cs = rng.standard_normal((4, 2, 16)), np.arange(4) + 3, table(9, 16)
    right = heads.rotate(x, cs, pos, False)
    assert np.abs(heads.rotate(x, cs, pos, True) - right).max() > 0.1          # the other pairing
    assert np.abs(heads.rotate(x, cs, pos + 1, False) - right).max() > 0.1     # one position off
    assert np.abs(heads.rotate(x, cs, pos, False, back=True) - right).max() > 0.1
    k = rng.standard_normal((9, 16))
    a = heads.attention(x[:, 0], k, k, 0.25, True, 0)[0]
    assert np.abs(heads.attention(x[:, 0], k, k, 0.25, False, 0)[0] - a).max() > 0.01
    assert np.abs(heads.attention(x[:, 0], k, k, 0.25, True, 3)[0] - a).max() > 0.01
    assert bf16.widen(bf16.round_rne(np.float32([1.0])))[0] == 1.0
