"""Pins of the 64-bit restatements of block norms, dropout and log probabilities."""
import numpy as np
import pytest

from oracle import decoder


def test_philox_known_words():
    """The published test vectors of the generator (all zeros, all ones, digits of pi)."""
    assert decoder.philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert decoder.philox([0xffffffff] * 4, [0xffffffff] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert decoder.philox([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_mask_is_the_generator():
    rng = [1, -2, 3, -4]
    m = decoder.keep_mask(rng, 3, 7, 0.5)
    for t in range(3):
        for c in range(7):
            i = 7 * t + c
            w = decoder.philox([i // 4, 0, 3, 2 ** 32 - 4], [1, 2 ** 32 - 2])[i % 4]
            assert m[t, c] == (w >= 2 ** 31)
    assert np.array_equal(decoder.keep_mask(rng, 2, 7, 0.5, first=1), m[1:])
    assert decoder.keep_mask(rng, 4, 5, 0.0).all()
    big = decoder.keep_mask(rng, 1, 8, 0.5, first=(1 << 35) // 8)
    assert [w >= 2 ** 31 for w in decoder.philox([0, 2, 3, 2 ** 32 - 4], [1, 2 ** 32 - 2])] == list(big[0, :4])


@pytest.mark.parametrize("post,gate,pre,res,drop", [
    (1, 0, 1, 1, 0), (1, 3, 1, 1, 1), (0, 1, 1, 1, 1), (0, 0, 0, 1, 1), (1, 1, 0, 0, 0), (0, 0, 1, 0, 0)])
def test_block_gradients_by_differences(post, gate, pre, res, drop):
    rng = np.random.default_rng(post + 2 * gate + 16 * pre)
    t, n, p = 6, 5, 0.5
    v = {"x": [rng.standard_normal((t, n)) for _ in range(2)], "r": rng.standard_normal((t, n)) if res else None,
         "post": 1 + rng.standard_normal(n) if post else None, "pre": 1 + rng.standard_normal(n) if pre else None,
         "gate": rng.standard_normal((gate, n) if gate > 1 else (n,)) if gate else None}
    keep = decoder.keep_mask([5, 6, 7, 8], t, n, p) if drop else None
    dh, dy = rng.standard_normal((t, n)), rng.standard_normal((t, n)) if pre else None

    def block():
        return decoder.Block(v["x"], v["r"], v["post"], v["gate"], v["pre"], 1e-3, 0.7, keep, p)

    def loss():
        b = block()
        return (b.h * dh).sum() + ((b.y * dy).sum() if pre else 0.0)

    grads = block().backward(dh, dy)
    for name, a in (("dx", v["x"][1]), ("dr", v["r"]), ("dpost", v["post"]), ("dgate", v["gate"]), ("dpre", v["pre"])):
        if a is None:
            continue
        g, mag = grads[name]
        assert g.shape == a.shape and (np.abs(g) <= mag * (1 + 1e-12) + 1e-300).all()
        for i in np.ndindex(a.shape):
            old, step = a[i], 1e-5
            a[i] = old + step
            up = loss()
            a[i] = old - step
            down = loss()
            a[i] = old
            assert abs((up - down) / (2 * step) - g[i]) <= 1e-6 * (1 + abs(g[i])), (name, i)


def test_log_probs_closed_forms():
    logp, lse, ent = decoder.log_probs(np.zeros((2, 8)))
    assert np.allclose(logp, -np.log(8)) and np.allclose(lse, np.log(8)) and np.allclose(ent, np.log(8))
    z = np.array([[0.0, -np.inf, np.log(3.0)], [-np.inf] * 3, [1.0, np.nan, 2.0], [np.inf, 0.0, 1.0]])
    logp, lse, ent = decoder.log_probs(z)
    assert np.allclose(np.exp(logp[0]), [0.25, 0, 0.75]) and np.isclose(lse[0], np.log(4.0))
    assert np.isclose(ent[0], 0.25 * np.log(4) + 0.75 * np.log(4 / 3))
    assert np.isneginf(logp[1]).all() and np.isneginf(lse[1]) and ent[1] == 0
    assert np.isnan(logp[2]).all() and np.isnan(ent[2]) and np.isnan(logp[3, 0])
    assert decoder.top(np.array([[1.0, 2.0, 2.0, 0.0], [-0.0, 0.0, np.nan, -np.inf]]), 3).tolist() == \
        [[1, 2, 0], [2, 0, 1]]


def test_log_probs_gradient_by_differences():
    rng = np.random.default_rng(3)
    z, ids = 2 * rng.standard_normal((4, 9)), np.array([[1, 1], [8, 0], [3, -100], [-100, -100]])
    dlp, dent, s = rng.standard_normal((4, 2)), rng.standard_normal(4), 1.3

    def loss(x):
        logp, _, ent = decoder.log_probs(x, s)
        return sum(dlp[i, c] * logp[i, ids[i, c]] for i in range(4) for c in range(2) if ids[i, c] >= 0) + \
            (ent * dent).sum()

    _, lse, ent = decoder.log_probs(z, s)
    g, mag = decoder.log_probs_backward(z, ids, dlp, lse, s, dent, ent)
    assert (np.abs(g) <= mag + 1e-15).all()
    for i in np.ndindex(z.shape):
        d = np.zeros_like(z)
        d[i] = 1e-5
        assert abs((loss(z + d) - loss(z - d)) / 2e-5 - g[i]) < 1e-7
