"""The check of attention results rejects what is wrong (on the CPU, mistakes planted in the oracle's results)."""
import numpy as np
import pytest

from oracle import bf16, heads

from attention_close import Rejected, check

CASES = [  # d, group, keys, queries, dtype, many rows: the long cases of the GPU tests and short ones
    (128, 64, 20000, 1, "bf16", False), (128, 64, 9000, 3, "bf16", True), (256, 64, 5000, 3, "bf16", True),
    (64, 32, 9000, 2, "fp32", False), (128, 64, 1000, 1, "bf16", False), (64, 64, 70, 2, "bf16", False),
    (64, 64, 64, 64, "bf16", True)]


def result(d, group, kv, n, dtype):
    rng = np.random.default_rng(60)
    size, offset = np.exp(0.4 * rng.standard_normal((1, d))), 0.5 * rng.standard_normal((1, d))
    k = (rng.standard_normal((kv, 1, d)) * size + offset).astype(np.float32)
    rec = heads.pack(k, rng.standard_normal((kv, 1, d)).astype(np.float32), group)
    q = rng.standard_normal((n, 1, d))
    q = bf16.widen64(bf16.round_rne(q)) if dtype == "bf16" else np.float64(np.float32(q))
    return q, rec


def rounded(x, dtype):
    return bf16.widen64(bf16.round_rne(x)) if dtype == "bf16" else np.float64(np.float32(x))


def attend(q, rec, d, group, keep=None, scale=None):
    k, v, _, _ = heads.unpack(rec, d, group)
    k, v = k[:, 0], v[:, 0]
    s = (d ** -0.5 if scale is None else scale) * (q[:, 0] @ k.T)
    s[~heads.visible(len(q), len(k), True, 0)] = -np.inf
    if keep is not None:
        s[:, ~keep] = -np.inf
    top = s.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):  # a row without keys gets NaN, which is wrong too
        p = np.exp(s - top)
        return (p @ v / p.sum(-1, keepdims=True))[:, None], (top[:, 0] + np.log(p.sum(-1)))[:, None]


@pytest.mark.parametrize("d,group,kv,n,dtype,many", CASES)
def test_right_results_pass_and_wrong_ones_do_not(d, group, kv, n, dtype, many):
    q, rec = result(d, group, kv, n, dtype)
    args = (q, rec, d, group, 1, d ** -0.5, dtype, True, 0, many)
    y, lse = attend(q, rec, d, group)
    check(rounded(y, dtype), lse, *args)
    wrong = {"zeros": (np.zeros_like(y), lse), "the mean of all values": (np.broadcast_to(
        heads.unpack(rec, d, group)[1].mean(0), y.shape), lse), "no log": (y, lse * 0)}
    j = np.arange(kv)
    piece = max(1, kv // 7)  # what one of several CTAs adds; a tile of a warp; a key
    for a, b in ((0, piece), (3 * piece, 4 * piece), (kv - piece, kv), (kv // 2, kv // 2 + 64)):
        if b - a < kv // 2:
            keep = ~((j >= a) & (j < b))
            part, part_lse = attend(q, rec, d, group, keep)
            wrong[f"without keys {a} to {b}"] = (part, part_lse)
            wrong[f"without the values of keys {a} to {b}"] = (part * np.exp(part_lse - lse)[..., None], lse)
    wrong["a scale 1 % off"] = attend(q, rec, d, group, scale=1.01 * d ** -0.5)
    for what, (bad, bad_lse) in wrong.items():
        with pytest.raises(Rejected):
            check(rounded(bad, dtype), bad_lse, *args)
            print(what)
        if what not in ("no log", "a scale 1 % off"):
            with pytest.raises(Rejected):  # by the output alone
                check(rounded(bad, dtype), None, *args)
                print(what, "(output)")


def test_fp16_operands_pass():
    """The prompt kernel's roundings, each to 11 bits, in numpy: within the bound; in 8 bits they are not."""
    for bits, ok in ((11, True), (8, False)):
        def cut(x):
            m, e = np.frexp(x)
            return np.ldexp(np.rint(m * 2.0 ** bits) / 2.0 ** bits, e)
        d, group, kv = 64, 64, 300
        q, rec = result(d, group, kv, 64, "bf16")
        k, v, _, _ = heads.unpack(rec, d, group)
        s = d ** -0.5 * (q[:, 0] @ cut(k[:, 0]).T)
        s[~heads.visible(64, kv, True, 0)] = -np.inf
        p = np.exp(s - s.max(-1, keepdims=True))
        y = (cut(p) @ cut(v[:, 0]) / p.sum(-1, keepdims=True))[:, None]
        args = (q, rec, d, group, 1, d ** -0.5, "fp32" if not ok else "bf16", True, 0, True)
        if ok:
            check(rounded(y, "bf16"), None, *args)
        else:
            with pytest.raises(Rejected):
                check(y, None, *args)
