"""Infinities and NaN among the channels of a head, in the head norms with rotation: where the definition's result
is finite the kernels' is, and infinities and NaN are those of the definition."""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from oracle import heads

from heads_helpers import draw, full, ints, sharded, table, whole

pytestmark = pytest.mark.gpu
EPS = 1e-6


def assert_same_kind(got, want, dtype):
    """NaN where NaN, infinities equal, the rest within the output's rounding and that of fp32 sums."""
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(np.isposinf(got), np.isposinf(want))
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want))
    f = np.isfinite(want)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    assert (np.abs(got[f] - want[f]) <= half * np.abs(want[f]) + 2.0 ** -18 * 16).all()  # inputs are below 8


def operands(d, rotary, dtype, seed):
    rng = np.random.default_rng(seed)
    mesh = tsl.DeviceMesh((2,), ("tp",))
    x = np.clip(draw(rng, (7, 4 * d), dtype), -4, 4)
    x[1, 3], x[2, d + rotary + 1], x[3, d - 1], x[4, 3 * d + rotary // 2] = np.inf, -np.inf, np.nan, np.inf
    x[5, 2 * d:2 * d + 3] = (np.inf, -np.inf, np.nan)
    x[6, rotary:d] = np.inf
    pos = np.array([5, 1, 0, 7, 2, 11, 3])
    return mesh, rng, x, table(12, rotary), pos


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 32), (128, 64), (128, 128), (256, 64), (80, 16), (48, 36)])
def test_rotation_alone(lib, d, rotary, interleaved, dtype):
    mesh, rng, x, cs, pos = operands(d, min(rotary, d - 2), dtype, 80) if rotary == d else operands(d, rotary, dtype, 80)
    cs = table(12, rotary)
    out, _ = tsl.tp_qk_norm_rope(sharded(x, mesh, dtype), cos_sin=whole(cs, mesh), positions=ints(pos, mesh), head_dim=d,
                                 interleaved=interleaved)
    with np.errstate(all="ignore"):
        want = heads.norm_rope(x.reshape(7, 4, d), None, cs, pos, interleaved, EPS)
    assert_same_kind(full(out).reshape(7, 4, d), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 32), (128, 64), (256, 64), (80, 16)])
def test_norm_and_rotation(lib, d, rotary, interleaved, dtype):
    mesh, rng, x, cs, pos = operands(d, rotary, dtype, 81)
    w = 1 + 0.1 * rng.standard_normal(d).astype(np.float32)
    out, _ = tsl.tp_qk_norm_rope(sharded(x, mesh, dtype), None, whole(w, mesh), cos_sin=whole(cs, mesh),
                                 positions=ints(pos, mesh), head_dim=d, interleaved=interleaved, eps=EPS)
    with np.errstate(all="ignore"):
        want = heads.norm_rope(x.reshape(7, 4, d), w, cs, pos, interleaved, EPS)
    assert_same_kind(full(out).reshape(7, 4, d), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_without_rotation(lib, dtype):
    mesh, rng, x, _, _ = operands(128, 64, dtype, 82)
    w = 1 + 0.1 * rng.standard_normal(128).astype(np.float32)
    out, _ = tsl.tp_qk_norm_rope(sharded(x, mesh, dtype), None, whole(w, mesh), head_dim=128, eps=EPS)
    with np.errstate(all="ignore"):
        want = heads.norm_rope(x.reshape(7, 4, 128), w, None, None, False, EPS)
    assert_same_kind(full(out).reshape(7, 4, 128), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 32), (128, 64), (256, 64), (80, 16)])
def test_gradients_of_the_rotation_alone(lib, d, rotary, interleaved, dtype):
    mesh, rng, dy, cs, pos = operands(d, rotary, dtype, 83)
    x = draw(rng, dy.shape, dtype)
    dq = tsl.tp_qk_norm_rope_backward(sharded(dy, mesh, dtype), None, sharded(x, mesh, dtype), cos_sin=whole(cs, mesh),
                                      positions=ints(pos, mesh), head_dim=d, interleaved=interleaved)[0]
    with np.errstate(all="ignore"):
        want = heads.norm_rope_backward(dy.reshape(7, 4, d), x.reshape(7, 4, d), None, cs, pos, interleaved, EPS)[0]
    assert_same_kind(full(dq).reshape(7, 4, d), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_weight_gradients_keep_their_channels(lib, interleaved, dtype):
    """An infinity in a gradient's unrotated channel reaches that channel of the weight's gradient alone."""
    rng = np.random.default_rng(84)
    mesh, d, rotary = tsl.DeviceMesh((2,), ("tp",)), 128, 64
    dy, x = draw(rng, (7, 4 * d), dtype), draw(rng, (7, 4 * d), dtype)
    dy[2, d + 100], dy[5, 127] = np.inf, -np.inf
    cs, pos = table(12, rotary), np.arange(7) + 1
    w = 1 + 0.1 * rng.standard_normal(d).astype(np.float32)
    dw = tsl.tp_qk_norm_rope_backward(sharded(dy, mesh, dtype), None, sharded(x, mesh, dtype), None, whole(w, mesh),
                                      cos_sin=whole(cs, mesh), positions=ints(pos, mesh), head_dim=d,
                                      interleaved=interleaved, eps=EPS)[2]
    got = dw.slots[0].double().cpu().numpy()
    with np.errstate(all="ignore"):
        _, want, _, size = heads.norm_rope_backward(dy.reshape(7, 4, d), x.reshape(7, 4, d), w, cs, pos, interleaved, EPS)
    f = np.isfinite(want)
    np.testing.assert_array_equal(np.isfinite(got), f)
    assert (np.abs(got[f] - want[f]) <= 2.0 ** -16 * size[f]).all()
