"""Block norms under weights, gates, residuals and gradients that are not finite: what the formula keeps finite stays so."""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from heads_helpers import DT, draw, strided, whole
from oracle import decoder
from test_gpu_block_norm import Case

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
R = tsl.Replicate()
INF, NAN = float("inf"), float("nan")


def same(a, e, tol):
    with np.errstate(invalid="ignore"):
        ok = (a == e) | (np.isnan(a) & np.isnan(e)) | (np.abs(a - e) <= tol)
    assert ok.all(), [(i.tolist(), a[tuple(i)], e[tuple(i)]) for i in np.argwhere(~ok)[:5]]


@pytest.mark.parametrize("dtype,stream", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("t", [3, 320])  # (few tokens: a vector a thread; many: rows read ahead)
@pytest.mark.parametrize("n,offset", [(9, 0), (40, 0), (1000, 0), (1152, 0), (1160, 1), (2568, 0), (4096, 0)])
def test_weights_of_the_first_channels(n, offset, t, dtype, stream):
    """An infinite or NaN weight of channels 0 to 7: channel counts with and without threads that have no last vector.

    Where dropout drops the channel, the row is that of a finite weight; where h is infinite, y is 0 in the others."""
    rng = np.random.default_rng(n)
    mesh = tsl.DeviceMesh((1,), ("tp",))
    x, r = draw(rng, (t, n), dtype), draw(rng, (t, n), stream)
    weights = {name: draw(rng, (n,), "fp32") for name in ("post", "gate", "pre")}
    seed = rng.integers(-2 ** 31, 2 ** 31, 4)
    keep = decoder.keep_mask(seed, t, n, 0.5)

    def rows(v, d):
        return tsl.DTensor([strided(torch.from_numpy(v).cuda().to(DT[d]), 0, offset)], mesh, [R], (t, n), DT[d])

    xd, rd, seed = rows(x, dtype), rows(r, stream), whole(torch.tensor(seed, dtype=torch.int32), mesh)
    for bad, channel in ((INF, 0), (NAN, 7), (-INF, 3)):
        for which in weights:
            w = {name: v.copy() for name, v in weights.items()}
            w[which][channel] = bad
            h, y = tsl.tp_block_norm(xd, rd, *(whole(v, mesh, torch.float32) for v in w.values()), dropout=0.5, rng=seed)
            h, y = h.slots[0].double().cpu().numpy(), y.slots[0].double().cpu().numpy()
            with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                e = decoder.Block([x], r, *w.values(), keep=keep, p=0.5)
                f = np.isfinite(e.h).all(1)
                # 20 roundings and two norms' sums, as many additions as a thread makes and 16 each; a norm's is of h,
                # whose terms may cancel, and is the worst row's ratio of magnitudes to values off
                ratio = ((e.abs_h[f] ** 2).sum(1) / (e.h[f] ** 2).sum(1)).max(initial=1.0)
                k = (20 + 2 * (-(-n // 32) + 16)) * ratio * 2.0 ** -24
                same(h, e.h, HALF[stream] * np.abs(e.h) + k * e.abs_h + 1e-37)
                same(y[f], e.y[f], HALF[dtype] * np.abs(e.y[f]) + k * e.abs_y[f] + 1e-37)
            if which != "pre":
                assert np.array_equal(f, ~keep[:, channel])
                others = np.arange(n) != channel
                assert np.isnan(y[~f][:, channel]).all()
                assert (np.isnan(y[~f]) if np.isnan(bad) else y[~f][:, others] == 0).all()


def check_gradients(case, dh):
    """Those of a case whose operands hold what is not finite, in all places where the formula has a value."""
    with np.errstate(invalid="ignore", over="ignore"):
        ref = case.ref.backward(dh, case.dy)
        for name, d in zip(("dx", "dr", "dpost", "dgate", "dpre"), case.backward()):
            if d is None:
                continue
            e, mag = ref[name]
            half = HALF[case.dtype if name == "dx" else case.stream if name == "dr" else case.wdtype]
            # as for finite operands: twice the forward's roundings, and sums over tokens
            k = 2 * case.k + (-(-case.t // 152) + 40) * 2.0 ** -24
            same(d.slots[0].double().cpu().numpy(), e, half * np.abs(e) + k * mag + 1e-37)
            assert np.isfinite(e).all() or name == "dr"


@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("n,dtype", [(1024, "bf16"), (1001, "fp32"), (4096, "bf16"), (12288, "bf16"), (20000, "bf16")])
def test_gradients_do_not_meet_a_residual_without_a_norm_of_it(n, dtype, drop):
    """Without pre_weight no gradient depends on h, whatever the residual holds."""
    case = Case(31, 9, n, dtype=dtype, pre=False, gate=3, drop=drop)
    for row, v in ((2, INF), (4, NAN), (7, -INF)):
        case.r.slots[0][row, n // 2:] = v
    check_gradients(case, case.dh)


@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("n,dtype", [(1024, "bf16"), (1001, "fp32"), (4096, "bf16"), (12288, "bf16"), (20000, "bf16")])
def test_gradients_of_dropped_elements_reach_the_residual_alone(n, dtype, pre):
    """Infinities and NaN of dh in dropped places: the residual's gradient has them there, the others stay finite."""
    case = Case(32, 9, n, dtype=dtype, pre=pre, gate=3, drop=0.5)
    dh = case.dh.copy()
    for row, v in ((1, INF), (4, NAN), (8, -INF)):
        dh[row, ~case.ref.keep[row]] = v
    case.gh.slots[0].copy_(torch.from_numpy(dh))
    check_gradients(case, dh)
