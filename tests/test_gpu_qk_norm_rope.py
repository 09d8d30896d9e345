"""GPU parity of dt_tp_qk_norm_rope and its backward against the fp64 oracle.

Tolerances, derived from the arithmetic: a row's sum of squares carries at
most 2^-20 (20 fp32 roundings of positive terms), its root half of that, and
five more roundings reach an output: 2^-19 of the pair's magnitude, plus half
an ulp of the output's type.  dx: 2^-17 of the sum of its terms' magnitudes
(two sums of D terms).  dw: at most 512 additions in a chain, 2^-15 of the
sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from oracle import heads

from heads_helpers import DT, draw, full, ints, sharded, table, whole

pytestmark = pytest.mark.gpu
EPS = 1e-6
HALF_ULP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -23}

# tokens, q heads, k heads, head_dim, rotary, parts, dtype, interleaved
CASES = [
    (1, 4, 1, 128, 128, 1, "bf16", False),
    (37, 8, 2, 128, 128, 2, "bf16", False),
    (37, 8, 2, 128, 128, 2, "bf16", True),
    (19, 4, 4, 64, 32, 4, "fp32", True),
    (19, 4, 4, 64, 32, 1, "fp32", False),
    (8, 28, 4, 80, 80, 4, "bf16", False),     # 5 lanes a head
    (8, 6, 2, 256, 64, 2, "bf16", False),
    (5, 3, 1, 512, 512, 1, "fp32", True),
    (7, 5, 1, 16, 16, 1, "bf16", False),
    (23, 4, 2, 100, 20, 2, "bf16", False),    # no multiple of 16: an element per lane
    (23, 4, 2, 33, 6, 1, "fp32", True),       # an odd width
    (3, 2, 1, 1000, 1000, 1, "bf16", False),
    (700, 16, 16, 128, 128, 4, "bf16", False),
    (4100, 32, 8, 128, 128, 4, "bf16", False),  # two heads per lane
    (2500, 24, 8, 64, 64, 1, "fp32", False),
]


def make(case, seed, extra=0, offset=0, weight_dtype=torch.float32):
    t, hq, hk, d, rot, p, dtype, inter = case
    rng = np.random.default_rng(seed)
    mesh = tsl.DeviceMesh((p,), ("tp",))
    scale = np.exp(rng.standard_normal((t, 1)) * 0.5)
    q, k = draw(rng, (t, hq * d), dtype) * 1.0, draw(rng, (t, hk * d), dtype)
    q = draw(rng, (t, hq * d), dtype, scale)
    w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(d)).to(weight_dtype) for _ in range(2)]
    cs, pos = table(t + 9, rot), rng.integers(0, t + 9, t)
    ops = dict(q=sharded(q, mesh, dtype, extra, offset), k=sharded(k, mesh, dtype, extra, offset),
               q_weight=whole(w[0], mesh), k_weight=whole(w[1], mesh), cos_sin=whole(cs, mesh),
               positions=ints(pos, mesh))
    return mesh, rng, (q, k), [x.double().numpy() for x in w], cs, pos, ops


def check_forward(case, out, xs, ws, cs, pos):
    t, hq, hk, d, rot, p, dtype, inter = case
    for y, x, w, h in zip(out, xs, ws, (hq, hk)):
        if x is None:
            continue
        e = heads.norm_rope(x.reshape(t, h, d), w, cs, pos, inter, EPS)
        mag = np.abs(e).copy()
        if cs is not None:
            ia, ib = heads.pairs_of(rot, inter)
            mag[..., ia] = mag[..., ib] = np.hypot(e[..., ia], e[..., ib])
        err = np.abs(full(y).reshape(t, h, d) - e)
        assert (err <= 2.0 ** -19 * mag + HALF_ULP[dtype] * np.abs(e) + 1e-37).all(), err.max()


@pytest.mark.parametrize("case", CASES)
def test_forward(lib, case):
    _, _, xs, ws, cs, pos, ops = make(case, 11)
    out = tsl.tp_qk_norm_rope(**ops, head_dim=case[3], eps=EPS, interleaved=case[7])
    assert tsl.read_device_status() == 0
    check_forward(case, out, xs, ws, cs, pos)


def check_backward(case, got, dys, xs, ws, cs, pos):
    t, hq, hk, d, rot, p, dtype, inter = case
    for i, h in enumerate((hq, hk)):
        dx, dw, size, wsize = heads.norm_rope_backward(dys[i].reshape(t, h, d), xs[i].reshape(t, h, d), ws[i], cs, pos,
                                                       inter, EPS)
        err = np.abs(full(got[i]).reshape(t, h, d) - dx)
        # a rotated gradient's error is relative to its pair; 2^-17 leaves room for that
        big = size.max(-1, keepdims=True)
        assert (err <= 2.0 ** -17 * np.maximum(size, big / 8) + HALF_ULP[dtype] * np.abs(dx) + 1e-37).all(), err.max()
        if ws[i] is not None:
            gw = got[2 + i].slots[0]
            ulp = 2.0 ** -8 if gw.dtype == torch.bfloat16 else 0.0
            err = np.abs(gw.double().cpu().numpy() - dw)
            assert (err <= 2.0 ** -15 * wsize + ulp * np.abs(dw)).all(), (err / wsize).max()


@pytest.mark.parametrize("case", CASES)
def test_backward(lib, case):
    mesh, rng, xs, ws, cs, pos, ops = make(case, 12)
    dys = [draw(rng, x.shape, case[6]) for x in xs]
    dyd = [sharded(y, mesh, case[6]) for y in dys]
    kw = dict(head_dim=case[3], eps=EPS, interleaved=case[7])
    got = tsl.tp_qk_norm_rope_backward(*dyd, **ops, **kw)
    assert tsl.read_device_status() == 0
    check_backward(case, got, dys, xs, ws, cs, pos)
    again = tsl.tp_qk_norm_rope_backward(*dyd, **ops, **kw)
    for a, b in zip(got, again):
        assert all(torch.equal(s, u) for s, u in zip(a.slots, b.slots))


@pytest.mark.parametrize("wd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("extra,offset", [(8, 0), (24, 8), (3, 0), (0, 1), (5, 3)])
def test_strides_and_offsets(lib, extra, offset, wd):
    """Pitched views, and rows off the 16-byte boundaries (the kernel of one element per lane)."""
    case = (13, 4, 2, 64, 64, 2, "bf16", False)
    mesh, rng, xs, ws, cs, pos, ops = make(case, 13, extra, offset, wd)
    out = [sharded(np.zeros_like(x), mesh, "bf16", extra, offset) for x in xs]
    tsl.tp_qk_norm_rope(**ops, head_dim=64, eps=EPS, out=tuple(out))
    check_forward(case, out, xs, ws, cs, pos)
    for o in out:  # the pitch's gap is untouched
        s = o.slots[0]
        gap = s.as_strided((s.shape[0], extra), s.stride(), s.storage_offset() + s.shape[1]) if extra else None
        assert gap is None or (gap[:-1] == 7).all()
    dys = [draw(rng, x.shape, "bf16") for x in xs]
    got = tsl.tp_qk_norm_rope_backward(*[sharded(y, mesh, "bf16", extra, offset) for y in dys], **ops, head_dim=64,
                                       eps=EPS)
    check_backward(case, got, dys, xs, ws, cs, pos)


@pytest.mark.parametrize("d", [64, 36])
@pytest.mark.parametrize("drop", ["k", "weights", "q_weight", "rotation"])
def test_optional_operands(lib, d, drop):
    case = (9, 4, 2, d, d, 2, "bf16", False)
    mesh, rng, xs, ws, cs, pos, ops = make(case, 14)
    xs, ws = list(xs), list(ws)
    if drop == "k":
        ops.update(k=None, k_weight=None)
        xs[1] = ws[1] = None
    elif drop == "rotation":
        ops.update(cos_sin=None, positions=None)
        cs = None
    else:
        ops.update(q_weight=None)
        ws[0] = None
        if drop == "weights":
            ops.update(k_weight=None)
            ws[1] = None
    out = tsl.tp_qk_norm_rope(**ops, head_dim=d, eps=EPS)
    check_forward(case, out, xs, ws, cs, pos)
    n = 1 if drop == "k" else 2
    dys = [draw(rng, x.shape, "bf16") for x in xs[:n]]
    dyd = [sharded(y, mesh, "bf16") for y in dys] + [None] * (2 - n)
    got = tsl.tp_qk_norm_rope_backward(*dyd, **ops, head_dim=d, eps=EPS)
    if drop == "k":
        assert got[1] is None and got[3] is None
        case, got, xs, ws = (9, 4, 0, d, d, 2, "bf16", False), got, xs[:1], ws[:1]
        dx, dw, size, wsize = heads.norm_rope_backward(dys[0].reshape(9, 4, d), xs[0].reshape(9, 4, d), ws[0], cs, pos,
                                                       False, EPS)
        assert (np.abs(got[2].slots[0].double().cpu().numpy() - dw) <= 2.0 ** -15 * wsize).all()
    else:
        check_backward(case, got, dys, xs, ws, cs, pos)


@pytest.mark.parametrize("d", [128, 40])
def test_positions_outside_the_table(lib, d):
    case = (6, 4, 2, d, d, 2, "bf16", False)
    mesh, rng, xs, ws, cs, pos, ops = make(case, 15)
    pos = pos.copy()
    pos[1], pos[4] = -1, cs.shape[0]
    ops["positions"] = ints(pos, mesh)
    out = tsl.tp_qk_norm_rope(**ops, head_dim=d, eps=EPS)
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX
    check_forward(case, out, xs, ws, cs, pos)
    assert (full(out[0])[[1, 4]] == 0).all()
    dys = [draw(rng, x.shape, "bf16") for x in xs]
    got = tsl.tp_qk_norm_rope_backward(*[sharded(y, mesh, "bf16") for y in dys], **ops, head_dim=d, eps=EPS)
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX
    check_backward(case, got, dys, xs, ws, cs, pos)


@pytest.mark.parametrize("case", [
    (6001, 13, 3, 64, 64, 1, "bf16", False),
    (5000, 5, 3, 80, 80, 1, "bf16", False),
    (3000, 9, 9, 256, 64, 1, "bf16", True),
    (2001, 11, 2, 128, 96, 1, "fp32", False),
])
def test_many_tokens(lib, case):
    """Several units a warp, with heads that do not fill the last block."""
    test_forward(lib, case)
    test_backward(lib, case)


@pytest.mark.parametrize("d", [128, 40])
def test_left_out_tokens_may_hold_nan(lib, d):
    """Tokens without a position add nothing to the weights' gradients, whatever they hold."""
    case = (6, 5, 3, d, d, 1, "bf16", False)
    mesh, rng, xs, ws, cs, pos, ops = make(case, 21)
    pos = pos.copy()
    pos[1], pos[4] = -1, cs.shape[0]
    ops["positions"] = ints(pos, mesh)
    dys = [draw(rng, x.shape, "bf16") for x in xs]
    dyd = [sharded(y, mesh, "bf16") for y in dys]
    for n in "qk":
        ops[n].slots[0][1] = float("nan")
        ops[n].slots[0][4] = float("inf")
    for y in dyd:
        y.slots[0][4] = float("nan")
    for x in xs + tuple(dys):
        x[[1, 4]] = 0
    got = tsl.tp_qk_norm_rope_backward(*dyd, **ops, head_dim=d, eps=EPS)
    assert tsl.read_device_status() == tsl._lib.DEV_ERR_INDEX
    check_backward(case, got, dys, xs, ws, cs, pos)


def test_gradient_against_differences(lib):
    """fp32, a small head: central differences of the kernel's own forward."""
    case = (2, 2, 1, 16, 8, 1, "fp32", False)
    mesh, rng, xs, ws, cs, pos, ops = make(case, 16)
    dys = [draw(rng, x.shape, "fp32") for x in xs]
    kw = dict(head_dim=16, eps=EPS)
    got = tsl.tp_qk_norm_rope_backward(*[sharded(y, mesh, "fp32") for y in dys], **ops, **kw)

    def loss():
        return sum((full(o) * y).sum() for o, y in zip(tsl.tp_qk_norm_rope(**ops, **kw), dys))

    h = 2.0 ** -7  # truncation h^2 |f'''| / 6 and rounding 2^-22 |f| / h are both below 1e-3
    for name, g in (("q", got[0]), ("k", got[1]), ("q_weight", got[2]), ("k_weight", got[3])):
        flat, gf = ops[name].slots[0].view(-1), g.slots[0].view(-1)
        for i in range(0, flat.numel(), 3):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            down = loss()
            flat[i] = keep
            assert abs((up - down) / (2 * h) - gf[i].item()) < 2e-3


def test_shared_key_heads_replicate_and_3d(lib):
    """k Replicate on tp beside a sharded q, and activations with two leading dims."""
    rng = np.random.default_rng(17)
    mesh = tsl.DeviceMesh((4,), ("tp",))
    q, k = draw(rng, (10, 8 * 64), "bf16"), draw(rng, (10, 64), "bf16")
    cs, pos = table(10, 64), np.arange(10)
    w = whole(np.ones(64, np.float32), mesh)
    q2 = sharded(q, mesh, "bf16")
    q3 = tsl.DTensor([s.view(2, 5, -1) for s in q2.slots], mesh, [tsl.Shard(2)], (2, 5, 8 * 64), torch.bfloat16)
    k3 = tsl.DTensor([sharded(k, mesh, "bf16", replicate=True).slots[0].view(2, 5, -1)], mesh, [tsl.Replicate()],
                     (2, 5, 64), torch.bfloat16)
    pos3 = tsl.DTensor([torch.tensor(pos, dtype=torch.int32).view(2, 5).cuda()], mesh, [tsl.Replicate()], (2, 5),
                       torch.int32)
    qo, ko = tsl.tp_qk_norm_rope(q3, k3, w, w, whole(cs, mesh), pos3, head_dim=64, eps=EPS)
    assert qo.gshape == (2, 5, 512) and len(ko.slots) == 1
    case = (10, 8, 1, 64, 64, 4, "bf16", False)
    flat = [tsl.DTensor([s.view(10, -1) for s in o.slots], mesh, o.placements[:0] + (pl,), (10, n), torch.bfloat16)
            for o, pl, n in ((qo, tsl.Shard(1), 512), (ko, tsl.Replicate(), 64))]
    check_forward(case, flat, (q, k), [np.ones(64)] * 2, cs, pos)


def test_on_another_stream_and_in_a_graph(lib):
    case = (33, 4, 2, 64, 64, 2, "bf16", False)
    mesh, rng, xs, ws, cs, pos, ops = make(case, 18)
    out = tuple(sharded(np.zeros_like(x), mesh, "bf16") for x in xs)
    kw = dict(head_dim=64, eps=EPS, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tsl.tp_qk_norm_rope(**ops, **kw)
    s.synchronize()
    check_forward(case, out, xs, ws, cs, pos)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsl.tp_qk_norm_rope(**ops, **kw)
    x2 = [draw(rng, x.shape, "bf16") for x in xs]
    for name, x in zip("qk", x2):
        for slot, new in zip(ops[name].slots, sharded(x, mesh, "bf16").slots):
            slot.copy_(new)
    g.replay()
    torch.cuda.synchronize()
    check_forward(case, out, x2, ws, cs, pos)


def test_no_tokens_gives_zero_weight_gradients(lib):
    mesh = tsl.DeviceMesh((2,), ("tp",))
    q = sharded(np.zeros((0, 256)), mesh, "bf16")
    w = whole(np.ones(64, np.float32), mesh)
    dw = whole(np.full(64, 5, np.float32), mesh)
    out = tsl.tp_qk_norm_rope_backward(q, None, q, None, w, None, head_dim=64, out=(q, None, dw, None))
    torch.cuda.synchronize()
    assert (out[2].slots[0] == 0).all()


def test_infinite_and_nan_rows_stay_in_their_rows(lib):
    case = (9, 4, 2, 128, 128, 2, "bf16", False)
    mesh, rng, xs, ws, cs, pos, ops = make(case, 19)
    q = xs[0].copy()
    q[3, 5], q[6, 200] = np.inf, np.nan
    ops["q"] = sharded(q, mesh, "bf16")
    out = tsl.tp_qk_norm_rope(**ops, head_dim=128, eps=EPS)
    y = full(out[0]).reshape(9, 4, 128)
    bad = np.zeros((9, 4), bool)
    bad[3, 0] = bad[6, 1] = True
    assert np.isnan(y[bad]).any(-1).all() and np.isfinite(y[~bad]).all() and DT["bf16"] == out[0].dtype
