"""Refusals and empty calls of the operators between blocks and behind the head, on the host (no GPU needed).

As for the operators on heads: CPU slots and a NULL stream, so a status other
than DT_ERR_CUDA comes from the checks before any launch.
"""
import ctypes as C

import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from tensor_sharded_linear_gb300 import _lib as L

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
MESH = tsl.DeviceMesh((2,), ("tp",))
R, S0, S1, PART = tsl.Replicate(), tsl.Shard(0), tsl.Shard(1), tsl.Partial()
INV, SHAPE, PLACE, UNSUP, CAP, ALIGN = (L.ERR_INVALID_ARG, L.ERR_SHAPE, L.ERR_PLACEMENT, L.ERR_UNSUPPORTED,
                                        L.ERR_CAPACITY, L.ERR_ALIGNMENT)


def dt(shape, pl=R, dtype=BF, mesh=MESH, materialize=False):
    d = tsl.DTensor.empty(mesh, [pl], shape, dtype, materialize_replicas=materialize, device="cpu")
    for s in d.slots:
        s.zero_()
    return d


def view(shape, strides, dtype=BF):
    """One Replicate slot with the given strides."""
    size = 1 + sum((s - 1) * st for s, st in zip(shape, strides))
    return tsl.DTensor([torch.zeros(size, dtype=dtype).as_strided(shape, strides)], MESH, [R], shape, dtype)


class Fake:
    """A descriptor of any shape whose slots are one byte (never read: the call is refused)."""

    def __init__(self, shape, pl=R, dtype=L.BF16):
        self.buf = (C.c_char * 64)()
        addr = (C.addressof(self.buf) + 15) // 16 * 16
        d = L.DTensorDesc()
        d.layout = tsl.api._layout(MESH, [pl], shape, {L.BF16: BF, L.FP32: F32, L.INT32: I32}[dtype], False)
        d.nslots = 1 if pl == R else 2
        self.ptrs = (C.c_void_p * 2)(addr, addr)
        d.slots = C.cast(self.ptrs, C.POINTER(C.c_void_p))
        self.d = d

    def _desc(self):
        return self.d


def ref(x):
    return None if x is None else C.byref(x._desc())


X = (6, 32)


def fwd(lib, eps=1e-6, scale=1.0, drop=0.0, tp=0, **kw):
    a = dict(x=dt(X, PART), r=dt(X, S0), post=dt((32,), R, F32), gate=dt((32,)), pre=dt((32,)), rng=None, h=dt(X, S0),
             y=dt(X))
    a.update(kw)
    return lib.dt_tp_block_norm(*(ref(a[k]) for k in ("x", "r", "post", "gate", "pre", "rng", "h", "y")), eps, scale,
                                drop, tp, None, None)


FWD_BAD = [
    (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV), (dict(eps=2.0), INV), (dict(scale=float("inf")), INV),
    (dict(drop=1.0), INV), (dict(drop=-0.1), INV), (dict(drop=float("nan")), INV), (dict(drop=0.5), INV),  # no rng
    (dict(drop=0.5, rng=dt((3,), R, I32)), INV), (dict(drop=0.5, rng=dt((4,), R, F32)), INV),
    (dict(drop=0.5, rng=dt((4,), S0, I32)), PLACE),
    (dict(tp=1), INV), (dict(tp=-1), PLACE),  # a Partial x needs tp
    (dict(x=None), INV), (dict(pre=None), INV), (dict(y=None), INV), (dict(h=None, y=None, pre=None), INV),
    (dict(x=dt(X, dtype=I32)), INV), (dict(x=dt((32,))), SHAPE), (dict(x=dt(X, S1)), PLACE),
    (dict(x=dt(X, tsl.Partial("max"))), UNSUP), (dict(r=dt(X, PART)), PLACE), (dict(h=dt(X, S1)), PLACE),
    (dict(r=dt((5, 32))), SHAPE), (dict(r=dt((6, 31))), SHAPE), (dict(y=dt((6, 1, 32))), SHAPE),
    (dict(h=dt(X, dtype=F32)), INV), (dict(r=dt(X, dtype=F32)), INV),          # h and the residual differ
    (dict(y=dt(X, dtype=F32)), INV), (dict(x=dt(X, dtype=F32), y=dt(X, dtype=F32)), UNSUP),
    (dict(post=dt((31,))), SHAPE), (dict(post=dt((1, 32))), SHAPE), (dict(post=dt((32,), S0)), PLACE),
    (dict(pre=dt((32,), R, I32)), INV), (dict(gate=dt((4, 32))), SHAPE), (dict(gate=dt((0, 32))), SHAPE),
    (dict(gate=dt((6, 31))), SHAPE), (dict(gate=dt((32,), R, I32)), INV),
    (dict(gate=view((2, 32), (33, 1))), UNSUP), (dict(r=view(X, (64, 2)), h=dt(X)), UNSUP),
    (dict(h=view(X, (16, 1))), UNSUP), (dict(h=dt(X, materialize=True)), UNSUP),
    (dict(x=dt(X, mesh=tsl.DeviceMesh((3,), ("tp",)))), SHAPE), (dict(pre=dt((32,), mesh=tsl.DeviceMesh((3,)))), SHAPE),
    (dict(x=Fake((2 ** 31, 32)), r=None), CAP), (dict(x=Fake((6, 2 ** 30 + 8)), r=None), CAP),
]


@pytest.mark.parametrize("i", range(len(FWD_BAD)))
def test_block_norm_refusals(lib, i):
    kw, want = FWD_BAD[i]
    n0 = lib.dt_launch_count()
    assert fwd(lib, **kw) == want, lib.dt_last_error()
    assert lib.dt_last_error() and lib.dt_launch_count() == n0


def bwd(lib, ws=0, ws_bytes=1 << 30, drop=0.0, **kw):
    a = dict(dh=dt(X, S0), dy=dt(X), x=dt(X, PART), r=dt(X, S0), post=dt((32,), R, F32), gate=dt((2, 32)), pre=dt((32,)),
             rng=None, dx=dt(X), dr=dt(X, S0), dpost=dt((32,)), dgate=dt((2, 32), R, F32), dpre=dt((32,)))
    a.update(kw)
    return lib.dt_tp_block_norm_backward(
        *(ref(a[k]) for k in ("dh", "dy", "x", "r", "post", "gate", "pre", "rng", "dx", "dr", "dpost", "dgate", "dpre")),
        1e-6, 1.0, drop, 0, ws, ws_bytes, None, None)


BWD_BAD = [
    (dict(dh=None, dy=None, pre=None, dpre=None), INV), (dict(dy=None), INV), (dict(pre=None), INV),
    (dict(dpre=None), INV), (dict(dpost=None), INV), (dict(post=None), INV), (dict(gate=None), INV),
    (dict(dgate=None), INV), (dict(r=None), INV), (dict(x=None), INV), (dict(drop=0.5), INV),
    (dict(dx=dt(X, PART)), PLACE), (dict(dx=dt(X, dtype=F32)), INV), (dict(dr=dt(X, dtype=F32)), INV),
    (dict(dh=dt(X, dtype=F32)), INV), (dict(dgate=dt((32,))), SHAPE), (dict(dgate=dt((3, 32))), SHAPE),
    (dict(dpost=dt((31,))), SHAPE), (dict(dpre=dt((32,), R, I32)), INV), (dict(dx=view(X, (1, 1))), UNSUP),
]


@pytest.mark.parametrize("i", range(len(BWD_BAD)))
def test_block_norm_backward_refusals(lib, i):
    kw, want = BWD_BAD[i]
    n0 = lib.dt_launch_count()
    assert bwd(lib, **kw) == want, lib.dt_last_error()
    assert lib.dt_last_error() and lib.dt_launch_count() == n0


def test_block_norm_nothing_to_do(lib):
    n0 = lib.dt_launch_count()
    z = (0, 32)
    assert fwd(lib, x=dt(z, PART), r=dt(z, S0), h=dt(z, S0), y=dt(z)) == L.OK
    z, w = (6, 0), dt((0,))
    assert fwd(lib, x=dt(z, PART), r=dt(z, S0), h=dt(z, S0), y=dt(z), post=w, gate=w, pre=w) == L.OK
    assert bwd(lib, x=dt(z, PART), r=dt(z, S0), dh=dt(z, S0), dy=dt(z), post=w, gate=w, pre=w, dx=dt(z), dr=dt(z),
               dpost=w, dgate=w, dpre=w) == L.OK
    assert lib.dt_launch_count() == n0


def test_block_norm_workspace_query(lib):
    n = C.c_size_t()
    q = lib.dt_tp_block_norm_backward_workspace_size
    assert q(10, 64, 0, C.byref(n)) == L.OK
    base = n.value
    assert q(10, 64, 5, C.byref(n)) == L.OK and n.value == base + 5 * 64 * 4
    assert q(10, 64, 10, C.byref(n)) == L.OK and n.value == base  # a gate per token needs no sums
    assert q(0, 64, 1, C.byref(n)) == L.OK
    for bad in ((-1, 64, 0), (10, -1, 0), (10, 64, -1), (2 ** 31, 64, 0), (10, 2 ** 31, 0)):
        assert q(*bad, C.byref(n)) == INV
    assert q(10, 64, 11, C.byref(n)) == SHAPE and q(10, 64, 0, None) == INV
    assert tsl.tp_block_norm_backward_workspace_bytes(dt(X)) == 0
    assert tsl.tp_block_norm_backward_workspace_bytes(dt((10, 64)), dt((64,)), dt((5, 64))) == base + 5 * 64 * 4


def test_block_norm_workspace_of_an_empty_batch_with_gate_rows(lib):
    """Five empty sequences, a gate row each: their gradients are zeros, from a workspace all the same."""
    n = C.c_size_t()
    assert lib.dt_tp_block_norm_backward_workspace_size(0, 64, 5, C.byref(n)) == L.OK
    assert tsl.tp_block_norm_backward_workspace_bytes(dt((5, 0, 64)), None, dt((5, 64))) == n.value
    assert n.value >= (3 + 5) * 64 * 4


Z = (6, 50)


def lp(lib, scale=1.0, ignore=-100, tp=0, **kw):
    a = dict(z=dt(Z, S1), ids=dt((6,), R, I32), logp=dt((6,), R, F32), lse=dt((6,), R, F32), ent=dt((6,), R, F32),
             top=dt((6, 5), R, F32), tids=dt((6, 5), R, I32))
    a.update(kw)
    return lib.dt_tp_log_probs(*(ref(a[k]) for k in ("z", "ids", "logp", "lse", "ent", "top", "tids")), scale, ignore, tp,
                               None, None)


LP_BAD = [
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(tp=1), INV), (dict(tp=-1), PLACE), (dict(z=None), INV), (dict(ids=None), INV), (dict(logp=None), INV),
    (dict(top=None), INV), (dict(tids=None), INV),
    (dict(ids=None, logp=None, lse=None, ent=None, top=None, tids=None), INV),
    (dict(z=dt(Z, S0)), PLACE), (dict(z=dt(Z, PART)), PLACE), (dict(z=dt(Z, S1, I32)), INV), (dict(z=dt((50,))), SHAPE),
    (dict(z=dt((6, 0))), SHAPE), (dict(z=view(Z, (100, 2))), UNSUP), (dict(z=Fake((6, 2 ** 31))), CAP),
    (dict(z=Fake((2 ** 31, 6))), CAP),
    (dict(ids=dt((6,), R, F32)), INV), (dict(ids=dt((5,), R, I32)), SHAPE), (dict(ids=dt((6, 2), R, I32)), SHAPE),
    (dict(ids=dt((6, 65), R, I32), logp=dt((6, 65), R, F32)), CAP), (dict(logp=dt((6,), R, BF)), INV),
    (dict(logp=dt((6, 2), R, F32)), SHAPE), (dict(ids=dt((6,), S0, I32)), PLACE), (dict(lse=dt((6, 1), R, F32)), SHAPE),
    (dict(lse=dt((6,), R, BF)), INV), (dict(ent=dt((7,), R, F32)), SHAPE),
    (dict(top=dt((6, 33), R, F32), tids=dt((6, 33), R, I32)), CAP), (dict(top=dt((6, 4), R, F32)), SHAPE),
    (dict(z=dt((6, 4), S1)), SHAPE),  # more alternatives than tokens
    (dict(tids=dt((6, 5), R, F32)), INV), (dict(lse=dt((6,), R, F32, materialize=True)), UNSUP),
    (dict(z=dt(Z, S1, mesh=tsl.DeviceMesh((3,), ("tp",)))), SHAPE),
]


@pytest.mark.parametrize("i", range(len(LP_BAD)))
def test_log_probs_refusals(lib, i):
    kw, want = LP_BAD[i]
    n0 = lib.dt_launch_count()
    assert lp(lib, **kw) == want, lib.dt_last_error()
    assert lib.dt_last_error() and lib.dt_launch_count() == n0


def test_log_probs_clusters_for_too_many_tokens(lib):
    """Rows whose alternatives need a cluster each, more of them than a grid has CTAs for."""
    t = 2 ** 28
    side = dict(ids=None, logp=None, lse=None, ent=None, top=Fake((t, 1), dtype=L.FP32), tids=Fake((t, 1), dtype=L.INT32))
    n0 = lib.dt_launch_count()
    assert lp(lib, z=Fake((t, 2 ** 21 + 1), S1), **side) == CAP
    assert lib.dt_last_error() and lib.dt_launch_count() == n0


def lpb(lib, scale=1.0, tp=0, **kw):
    a = dict(dlp=dt((6,), R, F32), dent=dt((6,), R, F32), z=dt(Z, S1), ids=dt((6,), R, I32), lse=dt((6,), R, F32),
             ent=dt((6,), R, F32), dz=dt(Z, S1))
    a.update(kw)
    return lib.dt_tp_log_probs_backward(*(ref(a[k]) for k in ("dlp", "dent", "z", "ids", "lse", "ent", "dz")), scale, -100,
                                        tp, None, None)


LPB_BAD = [
    (dict(scale=0.0), INV), (dict(z=None), INV), (dict(dz=None), INV), (dict(lse=None), INV), (dict(dlp=None), INV),
    (dict(ids=None), INV), (dict(ids=None, dlp=None, dent=None), INV), (dict(ent=None), INV),
    (dict(dz=dt(Z)), PLACE), (dict(dz=dt(Z, S1, F32)), INV), (dict(dz=dt((6, 49), S1)), SHAPE),
    (dict(dz=dt((5, 50), S1)), SHAPE), (dict(dlp=dt((6, 2), R, F32)), SHAPE), (dict(dlp=dt((6,), R, BF)), INV),
    (dict(dent=dt((5,), R, F32)), SHAPE), (dict(lse=dt((5,), R, F32)), SHAPE),
    (dict(z=dt((6, 0), S1), dz=dt((6, 0), S1)), SHAPE), (dict(dz=view(Z, (10, 1)), z=dt(Z)), UNSUP), (dict(tp=3), INV),
]


@pytest.mark.parametrize("i", range(len(LPB_BAD)))
def test_log_probs_backward_refusals(lib, i):
    kw, want = LPB_BAD[i]
    n0 = lib.dt_launch_count()
    assert lpb(lib, **kw) == want, lib.dt_last_error()
    assert lib.dt_last_error() and lib.dt_launch_count() == n0


def test_log_probs_no_tokens(lib):
    n0 = lib.dt_launch_count()
    e = lambda d, *s: dt((0, *s), R, d)  # noqa: E731
    assert lp(lib, z=dt((0, 50), S1), ids=e(I32), logp=e(F32), lse=e(F32), ent=e(F32), top=e(F32, 5), tids=e(I32, 5)) == L.OK
    assert lpb(lib, dlp=e(F32), dent=e(F32), z=dt((0, 50), S1), ids=e(I32), lse=e(F32), ent=e(F32),
               dz=dt((0, 50), S1)) == L.OK
    assert lib.dt_launch_count() == n0
