"""Refusals and empty calls of the operators on attention heads, on the host (no GPU needed).

The slots are CPU tensors and the stream is NULL: a call that passed its
checks and reached CUDA would fail with DT_ERR_CUDA, so each status below
comes from the checks before any launch.
"""
import ctypes as C

import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from tensor_sharded_linear_gb300 import _lib as L

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
P = 2
MESH = tsl.DeviceMesh((P,), ("tp",))
R, S0, S1 = tsl.Replicate(), tsl.Shard(0), tsl.Shard(1)


def dt(shape, pl=S1, dtype=BF, mesh=MESH):
    d = tsl.DTensor.empty(mesh, [pl], shape, dtype, device="cpu")
    for s in d.slots:
        s.zero_()
    return d


def ref(x):
    return None if x is None else C.byref(x._desc())


def norm(lib, head_dim=64, eps=1e-6, tp=0, **kw):
    a = dict(q=dt((5, 4 * 64)), k=dt((5, 2 * 64)), q_weight=dt((64,), R, F32), k_weight=dt((64,), R, BF),
             cos_sin=dt((9, 64), R, F32), positions=dt((5,), R, I32), q_out=dt((5, 4 * 64)), k_out=dt((5, 2 * 64)))
    a.update(kw)
    return lib.dt_tp_qk_norm_rope(ref(a["q"]), ref(a["k"]), ref(a["q_weight"]), ref(a["k_weight"]), ref(a["cos_sin"]),
                                  ref(a["positions"]), ref(a["q_out"]), ref(a["k_out"]), head_dim, eps, 0, tp, None,
                                  None)


NORM_BAD = [
    (dict(head_dim=0), L.ERR_UNSUPPORTED), (dict(head_dim=1025), L.ERR_UNSUPPORTED),
    (dict(eps=-1.0), L.ERR_INVALID_ARG), (dict(eps=float("nan")), L.ERR_INVALID_ARG),
    (dict(tp=1), L.ERR_INVALID_ARG),
    (dict(q=None), L.ERR_INVALID_ARG), (dict(q_out=None), L.ERR_INVALID_ARG),
    (dict(k=None), L.ERR_INVALID_ARG),                                  # its output and weight are still there
    (dict(cos_sin=None), L.ERR_INVALID_ARG), (dict(positions=None), L.ERR_INVALID_ARG),
    (dict(q_weight=None, k_weight=None, cos_sin=None, positions=None), L.ERR_INVALID_ARG),
    (dict(q=dt((5, 250))), L.ERR_SHAPE),                                # not whole heads
    (dict(q=dt((5, 3 * 64)), q_out=dt((5, 3 * 64))), L.ERR_SHAPE),      # shards of one and a half heads
    (dict(q=dt((6, 4 * 64))), L.ERR_SHAPE), (dict(k=dt((4, 2 * 64)), k_out=dt((4, 2 * 64))), L.ERR_SHAPE),
    (dict(q=dt((4 * 64,), tsl.Shard(0))), L.ERR_SHAPE),
    (dict(q=dt((5, 4 * 64), S0)), L.ERR_PLACEMENT), (dict(q=dt((5, 4 * 64), tsl.Partial())), L.ERR_PLACEMENT),
    (dict(q_out=dt((5, 4 * 64), dtype=F32)), L.ERR_INVALID_ARG), (dict(k=dt((5, 2 * 64), dtype=F32)), L.ERR_INVALID_ARG),
    (dict(q=dt((5, 4 * 64), dtype=I32)), L.ERR_INVALID_ARG),
    (dict(q_weight=dt((32,), R, F32)), L.ERR_SHAPE), (dict(q_weight=dt((64,), S0, F32)), L.ERR_PLACEMENT),
    (dict(q_weight=dt((64,), R, I32)), L.ERR_INVALID_ARG),
    (dict(cos_sin=dt((9, 66), R, F32)), L.ERR_SHAPE), (dict(cos_sin=dt((9, 33), R, F32)), L.ERR_SHAPE),
    (dict(cos_sin=dt((9, 64), R, BF)), L.ERR_INVALID_ARG), (dict(cos_sin=dt((0, 64), R, F32)), L.ERR_SHAPE),
    (dict(positions=dt((4,), R, I32)), L.ERR_SHAPE), (dict(positions=dt((5,), R, F32)), L.ERR_INVALID_ARG),
    (dict(q=dt((5, 4 * 64), mesh=tsl.DeviceMesh((4,), ("tp",)))), L.ERR_SHAPE),
]


@pytest.mark.parametrize("i", range(len(NORM_BAD)))
def test_norm_refusals(lib, i):
    kw, want = NORM_BAD[i]
    n0 = lib.dt_launch_count()
    assert norm(lib, **kw) == want, lib.dt_last_error()
    assert lib.dt_last_error() and lib.dt_launch_count() == n0


def test_norm_no_tokens(lib):
    n0 = lib.dt_launch_count()
    assert norm(lib, q=dt((0, 256)), k=dt((0, 128)), q_out=dt((0, 256)), k_out=dt((0, 128)),
                positions=dt((0,), R, I32)) == L.OK
    assert lib.dt_launch_count() == n0


def test_norm_overlapping_output_rows(lib):
    q = dt((5, 4 * 64))
    q.slots = [s[:1].expand(5, -1) for s in q.slots]  # a broadcast input is fine, an output is not
    assert norm(lib, q_out=q) == L.ERR_UNSUPPORTED
    q = tsl.DTensor([torch.zeros(5, 256, dtype=BF)[:, ::2], torch.zeros(5, 256, dtype=BF)[:, ::2]], MESH, [S1],
                    (5, 256), BF)
    assert norm(lib, q=q) == L.ERR_UNSUPPORTED


def test_norm_materialised_output(lib):
    o = tsl.DTensor.empty(MESH, [R], (5, 256), BF, materialize_replicas=True, device="cpu")
    assert norm(lib, q=dt((5, 256), R), q_out=o) == L.ERR_UNSUPPORTED


def test_backward_refusals(lib):
    q, k, w = dt((5, 256)), dt((5, 128)), dt((64,), R, F32)

    def call(dqw=w, ws=None, n=0, kw=w):
        return lib.dt_tp_qk_norm_rope_backward(ref(q), ref(k), ref(q), ref(k), ref(w), ref(kw), None, None, ref(dt((5, 256))),
                                               ref(dt((5, 128))), ref(dqw), ref(w), 64, 1e-6, 0, 0, ws, n, None, None)

    assert call(dqw=None) == L.ERR_INVALID_ARG and b"go together" in lib.dt_last_error()
    assert call(kw=None) == L.ERR_INVALID_ARG
    assert call() == L.ERR_INVALID_ARG and b"workspace" in lib.dt_last_error()
    n = C.c_size_t()
    assert lib.dt_tp_qk_norm_rope_backward_workspace_size(64, C.byref(n)) == L.OK and n.value > 0
    assert call(ws=0x1010, n=n.value) == L.ERR_ALIGNMENT
    assert lib.dt_tp_qk_norm_rope_backward_workspace_size(64, None) == L.ERR_INVALID_ARG
    assert lib.dt_tp_qk_norm_rope_backward_workspace_size(2000, C.byref(n)) == L.ERR_UNSUPPORTED


def test_record_words(lib):
    n = C.c_int32()
    for d, g, want in ((64, 64, 20), (64, 32, 20), (128, 64, 36), (128, 32, 40), (256, 64, 72), (256, 32, 80)):
        assert lib.dt_kv4_record_words(d, g, C.byref(n)) == L.OK and n.value == want
        assert tsl.kv4_record_words(d, g) == want
    for d, g in ((96, 32), (128, 128), (128, 0), (0, 64), (-64, 32)):
        assert lib.dt_kv4_record_words(d, g, C.byref(n)) == L.ERR_UNSUPPORTED
    assert lib.dt_kv4_record_words(64, 64, None) == L.ERR_INVALID_ARG
    with pytest.raises(tsl.DtError):
        tsl.kv4_cache(MESH, 4, 2, 16, head_dim=96, device="cpu")


def append(lib, head_dim=64, group=64, tp=0, **kw):
    a = dict(k=dt((6, 128)), v=dt((6, 128)), cache=dt((7, 2, 16, 20), S1, I32), page_table=dt((3, 2), R, I32),
             kv_lens=dt((3,), R, I32), q_starts=dt((4,), R, I32), cos_sin=dt((32, 64), R, F32), q=dt((6, 256)),
             q_out=dt((6, 256)), k_stored=None, v_stored=None)
    a.update(kw)
    return lib.dt_tp_kv4_append(*[ref(a[n]) for n in ("k", "v", "cache", "page_table", "kv_lens", "q_starts",
                                                      "cos_sin", "q", "q_out", "k_stored", "v_stored")],
                                head_dim, group, 0, tp, None, None)


APPEND_BAD = [
    (dict(head_dim=96), L.ERR_UNSUPPORTED), (dict(group=16), L.ERR_UNSUPPORTED),
    (dict(k=None), L.ERR_INVALID_ARG), (dict(v=None), L.ERR_INVALID_ARG), (dict(cache=None), L.ERR_INVALID_ARG),
    (dict(page_table=None), L.ERR_INVALID_ARG), (dict(kv_lens=None), L.ERR_INVALID_ARG),
    (dict(q=None), L.ERR_INVALID_ARG), (dict(q_out=None), L.ERR_INVALID_ARG),
    (dict(k_stored=dt((6, 128))), L.ERR_INVALID_ARG),
    (dict(v=dt((5, 128))), L.ERR_SHAPE), (dict(v=dt((6, 256))), L.ERR_SHAPE), (dict(q_out=dt((6, 128))), L.ERR_SHAPE),
    (dict(v=dt((6, 128), dtype=F32)), L.ERR_INVALID_ARG),
    (dict(cache=dt((7, 2, 16, 24), S1, I32)), L.ERR_SHAPE), (dict(cache=dt((7, 4, 16, 20), S1, I32)), L.ERR_SHAPE),
    (dict(cache=dt((7, 2, 0, 20), S1, I32)), L.ERR_SHAPE), (dict(cache=dt((7, 2, 16, 20), S1, F32)), L.ERR_INVALID_ARG),
    (dict(cache=dt((7, 2, 16, 20), S0, I32)), L.ERR_PLACEMENT),
    (dict(page_table=dt((3, 2), S0, I32)), L.ERR_PLACEMENT), (dict(page_table=dt((6,), R, I32)), L.ERR_SHAPE),
    (dict(page_table=dt((3, 0), R, I32)), L.ERR_SHAPE),
    (dict(kv_lens=dt((4,), R, I32)), L.ERR_SHAPE), (dict(q_starts=dt((3,), R, I32)), L.ERR_SHAPE),
    (dict(kv_lens=dt((3,), R, F32)), L.ERR_INVALID_ARG),
    (dict(k=dt((7, 128)), v=dt((7, 128)), q=None, q_out=None, q_starts=None), L.ERR_SHAPE),  # 7 tokens, 3 sequences
    (dict(cos_sin=dt((32, 8), R, F32)), L.ERR_SHAPE), (dict(cos_sin=dt((32, 80), R, F32)), L.ERR_SHAPE),
    (dict(cos_sin=dt((32, 64), R, BF)), L.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("i", range(len(APPEND_BAD)))
def test_append_refusals(lib, i):
    kw, want = APPEND_BAD[i]
    n0 = lib.dt_launch_count()
    assert append(lib, **kw) == want, lib.dt_last_error()
    assert lib.dt_last_error() and lib.dt_launch_count() == n0


def test_append_alignment(lib):
    k = dt((6, 128))
    k.slots = [torch.zeros(6 * 64 + 1, dtype=BF)[1:].view(6, 64) for _ in range(P)]
    assert append(lib, k=k) == L.ERR_ALIGNMENT
    c = dt((7, 2, 16, 20), S1, I32)
    c.slots = [torch.zeros(7 * 16 * 20 + 1, dtype=I32)[1:].view(7, 1, 16, 20) for _ in range(P)]
    assert append(lib, cache=c) == L.ERR_ALIGNMENT
    c.slots = [torch.zeros(7, 1, 32, 20, dtype=I32)[:, :, ::2] for _ in range(P)]
    assert append(lib, cache=c) == L.ERR_UNSUPPORTED


def test_append_no_tokens(lib):
    n0 = lib.dt_launch_count()
    e = dict(k=dt((0, 128)), v=dt((0, 128)), q=dt((0, 256)), q_out=dt((0, 256)))
    assert append(lib, **e) == L.OK
    assert append(lib, q_starts=None, **e) == L.OK
    assert append(lib, page_table=dt((0, 2), R, I32), kv_lens=dt((0,), R, I32), q_starts=dt((1,), R, I32), **e) == L.OK
    assert lib.dt_launch_count() == n0


def attention(lib, head_dim=64, group=64, tp=0, scale=0.125, causal=1, window=0, ws=None, n=0, **kw):
    a = dict(q=dt((6, 256)), cache=dt((7, 2, 16, 20), S1, I32), page_table=dt((3, 2), R, I32),
             kv_lens=dt((3,), R, I32), q_starts=dt((4,), R, I32), out=dt((6, 256)), lse=None)
    a.update(kw)
    return lib.dt_tp_kv4_attention(*[ref(a[x]) for x in ("q", "cache", "page_table", "kv_lens", "q_starts", "out",
                                                         "lse")], head_dim, group, scale, causal, window, tp, ws, n,
                                   None, None)


ATTN_BAD = [
    (dict(head_dim=96), L.ERR_UNSUPPORTED), (dict(group=128), L.ERR_UNSUPPORTED),
    (dict(q=None), L.ERR_INVALID_ARG), (dict(out=None), L.ERR_INVALID_ARG), (dict(cache=None), L.ERR_INVALID_ARG),
    (dict(kv_lens=None), L.ERR_INVALID_ARG), (dict(page_table=None), L.ERR_INVALID_ARG),
    (dict(scale=0.0), L.ERR_INVALID_ARG), (dict(scale=float("inf")), L.ERR_INVALID_ARG),
    (dict(scale=float("nan")), L.ERR_INVALID_ARG),
    (dict(window=-1), L.ERR_INVALID_ARG), (dict(window=4, causal=0), L.ERR_INVALID_ARG),
    (dict(out=dt((6, 128))), L.ERR_SHAPE), (dict(out=dt((6, 256), dtype=F32)), L.ERR_INVALID_ARG),
    (dict(lse=dt((6, 2), dtype=F32)), L.ERR_SHAPE), (dict(lse=dt((6, 4))), L.ERR_INVALID_ARG),
    (dict(cache=dt((7, 3, 16, 20), R, I32)), L.ERR_SHAPE),   # 4 query heads on 3 kv heads
    (dict(cache=dt((7, 0, 16, 20), R, I32)), L.ERR_SHAPE),
    (dict(q_starts=None, q=dt((7, 256)), out=dt((7, 256))), L.ERR_SHAPE),
    (dict(q=dt((6, 256), S0)), L.ERR_PLACEMENT),
]


@pytest.mark.parametrize("i", range(len(ATTN_BAD)))
def test_attention_refusals(lib, i):
    kw, want = ATTN_BAD[i]
    n0 = lib.dt_launch_count()
    assert attention(lib, **kw) == want, lib.dt_last_error()
    assert lib.dt_last_error() and lib.dt_launch_count() == n0


def test_attention_no_queries(lib):
    n0 = lib.dt_launch_count()
    assert attention(lib, q=dt((0, 256)), out=dt((0, 256))) == L.OK
    assert lib.dt_launch_count() == n0
    n = C.c_size_t(5)
    q, c, t = dt((0, 256)), dt((7, 2, 16, 20), S1, I32), dt((3, 2), R, I32)
    assert lib.dt_tp_kv4_attention_workspace_size(ref(q), ref(c), ref(t), 64, 64, 0, C.byref(n)) == L.OK
    assert n.value == 0
    assert lib.dt_tp_kv4_attention_workspace_size(ref(q), ref(c), ref(t), 64, 64, 0, None) == L.ERR_INVALID_ARG


def test_python_layer_raises(lib):
    with pytest.raises(tsl.DtError) as e:
        lse = tsl.DTensor([torch.zeros(6, 2), torch.zeros(6, 2)], MESH, [S1], (6, 4), F32)
        assert np.isfinite(lse.slots[0].numpy()).all()
        tsl.api.L.check(attention(lib, scale=-1.0, lse=lse), "tp_kv4_attention")
    assert e.value.status == L.ERR_INVALID_ARG and "scale" in str(e.value)


def test_descriptor_arguments_follow_the_slots(lib):
    """The argument is kept while every slot lies where it did with the strides it had."""
    from tensor_sharded_linear_gb300 import api
    mesh = tsl.DeviceMesh((2,), ("tp",), device="cpu")
    t = tsl.DTensor([torch.zeros(6, 64) for _ in range(2)], mesh, [tsl.Shard(1)], (6, 128), torch.float32)

    def seen():
        d = api._ref(t)._obj
        return [(d.slots[i], d.strides[2 * i], d.strides[2 * i + 1]) for i in range(2)]

    def held():
        return [(s.data_ptr(), *s.stride()) for s in t.slots]

    assert api._ref(None) is None
    first = api._ref(t)
    assert api._ref(t) is first and seen() == held()
    t.slots[1] = torch.zeros(6, 64)
    assert api._ref(t) is not first and seen() == held()
    wide = torch.zeros(6, 80)
    t.slots[0] = wide[:, :64]  # a pitch
    assert seen() == held()
    pitched = api._ref(t)
    assert api._ref(t) is pitched
    t.slots[0] = wide.view(-1)[:384].view(6, 64)  # the same address, contiguous
    assert seen() == held()
    t.slots[0] = wide[:, :64]
    assert seen() == held()
