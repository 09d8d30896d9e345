"""The end of a decoder asks for what it hands on, and for nothing else."""
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from tensor_sharded_linear_gb300 import api

R, S0, PART = tsl.Replicate(), tsl.Shard(0), tsl.Partial()


@pytest.mark.parametrize("place", [R, S0, PART])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [True, False])
def test_the_residual_stream_is_not_written(monkeypatch, place, stream, residual):
    mesh = tsl.DeviceMesh((2,), ("tp",))
    new = lambda pl, d, *s: tsl.DTensor.empty(mesh, [pl], s, d, device="cpu")  # noqa: E731
    x, w, head = new(place, torch.bfloat16, 6, 16), new(R, torch.float32, 16), new(tsl.Shard(1), torch.bfloat16, 16, 10)
    r = new(S0, stream, 6, 16) if residual else None
    seen = []

    def block_norm(*operands, out=None, **kw):
        seen.append(out)
        return out

    monkeypatch.setattr(api, "tp_block_norm", block_norm)
    monkeypatch.setattr(api, "column_parallel_linear", lambda a, *_, **__: seen.append(a))
    monkeypatch.setattr(api, "tp_log_probs", lambda *_, **__: None)
    tsl.tp_head_log_probs(x, head, residual=r, pre_weight=w)
    (h, y), into = seen
    assert h is None and into is y
    assert y.dtype == torch.bfloat16 and y.shape == (6, 16)
    assert y.placements == ((S0,) if residual else (R,) if place == PART else (place,))
