"""Limits of the operators on attention heads that are checked on the host (no GPU needed); slots are CPU tensors, so
each status comes from the checks before any launch."""
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from tensor_sharded_linear_gb300 import _lib as L

from test_heads_host import BF, F32, I32, MESH, R, S1, append, attention, dt, norm

HUGE = 2 ** 31 - 2 ** 16  # tokens, and (query, head) rows of a kv head: kernels add strides below 2^16 to their numbers


def rows(n, width, dtype=BF):
    """[n, width] over the mesh, every row the same memory."""
    slots = [torch.zeros(1, width // 2, dtype=dtype).expand(n, -1) for _ in range(2)]
    return tsl.DTensor(slots, MESH, [S1], (n, width), dtype)


@pytest.mark.parametrize("n", [HUGE, 2 ** 31 - 513])
def test_token_counts_near_32_bits(lib, n):
    one = dict(page_table=dt((1, 2), R, I32), kv_lens=dt((1,), R, I32), q_starts=dt((2,), R, I32))
    n0 = lib.dt_launch_count()
    assert append(lib, k=rows(n, 128), v=rows(n, 128), q=None, q_out=None, **one) == L.ERR_CAPACITY
    assert b"tokens" in lib.dt_last_error()
    assert attention(lib, q=rows(n, 256), **one) == L.ERR_CAPACITY
    assert norm(lib, q=rows(n, 256)) == L.ERR_CAPACITY
    assert lib.dt_launch_count() == n0


@pytest.mark.parametrize("n,want", [(HUGE // 8, L.ERR_CAPACITY), (HUGE // 8 - 1, L.ERR_SHAPE)])
def test_rows_per_kv_head_near_32_bits(lib, n, want):
    """8 query heads on each kv head; below the limit the call goes on to its next check, the output's shape."""
    one = dict(page_table=dt((1, 2), R, I32), kv_lens=dt((1,), R, I32), q_starts=dt((2,), R, I32))
    assert attention(lib, q=rows(n, 16 * 64), **one) == want


def test_append_with_an_empty_table(lib):
    """No rows of cosines and sines: refused, as the norms do, and not taken for "no rotation"."""
    n0 = lib.dt_launch_count()
    for rotary in (64, 32):
        assert append(lib, cos_sin=dt((0, rotary), R, F32)) == L.ERR_SHAPE
        assert b"no rows" in lib.dt_last_error()
    assert lib.dt_launch_count() == n0
    empty = dict(k=dt((0, 128)), v=dt((0, 128)), q=dt((0, 256)), q_out=dt((0, 256)))
    assert append(lib, cos_sin=dt((0, 64), R, F32), **empty) == L.OK
