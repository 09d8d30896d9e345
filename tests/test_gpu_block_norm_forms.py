"""Block norms and their gradients in each form of the kernels: types, parts, channel counts, alignment, dropout."""
import pytest

import tensor_sharded_linear_gb300 as tsl
from test_gpu_block_norm import PART, S0, Case, ids

pytestmark = pytest.mark.gpu
TYPES = [dict(), dict(stream="fp32"), dict(dtype="fp32")]


def run(c, seed=51):
    case = Case(seed, **c)
    case.check_forward(*case.forward())
    case.check_backward(case.backward())
    assert tsl.read_device_status() == 0


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("drop", [0.0, 0.2])
@pytest.mark.parametrize("n", [200, 1024, 2048, 2560, 4096, 7168, 8192, 8200, 16384])
def test_many_tokens(n, drop, types):
    """Rows read ahead forward; backward rings of five, three and one rows, on one CTA and on a pair."""
    run(dict(t=331, n=n, drop=drop, gate=-1, **types))


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("n,p,drop", [(1000, 2, 0.0), (2048, 8, 0.0), (4096, 4, 0.1), (8192, 3, 0.0), (12288, 2, 0.1)])
def test_partial_sums(n, p, drop, types):
    run(dict(t=160, n=n, p=p, place=PART, out=S0, drop=drop, gate=-1, **types))


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("n,p", [(8192, 4), (8192, 8), (8192, 16), (6144, 8), (4096, 16), (2048, 32), (16384, 8), (7000, 64)])
def test_many_partial_sums(n, p, types):
    """Parts of a row that fill the shared memory of an SM, of two, and more."""
    run(dict(t=5, n=n, p=p, place=PART, gate=-1, **types))


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("n,p", [(1001, 1), (1999, 4), (4093, 1), (8191, 2), (8197, 1), (16383, 3)])
def test_odd_channels(n, p, types):
    run(dict(t=37, n=n, p=p, place=PART if p > 1 else tsl.Replicate(), gate=-1, drop=0.1, **types))


@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("n", [9, 255, 1003, 4096])
def test_gradients_at_every_distance_from_a_16_byte_boundary(n, types):
    for offset in range(1, 9):
        run(dict(t=11, n=n, p=2, place=S0, out=S0, gate=11, extra=offset % 3, offset=offset, **types), 60 + offset)
