"""What attention over the low-bit caches may lose of small rows beside large and zero ones (bounds: lowbit_precision.py)."""
import pytest
import torch

from gpu_helpers import gpu, lib_ready
from lowbit_precision import Rows

pytestmark = gpu
FULL = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@pytest.mark.parametrize("power", [0, -10])
@pytest.mark.parametrize("split", [False, True])
def test_decode_zero_rows_set_no_unit(power, split):
    """A zero V row has the exponent 2^0, far above that of rows of ordinary size: they must keep their weights' bits.
    Every head pair has one head that looks at a single key and one that looks at many."""
    c = Rows([1500, 700, 33] if split else [700] * 40, [1] * (3 if split else 40), FULL, 0, 61)
    c.v_host *= 2.0 ** power
    c.v_host[:, 3::17] *= 0
    c.v_host[:, 100:140] *= 0                    # a whole warp's share
    c.upload()
    c.aim(range(0, 32, 2), lambda s, p: (p * 7 // 11) | 1)
    c.compare(False, f"2^{power}")


def test_decode_of_zero_rows_alone():
    c = Rows([600, 40], [1, 1], FULL, 0, 63)
    c.v_host *= 0
    c.upload()
    c.qd = c.q.cuda()
    out, lse = c.call(False)
    assert (out == 0).all() and lse.isfinite().all()
