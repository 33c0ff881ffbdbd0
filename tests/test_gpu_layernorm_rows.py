"""Layer norm over so many rows that every group of threads walks several of them,
in all of the kernels' forms, against the fp64 oracle.

Tolerances.  A normalised value as in the parity tests: under 2^-18 of the row's
largest, and one rounding of a bf16 output.  A column's sum over the rows: a term is
off by 2^-23 of itself (two roundings of (x - mean) rstd) and by what x - mean loses,
2^-24 of |x| and |mean|; a chain of at most 64 fp32 additions (a group's rows, a
block's groups) adds 64 x 2^-24 of the sum of magnitudes: together under 2^-17 of it
at worst and, the roundings being independent, under sqrt(64) x 2^-24 = 2^-21 of the
terms' root mean square times the square root of their number, with a factor 4 for
the largest of thousands of columns: 2^-19 of that."""
import numpy as np
import pytest
import torch

from oracle import delta as od
from retention_inputs import make_tensor
from tests.helpers import dev, host64
from tests.test_gpu_layernorm import rows_close

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


def test_partial_rows_are_added_in_64_bits():
    """Two rows that cancel, far above the others: what is lost beside them is lost
    in their own two blocks, not in the sum over the blocks.  8,192 rows on 148 blocks
    of four groups: block 0 and block 75."""
    rows, d = 8192, 2048
    x = torch.randn(rows, d, device="cuda").bfloat16()
    dy = torch.ones(rows, d, device="cuda", dtype=torch.bfloat16)
    dy[0], dy[300] = 2.0 ** 40, -(2.0 ** 40)
    _, mean, rstd = R.ret_layernorm_forward(x, want_stats=True)
    _, _, dbias = R.ret_layernorm_backward(dy, x, mean, rstd)
    assert (dbias - (rows - 2)).abs().max() <= 2 * -(-rows // 148)
