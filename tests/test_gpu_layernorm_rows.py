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


# rows, d: rows covered exactly by the groups' loads (512, 2,048, 8,192), with a
# remainder, and in single elements (1,001 and 37); groups of 32 to 512 threads
SHAPES = [(5000, 37), (5003, 64), (5000, 512), (3000, 1001), (2600, 1000), (3001, 2048), (1300, 4096), (700, 8192)]


@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_groups_walk_many_rows(rows, d, dtype, wtype):
    x = make_tensor(721, 1, (rows, d), dtype, 2.0)
    gain, bias = make_tensor(721, 2, (d,), wtype), make_tensor(721, 3, (d,), wtype)
    dy = make_tensor(721, 4, (rows, d), dtype)
    y, mean, rstd = R.ret_layernorm_forward(dev(x), dev(gain), dev(bias), eps=1e-3, want_stats=True)
    ry, rmean, rrstd = od.layernorm(x.f64, gain.f64, bias.f64, 1e-3)
    rows_close(y, ry, dtype)
    assert np.all(np.abs(host64(mean) - rmean) <= 2.0 ** -19 * np.abs(x.f64).mean(-1))
    assert np.all(np.abs(host64(rstd) / rrstd - 1) <= 2.0 ** -18)
    m, r = host64(mean)[:, None], host64(rstd)[:, None]
    dx, dgain, dbias = R.ret_layernorm_backward(dev(dy), dev(x), mean, rstd, dev(gain))
    rdx, rdg, rdb = od.layernorm_backward(dy.f64, x.f64, m[:, 0], r[:, 0], gain.f64)
    h = (x.f64 - m) * r
    t = np.abs(dy.f64 * gain.f64).max(-1, keepdims=True) * r * (1 + np.abs(h).max(-1, keepdims=True))
    assert np.all(np.abs(host64(dx) - rdx) <= 2.0 ** -18 * t + (2.0 ** -8 * np.abs(rdx) if dtype == "bf16" else 0))
    hx = np.abs(h) + (np.abs(x.f64) + np.abs(m)) * r
    for got, ref, terms in ((dgain, rdg, dy.f64 * hx), (dbias, rdb, dy.f64)):
        assert np.all(np.abs(host64(got) - ref) <= 2.0 ** -19 * np.sqrt((terms ** 2).sum(0)))
