"""GPU parity of the layer norm and its gradients against the fp64 oracle.

Tolerances.  Sums run in fp32 over at most 8,192 elements, in groups: each of
the about 24 levels of additions is off by 2^-24, so a sum by 24 x 2^-24 of
the sum of absolute values; a normalised value by that and a few roundings,
under 2^-18 of the row's largest.  bf16 outputs add one rounding, 2^-8 of the
value."""
import numpy as np
import pytest
import torch

from oracle import delta as od
from retention_inputs import make_tensor
from tests.helpers import dev, host64

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


def rows_close(got, ref, dtype, slack=2.0 ** -18):
    got = host64(got)
    assert got.shape == ref.shape and np.isfinite(got).all()
    bound = slack * np.abs(ref).max(-1, keepdims=True) + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0) + 1e-30
    assert np.all(np.abs(got - ref) <= bound), float((np.abs(got - ref) / bound).max())


SHAPES = [(1, 1), (1, 8), (3, 17), (5, 32), (64, 2048), (300, 1000), (37, 1001), (9, 4096), (3, 8192), (2, 8191), (700, 64)]


@pytest.mark.parametrize("dtype,wtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward_and_backward(rows, d, dtype, wtype):
    x = make_tensor(701, 1, (rows, d), dtype, 2.0)
    gain, bias = make_tensor(701, 2, (d,), wtype), make_tensor(701, 3, (d,), wtype)
    dy = make_tensor(701, 4, (rows, d), dtype)
    y, mean, rstd = R.ret_layernorm_forward(dev(x), dev(gain), dev(bias), eps=1e-3, want_stats=True)
    ry, rmean, rrstd = od.layernorm(x.f64, gain.f64, bias.f64, 1e-3)
    rows_close(y, ry, dtype)
    scale = np.abs(x.f64).mean(-1)
    assert np.all(np.abs(host64(mean) - rmean) <= 2.0 ** -19 * scale)
    assert np.all(np.abs(host64(rstd) / rrstd - 1) <= 2.0 ** -18)
    assert torch.equal(y, R.ret_layernorm_forward(dev(x), dev(gain), dev(bias), eps=1e-3))
    # the gradients, for the statistics that the call is given
    m, r = host64(mean), host64(rstd)
    dx, dgain, dbias = R.ret_layernorm_backward(dev(dy), dev(x), mean, rstd, dev(gain))
    rdx, rdg, rdb = od.layernorm_backward(dy.f64, x.f64, m, r, gain.f64)
    # two row averages subtract from dy gain: the row's largest term bounds the error
    t = np.abs(dy.f64 * gain.f64).max(-1, keepdims=True) * r[:, None] * (1 + np.abs((x.f64 - m[:, None]) * r[:, None]).max(-1, keepdims=True))
    bound = 2.0 ** -18 * t + (2.0 ** -8 * np.abs(rdx) if dtype == "bf16" else 0)
    assert np.all(np.abs(host64(dx) - rdx) <= bound)
    h = np.abs((x.f64 - m[:, None]) * r[:, None])
    # (x - mean) rounds to fp32 before the product: 2^-24 of |x| and |mean|
    hx = h + (np.abs(x.f64) + np.abs(m[:, None])) * r[:, None]
    assert np.all(np.abs(host64(dgain) - rdg) <= 2.0 ** -19 * (np.abs(dy.f64) * hx).sum(0))
    assert np.all(np.abs(host64(dbias) - rdb) <= 2.0 ** -19 * np.abs(dy.f64).sum(0))


def test_without_weights_and_single_gradients():
    x, dy = make_tensor(702, 1, (2, 50, 256), "bf16"), make_tensor(702, 2, (2, 50, 256), "bf16")
    y, mean, rstd = R.ret_layernorm_forward(dev(x), want_stats=True)
    assert y.shape == (2, 50, 256) and mean.shape == (2, 50)
    rows_close(y, od.layernorm(x.f64)[0], "bf16")
    dx, dgain, dbias = R.ret_layernorm_backward(dev(dy), dev(x), mean, rstd, want_weights=False)
    assert dgain is None and dbias is None
    full = R.ret_layernorm_backward(dev(dy), dev(x), mean, rstd)
    assert torch.equal(dx, full[0])
    only = torch.empty(256, dtype=torch.float32, device="cuda")
    _, none, got = R.ret_layernorm_backward(dev(dy), dev(x), mean, rstd, want_weights=False, dbias=only)
    assert none is None and torch.equal(got, full[2])


def test_the_same_bits_every_time():
    x, dy = make_tensor(703, 1, (4000, 520), "bf16"), make_tensor(703, 2, (4000, 520), "bf16")
    _, mean, rstd = R.ret_layernorm_forward(dev(x), want_stats=True)
    first = R.ret_layernorm_backward(dev(dy), dev(x), mean, rstd)
    for _ in range(3):
        for a, b in zip(first, R.ret_layernorm_backward(dev(dy), dev(x), mean, rstd)):
            assert torch.equal(a, b)


def test_large_mean_keeps_its_digits():
    """The variance is taken about the mean: rows around 1,000 with a spread of 1."""
    x = make_tensor(704, 1, (8, 2048), "f32")
    big = torch.from_numpy(x.stored + np.float32(1000)).cuda()
    y = R.ret_layernorm_forward(big)
    # the inputs themselves carry 2^-24 of 1,000, the mean as much again
    assert np.abs(host64(y) - od.layernorm(host64(big))[0]).max() < 1000 * 2.0 ** -22


def test_unaligned_rows_and_nan_rows():
    """A row pitch of no whole vector, a base off the 16-byte grid; a row of NaN stays alone."""
    x = make_tensor(705, 1, (6, 2048), "f32")
    flat = torch.empty(6 * 2048 + 1, dtype=torch.float32, device="cuda")
    view = flat[1:].view(6, 2048)
    view.copy_(dev(x))
    assert view.data_ptr() % 16
    rows_close(R.ret_layernorm_forward(view), od.layernorm(x.f64)[0], "f32")
    view[2] = float("nan")
    y = R.ret_layernorm_forward(view)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4, 5]]).all()


def test_replayed_from_a_graph_on_another_stream():
    x, dy = make_tensor(706, 1, (500, 768), "bf16"), make_tensor(706, 2, (500, 768), "bf16")
    xd, dyd = dev(x), dev(dy)
    _, mean, rstd = R.ret_layernorm_forward(xd, want_stats=True)
    want = R.ret_layernorm_backward(dyd, xd, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = R.ret_layernorm_backward(dyd, xd, mean, rstd)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
