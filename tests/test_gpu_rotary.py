"""GPU parity of the rotary positions against the fp64 oracle.

Tolerances.  bf16 output: one rounding, at most 2^-8 of the value, on top of
the fp32 ones.  fp32: the angle is reduced in 64 bits and rounded to fp32 (at
most 2^-24 pi), sine and cosine are good to 2 units (2^-22), two products and
a sum (2^-23): below 2^-20 of the pair's length."""
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


def check(got, ref, x, dtype, scale=1.0):
    """Element-wise: the pair's length bounds both products."""
    got, length = host64(got), np.abs(x).max(-1, keepdims=True) * 2 ** 0.5 * scale
    bound = 2.0 ** -20 * length + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0)
    assert np.all(np.abs(got - ref) <= bound), float((np.abs(got - ref) - bound).max())


CASES = [
    # B, N, H, Hk, d, rotary_dim
    (1, 1, 1, 1, 2, 2),
    (3, 5, 4, 2, 64, 64),
    (2, 130, 3, 1, 96, 24),       # parts of no whole vector in bf16
    (1, 257, 16, 16, 256, 128),
    (64, 1, 16, 4, 128, 32),      # one token for each of many sequences
    (2, 33, 2, 2, 10, 6),
    (1, 40, 2, 1, 520, 512),      # the widest turned part
]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,Hk,d,rd", CASES)
def test_matches_oracle(B, N, H, Hk, d, rd, dtype, layout):
    q, k = make_tensor(601, 1, (B, N, H, d), dtype), make_tensor(601, 2, (B, N, Hk, d), dtype)
    pos = np.random.default_rng(601).integers(0, 200000, (B, N))  # far ones among them
    freqs, scale = R.ret_rotary_frequencies(rd, scaling="yarn", factor=4.0)
    dpos = torch.from_numpy(pos).cuda()
    qo, ko = R.ret_rotary(dev(q), dev(k), freqs=freqs, positions=dpos, layout=layout, scale=scale)
    for got, x in ((qo, q), (ko, k)):
        check(got, od.rotary(x.f64, pos, freqs.numpy(), layout, scale), x.f64, dtype, scale)
        assert torch.equal(got[..., rd:].cpu(), dev(x)[..., rd:].cpu())
    # the transpose undoes the rotation up to scale^2
    back = R.ret_rotary(qo.float(), freqs=freqs, positions=dpos, layout=layout, scale=scale, inverse=True)
    check(back, od.rotary(host64(qo), pos, freqs.numpy(), layout, scale, inverse=True), host64(qo), "f32", scale)


def test_offset_in_place_and_the_older_entry_point():
    B, N, H, d = 2, 70, 3, 128
    x = make_tensor(602, 1, (B, N, H, d), "bf16")
    a, b = dev(x), dev(x)
    out = R.ret_rotary(a, pos_offset=5000, q_out=a)
    assert out is a
    R.ret_xpos_rotate(b, pos_offset=5000)
    ref = od.rotary(x.f64, np.broadcast_to(5000 + np.arange(N), (B, N)), R.ret_rotary_frequencies(d)[0].numpy())
    check(a, ref, x.f64, "bf16")
    check(b, ref, x.f64, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_slices_of_a_fused_projection_in_place(dtype, layout):
    """q and k are column slices of one [B, N, (H + 2 Hk) d] buffer; the v slice
    behind them stays as it is."""
    B, N, H, Hk, d = 2, 37, 4, 2, 64
    x = make_tensor(603, 1, (B, N, H + 2 * Hk, d), dtype)
    buf = dev(x)
    q, k, v = buf[:, :, :H], buf[:, :, H:H + Hk], buf[:, :, H + Hk:]
    keep = v.clone()
    R.ret_rotary(q, k, layout=layout, rotary_dim=32, pos_offset=3, q_out=q, k_out=k)
    ref = od.rotary(x.f64[:, :, :H + Hk], np.broadcast_to(3 + np.arange(N), (B, N)),
                    R.ret_rotary_frequencies(32)[0].numpy(), layout)
    check(buf[:, :, :H + Hk], ref, x.f64[:, :, :H + Hk], dtype)
    assert torch.equal(v, keep)


def test_other_orders_and_broadcast_inputs():
    """Head-major views, an odd row pitch, and one row broadcast over the heads."""
    B, N, H, d = 2, 19, 3, 16
    f = R.ret_rotary_frequencies(16)[0]
    pos = np.broadcast_to(np.arange(N), (B, N))
    x = make_tensor(604, 1, (B, H, N, d), "bf16")
    q = dev(x).transpose(1, 2)
    out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    R.ret_rotary(q, q_out=out)
    xt = x.f64.transpose(0, 2, 1, 3)
    check(out, od.rotary(xt, pos, f.numpy()), xt, "bf16")
    wide = torch.full((B, N, H, d + 3), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., :d] = q
    out = torch.full((B, N, H, d + 1), 7.0, dtype=torch.bfloat16, device="cuda")
    R.ret_rotary(wide[..., :d], q_out=out[..., :d])
    check(out[..., :d], od.rotary(xt, pos, f.numpy()), xt, "bf16")
    assert torch.all(out[..., d] == 7.0)
    one = q[:, :, :1].expand(B, N, H, d)
    got = R.ret_rotary(one)
    assert torch.equal(got[:, :, 0], got[:, :, 2])
    check(got[:, :, :1], od.rotary(host64(q[:, :, :1]), pos, f.numpy()), host64(q[:, :, :1]), "bf16")


def test_on_another_stream_and_in_a_graph():
    B, N, H, d = 1, 300, 8, 256
    x = make_tensor(605, 1, (B, N, H, d), "bf16")
    q = dev(x)
    want = R.ret_rotary(q, layout="half")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    R.ret_rotary(q, layout="half", q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        R.ret_rotary(q, layout="half", q_out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
