"""The number format of the chunked gated delta rule, and its blocks of several
groups of columns.

Every tile is brought near one by a power of two before it is split into fp16
terms, so a power of two on an input is a power of two on the result, bit for
bit; the tolerances of the other cases are those of the parity tests."""
import numpy as np
import pytest
import torch

from oracle import delta as od
from retention_inputs import make_tensor
from tests.helpers import dev, err_out, err_state, host64
from tests.test_gpu_delta import TOL_SPLIT, cuda, f64, inputs
from tests.test_gpu_delta_backward import check

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


def forward(c, s0):
    return R.ret_delta_forward_chunkwise(**c, initial_state=s0, out_dtype=torch.float32, want_final_state=True)


@pytest.mark.parametrize("e", [-40, 40])
@pytest.mark.parametrize("dk", [64, 256])
def test_values_and_states_scale_exactly(dk, e):
    f, s0 = inputs(821, 2, 140, 1, 2, dk, 40, "bf16")
    c, s0 = cuda(f), s0.cuda()
    out, S = forward(c, s0)
    c["v"] = c["v"] * 2.0 ** e
    out2, S2 = forward(c, s0 * 2.0 ** e)
    assert torch.equal(out2, out * 2.0 ** e) and torch.equal(S2, S * 2.0 ** e)


@pytest.mark.parametrize("a,b", [(-7, 3), (9, -5)])
def test_keys_and_queries_scale_exactly(a, b):
    """k 2^a with beta 2^-2a and v 2^a is the same rule; q 2^b scales the output."""
    f, s0 = inputs(822, 2, 140, 1, 2, 128, 40, "bf16")
    c, s0 = cuda(f), s0.cuda()
    out, S = forward(c, s0)
    c["k"], c["v"], c["beta"] = c["k"] * 2.0 ** a, c["v"] * 2.0 ** a, c["beta"] * 2.0 ** (-2 * a)
    c["q"] = c["q"] * 2.0 ** b
    out2, S2 = forward(c, s0)
    assert torch.equal(out2, out * 2.0 ** b) and torch.equal(S2, S)


@pytest.mark.parametrize("e", [-30, 30])
@pytest.mark.parametrize("Hk", [1, 2])
def test_gradients_scale_exactly(Hk, e):
    f, s0 = inputs(823, 2, 140, Hk, 2, 128, 40, "bf16")
    c = cuda(f)
    dout, dS = dev(make_tensor(823, 4, (2, 140, 2, 40), "bf16")), dev(make_tensor(823, 5, (2, 2, 128, 40), "f32", 0.3))
    a = R.ret_delta_backward_chunkwise(**c, dout=dout, initial_state=s0.cuda(), dfinal_state=dS)
    b = R.ret_delta_backward_chunkwise(**c, dout=dout * 2.0 ** e, initial_state=s0.cuda(), dfinal_state=dS * 2.0 ** e)
    for x, y in zip(a, b):
        assert torch.equal(y, x * 2.0 ** e)


def test_rows_of_different_magnitude():
    """Key norms from 2^-6 to 2^6 (with beta to match), values over 2^12, zero keys and values."""
    B, N, H = 1, 200, 2
    f, s0 = inputs(824, B, N, H, H, 64, 64, "bf16")
    r = np.random.default_rng(824)
    e = torch.from_numpy(r.integers(-6, 7, (B, N, H))).float()
    f["k"] = (f["k"].float() * 2.0 ** e[..., None]).to(torch.bfloat16)
    f["beta"] = f["beta"] * 2.0 ** (-2 * e)
    f["v"] = (f["v"].float() * 2.0 ** (e[..., None] + torch.from_numpy(r.integers(-6, 7, (B, N, H, 1))).float())).to(torch.bfloat16)
    f["k"][0, 20:23] = 0
    f["v"][0, 50:120] = 0
    f["q"][0, 70] = 0
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0))
    out, S = forward(cuda(f), s0.cuda())
    assert err_out(host64(out), ref) < TOL_SPLIT
    assert err_state(host64(S), Sref) < TOL_SPLIT


@pytest.mark.parametrize("dk", [64, 256])
def test_one_key_with_equal_elements(dk):
    """The largest products that the scales allow: every key the same, its elements
    and the state's too, beta |k|^2 = 2, so that the state turns round at each token.

    Tolerance: the factors of a product are off by 2^-22.  A correction sums 64
    terms T r with |T| = 2: 8 x 2 x 2^-22 = 2^-18 of independent errors; the state
    sums 64 of those times beta k k = 2: 2^-14 a chunk, less than 2^-13 in three."""
    B, N, H, dv = 1, 140, 1, 24
    f, _ = inputs(825, B, N, H, H, dk, dv, "bf16")
    e = 2 - 2.0 ** -6
    f["k"] = torch.full_like(f["k"], e)
    f["beta"] = torch.full_like(f["beta"], 2 / (dk * e ** 2))
    f["g"] = torch.zeros_like(f["g"])
    s0, dS = (torch.full((B, H, dk, dv), e) for _ in range(2))
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0))
    out, S = forward(cuda(f), s0.cuda())
    assert err_out(host64(out), ref) < 2.0 ** -13
    assert err_state(host64(S), Sref) < 2.0 ** -13
    dout = make_tensor(825, 4, (B, N, H, dv), "bf16")
    grads = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), initial_state=s0.cuda(), dfinal_state=dS.cuda())
    assert all(torch.isfinite(x).all() for x in grads)


def test_all_zero_inputs():
    B, N, H, dk, dv = 1, 70, 2, 64, 24
    z = {"q": torch.zeros(B, N, H, dk), "k": torch.zeros(B, N, H, dk), "v": torch.zeros(B, N, H, dv)}
    c = {n: t.bfloat16().cuda() for n, t in z.items()}
    c["g"], c["beta"] = torch.zeros(B, N, H, device="cuda"), torch.ones(B, N, H, device="cuda")
    s0 = torch.randn(B, H, dk, dv, device="cuda")
    out, S = forward(c, s0)
    assert not out.any() and torch.equal(S, s0)
    grads = R.ret_delta_backward_chunkwise(**c, dout=torch.zeros_like(c["v"]), initial_state=s0, dfinal_state=s0)
    for x in grads[:3] + grads[4:5]:
        assert not x.any()
    # the state's gradient passes through; a gate's is <dS, S>
    assert torch.equal(grads[5], s0)
    assert torch.allclose(grads[3], (s0 * s0).sum((2, 3))[:, None].expand(B, N, H), rtol=2.0 ** -17)


MANY = [
    # B, N, Hk, H, dk, dv: several groups of 16 columns to a block, the last block's partly behind dv
    (4, 130, 8, 16, 128, 72),
    (3, 70, 8, 16, 64, 200),
    (2, 66, 8, 16, 256, 168),
    (5, 65, 16, 16, 64, 40),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,N,Hk,H,dk,dv", MANY)
def test_blocks_of_several_groups(B, N, Hk, H, dk, dv, out_dtype):
    f, s0 = inputs(825, B, N, Hk, H, dk, dv, "bf16")
    lens = [N, 1, 0, N - 1, N + 3][:B]
    out = torch.full((B, N, H, dv), -7.0, dtype=out_dtype, device="cuda")
    _, S = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda(), out=out, want_final_state=True,
                                         lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0), lengths=lens)
    assert err_state(host64(S), Sref) < TOL_SPLIT
    got = host64(out)
    for b, n in enumerate(lens):
        n = min(n, N)
        assert (got[b, n:] == -7).all()
        if out_dtype == torch.float32 and n:
            assert err_out(got[b:b + 1, :n], ref[b:b + 1, :n]) < TOL_SPLIT
        elif n:  # one rounding, on top of the fp16 terms' 2^-10 of a row's length
            assert np.all(np.abs(got[b, :n] - ref[b, :n]) <= 2.0 ** -8 * np.abs(ref[b, :n]) + 2.0 ** -10 * np.abs(ref[b, :n]).max(-1, keepdims=True))


@pytest.mark.parametrize("B,N,Hk,H,dk,dv", MANY)
def test_gradients_of_several_groups(B, N, Hk, H, dk, dv):
    f, s0 = inputs(826, B, N, Hk, H, dk, dv, "bf16")
    dout, dS = make_tensor(826, 4, (B, N, H, dv), "bf16"), make_tensor(826, 5, (B, H, dk, dv), "f32", 0.3)
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), initial_state=s0.cuda(), dfinal_state=dev(dS))
    check(got, od.delta_backward(**f64(f), dout=dout.f64, initial_state=host64(s0), dfinal_state=dS.f64), f64(f))
