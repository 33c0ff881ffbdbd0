"""GPU parity of the gated delta rule's gradients against the fp64 oracle, and
of a whole pre-norm block step: norm, projections, positions, the rule, and
back.

Tolerances.  Every fp32 factor of a product is two fp16 terms (2^-22 of the
value at most, the product of the second terms, 2^-22, left out: 2^-21 a
product); a gradient passes at most eight products (state and corrections of
the forward; dU, dY and the state's gradient; the scores; the last product):
2^-18 of the slice's norm, and as much again for the fp32 sums: 2^-17.  dg sums
differences of row products that are up to ten times the result (their norm is
in the test), so it is held to 2^-17 of theirs.  A bf16 gradient adds one
rounding: 2^-8 of each value."""
import numpy as np
import pytest
import torch

from oracle import delta as od
from retention_inputs import make_tensor
from tests.helpers import dev, err_out, err_state, host64
from tests.test_gpu_delta import cuda, f64, inputs

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -17
R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state")


def check(got, ref, f, tol=TOL, rows=slice(None)):
    for name, x in zip(NAMES, got):
        if x is None:
            continue
        x, r = host64(x), ref[name]
        if name == "dinitial_state":
            assert err_state(x, r) < tol, name
            continue
        x, r = x[:, rows], r[:, rows]
        assert np.isfinite(x).all(), name
        if name in ("dg", "dbeta"):
            # per head; the row products that dg sums: |q dq| + |k dk|
            H, Hk = r.shape[2], ref["dq"].shape[2]
            terms = np.abs((f["q"] * ref["dq"]).sum(-1)) + np.abs((f["k"] * ref["dk"]).sum(-1))
            terms = np.repeat(terms, H // Hk, axis=2)[:, rows]
            scale = np.linalg.norm(r, axis=1) + (np.linalg.norm(terms, axis=1) if name == "dg" else 0)
            assert np.all(np.linalg.norm(x - r, axis=1) <= tol * scale + 1e-12), (name, (np.linalg.norm(x - r, axis=1) / scale).max())
        else:
            assert err_out(x, r) < tol, (name, err_out(x, r))


SHAPES = [
    # B, N, Hk, H, dk, dv
    (1, 1, 1, 1, 64, 64),
    (2, 64, 1, 1, 64, 64),
    (1, 65, 1, 2, 128, 64),
    (2, 200, 2, 4, 128, 128),
    (1, 190, 1, 3, 64, 72),
    (1, 150, 1, 1, 256, 136),
    (1, 130, 2, 4, 256, 64),
    (1, 300, 2, 2, 64, 8),
]


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,N,Hk,H,dk,dv", SHAPES)
def test_gradients(B, N, Hk, H, dk, dv, state):
    f, s0 = inputs(901, B, N, Hk, H, dk, dv, "bf16")
    dout = make_tensor(901, 4, (B, N, H, dv), "bf16")
    dS = make_tensor(901, 5, (B, H, dk, dv), "f32", 0.3)
    kw = dict(initial_state=s0.cuda(), dfinal_state=dev(dS)) if state else {}
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), **kw)
    assert (got[5] is not None) == state
    ref = od.delta_backward(**f64(f), dout=dout.f64, **({"initial_state": host64(s0), "dfinal_state": dS.f64} if state else {}))
    check(got, ref, f64(f))
    # bf16 gradients are the fp32 ones rounded once; the others the same
    half = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), grad_dtype=torch.bfloat16, **kw)
    for a, b in zip(half[:3], got[:3]):
        assert torch.equal(a, b.to(torch.bfloat16))
    for a, b in zip(half[3:], got[3:]):
        assert a is b is None or torch.equal(a, b)


def test_initial_state_gradient_without_a_state():
    f, _ = inputs(902, 1, 100, 1, 1, 64, 64, "bf16")
    dout = make_tensor(902, 4, (1, 100, 1, 64), "bf16")
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), want_dinitial_state=True)
    ref = od.delta_backward(**f64(f), dout=dout.f64)
    check(got, ref, f64(f))


def test_against_differences():
    """Directional differences of the GPU's own forward (fp32 out) along a random
    direction of every input.  The forward is good to 2^-14 of its norm; with a
    loss of norm |out| |dout| and steps of 2^-4 that is an error of
    2^-14 x 2^4 x |out| |dout| x 2 in a difference, and the step's own curvature
    is removed to third order by the central difference."""
    B, N, Hk, H, dk, dv = 1, 100, 1, 2, 64, 64
    f, s0 = inputs(903, B, N, Hk, H, dk, dv, "bf16")
    dout = make_tensor(903, 4, (B, N, H, dv), "bf16")
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), initial_state=s0.cuda())
    r = np.random.default_rng(903)

    def loss(fd, s):
        o, _ = od.delta_forward(**fd, initial_state=s)
        return (o * dout.f64).sum()

    base = f64(f)
    for name, grad in zip(("q", "k", "v", "g", "beta", "s"), got):
        x = host64(s0) if name == "s" else base[name]
        u = r.standard_normal(x.shape)
        h = 1e-5
        vals = [loss(base, x + d * h * u) if name == "s" else loss({**base, name: x + d * h * u}, host64(s0)) for d in (1, -1)]
        num = (vals[0] - vals[1]) / (2 * h)
        exact = (host64(grad) * u).sum()
        # random direction: the error of the sum is tol x the gradient's norm x a few
        assert abs(num - exact) < 5 * TOL * np.linalg.norm(host64(grad)) * np.abs(u).max() + 1e-6


@pytest.mark.parametrize("N,dk,dv,g", [(1, 64, 40, -25.0), (1, 256, 168, -25.0), (5, 128, 64, -20.0), (66, 64, 64, -20.0)])
def test_gates_behind_a_strong_decay(N, dk, dv, g):
    """dg itself, not next to the row products: what passes a decay of e^-25 is
    e^-25 of them.  It is the sum of four kinds of paths, each off by 2^-17 of its
    norm; over the heads their norms and the sum's are alike: 4 x 2^-17."""
    B, H = 2, 4
    f, s0 = inputs(909, B, N, H, H, dk, dv, "bf16")
    f["g"] = torch.full_like(f["g"], g)
    dout, dS = make_tensor(909, 4, (B, N, H, dv), "bf16"), make_tensor(909, 5, (B, H, dk, dv), "f32", 0.3)
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), initial_state=s0.cuda(), dfinal_state=dev(dS))
    ref = od.delta_backward(**f64(f), dout=dout.f64, initial_state=host64(s0), dfinal_state=dS.f64)
    assert np.linalg.norm(host64(got[3]) - ref["dg"]) < 2.0 ** -15 * np.linalg.norm(ref["dg"])


def test_calls_on_several_streams_together():
    """Calls that share the GPU wait longer within a block; the results stay the
    same bits.  Blocks of two groups of columns (the first shape) and of one."""
    sets = []
    for B, N, Hk, H, dk, dv in ((3, 300, 2, 6, 64, 200), (2, 400, 4, 8, 128, 200), (2, 700, 2, 4, 128, 128), (1, 500, 4, 4, 256, 96)):
        f, s0 = inputs(910, B, N, Hk, H, dk, dv, "bf16")
        sets.append((cuda(f), s0.cuda(), dev(make_tensor(910, 4, (B, N, H, dv), "bf16"))))

    def run(c, s0, dout):
        out, S = R.ret_delta_forward_chunkwise(**c, initial_state=s0, want_final_state=True)
        return [out, S, *R.ret_delta_backward_chunkwise(**c, dout=dout, initial_state=s0, dfinal_state=s0)]

    ref = [run(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(100):
        got = []
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got.append([run(*sets[(i + j) % 4]) for j in range(4)])
        torch.cuda.synchronize()
        for i in range(4):
            for j in range(4):
                for n, (a, b) in enumerate(zip(got[i][j], ref[(i + j) % 4])):
                    assert torch.equal(a, b), ((i + j) % 4, n)


def test_lengths_and_nan_in_padded_rows():
    B, N, Hk, H, dk, dv = 7, 150, 1, 2, 64, 64
    f, s0 = inputs(904, B, N, Hk, H, dk, dv, "bf16")
    lens = [0, 1, 63, 64, 65, 150, 999]
    clamped = [min(n, N) for n in lens]
    dout = dev(make_tensor(904, 4, (B, N, H, dv), "bf16"))
    dS = make_tensor(904, 5, (B, H, dk, dv), "f32", 0.3)
    ref = od.delta_backward(**f64(f), dout=host64(dout), lengths=clamped, initial_state=host64(s0), dfinal_state=dS.f64)
    for b, n in enumerate(clamped):
        for i, name in enumerate(("q", "k", "v", "g", "beta")):
            f[name][b, n:] = (float("nan"), float("inf"), -float("inf"))[(b + i) % 3]
        dout[b, n:] = float("nan")
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dout, initial_state=s0.cuda(), dfinal_state=dev(dS),
                                         lengths=torch.tensor(lens, dtype=torch.int32).cuda())
    clean = f64(f)
    for b, n in enumerate(clamped):
        for name in ("q", "k"):
            clean[name][b, n:] = 0
    check(got, ref, clean)
    for b, n in enumerate(clamped):
        for x in got[:5]:
            assert torch.all(x[b, n:] == 0)
    assert torch.equal(got[5][0].cpu(), torch.from_numpy(dS.stored[0]))  # nothing happened to it


def test_gates_at_their_ends():
    B, N, Hk, H, dk, dv = 1, 150, 1, 3, 64, 64
    f, s0 = inputs(905, B, N, Hk, H, dk, dv, "bf16")
    f["beta"][0, 10:20] = 0.0
    f["beta"][0, 30:90] = 1.0
    f["g"][..., 0] = 0.0
    f["g"][0, 40:42, 1] = -float("inf")
    f["g"][0, 100, 2] = torch.finfo(torch.float32).min
    f["g"][0, 64, 2] = -87.0
    dout = make_tensor(905, 4, (B, N, H, dv), "bf16")
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), initial_state=s0.cuda())
    ref = od.delta_backward(**f64(f), dout=dout.f64, initial_state=host64(s0))
    check(got, ref, f64(f))


def test_same_bits_streams_and_graphs():
    """Four calls on two streams give the bits of one call alone; a captured call
    replays, with an eager call on other inputs between."""
    B, N, Hk, H, dk, dv = 1, 330, 1, 2, 128, 128
    f, s0 = inputs(906, B, N, Hk, H, dk, dv, "bf16")
    c, dout = cuda(f), dev(make_tensor(906, 4, (B, N, H, dv), "bf16"))
    s0 = s0.cuda()
    want = R.ret_delta_backward_chunkwise(**c, dout=dout, initial_state=s0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            got.append(R.ret_delta_backward_chunkwise(**c, dout=dout, initial_state=s0))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(want, g):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        kept = R.ret_delta_backward_chunkwise(**c, dout=dout, initial_state=s0)
    other = R.ret_delta_backward_chunkwise(**c, dout=dout.flip(1).contiguous())
    assert not torch.equal(other[0], want[0])
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, kept):
        assert torch.equal(a, b)


def test_a_block_step_forward_and_back():
    """Pre-norm block step of two sequences: h = LN(x); q, k, v = h W; positions on
    q and k; the rule; then every gradient back to x and the norm's weights.  Each
    operator's result against the oracle applied to what that operator was given,
    and the gradients of the norm's weights against the oracle's whole chain (bf16
    hand-overs between the operators, each 2^-8 at most: five of them on the way
    there and six back, 11 x 2^-8 = 4.3e-2 of the norm)."""
    B, N, H, d, dm = 2, 90, 2, 64, 128
    x, gain, bias = make_tensor(907, 1, (B, N, dm), "bf16"), make_tensor(907, 2, (dm,), "bf16"), make_tensor(907, 3, (dm,), "bf16")
    W = [make_tensor(907, 10 + i, (dm, H * d), "bf16", dm ** -0.5 * (0.3 if i < 2 else 1.0)) for i in range(3)]
    f, _ = inputs(907, B, N, H, H, d, d, "bf16")
    g, beta = f["g"].cuda(), f["beta"].cuda()
    f64w = [w.f64 for w in W]
    freqs, _ = R.ret_rotary_frequencies(d // 2)
    pos = torch.tensor([[0], [1000]]).cuda() + torch.arange(N, device="cuda")
    h, mean, rstd = R.ret_layernorm_forward(dev(x), dev(gain), dev(bias), want_stats=True)
    q, k, v = (R.ret_linear_bf16(h.view(B * N, dm), dev(w), out_dtype=torch.bfloat16).view(B, N, H, d) for w in W)
    qr, kr = R.ret_rotary(q, k, freqs=freqs, positions=pos, layout="half")
    kr = (kr.float() / kr.float().norm(dim=-1, keepdim=True).clamp_min(1.0)).to(torch.bfloat16)  # |k| <= 1: stable
    out = R.ret_delta_forward_chunkwise(qr, kr, v, g, beta)
    ref, _ = od.delta_forward(host64(qr), host64(kr), host64(v), host64(g), host64(beta))
    assert err_out(host64(out), ref) < 5e-3
    dout = dev(make_tensor(907, 4, (B, N, H, d), "bf16"))
    dqr, dkr, dvv, dg, dbeta, _ = R.ret_delta_backward_chunkwise(qr, kr, v, g, beta, dout, grad_dtype=torch.bfloat16)
    rb = od.delta_backward(host64(qr), host64(kr), host64(v), host64(g), host64(beta), host64(dout))
    for a, n in ((dqr, "dq"), (dvv, "dv")):
        assert err_out(host64(a), rb[n]) < 5e-3
    dq = R.ret_rotary(dqr, freqs=freqs, positions=pos, layout="half", inverse=True)
    assert err_out(host64(dq), od.rotary(host64(dqr), host64(pos), freqs.numpy(), "half", inverse=True)) < 2.0 ** -8
    # back through W_q and W_v to the norm (k is left out: its clamp is torch's)
    dh = sum(R.ret_linear_bf16(t.reshape(B * N, H * d), dev(w).t().contiguous(), out_dtype=torch.float32)
             for t, w in ((dq, W[0]), (dvv, W[2]))).view(B, N, dm).to(torch.bfloat16)
    dx, dgain, dbias = R.ret_layernorm_backward(dh, dev(x), mean, rstd, dev(gain))
    R.ret_check_device_error()
    back = od.rotary(rb["dq"], host64(pos), freqs.numpy(), "half", inverse=True).reshape(B * N, -1) @ f64w[0].T + \
        rb["dv"].reshape(B * N, -1) @ f64w[2].T
    hx, hm, hr = od.layernorm(x.f64, gain.f64, bias.f64)
    rdx, rdg, rdb = od.layernorm_backward(back.reshape(B, N, dm), x.f64, hm, hr, gain.f64)
    for a, r_ in ((dx, rdx), (dgain, rdg), (dbias, rdb)):
        assert np.linalg.norm(host64(a) - r_) < 11 * 2.0 ** -8 * np.linalg.norm(r_)
