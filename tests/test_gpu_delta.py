"""GPU parity of the gated delta rule against the fp64 oracle.

Tolerances (relative L2 of a (sequence, head) slice).
* fp32 inputs, token by token, and one decode step: fp32 arithmetic, the
  suite's 1e-5.
* bf16 inputs in chunks, fp32 results (out, states): every fp32 factor of a
  product is two fp16 terms, off by at most 2^-22 of the value (each term's
  rounding is at most 2^-11 of what it rounds), and the product of the two
  second terms, 2^-22 again, is left out: 2^-21 a product.  A result passes
  four products (the state, T, the corrections, the scores), 2^-19, and as much
  again for the fp32 sums: 2^-18.
* a bf16 out: its own rounding, at most 2^-8 of the value and 1.7e-3 of a
  slice's norm, and one fp16 term each of the state, the corrections and the
  scores, 2^-11 of a value at most; the suite's 5e-3."""
import numpy as np
import pytest
import torch

from oracle import delta as od
from retention_inputs import make_tensor
from tests.helpers import TOL_BF16, TOL_F32, dev, err_out, err_state, host64

pytestmark = pytest.mark.gpu

TOL_SPLIT = 2.0 ** -18
R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


def inputs(seed, B, N, Hk, H, dk, dv, dtype, fast=0.5):
    """Unit keys, queries of length dk^-1/2; decays from slow (0.003 a token) to ``fast`` per head."""
    r = np.random.default_rng(seed)

    def unit(*shape):
        x = r.standard_normal(shape)
        return x / np.linalg.norm(x, axis=-1, keepdims=True)

    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    f = {"q": torch.from_numpy(unit(B, N, Hk, dk) * dk ** -0.5).to(t), "k": torch.from_numpy(unit(B, N, Hk, dk)).to(t),
         "v": torch.from_numpy(r.standard_normal((B, N, H, dv))).to(t)}
    rate = np.exp(np.linspace(np.log(0.003), np.log(fast), H))
    f["g"] = torch.from_numpy(-rate * np.log1p(np.exp(r.standard_normal((B, N, H))))).float()
    f["beta"] = torch.from_numpy(1 / (1 + np.exp(-r.standard_normal((B, N, H))))).float()
    return f, torch.from_numpy(0.3 * r.standard_normal((B, H, dk, dv))).float()


def cuda(f):
    return {n: t.cuda() for n, t in f.items()}


def f64(f):
    return {n: host64(t) for n, t in f.items()}


SHAPES = [
    # B, N, Hk, H, dk, dv
    (1, 1, 1, 1, 64, 64),
    (2, 63, 1, 2, 64, 128),
    (1, 64, 2, 2, 128, 64),
    (1, 65, 1, 1, 256, 64),
    (2, 200, 2, 4, 128, 128),
    (1, 500, 1, 3, 64, 72),       # a slice of eight columns
    (1, 300, 1, 1, 256, 200),
    (1, 700, 2, 2, 128, 8),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,N,Hk,H,dk,dv", SHAPES)
def test_chunked_forward(B, N, Hk, H, dk, dv, state, out_dtype):
    f, s0 = inputs(801, B, N, Hk, H, dk, dv, "bf16")
    assert R.ret_delta_workspace_bytes(B, N, Hk, H, dk, dv) > 0
    out, S = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda() if state else None, out_dtype=out_dtype,
                                           want_final_state=True)
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0) if state else None)
    assert err_state(host64(S), Sref) < TOL_SPLIT
    if out_dtype == torch.float32:
        assert err_out(host64(out), ref) < TOL_SPLIT
    elif N > 1:
        assert err_out(host64(out), ref) < TOL_BF16
    # a call without the state writes the same output
    again = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda() if state else None, out_dtype=out_dtype)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype,B,N,Hk,H,dk,dv", [
    ("f32", 1, 64, 8, 8, 16, 16),     # the fp32 exercise shape
    ("f32", 2, 50, 2, 4, 128, 64),
    ("f32", 1, 33, 1, 1, 256, 7),
    ("f32", 1, 3, 1, 1, 1, 1),
    ("bf16", 1, 40, 1, 2, 100, 64),   # dk off the chunked path
    ("bf16", 2, 20, 1, 1, 64, 33),    # dv off the chunked path
])
def test_token_by_token_forward(dtype, B, N, Hk, H, dk, dv):
    f, s0 = inputs(802, B, N, Hk, H, dk, dv, dtype)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    assert R.ret_delta_workspace_bytes(B, N, Hk, H, dk, dv, t) == 0
    out, S = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda(), out_dtype=torch.float32,
                                           want_final_state=True)
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0))
    assert err_out(host64(out), ref) < TOL_F32
    assert err_state(host64(S), Sref) < TOL_F32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_leave_padded_rows_alone(dtype):
    """Lengths of zero, one, whole chunks and their neighbours, beyond N and
    below zero; the padded rows hold NaN and infinities, and out keeps what it held."""
    B, N, Hk, H, dk, dv = 8, 200, 1, 2, 64, 64
    f, s0 = inputs(803, B, N, Hk, H, dk, dv, dtype)
    lens = [0, 1, 63, 64, 65, 200, 500, -3]
    clamped = [min(max(n, 0), N) for n in lens]
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0), lengths=clamped)
    for b, n in enumerate(clamped):
        for i, name in enumerate(("q", "k", "v", "g", "beta")):
            f[name][b, n:] = (float("nan"), float("inf"), -float("inf"))[(b + i) % 3]
    out = torch.full((B, N, H, dv), 7.0, dtype=torch.float32, device="cuda")
    _, S = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda(), out=out, want_final_state=True,
                                         lengths=torch.tensor(lens, dtype=torch.int32).cuda())
    tol = TOL_SPLIT if dtype == "bf16" else TOL_F32
    assert err_state(host64(S), Sref) < tol
    assert torch.equal(S[0].cpu(), s0[0]) and torch.equal(S[7].cpu(), s0[7])
    for b, n in enumerate(clamped):
        assert torch.all(out[b, n:] == 7.0)
        if n:
            assert err_out(host64(out[b:b + 1, :n]), ref[b:b + 1, :n]) < tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_split_sequence_and_state_in_place(dtype):
    B, N, Hk, H, dk, dv = 1, 300, 2, 2, 128, 64
    f, s0 = inputs(804, B, N, Hk, H, dk, dv, dtype)
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0))
    S, outs = s0.cuda(), []
    for a, b in ((0, 1), (1, 130), (130, 194), (194, 300)):
        part = {n: t[:, a:b].contiguous() for n, t in cuda(f).items()}
        o, S2 = R.ret_delta_forward_chunkwise(**part, initial_state=S, final_state=S, out_dtype=torch.float32)
        assert S2 is S
        outs.append(o)
    tol = TOL_SPLIT if dtype == "bf16" else TOL_F32
    assert err_out(host64(torch.cat(outs, 1)), ref) < tol
    assert err_state(host64(S), Sref) < tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_at_their_ends(dtype):
    """beta 0 and 1, g 0 (nothing forgotten), -inf and the lowest finite value (the state dropped)."""
    B, N, Hk, H, dk, dv = 1, 150, 1, 3, 64, 64
    f, s0 = inputs(805, B, N, Hk, H, dk, dv, dtype)
    f["beta"][0, 10:20] = 0.0
    f["beta"][0, 30:90] = 1.0
    f["g"][..., 0] = 0.0
    f["g"][0, 40, 1] = -float("inf")
    f["g"][0, 41, 1] = -float("inf")
    f["g"][0, 100, 2] = torch.finfo(torch.float32).min
    f["g"][0, 64, 2] = -87.0
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0))
    out, S = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda(), out_dtype=torch.float32,
                                           want_final_state=True)
    tol = TOL_SPLIT if dtype == "bf16" else TOL_F32
    assert err_out(host64(out), ref) < tol
    assert err_state(host64(S), Sref) < tol


def test_no_token_reads_a_later_one():
    """Up to the number format: a chunk's tiles are brought near one by a power
    of two that all of its tokens decide, so a later token can change which of
    the bits beyond the 22nd an earlier one loses."""
    B, N, Hk, H, dk, dv = 1, 190, 1, 1, 128, 64
    f, _ = inputs(806, B, N, Hk, H, dk, dv, "bf16")
    a = R.ret_delta_forward_chunkwise(**cuda(f), out_dtype=torch.float32)
    cut = 100
    for n in ("q", "k", "v", "g", "beta"):
        f[n][:, cut:] = f[n][:, cut:].flip(1) if n != "g" else f[n][:, cut:] * 3
    b = R.ret_delta_forward_chunkwise(**cuda(f), out_dtype=torch.float32)
    assert torch.equal(a[:, :64], b[:, :64])  # the chunk before
    assert err_out(host64(a[:, :cut]), host64(b[:, :cut])) < TOL_SPLIT
    assert not torch.equal(a[:, cut:], b[:, cut:])


@pytest.mark.parametrize("B,Hk,H,dk,dv,dtype,out_dtype", [
    (1, 1, 1, 1, 4, "f32", torch.float32),
    (1, 8, 16, 128, 128, "bf16", torch.bfloat16),
    (3, 2, 2, 100, 36, "bf16", torch.float32),
    (64, 4, 4, 256, 512, "bf16", torch.float32),   # many columns: the wide form
    (40, 2, 4, 64, 192, "f32", torch.bfloat16),
    (2, 1, 5, 256, 20, "f32", torch.float32),
])
def test_decode_step(B, Hk, H, dk, dv, dtype, out_dtype):
    f, s0 = inputs(807, B, 3, Hk, H, dk, dv, dtype)
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0))
    S = s0.cuda()
    for t in range(3):
        step = {n: x[:, t].contiguous().cuda() for n, x in f.items()}
        o = R.ret_delta_decode_step(**step, state=S, out_dtype=out_dtype)
        if out_dtype == torch.float32:
            assert err_out(host64(o)[:, None], ref[:, t:t + 1]) < TOL_F32
        else:  # one rounding of the output
            assert np.all(np.abs(host64(o) - ref[:, t]) <= 2.0 ** -8 * np.abs(ref[:, t]) + 1e-5 * np.abs(ref[:, t]).max())
    assert err_state(host64(S), Sref) < TOL_F32


def test_prefill_then_decode():
    B, N, Hk, H, dk, dv = 2, 133, 2, 4, 128, 128
    f, _ = inputs(808, B, N + 4, Hk, H, dk, dv, "bf16")
    ref, Sref = od.delta_forward(**f64(f))
    c = cuda(f)
    out, S = R.ret_delta_forward_chunkwise(**{n: t[:, :N].contiguous() for n, t in c.items()}, out_dtype=torch.float32,
                                           want_final_state=True)
    outs = [out]
    for t in range(N, N + 4):
        outs.append(R.ret_delta_decode_step(**{n: x[:, t].contiguous() for n, x in c.items()}, state=S)[:, None])
    assert err_out(host64(torch.cat(outs, 1)), ref) < TOL_SPLIT
    assert err_state(host64(S), Sref) < TOL_SPLIT


def test_two_streams_at_once_and_a_graph():
    """Two calls side by side with workspaces of their own give the bits of calls
    alone; a captured prefill and decode step replay."""
    fs = [inputs(s, 1, 400, 2, 2, 128, 128, "bf16")[0] for s in (809, 810)]
    cs = [cuda(f) for f in fs]
    want = [R.ret_delta_forward_chunkwise(**c, want_final_state=True) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append([R.ret_delta_forward_chunkwise(**c, want_final_state=True) for _ in range(4)])
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        for g in gs:
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
    c = cs[0]
    step = {n: t[:, 0].contiguous() for n, t in c.items()}
    S = want[0][1].clone()
    o_want = R.ret_delta_decode_step(**step, state=S)
    ws = torch.empty(R.ret_delta_workspace_bytes(1, 400, 2, 2, 128, 128), dtype=torch.uint8, device="cuda")
    out, fin = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    o = torch.empty_like(o_want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        R.ret_delta_forward_chunkwise(**c, out=out, final_state=fin, workspace=ws)
        R.ret_delta_decode_step(**step, state=fin, out=o)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0][0]) and torch.equal(fin, S) and torch.equal(o, o_want)
