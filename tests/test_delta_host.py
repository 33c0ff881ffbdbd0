"""Host-side checks of the rotary, layer norm and delta-rule entry points: what
they refuse, before anything is launched, and the sizes of their workspaces."""
import ctypes
import math

import pytest
import torch

import linear_recurrent_sequence_chunkwise_b200 as R
from tests.test_abi_host import needs_no_gpu

F32, BF16 = R.RET_F32, R.RET_BF16
INVALID, UNSUPPORTED = R.RET_ERR_INVALID_ARG, R.RET_ERR_UNSUPPORTED


def at(i, off=0):
    """A made-up, far apart device address (never read: the call is refused first)."""
    return ctypes.c_void_p((i << 40) + off)


def refused(status, want):
    assert status == want, (status, R.ret_last_error_string())
    assert R.ret_last_error_string()


# -------------------------------------------------------------------- rotary

def strides(*s):
    return (ctypes.c_int64 * 3)(*s) if s else None


FREQS = (ctypes.c_double * 256)(*[1.0 / (1 + i) for i in range(256)])


def rotary(q=at(1), k=at(2), qo=at(3), ko=at(4), qs=None, ks=None, qos=None, kos=None, freqs=FREQS, scale=1.0, pos=at(5), layout=0,
           B=2, N=3, H=4, Hk=2, d=64, rd=32, dt=BF16):
    return R.lib.ret_rotary(q, k, qo, ko, qs, ks, qos, kos, freqs, scale, pos, 0, 0, layout, B, N, H, Hk, d, rd, dt, None)


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(qo=None), dict(freqs=None), dict(k=None), dict(ko=None), dict(dt=7), dict(B=0), dict(N=0), dict(H=0),
    dict(Hk=0), dict(d=63, rd=32), dict(rd=0), dict(rd=31), dict(rd=66), dict(d=1024, rd=514), dict(layout=2), dict(scale=math.inf),
    dict(scale=math.nan), dict(freqs=(ctypes.c_double * 16)(*([1.0] * 15 + [math.nan]))), dict(H=65536), dict(q=at(1, 1)),
    dict(pos=at(5, 4)), dict(N=1 << 31 - 1, B=1 << 30),
    dict(qo=at(1, 2)),                          # overlaps its input by part
    dict(ko=at(3)),                             # the outputs overlap
    dict(qo=at(2)),                             # q's output is k
    dict(pos=at(3, 8)),                         # positions in an output
    dict(qos=strides(0, 256, 64)),              # rows of an output share elements
    dict(qos=strides(768, 256, 32)),
    dict(qs=strides(-1, 256, 64)),
])
def test_rotary_refusals(kw):
    refused(rotary(**kw), INVALID)


@pytest.mark.parametrize("kw", [dict(rd=0), dict(rd=7), dict(base=0.0), dict(base=math.inf), dict(scaling=3), dict(scaling=1, factor=0.5),
                                dict(scaling=2, base=1.0, factor=2.0), dict(scaling=2, original=0.0, factor=2.0),
                                dict(scaling=2, fast=1.0, slow=2.0, factor=2.0)])
def test_rotary_frequency_refusals(kw):
    a = dict(rd=32, base=1e4, scaling=0, factor=1.0, original=4096.0, fast=32.0, slow=1.0)
    a.update(kw)
    out, scale = (ctypes.c_double * 256)(), ctypes.c_double()
    refused(R.lib.ret_rotary_frequencies(a["rd"], a["base"], a["scaling"], a["factor"], a["original"], a["fast"], a["slow"],
                                         ctypes.cast(out, ctypes.c_void_p), ctypes.byref(scale)), INVALID)


# ---------------------------------------------------------------- layer norm

def ln_forward(x=at(1), gain=at(2), bias=at(3), eps=1e-5, rows=8, d=64, y=at(4), mean=at(5), rstd=at(6), dt=BF16, w=BF16):
    return R.lib.ret_layernorm_forward(x, gain, bias, eps, rows, d, y, mean, rstd, dt, w, None)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(rows=0), INVALID),
    (dict(d=0), INVALID), (dict(dt=3), INVALID), (dict(w=3), INVALID), (dict(rows=1 << 31), INVALID), (dict(d=8193), UNSUPPORTED),
    (dict(x=at(1, 1)), INVALID), (dict(gain=at(2, 1)), INVALID), (dict(mean=at(5, 2)), INVALID), (dict(y=at(1, 2)), INVALID),
    (dict(y=at(1)), INVALID), (dict(mean=at(6)), INVALID), (dict(rstd=at(4)), INVALID), (dict(y=at(2, 64)), INVALID),
])
def test_layernorm_forward_refusals(kw, status):
    refused(ln_forward(**kw), status)


def ln_backward(dy=at(1), x=at(2), mean=at(3), rstd=at(4), gain=at(5), rows=8, d=64, dx=at(6), dgain=at(7), dbias=at(8), dt=BF16, w=F32,
                ws=at(9), nbytes=1 << 20):
    return R.lib.ret_layernorm_backward(dy, x, mean, rstd, gain, rows, d, dx, dgain, dbias, dt, w, ws, nbytes, None)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dx=None, dgain=None, dbias=None), INVALID), (dict(ws=None), INVALID), (dict(nbytes=16), INVALID), (dict(ws=at(9, 8)), INVALID),
    (dict(d=8193), UNSUPPORTED), (dict(dx=at(1)), INVALID), (dict(dgain=at(8)), INVALID), (dict(ws=at(6)), INVALID), (dict(rows=-1), INVALID),
])
def test_layernorm_backward_refusals(kw, status):
    refused(ln_backward(**kw), status)


def test_layernorm_workspace():
    size = R.ret_layernorm_backward_workspace_bytes
    assert size(1, 64) == 2 * 64 * 4 and size(0, 64) == 0 and size(64, 8193) == 0
    assert size(10 ** 6, 2048) == size(10 ** 9, 2048) == 296 * 2 * 2048 * 4  # a partial row for each block


# ---------------------------------------------------------------- delta rule

def forward(q=at(1), k=at(2), v=at(3), g=at(4), beta=at(5), lens=None, s0=None, B=2, N=70, Hk=2, H=4, dk=64, dv=64, out=at(6), fs=at(7),
            dt=BF16, odt=BF16, ws=at(8), nbytes=1 << 30):
    return R.lib.ret_delta_forward_chunkwise(q, k, v, g, beta, lens, s0, B, N, Hk, H, dk, dv, out, fs, None, dt, odt, ws, nbytes)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID), (dict(beta=None), INVALID),
    (dict(out=None), INVALID), (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(H=3), INVALID), (dict(Hk=0), INVALID), (dict(dk=0), INVALID),
    (dict(dv=0), INVALID), (dict(dk=257), UNSUPPORTED), (dict(dt=5), INVALID), (dict(odt=5), INVALID), (dict(B=65536), INVALID),
    (dict(H=65536, Hk=65536), INVALID), (dict(N=1 << 30, H=1 << 14, Hk=1), INVALID), (dict(q=at(1, 8)), INVALID), (dict(out=at(6, 2)), INVALID),
    (dict(g=at(4, 2)), INVALID), (dict(lens=at(9, 2)), INVALID), (dict(ws=None), INVALID), (dict(nbytes=1000), INVALID),
    (dict(ws=at(8, 16)), INVALID), (dict(out=at(3)), INVALID), (dict(out=at(1)), INVALID), (dict(fs=at(6)), INVALID), (dict(ws=at(7)), INVALID),
    (dict(s0=at(7, 16)), INVALID),              # the states overlap by part
    (dict(lens=at(6)), INVALID),
])
def test_delta_forward_refusals(kw, status):
    refused(forward(**kw), status)


def decode(q=at(1), k=at(2), v=at(3), g=at(4), beta=at(5), state=at(6), out=at(7), B=2, Hk=2, H=4, dk=64, dv=64, dt=BF16, odt=BF16):
    return R.lib.ret_delta_decode_step(q, k, v, g, beta, state, out, None, B, Hk, H, dk, dv, dt, odt)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(state=None), INVALID), (dict(out=None), INVALID), (dict(dv=66), INVALID), (dict(dk=260), UNSUPPORTED), (dict(H=5), INVALID),
    (dict(out=at(6)), INVALID), (dict(state=at(1)), INVALID), (dict(state=at(6, 4)), INVALID), (dict(v=at(7)), INVALID), (dict(B=0), INVALID),
])
def test_delta_decode_refusals(kw, status):
    refused(decode(**kw), status)


def backward(q=at(1), k=at(2), v=at(3), g=at(4), beta=at(5), dout=at(6), lens=None, s0=None, dfs=None, B=2, N=70, Hk=2, H=4, dk=64, dv=64,
             dq=at(7), dkk=at(8), dvv=at(9), dg=at(10), db=at(11), ds0=None, dt=BF16, gdt=F32, ws=at(12), nbytes=1 << 32):
    return R.lib.ret_delta_backward_chunkwise(q, k, v, g, beta, dout, lens, s0, dfs, B, N, Hk, H, dk, dv, dq, dkk, dvv, dg, db, ds0, None,
                                              dt, gdt, ws, nbytes)


@needs_no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(dout=None), INVALID), (dict(dq=None), INVALID), (dict(dkk=None), INVALID), (dict(dvv=None), INVALID), (dict(dg=None), INVALID),
    (dict(db=None), INVALID), (dict(gdt=4), INVALID), (dict(B=32768), INVALID), (dict(dt=F32), UNSUPPORTED), (dict(dk=100), UNSUPPORTED),
    (dict(dv=12), UNSUPPORTED), (dict(ws=None), INVALID), (dict(nbytes=4096), INVALID), (dict(dq=at(8)), INVALID), (dict(dvv=at(6)), INVALID),
    (dict(dg=at(4)), INVALID), (dict(ws=at(1)), INVALID), (dict(ds0=at(11)), INVALID), (dict(dg=at(10, 8)), INVALID),
    (dict(dfs=at(13, 4)), INVALID), (dict(s0=at(7)), INVALID),
])
def test_delta_backward_refusals(kw, status):
    refused(backward(**kw), status)


def test_delta_workspaces():
    fwd, bwd = R.ret_delta_workspace_bytes, R.ret_delta_backward_workspace_bytes
    for size in (fwd, bwd):
        assert size(1, 64, 1, 1, 64, 64) > 0 and size(1, 65, 1, 1, 64, 64) == 2 * size(1, 64, 1, 1, 64, 64) or size is bwd
        assert size(0, 64, 1, 1, 64, 64) == size(1, 64, 2, 3, 64, 64) == 0
        assert size(1, 64, 1, 1, 96, 64) == size(1, 64, 1, 1, 64, 60) == size(1, 64, 1, 1, 64, 64, torch.float32) == 0
    assert bwd(1, 64, 1, 2, 64, 64) > fwd(1, 64, 1, 2, 64, 64)
    # far past 32 bits without wrapping
    assert bwd(64, 1 << 20, 16, 16, 256, 512) > 1 << 40


# ---------------------------------------------------------------- the binding

def test_binding_refuses_on_host_tensors():
    """Wrong shapes, dtypes and places are refused by name before a pointer is taken."""
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="gain must have shape"):
        R.ret_layernorm_forward(x, torch.zeros(7))
    with pytest.raises(TypeError, match="gain must be"):
        R.ret_layernorm_forward(x, torch.zeros(8, dtype=torch.float16))
    with pytest.raises(ValueError, match="at least one row"):
        R.ret_layernorm_forward(torch.zeros(0, 8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        R.ret_layernorm_forward(x)
    with pytest.raises(ValueError, match="rstd must have shape"):
        R.ret_layernorm_backward(x, x, torch.zeros(4), torch.zeros(8))
    q, k = torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, 2, 8)
    with pytest.raises(ValueError, match="layout"):
        R.ret_rotary(q, layout="pairs")
    with pytest.raises(ValueError, match="expected q"):
        R.ret_rotary(q, k[:, :2])
    with pytest.raises(TypeError, match="share a dtype"):
        R.ret_rotary(q, k.bfloat16())
    with pytest.raises(ValueError, match="k_out without k"):
        R.ret_rotary(q, k_out=k)
    with pytest.raises(ValueError, match="float64 vector"):
        R.ret_rotary(q, freqs=torch.zeros(4))
    with pytest.raises(ValueError, match="expected 2"):
        R.ret_rotary(q, freqs=torch.zeros(3, dtype=torch.float64), rotary_dim=4)
    with pytest.raises(ValueError, match="scaling"):
        R.ret_rotary_frequencies(8, scaling="cubic")
    v, g = torch.zeros(2, 3, 4, 16), torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="expected q, k"):
        R.ret_delta_forward_chunkwise(k, q, v, g, g)
    with pytest.raises(ValueError, match="beta must have shape"):
        R.ret_delta_forward_chunkwise(k, k, v, g, g[..., :2])
    with pytest.raises(TypeError, match="g must be"):
        R.ret_delta_forward_chunkwise(k, k, v, g.bfloat16(), g)
    with pytest.raises(TypeError, match="lengths must be"):
        R.ret_delta_forward_chunkwise(k, k, v, g, g, lengths=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="initial_state must have shape"):
        R.ret_delta_forward_chunkwise(k, k, v, g, g, initial_state=torch.zeros(2, 4, 16, 8))
    with pytest.raises(TypeError, match="dout must be"):
        R.ret_delta_backward_chunkwise(k, k, v, g, g, v.bfloat16())
    with pytest.raises(ValueError, match="dk must have shape"):
        R.ret_delta_backward_chunkwise(k, k, v, g, g, v, dk=q)
    with pytest.raises(ValueError, match="state must"):
        R.ret_delta_decode_step(k[:, 0], k[:, 0], v[:, 0], g[:, 0], g[:, 0], None)
    with pytest.raises(ValueError, match="state must have shape"):
        R.ret_delta_decode_step(k[:, 0], k[:, 0], v[:, 0], g[:, 0], g[:, 0], torch.zeros(2, 4, 16, 8))


def test_direct_binding_leaves_odd_arguments_to_the_general_way():
    """It answers None, and raises nothing, whatever it is given."""
    x = torch.zeros(4, 8)
    for fn, n in ((R._binding.layernorm_forward, 5), (R._binding.layernorm_backward, 5), (R._binding.delta_decode_step, 7),
                  (R._binding.rotary, 8), (R._binding.delta_forward, 10), (R._binding.delta_backward, 11)):
        for args in ([], [None] * n, [x] * n, ["a"] * n, [3] * n, [x] * (n + 1)):
            assert fn(*args) is None
