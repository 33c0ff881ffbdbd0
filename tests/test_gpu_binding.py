"""The short calls' direct binding against the general way through ctypes: the
same bits, the same refusals, the caller's stream and graphs; and workspaces
that the calls make for themselves, on a stream of the caller's choice."""
import pytest
import torch

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


def normal(*shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(len(shape) * 1000 + shape[-1])
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def calls():
    """(name, a call that the binding takes, the same with an output or a stream passed in)."""
    s = torch.cuda.current_stream()
    for dt in (torch.bfloat16, torch.float32):
        x, gain, bias = normal(5, 3, 96, dtype=dt), normal(96, dtype=dt), normal(96, dtype=dt)
        for stats in (False, True):
            yield "layernorm_forward", lambda s=None, x=x, stats=stats: R.ret_layernorm_forward(x, gain, bias, want_stats=stats, stream=s)
        yield "layernorm_forward", lambda s=None, x=x: R.ret_layernorm_forward(x, stream=s)
        _, mean, rstd = R.ret_layernorm_forward(x, want_stats=True, stream=s)
        dy = normal(5, 3, 96, dtype=dt)
        yield "layernorm_backward", lambda s=None, x=x, dy=dy, m=mean, r=rstd: R.ret_layernorm_backward(dy, x, m, r, gain.to(x.dtype), stream=s)
        q, k = normal(2, 7, 4, 64, dtype=dt), normal(2, 7, 2, 64, dtype=dt)
        freqs, scale = R.ret_rotary_frequencies(32, scaling="yarn", factor=2.0)
        pos = torch.randint(0, 9999, (2, 7), device="cuda")
        for layout in ("half", "interleaved"):
            yield "rotary", lambda s=None, q=q, k=k, l=layout: R.ret_rotary(q, k, freqs=freqs, positions=pos, layout=l, scale=scale, stream=s)
            yield "rotary", lambda s=None, q=q, l=layout: R.ret_rotary(q, freqs=freqs, pos_offset=5, layout=l, inverse=True, stream=s)
        q, k, v = normal(3, 2, 64, dtype=dt), normal(3, 2, 64, dtype=dt) / 8, normal(3, 4, 32, dtype=dt)
        g, beta, S0 = -normal(3, 4, dtype=torch.float32).abs(), normal(3, 4, dtype=torch.float32).sigmoid(), normal(3, 4, 64, 32, dtype=torch.float32)

        def step(s=None, q=q, k=k, v=v, out=None):
            S = S0.clone()
            return R.ret_delta_decode_step(q, k, v, g, beta, S, out_dtype=out, stream=s), S
        qs, ks, vs = normal(2, 70, 2, 64, dtype=dt) / 8, normal(2, 70, 2, 64, dtype=dt) / 8, normal(2, 70, 4, 40, dtype=dt)
        gs, bs = -normal(2, 70, 4, dtype=torch.float32).abs(), normal(2, 70, 4, dtype=torch.float32).sigmoid()
        lens, s0, do = torch.tensor([70, 33], dtype=torch.int32, device="cuda"), normal(2, 4, 64, 40, dtype=torch.float32), normal(2, 70, 4, 40, dtype=dt)
        for kw in ({}, {"lengths": lens, "initial_state": s0, "want_final_state": True, "out_dtype": torch.float32}):
            # rows behind an end are not written: the same zeros in both
            yield "delta_forward", lambda s=None, q=qs, k=ks, v=vs, kw=kw: R.ret_delta_forward_chunkwise(
                q, k, v, gs, bs, out=torch.zeros(2, 70, 4, 40, dtype=kw.get("out_dtype", q.dtype), device="cuda"), stream=s, **kw)
        if dt == torch.bfloat16:
            for kw in ({}, {"lengths": lens, "initial_state": s0, "dfinal_state": s0, "grad_dtype": torch.bfloat16}, {"want_dinitial_state": True}):
                yield "delta_backward", lambda s=None, kw=kw, q=qs, k=ks, v=vs, d=do: R.ret_delta_backward_chunkwise(q, k, v, gs, bs, d, stream=s, **kw)
        yield "delta_decode_step", step
        yield "delta_decode_step", lambda s=None, step=step: step(s, out=torch.bfloat16)


def as_list(r):
    return list(r) if isinstance(r, tuple) else [r]


def test_both_ways_give_the_same(monkeypatch):
    taken = {}
    for name in ("rotary", "layernorm_forward", "layernorm_backward", "delta_decode_step", "delta_forward", "delta_backward"):
        real = getattr(R._binding, name)

        def count(*a, real=real, name=name):
            r = real(*a)
            taken[name] = taken.get(name, 0) + (r is not None)
            return r
        monkeypatch.setattr(R._binding, name, count)
    for name, call in calls():
        before = taken.get(name, 0)
        direct = as_list(call())
        assert taken[name] == before + 1, name
        general = as_list(call(torch.cuda.current_stream()))
        assert taken[name] == before + 1, name
        for a, b in zip(direct, general, strict=True):
            assert (a is None) == (b is None)
            if a is None:
                continue
            assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b), name


def test_current_stream_and_graph():
    x = normal(40, 512)
    want = R.ret_layernorm_forward(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        y = R.ret_layernorm_forward(x)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = R.ret_layernorm_forward(x)
    z.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, want)


def test_refusals_are_worded_by_the_general_way():
    x = normal(4, 64)
    with pytest.raises(ValueError, match="gain must have shape"):
        R.ret_layernorm_forward(x, normal(32))
    with pytest.raises(TypeError, match="share a dtype"):
        R.ret_layernorm_forward(x, normal(64), normal(64).float())
    with pytest.raises(R.RetentionError, match="eps"):
        R.ret_layernorm_forward(x, eps=-1.0)
    with pytest.raises(ValueError, match="mean must have shape"):
        R.ret_layernorm_backward(x, x, torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError, match="must be a CUDA tensor|on cpu"):
        R.ret_layernorm_forward(x, normal(64).cpu())
    q = normal(2, 3, 4, 64)
    with pytest.raises(ValueError, match="positions must have shape"):
        R.ret_rotary(q, freqs=R.ret_rotary_frequencies(64)[0], positions=torch.zeros(2, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(R.RetentionError, match="rotary_dim"):
        R.ret_rotary(q, freqs=torch.ones(40, dtype=torch.float64))
    with pytest.raises(ValueError, match="state must have shape"):
        g = torch.zeros(2, 4, device="cuda")
        R.ret_delta_decode_step(normal(2, 4, 64), normal(2, 4, 64), normal(2, 4, 32), g, g, torch.zeros(2, 4, 32, 64, device="cuda"))
    # a view that is not contiguous is the general way's
    assert torch.equal(R.ret_rotary(q[:, :2], freqs=R.ret_rotary_frequencies(64)[0]),
                       R.ret_rotary(q[:, :2].contiguous(), freqs=R.ret_rotary_frequencies(64)[0]))


def test_own_workspace_on_a_passed_stream():
    """A workspace that a call makes is free when the call returns, while its
    kernels wait on the passed stream: memory of another stream must not be
    the same."""
    x, dy = normal(600, 512), normal(600, 512) + 1
    _, mean, rstd = R.ret_layernorm_forward(x, want_stats=True)
    want = R.ret_layernorm_backward(dy, x, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    out = [torch.empty_like(t) for t in want]
    R.ret_layernorm_backward(dy, x, mean, rstd, dx=out[0], dgain=out[1], dbias=out[2], stream=s)
    n = R.ret_layernorm_backward_workspace_bytes(600, 512)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert junk and all(torch.equal(a, b) for a, b in zip(want, out))
