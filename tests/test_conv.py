"""The causal depthwise convolution: sscan_conv_fwd, sscan_conv_bwd, sscan_conv_step."""
import ctypes

import pytest
import torch

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R

# Outputs: K + 1 products and sums of terms no larger than sum |W x| + |bias|, which here is
# at most ~8 times the largest output, each rounded to 2^-24, and SiLU's exponential and
# reciprocal (a few 2^-23): below 2^-18 of the largest output.  Then one rounding to the I/O
# type.  du adds K such products again and SiLU' (two more products).  Parameter gradients
# are fp32 sums over tokens: S terms of size up to ~16 times the mean, in tiles of 256 and
# then 32 rows in turn; the roundings are below 2^-24 * (number of serial additions <= 600)
# of the largest partial sum, which stays within ~8 times the result for the sizes here.
F32 = 2.0 ** -18
SUMS = 600 * 8 * 2.0 ** -24


def tol(t):
    return F32 + R.HALF_STEP[t.dtype]


SHAPES = [(1, 1, 1, 4), (2, 2, 8, 4), (1, 3, 16, 2), (3, 33, 24, 3), (2, 64, 40, 4), (1, 257, 130, 4), (2, 300, 17, 3),
          (1, 1000, 5, 2), (5, 31, 1536, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,D,K", SHAPES)
@pytest.mark.parametrize("silu,state,biases", [(True, True, True), (False, False, True), (True, False, False)])
def test_forward_and_backward(cuda_device, io, batch, L, D, K, silu, state, biases):
    x = R.inputs("conv", 11 * L + D, io, cuda_device, state, biases, batch=batch, length=L, dim=D, taps=K)
    dout = torch.randn(batch, L, D, generator=torch.Generator().manual_seed(L)).to(x["u"].dtype).to(cuda_device)
    out, last = sb.sscan_conv_fwd(**x, silu=silu, return_last_state=True)
    ref, ref_last = R.conv(**{k: R.d64(v) for k, v in x.items()}, silu=silu)
    assert R.off(out, ref) <= tol(out)
    assert torch.equal(R.d64(last), ref_last)          # copies
    g = sb.sscan_conv_bwd(x["u"], x["weight"], dout, x["bias"], x["state0"], silu=silu)
    want = R.grads("conv", x, dout, silu=silu)
    assert set(g) == {"du", "dweight"} | ({"dbias"} if biases else set()) | ({"dstate0"} if state else set())
    for k, v in g.items():
        assert R.off(v, want[k[1:]]) <= (SUMS if k in ("dweight", "dbias") else tol(v)), k


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unaligned_pointers(cuda_device, io):
    x = R.inputs("conv", 5, io, cuda_device, batch=2, length=70, dim=64, taps=4)
    dout = torch.randn_like(x["u"])
    y = {k: R.shifted(v) if k in ("u", "state0") else v for k, v in x.items()}
    a, la = sb.sscan_conv_fwd(**x, return_last_state=True)
    b, lb = sb.sscan_conv_fwd(**y, return_last_state=True)
    assert torch.equal(a, b) and torch.equal(la, lb)   # the access width changes no arithmetic
    ga = sb.sscan_conv_bwd(x["u"], x["weight"], dout, x["bias"], x["state0"])
    gb = sb.sscan_conv_bwd(y["u"], y["weight"], R.shifted(dout), y["bias"], y["state0"])
    assert all(torch.equal(ga[k], gb[k]) for k in ga)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 33])
def test_steps_and_segments_equal_one_forward(cuda_device, io, D):
    x = R.inputs("conv", 3, io, cuda_device, batch=3, length=41, dim=D, taps=4)
    full, last = sb.sscan_conv_fwd(**x, return_last_state=True)
    state, outs = x["state0"].clone(), []
    for t in range(41):
        outs.append(sb.sscan_conv_step(x["u"][:, t].contiguous(), x["weight"], state, x["bias"]))
    # the same products in another order (the step adds oldest first): roundings only
    assert R.off(torch.stack(outs, 1), full) <= 2 * tol(full)
    assert torch.equal(state, last)
    a, s = sb.sscan_conv_fwd(x["u"][:, :7].contiguous(), x["weight"], x["bias"], x["state0"], return_last_state=True)
    b, s = sb.sscan_conv_fwd(x["u"][:, 7:].contiguous(), x["weight"], x["bias"], s, return_last_state=True)
    assert torch.equal(torch.cat([a, b], 1), full) and torch.equal(s, last)


@pytest.mark.gpu
def test_later_and_other_rows_do_not_leak(cuda_device):
    """A NaN at step t reaches steps t .. t+K-1 of its own channel and batch row only."""
    x = R.inputs("conv", 8, "bf16", cuda_device, batch=2, length=100, dim=16, taps=4)
    clean = sb.sscan_conv_fwd(**x)
    x["u"][1, 50, 3] = float("nan")
    out = sb.sscan_conv_fwd(**x)
    bad = torch.isnan(out)
    assert bad[1, 50:54, 3].all() and int(bad.sum()) == 4
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.gpu
def test_empty_sizes(cuda_device):
    for batch, L, D in ((0, 5, 4), (2, 0, 4), (2, 5, 0)):
        x = R.inputs("conv", 1, "bf16", cuda_device, batch=batch, length=L, dim=D, taps=3)
        out, last = sb.sscan_conv_fwd(**x, return_last_state=True)
        assert out.shape == x["u"].shape
        if L == 0:
            assert torch.equal(last, x["state0"])
        g = sb.sscan_conv_bwd(x["u"], x["weight"], torch.empty_like(x["u"]), x["bias"], x["state0"])
        assert all((v == 0).all() for v in g.values())


@pytest.mark.gpu
def test_repeats_and_graph_and_stream(cuda_device):
    """Two runs give the same bits; a captured call replays on new values; a call on another
    stream, with its own workspace, gives the same result."""
    x = R.inputs("conv", 9, "bf16", cuda_device, batch=2, length=700, dim=96, taps=4)
    dout = torch.randn_like(x["u"])

    def both(stream=None):
        out = sb.sscan_conv_fwd(**x, stream=stream)
        return [out] + list(sb.sscan_conv_bwd(x["u"], x["weight"], dout, x["bias"], x["state0"], stream=stream).values())
    first = both()
    assert all(torch.equal(a, b) for a, b in zip(first, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    x["u"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, both()))


def test_binding_refuses():
    u, w = torch.zeros(1, 4, 6), torch.zeros(6, 4)
    with pytest.raises(ValueError, match="CUDA"):
        sb.sscan_conv_fwd(u, w)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sb.sscan_conv_fwd(u.half(), w)
    with pytest.raises(ValueError, match="must be"):
        sb.sscan_conv_fwd(u[0], w)
    with pytest.raises(ValueError, match="must be"):
        sb.sscan_conv_step(u, w, u)


@pytest.mark.gpu
def test_binding_refuses_on_device(cuda_device):
    x = R.inputs("conv", 9, "f32", cuda_device, batch=2, length=8, dim=6, taps=4)
    u, w, b, s = x["u"], x["weight"], x["bias"], x["state0"]
    for bad in (lambda: sb.sscan_conv_fwd(u, w[:5]), lambda: sb.sscan_conv_fwd(u, w.bfloat16()),
                lambda: sb.sscan_conv_fwd(u, w, b, s[:, :2]), lambda: sb.sscan_conv_fwd(u, w, b, s.bfloat16()),
                lambda: sb.sscan_conv_fwd(u.transpose(0, 1), w), lambda: sb.sscan_conv_fwd(u, w, b[:5]),
                lambda: sb.sscan_conv_fwd(u, w, out=torch.empty(2, 8, 7, device=cuda_device)),
                lambda: sb.sscan_conv_bwd(u, w, u.bfloat16()), lambda: sb.sscan_conv_bwd(u, w, None),
                lambda: sb.sscan_conv_step(u[:, 0].contiguous(), w, None)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(sb.SscanError, match="taps"):
        sb.sscan_conv_fwd(u, torch.zeros(6, 5, device=cuda_device))
    with pytest.raises(sb.SscanError, match="workspace"):
        sb.sscan_conv_bwd(u, w, u, workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device)[:16])


def test_c_entry_refuses():
    """Host checks through the C interface; no pointer here is dereferenced."""
    lib = sb.load_library()
    fake = ctypes.c_void_p(0x10000)

    def fwd(prob, *p):
        return lib.sscan_conv_fwd(prob, *p, None)
    ok = sb.ConvProblem(2, 8, 6, 4, 0, 1)
    assert lib.sscan_conv_fwd(None, *([fake] * 6), None) == 1
    assert fwd(ok, None, fake, None, None, fake, None) == 1 and b"required" in lib.sscan_last_error()
    assert fwd(sb.ConvProblem(-1, 8, 6, 4, 0, 1), *([fake] * 6)) == 1
    assert fwd(sb.ConvProblem(2, 8, 6, 0, 0, 1), *([fake] * 6)) == 1
    assert fwd(sb.ConvProblem(2, 8, 6, 5, 0, 1), *([fake] * 6)) == 2
    assert fwd(sb.ConvProblem(2, 8, 6, 4, 2, 1), *([fake] * 6)) == 1
    assert fwd(sb.ConvProblem(2, 8, 6, 4, 0, 2), *([fake] * 6)) == 1
    assert fwd(sb.ConvProblem(1 << 20, 1 << 20, 6, 4, 0, 1), *([fake] * 6)) == 2
    need = lib.sscan_conv_workspace_size(ok, sb.SSCAN_OP_BWD)
    assert need > 0 and need % 256 == 0
    assert lib.sscan_conv_workspace_size(ok, sb.SSCAN_OP_FWD) == 0
    args = [fake, fake, fake, fake, fake, fake, fake, fake, fake]
    assert lib.sscan_conv_bwd(ok, *args, None, 0, None) == 3
    assert lib.sscan_conv_bwd(ok, *args, fake, need - 1, None) == 3
    assert lib.sscan_conv_bwd(ok, fake, fake, None, fake, fake, fake, fake, fake, None, fake, need, None) == 1
    assert b"dbias" in lib.sscan_last_error()
    assert lib.sscan_conv_bwd(ok, fake, fake, fake, None, fake, fake, fake, None, fake, fake, need, None) == 1
    assert lib.sscan_conv_step(ok, fake, fake, None, fake, fake, None) == 1 and b"seqlen" in lib.sscan_last_error()
    one = sb.ConvProblem(2, 1, 6, 4, 0, 1)
    assert lib.sscan_conv_step(one, fake, fake, None, None, fake, None) == 1


def test_reference_gradient_matches_differences():
    x = {k: R.d64(v) for k, v in R.inputs("conv", 2, batch=2, length=9, dim=3, taps=4).items()}
    dout = torch.randn(2, 9, 3, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    R_check_differences("conv", x, dout)


def R_check_differences(op, x, dout, **kw):
    """Directional central differences of the 64-bit reference against its gradients: with
    steps of 1e-6 the truncation is ~1e-12 and the roundings ~1e-9 of the sums involved."""
    g = R.grads(op, x, dout, **kw)
    gen = torch.Generator().manual_seed(7)
    for k, v in x.items():
        if v is None:
            continue
        step = torch.randn(v.shape, dtype=torch.float64, generator=gen) * 1e-6
        f = [(R.FN[op](**{**x, k: v + sign * step}, **kw)[0] * dout).sum() for sign in (1, -1)]
        want = float((g[k] * step).sum())
        assert abs(float(f[0] - f[1]) / 2 - want) <= 1e-6 * abs(want) + 1e-12, k
