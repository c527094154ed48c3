"""The layers around the scan used together, as a block uses them: the convolution feeds a scan or a
recurrence, forward and backward; generation continues from what prefill leaves."""
import pytest
import torch

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R

# Each layer is within its own test's tolerance of its reference; here the output of one (rounded to
# bf16 in between) feeds the next, whose gain on the largest value is below 4.
TOL = {"f32": 4 * 2.0 ** -13, "bf16": 4 * 4 * 2.0 ** -8}


def _inputs(io, device, batch=2, L=150, H=3, P=16, N=16):
    c = R.inputs("conv", 1, io, device, batch=batch, length=L, dim=H * P, taps=4)
    h = R.inputs("heads", 2, io, device, batch=batch, length=L, heads=H, headdim=P, dstate=N, groups=1)
    g = R.inputs("gated", 3, io, device, batch=batch, length=L, dim=H * P)
    return c, h, g


def _chain(c, h, g, ops):
    """conv -> heads -> gated on its output; (out, conv window, heads state, gated state)"""
    conv, heads, gated = ops
    b, L, D = c["u"].shape
    y, window = conv(c)
    o, state = heads({**h, "u": y.reshape(h["u"].shape)})
    r, last = gated({**g, "u": o.reshape(b, L, D)})
    return r, window, state, last


OWN = (lambda x: sb.sscan_conv_fwd(**x, return_last_state=True), lambda x: sb.sscan_heads_fwd(**x, return_last_state=True),
       lambda x: sb.sscan_gated_fwd(**x, return_last_state=True))
REF = tuple(lambda x, f=f: f(**x) for f in (R.conv, R.heads, R.gated))


def _d64(x):
    return {k: R.d64(v) for k, v in x.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prefill_then_generation(cuda_device, io):
    c, h, g = _inputs(io, cuda_device)
    full = _chain(c, h, g, OWN)
    for got, want in zip(full, _chain(_d64(c), _d64(h), _d64(g), REF)):
        assert R.off(got, want) <= TOL[io]
    # the first 100 tokens at once, the others one by one
    def head(x):
        return {k: v[:, :100].contiguous() if v.dim() > 1 and v.shape[1] == 150 else v for k, v in x.items()}
    out, window, state, last = _chain(head(c), head(h), head(g), OWN)
    outs = [out]
    for t in range(100, 150):
        ct, ht, gt = (R.token(x, t) for x in (c, h, g))
        y = sb.sscan_conv_step(ct["u"], c["weight"], window, c["bias"])
        o = sb.sscan_heads_step(y.view(ht["u"].shape), ht["delta_raw"], h["A"], ht["B"], ht["C"], state, h["delta_bias"],
                                h["D_skip"], ht["z"])
        outs.append(sb.sscan_gated_step(o.view(gt["u"].shape), gt["a_raw"], gt["i_raw"], g["Lam"], last, g["a_bias"],
                                        g["i_bias"])[:, None])
    for got, want in zip((torch.cat(outs, 1), window, state, last), full):
        assert R.off(got, want) <= TOL[io]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_through_the_block(cuda_device, io):
    c, h, g = _inputs(io, cuda_device, L=70)
    b, L, D = c["u"].shape
    y = sb.sscan_conv_fwd(**c)
    o = sb.sscan_heads_fwd(**{**h, "u": y.view(h["u"].shape)})
    dout = torch.randn(b, L, D, generator=torch.Generator().manual_seed(4)).to(c["u"].dtype).to(cuda_device)
    dg = sb.sscan_gated_bwd(o.view(b, L, D), g["a_raw"], g["i_raw"], g["Lam"], dout, g["a_bias"], g["i_bias"], g["h0"])
    dh = sb.sscan_heads_bwd(y.view(h["u"].shape), h["delta_raw"], h["A"], h["B"], h["C"], dg["du"].view(h["u"].shape),
                            h["delta_bias"], h["D_skip"], h["z"], h["h0"])
    dc = sb.sscan_conv_bwd(c["u"], c["weight"], dh["du"].view(b, L, D), c["bias"], c["state0"])
    leaf = [{k: R.d64(v).requires_grad_() for k, v in x.items()} for x in (c, h, g)]
    # heads and gated take the chain's values, so their own u is not a leaf of it
    out = _chain(*leaf, REF)[0]
    (out * R.d64(dout)).sum().backward()
    for got, want in ((dc["du"], leaf[0]["u"]), (dc["dweight"], leaf[0]["weight"]), (dc["dstate0"], leaf[0]["state0"]),
                      (dh["dB"], leaf[1]["B"]), (dh["dz"], leaf[1]["z"]), (dh["dh0"], leaf[1]["h0"]),
                      (dh["ddelta_raw"], leaf[1]["delta_raw"]), (dg["da_raw"], leaf[2]["a_raw"]), (dg["dh0"], leaf[2]["h0"])):
        assert R.off(got, want.grad) <= TOL[io]


@pytest.mark.gpu
def test_convolution_feeds_the_selective_scan(cuda_device):
    """The input branch of the layer: convolution with SiLU, then sscan_fwd on its output equals
    sscan_fwd with the SiLU of the convolution left to SSCAN_INPUT_SILU."""
    from selective_state_space_33_b200 import workloads as W
    x = W.to_device(W.small_case(2, 200, 64, 16, io="f32", seed=3), cuda_device)
    c = R.inputs("conv", 4, "f32", cuda_device, batch=2, length=200, dim=64, taps=4)
    c["u"] = x["u"]
    rest = [x[k] for k in ("delta_raw", "A", "B", "C", "delta_bias", "D_skip", "z")]
    a = sb.sscan_fwd(sb.sscan_conv_fwd(**c, silu=True), *rest)
    b = sb.sscan_fwd(sb.sscan_conv_fwd(**c, silu=False), *rest, input_silu=True)
    assert R.off(a, b) <= 2.0 ** -16                     # two forms of one SiLU, then the same scan


@pytest.mark.gpu
def test_two_streams_at_once(cuda_device):
    """Calls on two streams that overlap, each with its own (default) workspace."""
    c, h, g = _inputs("bf16", cuda_device, L=3000)
    want = _chain(c, h, g, OWN)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([_chain(c, h, g, OWN) for _ in range(3)])
    torch.cuda.synchronize()
    for runs in got:
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
    assert sb.device_status() == 0
