"""The gated recurrence where the decay is strong (a = exp(-s) far below 1) and where gates are closed:
every result keeps its relative precision, however small it is."""
import pytest
import torch

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R

EPS = 2.0 ** -24


def relative(got, ref):
    """|got - ref| / |ref| for each element (none of ref is 0)"""
    got, ref = R.d64(got), R.d64(ref)
    assert got.shape == ref.shape and (ref != 0).all()
    return (got - ref).abs() / ref.abs()


def strong(io, device, L=6, D=64, rate=8.0):
    """Decay rates from 0.35 to 60 per step; signs such that no sum below cancels: u and dout alternate,
    so h_{t-1} and u_t have opposite signs, and ds has one sign throughout."""
    c = torch.linspace(0.35, 60.0, D, dtype=torch.float64)
    gen = torch.Generator().manual_seed(3)
    dt = R.DTYPES[io]
    sign = torch.tensor([(-1.0) ** t for t in range(L)])[None, :, None].expand(2, L, D)
    x = {"u": sign.to(dt).contiguous(), "a_raw": (2 * torch.rand(2, L, D, generator=gen) - 1).to(dt),
         "i_raw": torch.full((2, L, D), 0.25).to(dt), "Lam": torch.log(torch.expm1(c / rate)).float(),
         "h0": torch.zeros(2, D)}
    x = {k: v.to(device) for k, v in x.items()}
    s = rate * torch.logaddexp(R.d64(x["Lam"]), torch.zeros(D, dtype=torch.float64)) * torch.sigmoid(R.d64(x["a_raw"]))
    return x, x["u"].clone(), s


# s = c r: c carries two functions of 2 ulp and a product (9 * 2^-24), r an exponential of 2 ulp whose
# argument is below 2, a sum, a reciprocal of 1 ulp and two products (10 * 2^-24), their product one more:
# 20 * 2^-24.  a = exp(-s): 20 s from s, 2 s from the argument's rounding, 4 for the exponential.
# With |a_raw| <= 1 the factor 1 - r (r <= 0.74) adds 30 * 2^-24; e = 1 - a >= 0.1 and the slope term
# 1 / m take (22 s + 4) a / e <= 100; g = 1 - a |g| >= 0.1 as much again, and h two of them.
def limit(s):
    return (32 * s + 400) * EPS


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_decay_keeps_the_gradients_relative_precision(cuda_device, io):
    x, dout, s = strong(io, cuda_device)
    g = sb.sscan_gated_bwd(x["u"], x["a_raw"], x["i_raw"], x["Lam"], dout, h0=x["h0"])
    want = R.grads("gated", x, dout)
    assert (relative(g["dh0"], want["h0"]) <= limit(s[:, 0])).all()
    # h before the first step is 0, so its da_raw is the slope of m alone, e (a / m) i u s (1 - r) with e = dh0:
    # two factors a, and below 2^-126 nothing in fp32.  (The reference's derivative of expm1 is
    # 1 + expm1, which has no digits left there.)
    r, i = torch.sigmoid(R.d64(x["a_raw"])[:, 0]), torch.sigmoid(R.d64(x["i_raw"])[:, 0])
    s0 = s[:, 0]
    first = want["h0"] * torch.exp(-s0) / torch.sqrt(1 - torch.exp(-2 * s0)) * i * R.d64(x["u"])[:, 0] * s0 * (1 - r)
    assert ((R.d64(g["da_raw"])[:, 0] - first).abs() <= first.abs() * (2 * limit(s0) + R.HALF_STEP[dout.dtype]) + 2.0 ** -126).all()
    assert (relative(g["da_raw"][:, 1:], want["a_raw"][:, 1:]) <= limit(s[:, 1:]) + R.HALF_STEP[dout.dtype]).all()
    assert (relative(g["dLam"], want["Lam"]) <= limit(s.amax((0, 1)))).all()
    assert sb.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_decay_of_a_state(cuda_device, io):
    """u = 0: one token leaves a h, by the forward and by the step."""
    x, _, s = strong(io, cuda_device, L=1)
    x["u"].zero_()
    x["h0"].fill_(1.0)
    _, last = sb.sscan_gated_fwd(**x, return_last_state=True)
    a = torch.exp(-s[:, 0])
    assert (relative(last, a) <= limit(s[:, 0])).all()
    state = x["h0"].clone()
    sb.sscan_gated_step(x["u"][:, 0].contiguous(), x["a_raw"][:, 0].contiguous(), x["i_raw"][:, 0].contiguous(), x["Lam"],
                        state)
    assert (relative(state, a) <= limit(s[:, 0])).all()


# m = sqrt(2 s) with s = c r: half of s's 20 * 2^-24 and a root, a product with i (10 * 2^-24) and with u: below
# 64 * 2^-24 of a term.  L terms of one sign add up; each step rounds a (half of 2^-24 for a in [1/2, 1]) and the sum
# (as much): at most L * 2^-24 of the result.
def closed_limit(L, dtype=torch.float32):
    return (L + 64) * EPS + (R.HALF_STEP[dtype] if dtype != torch.float32 else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 70, 33])
@pytest.mark.parametrize("gate,value", [("a_raw", -45.0), ("a_raw", -70.0), ("i_raw", -43.0), ("i_raw", -60.0)])
def test_a_nearly_closed_gate_lets_through_what_it_should(cuda_device, io, D, gate, value):
    """A decay gate at exp(-45) keeps a state and adds next to nothing to it, an input gate at exp(-60) adds
    next to nothing to any: over 2000 steps both stay at what the definition gives, not at a
    floor of the sigmoid."""
    L = 2000
    x = R.inputs("gated", 5, io, cuda_device, biases=False, batch=2, length=L, dim=D)
    x["h0"].zero_()
    x["u"] = x["u"].abs() + 0.5
    x["i_raw"].fill_(0.5)
    x["a_raw"].fill_(0.5)
    x[gate].fill_(value)
    out, last = sb.sscan_gated_fwd(**x, return_last_state=True)
    ref, ref_last = R.gated(**{k: R.d64(v) for k, v in x.items()})
    assert (relative(last, ref_last) <= closed_limit(L)).all()
    assert (relative(out, ref) <= closed_limit(L, out.dtype)).all()
    dout = torch.rand_like(x["u"]) + 0.5
    g = sb.sscan_gated_bwd(x["u"], x["a_raw"], x["i_raw"], x["Lam"], dout, h0=x["h0"])
    want = R.grads("gated", x, dout)
    # no sum of these cancels: every term is of one sign
    for k in ("du", "di_raw"):
        assert (relative(g[k], want[k[1:]]) <= 2 * closed_limit(L, dout.dtype)).all(), k
    state = x["h0"].clone()
    for t in range(3):
        p = R.token(x, t)
        sb.sscan_gated_step(p["u"], p["a_raw"], p["i_raw"], x["Lam"], state)
    assert (relative(state, R.d64(ref[:, 2])) <= closed_limit(3)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 33])
def test_a_closed_gate_is_closed(cuda_device, io, D):
    """-inf: nothing enters, exactly; a decay gate of -inf keeps the state, exactly, and takes no gradient."""
    x = R.inputs("gated", 6, io, cuda_device, batch=2, length=300, dim=D)
    y = {**x, "i_raw": torch.full_like(x["i_raw"], -float("inf")), "h0": torch.zeros_like(x["h0"])}
    assert (sb.sscan_gated_fwd(**y) == 0).all()
    y = {**x, "a_raw": torch.full_like(x["a_raw"], -float("inf"))}
    out, last = sb.sscan_gated_fwd(**y, return_last_state=True)
    assert torch.equal(last, x["h0"])
    assert torch.equal(out, x["h0"].to(out.dtype)[:, None].expand_as(out))
    dout = torch.ones_like(x["u"])
    g = sb.sscan_gated_bwd(y["u"], y["a_raw"], y["i_raw"], y["Lam"], dout, y["a_bias"], y["i_bias"], y["h0"])
    assert all((g[k] == 0).all() for k in ("du", "da_raw", "di_raw", "da_bias", "di_bias", "dLam"))
    assert (g["dh0"] == 300).all()
    state, p = x["h0"].clone(), R.token(y, 0)
    sb.sscan_gated_step(p["u"], p["a_raw"], p["i_raw"], x["Lam"], state, x["a_bias"], x["i_bias"])
    assert torch.equal(state, x["h0"])
    # one masked stretch among ordinary tokens
    z = {k: v.clone() for k, v in x.items()}
    z["a_raw"][:, 100:200] = -float("inf")
    out = sb.sscan_gated_fwd(**z)
    # the state after each warp's 16 steps is put together from maps (a few fused products, exact but for
    # their roundings: 16 * 2^-24 at most over the warps of a tile), then rounded
    assert R.off(out[:, 100:200], out[:, 99:100].expand(-1, 100, -1)) <= 16 * EPS + (2 * R.HALF_STEP[out.dtype] if io == "bf16" else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 33])
@pytest.mark.parametrize("name,value", [("a_raw", float("nan")), ("a_raw", -float("inf")), ("i_raw", float("nan")),
                                        ("i_raw", -100.0)])
def test_one_extreme_gate_changes_nothing_else(cuda_device, io, D, name, value):
    """Bit for bit: not the channel beside it, not the steps before it, not another batch row."""
    x = R.inputs("gated", 8, io, cuda_device, batch=2, length=300, dim=D)
    clean = sb.sscan_gated_fwd(**x)
    x[name][1, 150, 3] = value
    out = sb.sscan_gated_fwd(**x)
    same = torch.ones_like(out, dtype=torch.bool)
    same[1, 150:, 3] = False
    assert torch.equal(out[same], clean[same])
    assert bool(torch.isnan(out[1, 150:, 3]).all()) == (value != value) and not torch.isnan(out[same]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_both_gates_at_every_extreme(cuda_device, io, shift):
    """One token, every pair of raw values from -inf to inf; by two channels per lane, or one (an odd start)."""
    values = torch.tensor([-float("inf"), -200.0, -90.0, -87.5, -75.0, -60.0, -42.0, -20.0, 0.0, 20.0, 90.0, float("inf")])
    a, i = (v.flatten() for v in torch.meshgrid(values, values, indexing="ij"))
    dt = R.DTYPES[io]
    x = {"u": torch.full((1, 1, a.numel()), 2.0).to(dt), "a_raw": a.to(dt)[None, None], "i_raw": i.to(dt)[None, None],
         "Lam": torch.full((a.numel(),), -2.0), "h0": torch.zeros(1, a.numel())}
    x = {k: v.to(cuda_device) for k, v in x.items()}
    ref = R.gated(**{k: R.d64(v) for k, v in x.items()})[0]
    if shift:
        x.update({k: R.shifted(x[k]) for k in ("u", "a_raw", "i_raw")})
    out, last = sb.sscan_gated_fwd(**x, return_last_state=True)
    state = x["h0"].clone()
    step = sb.sscan_gated_step(x["u"][:, 0], x["a_raw"][:, 0], x["i_raw"][:, 0], x["Lam"], state)
    # x = m i u in a few roundings; a gate below 2^-126 is 0, as are two whose product is below 2^-226, and sqrt(2 c r) i u with
    # either left out is below 2^-61 (r = 2^-126 alone) or 2^-98
    for got in (last, state):
        assert ((R.d64(got) - ref[:, 0]).abs() <= 64 * EPS * ref[:, 0].abs() + 2.0 ** -61).all()
        assert (got[0, i.to(cuda_device) == -float("inf")] == 0).all() and (got[0, a.to(cuda_device) == -float("inf")] == 0).all()
    half = R.HALF_STEP[dt]
    assert ((R.d64(out) - ref).abs() <= (64 * EPS + half) * ref.abs() + 2.0 ** -61).all()
    assert torch.equal(step, state.to(dt))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 33])
def test_open_gates_to_a_few_roundings(cuda_device, D):
    """One token with gates of ordinary size, element by element: h = m i u and a h0 in fp32."""
    x = R.inputs("gated", 21, "f32", cuda_device, batch=64, length=1, dim=D)
    x["h0"].zero_()
    _, last = sb.sscan_gated_fwd(**x, return_last_state=True)
    _, ref = R.gated(**{k: R.d64(v) for k, v in x.items()})
    # i: its exponent is rounded to half a step of a number below 8 (2^-22, times ln 2) as is the bias's product (as
    # much), an exponential of 2 ulp, a sum, a reciprocal of 1 ulp and four products: 22 * 2^-24; m: half of r's as many
    # and of c's 9, a root of 2 ulp and three products: 23; two products
    limit = 47 * EPS
    assert (relative(last, ref) <= limit).all()
    state = x["h0"].clone()
    sb.sscan_gated_step(*(x[k][:, 0].contiguous() for k in ("u", "a_raw", "i_raw")), x["Lam"], state, x["a_bias"], x["i_bias"])
    assert (relative(state, ref) <= limit).all()
