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
