"""The heads gradients at the precision their kernels are written for: what enters a parameter's
gradient carries 24 bits, and what the heads of a group share is summed in fp32 before it is rounded."""
import pytest
import torch

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R
from .test_heads import NAMES, bwd, case, randn_like


def per_token(x, dout):
    """What each token adds to dA, ddelta_bias and dD, in 64 bits: (batch, L, heads) each; and dh0."""
    x = {k: R.d64(v) for k, v in x.items()}
    b, L, H, P = x["u"].shape
    leaf = {k: x[k].expand(b, L, H).clone().requires_grad_() for k in ("A", "delta_bias", "D_skip")}
    h0 = x["h0"].requires_grad_()
    S, out = h0, []
    for t in range(L):
        A = leaf["A"][:, t]
        dl = x["delta_raw"][:, t] + leaf["delta_bias"][:, t]
        dl = torch.logaddexp(dl, torch.zeros_like(dl))
        w = torch.expm1(dl * A) / A
        Bt, Ct = (x[n][:, t].repeat_interleave(H // x["B"].shape[2], 1) for n in "BC")
        S = torch.exp(dl * A)[..., None, None] * S + (w[..., None] * x["u"][:, t])[..., None] * Bt[:, :, None]
        y = (S * Ct[:, :, None]).sum(-1) + leaf["D_skip"][:, t][..., None] * x["u"][:, t]
        out.append(y if x["z"] is None else y * torch.nn.functional.silu(x["z"][:, t]))
    g = torch.autograd.grad((torch.stack(out, 1) * R.d64(dout)).sum(), [*leaf.values(), h0])
    return dict(zip(("dA", "ddelta_bias", "dD", "dh0"), g))


# A token's term rounds an operand in three parts (2^-24), has two factors of an exponential of 2 ulp
# (2^-22 each) and some four products and sums: 13 * 2^-24, not of either sign (the tensor core's sums
# truncate).  The fp32 sums over a chunk's steps, then over rows of partial sums, add 3 * 2^-24 of the sizes.
# So a parameter gradient is within 16 * 2^-24 of the sum of its terms' sizes.  (Not of its own value: that
# is up to 90 times smaller here where the terms cancel.  With one head of 300 tokens and seed 100, dA is
# -41.0 and its terms' sizes add up to 763, so 2^-22 of each term is already 4.4e-6 of the value.)
# Two parts (2^-17) would be 128 * 2^-24 for each term.
SUM = 16 * 2.0 ** -24
# dh0 is not a sum over tokens but the adjoint after L steps: each chunk's three-part products and its
# decay leave some 2^-22 of the largest entry, of which the last few chunks' add up.
STATE = 2.0 ** -19


# one head alone (no other head's larger gradient in the maximum), heads in one group, 128 states,
# an odd width; lengths of one and of many chunks
SHAPES = [(1, 300, 1, 64, 64, 1), (2, 700, 1, 64, 16, 1), (1, 500, 1, 33, 24, 1), (2, 515, 6, 40, 24, 2),
          (1, 400, 2, 64, 128, 1), (1, 64, 1, 64, 32, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_parameter_gradients_carry_24_bits(cuda_device, io, gate, shape):
    bad = {}
    for seed in range(4):
        x = case(shape, 100 + seed, io, cuda_device, gate=gate)
        dout = randn_like(x["u"], seed)
        g = bwd(x, dout)
        terms = per_token(x, dout)
        for k in ("dA", "ddelta_bias", "dD"):
            e = (R.d64(g[k]) - terms[k].sum((0, 1))).abs() / terms[k].abs().sum((0, 1))
            if not (e <= SUM).all():
                bad[seed, k] = float(e.max())
        if not R.off(g["dh0"], terms["dh0"]) <= STATE:
            bad[seed, "dh0"] = R.off(g["dh0"], terms["dh0"])
    assert not bad, bad
    assert sb.device_status() == 0


# One token: dB = sum over the heads of M2 C with M2 = w dy . u, in fp32 up to its two parts of 2^-17 and
# then rounded once; the heads' terms are of either sign, so their sizes add up to at most some 8
# times the result for 24 heads.
@pytest.mark.gpu
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("L", [1, 2])
def test_shared_b_and_c_are_rounded_once(cuda_device, gate, L):
    bad = {}
    for seed in range(8):
        x = case((1, L, 24, 64, 64, 1), 200 + seed, "bf16", cuda_device, gate=gate, state=False)
        dout = randn_like(x["u"], seed)
        g = bwd(x, dout)
        want = R.grads("heads", x, dout)
        for k in ("dB", "dC"):
            e = R.off(g[k], want[NAMES[k]])
            if not e <= R.HALF_STEP[torch.bfloat16] + 8 * 2.0 ** -17:
                bad[seed, k] = e
    assert not bad, bad
    assert sb.device_status() == 0
