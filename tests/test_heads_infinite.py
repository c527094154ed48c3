"""Infinities in the heads forward: the state becomes what the recurrence makes of it, an infinity with
its sign where the recurrence has one."""
import pytest
import torch

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R
from .test_heads import F32, PAIR, case

# batch, L, heads, P, N, groups: 16 and 33 states by mma.sync, 64 and 128 by tcgen05 (bf16); a sequence
# in segments by either; segments handed on
SHAPES = [(2, 150, 2, 16, 16, 1), (2, 150, 2, 20, 33, 1), (2, 150, 2, 16, 64, 1), (2, 150, 2, 16, 128, 1),
          (2, 2500, 2, 16, 16, 1), (2, 2500, 2, 16, 64, 1), (8, 600, 60, 9, 12, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("name", ["u", "B", "h0"])
def test_state_is_infinite_where_the_recurrence_is(cuda_device, io, shape, name):
    x = case(shape, 9, io, cuda_device)
    x[name] = x[name].clone()
    x[name][{"u": (1, 70, 1, 3), "B": (1, 70, 0, 2), "h0": (1, 1, 3, 2)}[name]] = float("inf")
    out, got = sb.sscan_heads_fwd(**x, return_last_state=True)
    assert sb.device_status() == 0
    ref_out, ref = R.heads(**{k: R.d64(v) for k, v in x.items()})
    got = R.d64(got)
    assert torch.isinf(ref).any() and not torch.isnan(ref).any()
    assert torch.equal(torch.isinf(got), torch.isinf(ref))
    assert torch.equal(torch.sign(got[torch.isinf(ref)]), torch.sign(ref[torch.isinf(ref)]))
    fine = torch.isfinite(ref)
    assert float((got - ref)[fine].abs().max() / ref[fine].abs().max()) <= (PAIR if io == "bf16" else F32)
    # an output is finite exactly where the recurrence's is
    assert torch.equal(torch.isfinite(R.d64(out)), torch.isfinite(ref_out))
