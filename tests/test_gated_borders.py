"""The gated recurrence across every border of its carry, in the forms that the lengths and widths of
test_gated.py leave out.  A forward tile is 128 steps, a backward tile 64, by 64 channels (32 on an odd
width); 8 tiles make a group and 8 groups a hop.  So groups close every 1024 steps forward and 512
backward, and hops every 8192 and 4096."""
import pytest
import torch

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R
from .test_gated import F32, NAMES, args, randn_like, sums, tol

# rows on 16-byte boundaries (TMA) over several channel blocks and batch rows, one step past a
# group, a few tiles past one, one step past a hop, several hops; then 70 and 33 channels (plain loads, two
# and one channel per lane)
SHAPES = [(2, 1025, 96), (2, 1153, 136), (3, 2048, 128), (2, 8193, 96), (1, 16500, 136), (2, 8193, 70), (2, 4161, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,D", SHAPES)
def test_across_groups_and_hops(cuda_device, io, batch, L, D):
    x = R.inputs("gated", L + D, io, cuda_device, batch=batch, length=L, dim=D)
    dout = randn_like(x["u"], L)
    out, last, saved = sb.sscan_gated_fwd(**x, return_last_state=True, return_checkpoints=True)
    ref, ref_last = R.gated(**{k: R.d64(v) for k, v in x.items()})
    assert R.off(out, ref) <= tol(out)
    assert R.off(last, ref_last) <= F32
    # the saved states are those before every 64th step
    before = torch.cat([R.d64(x["h0"])[:, None], ref[:, 63:-1:64]], 1)
    assert R.off(saved, before) <= F32
    first, rest = args(x)
    g = sb.sscan_gated_bwd(*first, dout, *rest, checkpoints=saved)
    want = R.grads("gated", x, dout)
    for k, v in g.items():
        assert R.off(v, want[NAMES[k]]) <= (sums(batch * L) if k in ("dLam", "da_bias", "di_bias") else tol(v)), k
    assert sb.device_status() == 0
