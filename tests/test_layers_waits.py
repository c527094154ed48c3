"""The bounded waits of the layers' kernels run out without a fault: each is made to wait, with a short limit, for
something that nothing sets, and must raise the device status bit and leave the context usable."""
import pytest

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R
from .test_gated import F32


@pytest.mark.gpu
@pytest.mark.parametrize("wait", list(sb.LAYER_WAITS))
def test_a_wait_that_runs_out_is_reported(cuda_device, wait):
    sb.device_status(clear=True)
    assert sb.device_status() == 0
    sb.probe_layer_wait_timeout(wait, 1000)
    assert sb.device_status(clear=True) == 4
    assert sb.device_status() == 0
    # kernels with the same waits, right after: the carry over several hops, handed-on segments, tcgen05
    x = R.inputs("gated", 3, "f32", cuda_device, batch=1, length=9000, dim=8)
    out = sb.sscan_gated_fwd(**x)
    assert R.off(out, R.gated(**{k: R.d64(v) for k, v in x.items()})[0]) <= F32 + 2.0 ** -24
    for shape in (dict(batch=8, length=600, heads=60, headdim=8, dstate=8), dict(batch=1, length=300, heads=2, headdim=16, dstate=64)):
        y = R.inputs("heads", 4, "bf16", cuda_device, groups=1, **shape)
        ref = R.heads(**{k: R.d64(v) for k, v in y.items()})[0]
        assert R.off(sb.sscan_heads_fwd(**y), ref) <= 4 * 2.0 ** -8
    assert sb.device_status() == 0


def test_probe_refuses():
    """Checked on the host before any launch."""
    lib = sb.load_library()
    for wait, polls in ((0, 0), (0, (1 << 20) + 1), (3, 10), (-1, 10)):
        assert lib.sscan_probe_layer_wait_timeout(wait, polls, None) == 1
