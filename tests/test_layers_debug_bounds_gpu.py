"""The debug build (index checks into the workspace of the carry compiled in) on the gated recurrence
over several groups of tiles, forward and backward, and on the layers beside it: the same results as the
release build, with the status word clear."""
import ctypes

import pytest
import torch

from selective_state_space_33_b200 import binding as sb
from selective_state_space_33_b200 import build as lib_build

from . import layer_refs as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [70, 33])
def test_same_results_and_no_bad_index(cuda_device, monkeypatch, D):
    x = R.inputs("gated", 5, "bf16", cuda_device, batch=2, length=9000, dim=D)
    h = R.inputs("heads", 6, "bf16", cuda_device, batch=1, length=700, heads=2, headdim=16, dstate=40, groups=1)
    c = R.inputs("conv", 7, "bf16", cuda_device, batch=2, length=300, dim=D, taps=3)

    def run():
        first = [x[k] for k in ("u", "a_raw", "i_raw", "Lam")]
        rest = [x[k] for k in ("a_bias", "i_bias", "h0")]
        r = [sb.sscan_gated_fwd(**x)] + list(sb.sscan_gated_bwd(*first, x["u"], *rest).values())
        r.append(sb.sscan_heads_fwd(**h))
        r += list(sb.sscan_heads_bwd(*[h[k] for k in ("u", "delta_raw", "A", "B", "C")], h["u"],
                                     *[h[k] for k in ("delta_bias", "D_skip", "z", "h0")]).values())
        return r + [sb.sscan_conv_fwd(**c)] + list(sb.sscan_conv_bwd(c["u"], c["weight"], c["u"], c["bias"], c["state0"]).values())
    want = run()
    dbg = sb.load_library(lib_build.build(debug=True))
    monkeypatch.setattr(sb, "_lib", dbg)
    flags = ctypes.c_uint(0)
    dbg.sscan_device_status(1, ctypes.byref(flags))
    got = run()
    torch.cuda.synchronize()
    assert dbg.sscan_device_status(1, ctypes.byref(flags)) == 0 and flags.value == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
