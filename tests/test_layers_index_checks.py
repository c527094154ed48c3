"""The debug build's index checks in the layers' kernels.  They exist: with every array counted one element shorter
than it is, each operator's accesses to the last elements are reported (and skipped; none leaves its array).
And they pass: on split and handed-on sequences, several head shares, checkpoints of the caller's, states and
steps, the debug library gives the release library's results with a clear status word."""
import ctypes

import pytest
import torch

from selective_state_space_33_b200 import binding as sb
from selective_state_space_33_b200 import build as lib_build

from . import layer_refs as R


def conv(dev, io, kind, **s):
    x = R.inputs("conv", 1, io, dev, **{**dict(batch=2, length=70, dim=40, taps=4), **s})
    if kind == "fwd":
        return lambda: list(sb.sscan_conv_fwd(**x, return_last_state=True))
    if kind == "bwd":
        return lambda: list(sb.sscan_conv_bwd(x["u"], x["weight"], x["u"], x["bias"], x["state0"]).values())

    def step():
        state = x["state0"].clone()
        return [sb.sscan_conv_step(x["u"][:, 0].contiguous(), x["weight"], state, x["bias"]), state]
    return step


def gated(dev, io, kind, **s):
    x = R.inputs("gated", 2, io, dev, **{**dict(batch=2, length=300, dim=40), **s})
    first, rest = [x[k] for k in ("u", "a_raw", "i_raw", "Lam")], [x[k] for k in ("a_bias", "i_bias", "h0")]
    if kind == "fwd":
        return lambda: list(sb.sscan_gated_fwd(**x, return_last_state=True, return_checkpoints=True))
    if kind == "bwd":
        return lambda: list(sb.sscan_gated_bwd(*first, x["u"], *rest).values())

    def step():
        p, state = R.token(x, 0), x["h0"].clone()
        return [sb.sscan_gated_step(p["u"], p["a_raw"], p["i_raw"], x["Lam"], state, *rest[:2]), state]
    return step


def heads(dev, io, kind, **s):
    x = R.inputs("heads", 3, io, dev, **{**dict(batch=2, length=100, heads=4, headdim=16, dstate=16, groups=2), **s})
    first, rest = [x[k] for k in ("u", "delta_raw", "A", "B", "C")], [x[k] for k in ("delta_bias", "D_skip", "z", "h0")]
    if kind == "fwd":
        return lambda: list(sb.sscan_heads_fwd(**x, return_last_state=True))
    if kind == "bwd":
        return lambda: list(sb.sscan_heads_bwd(*first, x["u"], *rest).values())

    def step():
        p, state = R.token(x, 0), x["h0"].clone()
        return [sb.sscan_heads_step(p["u"], p["delta_raw"], x["A"], p["B"], p["C"], state, x["delta_bias"], x["D_skip"],
                                    p["z"]), state]
    return step


# every kernel: forms by type, width and states; sequences split, handed on, in one piece; head shares
CASES = [(conv, "fwd", {}), (conv, "fwd", dict(dim=33, taps=3)), (conv, "fwd", dict(length=2)), (conv, "bwd", {}),
         (conv, "bwd", dict(dim=33, taps=2, length=700)), (conv, "step", dict(length=1)), (conv, "step", dict(length=1, dim=33)),
         (gated, "fwd", {}), (gated, "fwd", dict(dim=33)), (gated, "fwd", dict(length=9000, dim=72)), (gated, "bwd", {}),
         (gated, "bwd", dict(dim=33)), (gated, "bwd", dict(length=5000, dim=72)), (gated, "step", dict(length=1)),
         (gated, "step", dict(length=1, dim=33)),
         (heads, "fwd", {}), (heads, "fwd", dict(dstate=64)), (heads, "fwd", dict(dstate=100, headdim=20)),
         (heads, "fwd", dict(batch=1, length=3000)), (heads, "fwd", dict(batch=1, length=3000, dstate=128)),
         (heads, "fwd", dict(batch=8, length=600, heads=60, headdim=8, dstate=8)),
         (heads, "bwd", {}), (heads, "bwd", dict(dstate=64)), (heads, "bwd", dict(dstate=21, headdim=20)),
         (heads, "bwd", dict(batch=1, length=700, heads=12, groups=1)), (heads, "step", dict(length=1)),
         (heads, "step", dict(length=1, dstate=21)), (heads, "step", dict(length=1, dstate=128))]
IDS = [f"{f.__name__}-{k}-" + "-".join(f"{a}{b}" for a, b in s.items()) for f, k, s in CASES]


@pytest.fixture
def debug(monkeypatch):
    dbg = sb.load_library(lib_build.build(debug=True))
    dbg.sscan_debug_shorten.argtypes = [ctypes.c_int64]
    dbg.sscan_debug_shorten.restype = ctypes.c_int
    flags = ctypes.c_uint(0)

    def run(fn, shorten=0):
        """(results, status bits) of fn on the debug library"""
        with monkeypatch.context() as m:
            m.setattr(sb, "_lib", dbg)
            dbg.sscan_device_status(1, ctypes.byref(flags))
            assert dbg.sscan_debug_shorten(shorten) == 0
            try:
                out = fn()
                torch.cuda.synchronize()
            finally:
                assert dbg.sscan_debug_shorten(0) == 0
            dbg.sscan_device_status(1, ctypes.byref(flags))
            return out, flags.value
    return run


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("op,kind,sizes", CASES, ids=IDS)
def test_checks_are_there_and_pass(cuda_device, debug, io, op, kind, sizes):
    fn = op(cuda_device, io, kind, **sizes)
    want = fn()
    got, bits = debug(fn)
    assert bits == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    _, bits = debug(fn, shorten=1)
    assert bits == 8, bits
    got, bits = debug(fn)                                # and as before
    assert bits == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_release_build_has_no_checks_to_shorten():
    lib = sb.load_library()
    assert lib.sscan_debug_shorten(ctypes.c_int64(1)) == 2
    assert lib.sscan_debug_shorten(ctypes.c_int64(-1)) == 1
