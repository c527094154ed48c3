"""The gated linear recurrence: sscan_gated_fwd, sscan_gated_bwd, sscan_gated_step."""
import ctypes

import pytest
import torch

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R
from .test_conv import R_check_differences

# exp(-rate softplus(Lam)) is at most 0.999 here and r about 1/2, so a state remembers some
# M = 2000 steps.  a = 1 + expm1(-s) carries one rounding of 2^-24 per step and the input a
# few 2^-24 (sigmoid: exponential, sum, reciprocal; the square root; two products: 8 in all),
# so |dh| <= M (2^-24 |h| + 8 * 2^-24 |x|) with |x| <= |h|max / sqrt(M) or so: M * 2^-24 = 1.2e-4
# bounds it.  The adjoint runs the same recurrence.  Each result is then rounded once.
F32 = 2000 * 2.0 ** -24


def sums(tokens):
    """Sums over T tokens of terms with that error and of either sign: the sum of T sizes is some
    sqrt(T) times the size of a sum of T random signs; twice that."""
    return F32 * max(8, 2 * tokens ** 0.5)


def tol(t):
    return F32 + R.HALF_STEP[t.dtype]


NAMES = {"du": "u", "da_raw": "a_raw", "di_raw": "i_raw", "dLam": "Lam", "da_bias": "a_bias", "di_bias": "i_bias",
         "dh0": "h0"}
# lengths around the 64-step tile and the 32-tile group of the carry; widths off 2 and 64
SHAPES = [(1, 1, 1), (2, 5, 64), (1, 63, 66), (3, 64, 34), (2, 65, 33), (1, 128, 130), (2, 200, 62), (1, 2049, 6),
          (1, 4229, 3), (2, 777, 96)]


def args(x):
    return [x[k] for k in ("u", "a_raw", "i_raw", "Lam")], [x[k] for k in ("a_bias", "i_bias", "h0")]


def randn_like(t, seed):
    return torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)).to(t.dtype).to(t.device)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,D", SHAPES)
@pytest.mark.parametrize("state,biases", [(True, True), (False, False)])
def test_forward_and_backward(cuda_device, io, batch, L, D, state, biases):
    x = R.inputs("gated", L + D, io, cuda_device, state, biases, batch=batch, length=L, dim=D)
    dout = randn_like(x["u"], L)
    out, last, saved = sb.sscan_gated_fwd(**x, return_last_state=True, return_checkpoints=True)
    ref, ref_last = R.gated(**{k: R.d64(v) for k, v in x.items()})
    assert R.off(out, ref) <= tol(out)
    assert R.off(last, ref_last) <= F32
    first, rest = args(x)
    g = sb.sscan_gated_bwd(*first, dout, *rest, checkpoints=saved)
    again = sb.sscan_gated_bwd(*first, dout, *rest)      # checkpoints rebuilt by a pass of their own
    assert set(g) == {"du", "da_raw", "di_raw", "dLam", "dh0"} | ({"da_bias", "di_bias"} if biases else set())
    assert all(torch.equal(g[k], again[k]) for k in g)
    if x["h0"] is None:
        x["h0"] = torch.zeros(batch, D, device=cuda_device)
    want = R.grads("gated", x, dout)
    for k, v in g.items():
        assert R.off(v, want[NAMES[k]]) <= (sums(batch * L) if k in ("dLam", "da_bias", "di_bias") else tol(v)), k
    assert sb.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rate", [0.5, 20.0])
def test_rates_and_extreme_gates(cuda_device, rate):
    """Gates at +-30 and +-inf, Lam from -20 to 20: a from exactly 1 (s = 0) to exactly 0.  Every
    result stays finite and right; an i_raw of -inf masks the input, an a_raw of -inf keeps the
    state (up to 2^-24 per step)."""
    x = R.inputs("gated", 4, "f32", cuda_device, batch=2, length=150, dim=40)
    x["Lam"] = torch.linspace(-20, 20, 40, device=cuda_device)
    x["a_raw"][:, ::7] = 30
    x["a_raw"][:, 1::7] = -30
    x["i_raw"][:, 2::7] = -float("inf")
    x["i_raw"][:, 3::7] = 30
    out, last = sb.sscan_gated_fwd(**x, rate=rate, return_last_state=True)
    ref, ref_last = R.gated(**{k: R.d64(v) for k, v in x.items()}, rate=rate)
    assert R.off(out, ref) <= F32 and R.off(last, ref_last) <= F32
    x["a_raw"][:, 10:] = -float("inf")
    out = sb.sscan_gated_fwd(**x, rate=rate)
    assert R.off(out[:, -1], out[:, 9]) <= 140 * 2.0 ** -24
    first, rest = args(x)
    g = sb.sscan_gated_bwd(*first, randn_like(x["u"], 1), *rest, rate=rate)
    assert all(torch.isfinite(v).all() for v in g.values())


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_sequence_in_many_groups(cuda_device, io):
    """40000 steps: 20 hops of the carry between groups of tiles; the end state and the
    gradients against one 64-bit recurrence."""
    x = R.inputs("gated", 12, io, cuda_device, batch=1, length=40000, dim=4)
    dout = randn_like(x["u"], 3)
    out, last = sb.sscan_gated_fwd(**x, return_last_state=True)
    ref, ref_last = R.gated(**{k: R.d64(v) for k, v in x.items()})
    assert R.off(out, ref) <= tol(out) and R.off(last, ref_last) <= F32
    first, rest = args(x)
    g = sb.sscan_gated_bwd(*first, dout, *rest)
    want = R.grads("gated", x, dout)
    for k, v in g.items():
        assert R.off(v, want[NAMES[k]]) <= (sums(40000) if k in ("dLam", "da_bias", "di_bias") else tol(v)), k
    assert sb.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 33])
def test_steps_and_segments_equal_one_forward(cuda_device, io, D):
    x = R.inputs("gated", 3, io, cuda_device, batch=3, length=70, dim=D)
    full, last = sb.sscan_gated_fwd(**x, return_last_state=True)
    first, rest = args(x)
    state, outs = x["h0"].clone(), []
    for t in range(70):
        p = R.token(x, t)
        outs.append(sb.sscan_gated_step(p["u"], p["a_raw"], p["i_raw"], x["Lam"], state, x["a_bias"], x["i_bias"]))
    assert R.off(torch.stack(outs, 1), full) <= 2 * tol(full)
    assert R.off(state, last) <= F32
    h, parts = x["h0"], []
    for cut in (slice(0, 13), slice(13, 70)):
        seg = [t[:, cut].contiguous() for t in first[:3]]
        o, h = sb.sscan_gated_fwd(*seg, x["Lam"], x["a_bias"], x["i_bias"], h, return_last_state=True)
        parts.append(o)
    assert R.off(torch.cat(parts, 1), full) <= 2 * tol(full) and R.off(h, last) <= F32


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unaligned_pointers(cuda_device, io):
    x = R.inputs("gated", 6, io, cuda_device, batch=2, length=300, dim=64)
    dout = randn_like(x["u"], 2)
    y = {k: R.shifted(v) if k in ("u", "a_raw", "i_raw") else v for k, v in x.items()}
    a, b = sb.sscan_gated_fwd(**x), sb.sscan_gated_fwd(**y)
    assert torch.equal(a, b)                              # the access width changes no arithmetic
    ga, gb = (sb.sscan_gated_bwd(*args(v)[0], dout, *args(v)[1]) for v in (x, y))
    assert all(torch.equal(ga[k], gb[k]) for k in ga)


@pytest.mark.gpu
def test_a_nan_stays_in_its_own_future(cuda_device):
    x = R.inputs("gated", 8, "bf16", cuda_device, batch=2, length=300, dim=16)
    clean = sb.sscan_gated_fwd(**x)
    x["u"][1, 150, 3] = float("nan")
    out = sb.sscan_gated_fwd(**x)
    bad = torch.isnan(out)
    assert bad[1, 150:, 3].all() and int(bad.sum()) == 150
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.gpu
def test_repeats_graphs_and_streams(cuda_device):
    """Two runs give the same bits, whatever the tiles' timing; two captured graphs that share a
    caller's workspace replay one after the other on new values; a call on another stream."""
    x = R.inputs("gated", 9, "bf16", cuda_device, batch=2, length=5000, dim=70)
    dout = randn_like(x["u"], 5)
    first, rest = args(x)
    prob = sb.GatedProblem(2, 5000, 70, 1, 8.0)
    ws = torch.empty(sb.load_library().sscan_gated_workspace_size(prob, sb.SSCAN_OP_BWD), dtype=torch.uint8,
                     device=cuda_device)

    def fwd(**kw):
        return list(sb.sscan_gated_fwd(**x, return_last_state=True, **kw))

    def bwd(**kw):
        return list(sb.sscan_gated_bwd(*first, dout, *rest, **kw).values())
    want = fwd() + bwd()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, fwd() + bwd()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fwd(stream=side) + bwd(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs, held = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr, fn in zip(graphs, (fwd, bwd)):
        with torch.cuda.graph(gr):
            held += fn(workspace=ws)
    x["u"].neg_()
    for gr in graphs * 2:
        gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, fwd() + bwd()))
    assert sb.device_status() == 0


@pytest.mark.gpu
def test_empty_sizes(cuda_device):
    for batch, L, D in ((0, 5, 4), (2, 0, 4), (2, 5, 0)):
        x = R.inputs("gated", 1, "bf16", cuda_device, batch=batch, length=L, dim=D)
        out, last = sb.sscan_gated_fwd(**x, return_last_state=True)
        assert out.shape == x["u"].shape
        if L == 0:
            assert torch.equal(last, x["h0"])
        first, rest = args(x)
        g = sb.sscan_gated_bwd(*first, torch.empty_like(x["u"]), *rest)
        assert all((v == 0).all() for v in g.values())


def test_binding_refuses():
    u, lam = torch.zeros(1, 4, 6), torch.zeros(6)
    with pytest.raises(ValueError, match="CUDA"):
        sb.sscan_gated_fwd(u, u, u, lam)
    with pytest.raises(TypeError):
        sb.sscan_gated_fwd(u.half(), u, u, lam)
    with pytest.raises(ValueError):
        sb.sscan_gated_step(u, u, u, lam, lam)


@pytest.mark.gpu
def test_binding_refuses_on_device(cuda_device):
    x = R.inputs("gated", 9, "f32", cuda_device, batch=2, length=100, dim=6)
    (u, a, i, lam), (ab, ib, h0) = args(x)
    for bad in (lambda: sb.sscan_gated_fwd(u, a[:, :99], i, lam), lambda: sb.sscan_gated_fwd(u, a.bfloat16(), i, lam),
                lambda: sb.sscan_gated_fwd(u, a, i, lam[:5]), lambda: sb.sscan_gated_fwd(u, a, i, None),
                lambda: sb.sscan_gated_fwd(u, a, i, lam, ab, ib, h0.bfloat16()),
                lambda: sb.sscan_gated_fwd(u.transpose(0, 1), a, i, lam),
                lambda: sb.sscan_gated_bwd(u, a, i, lam, None), lambda: sb.sscan_gated_bwd(u, a, i, lam, u[:1]),
                lambda: sb.sscan_gated_bwd(u, a, i, lam, u, checkpoints=torch.zeros(2, 3, 6, device=cuda_device)),
                lambda: sb.sscan_gated_step(u[:, 0].contiguous(), a[:, 0].contiguous(), i[:, 0].contiguous(), lam, None)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for rate in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(sb.SscanError, match="rate"):
            sb.sscan_gated_fwd(u, a, i, lam, rate=rate)
    with pytest.raises(sb.SscanError, match="workspace"):
        sb.sscan_gated_bwd(u, a, i, lam, u, workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device)[:16])


def test_c_entry_refuses():
    lib = sb.load_library()
    fake = ctypes.c_void_p(0x10000)
    ok = sb.GatedProblem(2, 200, 6, 0, 8.0)
    assert lib.sscan_gated_fwd(None, *([fake] * 10), fake, 1 << 20, None) == 1
    assert lib.sscan_gated_fwd(sb.GatedProblem(2, -1, 6, 0, 8.0), *([fake] * 10), fake, 1 << 20, None) == 1
    assert lib.sscan_gated_fwd(sb.GatedProblem(2, 100, 6, 3, 8.0), *([fake] * 10), fake, 1 << 20, None) == 1
    assert lib.sscan_gated_fwd(sb.GatedProblem(1 << 20, 1 << 17, 64, 0, 8.0), *([fake] * 10), fake, 1 << 20, None) == 2
    need = lib.sscan_gated_workspace_size(ok, sb.SSCAN_OP_FWD)
    assert need > 0 and need % 256 == 0
    # one tile needs no carry
    assert lib.sscan_gated_workspace_size(sb.GatedProblem(2, 64, 6, 0, 8.0), sb.SSCAN_OP_FWD) == 0
    assert lib.sscan_gated_checkpoints(ok) == 4
    assert lib.sscan_gated_fwd(ok, *([fake] * 10), None, 0, None) == 3
    assert lib.sscan_gated_fwd(ok, *([fake] * 10), fake, need - 1, None) == 3
    assert lib.sscan_gated_fwd(ok, fake, None, *([fake] * 8), fake, need, None) == 1
    args_ = [fake] * 16
    args_[4] = None                                       # a_bias, with da_bias given
    assert lib.sscan_gated_bwd(ok, *args_, fake, 1 << 30, None) == 1 and b"da_bias" in lib.sscan_last_error()
    assert lib.sscan_gated_step(ok, *([fake] * 8), None) == 1 and b"seqlen" in lib.sscan_last_error()


def test_reference_gradient_matches_differences():
    x = {k: R.d64(v) for k, v in R.inputs("gated", 2, batch=2, length=9, dim=3).items()}
    dout = torch.randn(2, 9, 3, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    R_check_differences("gated", x, dout)
