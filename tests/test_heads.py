"""The multi-head linear recurrence: sscan_heads_fwd, sscan_heads_bwd, sscan_heads_step."""
import ctypes

import pytest
import torch

from selective_state_space_33_b200 import binding as sb

from . import layer_refs as R
from .test_conv import R_check_differences

# fp32: products of two-part tf32 operands leave out 2^-22 of each term and accumulate in
# fp32; the longest sums here have 64 + 128 + 64 terms, the sum of whose sizes is within ~16
# times the largest result: 16 * (2^-22 + 256 * 2^-24 / 16) ~ 2e-5; exponentials and step
# sizes add a few 2^-23 per step of a memory of at most some 1000 steps.  In all 2^-13.
F32 = 2.0 ** -13
# bf16: a result is rounded once (2^-8 at most); on the way the entries of M, and in the
# backward dy and the states, are rounded to bf16 once more, each at most 2^-8 of its term,
# with signs that do not align: three such contributions against the largest result.
BF16 = 4 * 2.0 ** -8
# fp32 results of bf16 inputs: their inexact factors go in as two bf16 parts, 2^-16 of each
# term at most, the sum of sizes within ~16 times the result.
PAIR = 16 * 2.0 ** -16


def tol(t):
    return BF16 if t.dtype == torch.bfloat16 else F32


def sums(tokens, io):
    """Parameter gradients, sums over tokens of either sign: the sum of T sizes is some sqrt(T)
    times that of a sum of T random signs."""
    return (PAIR if io == "bf16" else F32) * max(4, tokens ** 0.5 / 4)


NAMES = {"du": "u", "ddelta_raw": "delta_raw", "dA": "A", "dB": "B", "dC": "C", "ddelta_bias": "delta_bias",
         "dD": "D_skip", "dz": "z", "dh0": "h0"}
# batch, L, heads, P, N, groups: around the 64-step chunk; P, N off every multiple
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 7, 3, 64, 16, 1), (1, 63, 2, 16, 40, 2), (2, 64, 4, 33, 5, 2), (1, 65, 1, 64, 128, 1),
          (1, 200, 6, 40, 24, 3), (2, 130, 2, 64, 64, 1), (1, 321, 2, 8, 100, 1), (1, 700, 2, 20, 16, 1),
          # more than 32 states on 16-byte rows, around the 128-step chunk of the tensor-core forward
          (1, 128, 2, 64, 128, 1), (2, 129, 1, 48, 72, 1), (1, 255, 4, 64, 64, 2), (1, 700, 2, 64, 128, 1),
          (1, 1100, 3, 16, 48, 3)]


def case(shape, seed, io, device, **kw):
    batch, L, H, P, N, G = shape
    return R.inputs("heads", seed, io, device, batch=batch, length=L, heads=H, headdim=P, dstate=N, groups=G, **kw)


def bwd(x, dout, **kw):
    return sb.sscan_heads_bwd(*[x[k] for k in ("u", "delta_raw", "A", "B", "C")], dout,
                              *[x[k] for k in ("delta_bias", "D_skip", "z", "h0")], **kw)


def randn_like(t, seed):
    return torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)).to(t.dtype).to(t.device)


def check_backward(x, dout, io, tokens, **kw):
    g = bwd(x, dout, **({"delta_softplus": kw["softplus"]} if kw else {}))
    given = dict(x)
    if x["h0"] is None:
        given["h0"] = torch.zeros_like(g["dh0"])
    want = R.grads("heads", given, dout, **kw)
    assert {NAMES[k] for k in g} == {k for k, v in given.items() if v is not None}
    bad = {}
    for k, v in g.items():
        limit = sums(tokens, io) if k in ("dA", "ddelta_bias", "dD") else (PAIR if io == "bf16" else F32) if k == "dh0" \
            else tol(v)
        e = R.off(v, want[NAMES[k]])
        if not e <= limit:
            bad[k] = (e, limit)
    assert not bad, bad


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("full", [True, False])
def test_forward_and_backward(cuda_device, io, shape, full):
    x = case(shape, sum(shape), io, cuda_device, state=full, biases=full, gate=full)
    out, last = sb.sscan_heads_fwd(**x, return_last_state=True)
    ref, ref_last = R.heads(**{k: R.d64(v) for k, v in x.items()})
    assert R.off(out, ref) <= tol(out)
    assert R.off(last, ref_last) <= (PAIR if io == "bf16" else F32)
    check_backward(x, randn_like(x["u"], 1), io, shape[0] * shape[1])


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_split_sequence(cuda_device, io):
    """5000 steps of two heads: 20 segments in the forward pass, 79 chunks in the backward."""
    x = case((1, 5000, 2, 24, 16, 1), 5, io, cuda_device)
    out, last = sb.sscan_heads_fwd(**x, return_last_state=True)
    assert sb.load_library().sscan_last_launch_count() == 3
    ref, ref_last = R.heads(**{k: R.d64(v) for k, v in x.items()})
    assert R.off(out, ref) <= tol(out)
    assert R.off(last, ref_last) <= (PAIR if io == "bf16" else F32)
    check_backward(x, randn_like(x["u"], 1), io, 5000)


@pytest.mark.gpu
@pytest.mark.parametrize("io,shape", [("f32", (8, 1100, 64, 8, 4, 1)), ("bf16", (8, 1100, 64, 8, 4, 1)),
                                      ("f32", (4, 600, 40, 8, 80, 1)), ("bf16", (8, 600, 60, 9, 40, 2))])
def test_more_pairs_than_blocks(cuda_device, io, shape):
    """More (batch, head) pairs than the GPU holds blocks: segments of 512 steps hand their state on;
    twice the same bits, and a captured call replays."""
    x = case(shape, 21, io, cuda_device)
    out, last = sb.sscan_heads_fwd(**x, return_last_state=True)
    ref, ref_last = R.heads(**{k: R.d64(v) for k, v in x.items()})
    assert R.off(out, ref) <= tol(out)
    assert R.off(last, ref_last) <= (PAIR if io == "bf16" else F32)
    again, last2 = sb.sscan_heads_fwd(**x, return_last_state=True)
    assert torch.equal(out, again) and torch.equal(last, last2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = sb.sscan_heads_fwd(**x)
    for _ in range(3):
        held.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, out)
    assert sb.device_status() == 0


@pytest.mark.gpu
def test_plain_step_sizes_and_zero_decay(cuda_device):
    """Without softplus (step sizes of either sign, growing states among them) and with A = 0,
    where the weight of the input is the step size itself."""
    x = case((2, 100, 4, 16, 16, 1), 6, "f32", cuda_device, biases=False)
    x["delta_raw"] *= 0.05
    x["A"][0] = 0.0
    out = sb.sscan_heads_fwd(**x, delta_softplus=False)
    ref, _ = R.heads(**{k: R.d64(v) for k, v in x.items()}, softplus=False)
    assert R.off(out, ref) <= F32
    x["A"][0] = -1e-4  # the reference's derivative at exactly 0 is not defined by its division
    check_backward(x, randn_like(x["u"], 2), "f32", 200, softplus=False)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_steps_that_forget_everything(cuda_device, io):
    """Step sizes up to 1000 with A = -16: q down to -16000, among ordinary ones.  The running sum
    inside a chunk reaches -1e6 while differences of it stay of order one."""
    x = case((1, 150, 2, 16, 16, 1), 8, io, cuda_device)
    x["A"][:] = -16
    x["delta_raw"][:, ::5] = 1000
    out, last = sb.sscan_heads_fwd(**x, return_last_state=True)
    ref, ref_last = R.heads(**{k: R.d64(v) for k, v in x.items()})
    assert R.off(out, ref) <= tol(out)
    assert R.off(last, ref_last) <= (PAIR if io == "bf16" else F32)
    check_backward(x, randn_like(x["u"], 2), io, 150)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", [(64, 16), (20, 33), (64, 128)])
def test_steps_and_segments_equal_one_forward(cuda_device, io, P, N):
    x = case((2, 90, 4, P, N, 2), 3, io, cuda_device)
    full, last = sb.sscan_heads_fwd(**x, return_last_state=True)
    state, outs = x["h0"].clone(), []
    for t in range(90):
        p = R.token(x, t)
        outs.append(sb.sscan_heads_step(p["u"], p["delta_raw"], x["A"], p["B"], p["C"], state, x["delta_bias"],
                                        x["D_skip"], p["z"]))
    assert R.off(torch.stack(outs, 1), full) <= 2 * tol(full)
    assert R.off(state, last) <= 2 * (PAIR if io == "bf16" else F32)
    h, parts = x["h0"], []
    for cut in (slice(0, 31), slice(31, 90)):
        seg = {k: x[k][:, cut].contiguous() for k in ("u", "delta_raw", "B", "C", "z")}
        o, h = sb.sscan_heads_fwd(**{**x, **seg, "h0": h}, return_last_state=True)
        parts.append(o)
    assert R.off(torch.cat(parts, 1), full) <= 2 * tol(full)
    assert R.off(h, last) <= 2 * (PAIR if io == "bf16" else F32)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("N", [16, 64])
def test_a_value_that_is_not_finite_stays_in_its_own_future(cuda_device, io, value, N):
    x = case((2, 150, 2, 16, N, 1), 9, io, cuda_device)
    clean = sb.sscan_heads_fwd(**x)
    for name, at in (("u", (1, 70, 1, 3)), ("B", (1, 70, 0, 2)), ("C", (1, 70, 0, 2)), ("z", (1, 70, 1, 3)),
                     ("delta_raw", (1, 70, 1)), ("delta_raw", (1, 71, 1))):
        y = dict(x)
        y[name] = x[name].clone()
        y[name][at] = value
        out = sb.sscan_heads_fwd(**y)
        assert sb.device_status() == 0
        assert torch.equal(out[0], clean[0]), name
        assert torch.equal(out[1, :70], clean[1, :70]), name
        if name in ("u", "z", "delta_raw"):              # the other head
            assert torch.equal(out[1, :, 0], clean[1, :, 0]), name
        if name == "u":                                  # the other channels, and this one from step 70 on
            keep = [p for p in range(16) if p != 3]
            assert torch.equal(out[1, :, 1, keep], clean[1, :, 1, keep])
            assert not torch.isfinite(out[1, 70:, 1, 3]).any()
        if name in ("C", "z"):                           # one step only
            assert torch.equal(out[1, 71:], clean[1, 71:]), name


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_unaligned_pointers(cuda_device, io):
    x = case((2, 100, 2, 64, 16, 1), 6, io, cuda_device)
    dout = randn_like(x["u"], 2)
    y = {k: R.shifted(v) if k in ("u", "B", "C", "z", "delta_raw") else v for k, v in x.items()}
    assert torch.equal(sb.sscan_heads_fwd(**x), sb.sscan_heads_fwd(**y))
    ga, gb = bwd(x, dout), bwd(y, R.shifted(dout))
    assert all(torch.equal(ga[k], gb[k]) for k in ga)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["u", "B", "C", "z", "dout", "out"])
def test_one_unaligned_pointer(cuda_device, io, name):
    """Wide accesses need every tensor they touch on a 16-byte boundary, not the first one only."""
    x = case((1, 70, 2, 64, 32, 1), 16, io, cuda_device)
    dout = randn_like(x["u"], 2)
    want, grads = sb.sscan_heads_fwd(**x), bwd(x, dout)
    if name == "dout":
        dout = R.shifted(dout)
    elif name != "out":
        x[name] = R.shifted(x[name])
    out = R.shifted(torch.empty_like(want)) if name == "out" else None
    assert torch.equal(sb.sscan_heads_fwd(**x, out=out), want)
    again = bwd(x, dout)
    assert all(torch.equal(grads[k], again[k]) for k in grads)


@pytest.mark.gpu
def test_repeats_graphs_and_streams(cuda_device):
    x = case((2, 3000, 4, 32, 32, 2), 9, "bf16", cuda_device)
    dout = randn_like(x["u"], 5)
    prob = sb.HeadsProblem(2, 3000, 4, 32, 32, 2, 1, 1)
    lib = sb.load_library()
    ws = torch.empty(max(lib.sscan_heads_workspace_size(prob, op) for op in (sb.SSCAN_OP_FWD, sb.SSCAN_OP_BWD)),
                     dtype=torch.uint8, device=cuda_device)

    def fwd_(**kw):
        return list(sb.sscan_heads_fwd(**x, return_last_state=True, **kw))

    def bwd_(**kw):
        return list(bwd(x, dout, **kw).values())
    want = fwd_() + bwd_()
    assert all(torch.equal(a, b) for a, b in zip(want, fwd_() + bwd_()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fwd_(stream=side) + bwd_(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs, held = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr, fn in zip(graphs, (fwd_, bwd_)):
        with torch.cuda.graph(gr):
            held += fn(workspace=ws)
    x["u"].neg_()
    for gr in graphs * 2:
        gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, fwd_() + bwd_()))


@pytest.mark.gpu
def test_empty_sizes(cuda_device):
    for shape in ((0, 5, 2, 4, 4, 1), (2, 0, 2, 4, 4, 1)):
        x = case(shape, 1, "bf16", cuda_device)
        out, last = sb.sscan_heads_fwd(**x, return_last_state=True)
        assert out.shape == x["u"].shape
        if shape[1] == 0:
            assert torch.equal(last, x["h0"])
        g = bwd(x, torch.empty_like(x["u"]))
        assert all((v == 0).all() for v in g.values())


def test_binding_refuses():
    u, d, A, B = torch.zeros(1, 4, 2, 6), torch.zeros(1, 4, 2), torch.zeros(2), torch.zeros(1, 4, 1, 8)
    with pytest.raises(ValueError, match="CUDA"):
        sb.sscan_heads_fwd(u, d, A, B, B)
    with pytest.raises(TypeError):
        sb.sscan_heads_fwd(u.half(), d, A, B, B)
    with pytest.raises(ValueError):
        sb.sscan_heads_fwd(u[0], d, A, B, B)


@pytest.mark.gpu
def test_binding_refuses_on_device(cuda_device):
    x = case((2, 8, 4, 6, 8, 2), 9, "f32", cuda_device)
    for k, v in (("delta_raw", x["delta_raw"][:, :7]), ("A", x["A"][:3]), ("A", x["A"].bfloat16()), ("B", x["B"][0]),
                 ("C", x["C"][..., :7]), ("z", x["z"].bfloat16()), ("h0", x["h0"][:1]), ("u", x["u"].transpose(0, 1)),
                 ("A", None), ("D_skip", x["D_skip"][:1])):
        with pytest.raises((ValueError, TypeError)):
            sb.sscan_heads_fwd(**{**x, k: v})
    with pytest.raises((ValueError, TypeError)):
        bwd(x, None)
    with pytest.raises(sb.SscanError, match="multiple"):
        sb.sscan_heads_fwd(**{**x, "B": x["B"].repeat(1, 1, 3, 1)[:, :, :3].contiguous(),
                              "C": x["C"].repeat(1, 1, 3, 1)[:, :, :3].contiguous()})
    with pytest.raises(sb.SscanError, match="workspace"):
        bwd(x, x["u"], workspace=torch.empty(256, dtype=torch.uint8, device=cuda_device)[:16])


def test_c_entry_refuses():
    lib = sb.load_library()
    fake = ctypes.c_void_p(0x10000)

    def fwd(prob, args=None):
        return lib.sscan_heads_fwd(prob, *(args or [fake] * 11), fake, 1 << 30, None)
    P = sb.HeadsProblem
    assert lib.sscan_heads_fwd(None, *([fake] * 11), fake, 0, None) == 1
    for bad, rc in (((-1, 8, 4, 8, 8, 1, 0, 1), 1), ((2, 8, 4, 0, 8, 1, 0, 1), 1), ((2, 8, 4, 65, 8, 1, 0, 1), 2),
                    ((2, 8, 4, 8, 129, 1, 0, 1), 2), ((2, 8, 4, 8, 8, 3, 0, 1), 1), ((2, 8, 4, 8, 8, 1, 5, 1), 1),
                    ((2, 8, 4, 8, 8, 1, 0, 2), 1), ((70000, 8, 4, 8, 8, 1, 0, 1), 2),
                    ((1, 1 << 36, 64, 8, 8, 1, 0, 1), 2)):
        assert fwd(P(*bad)) == rc, bad
    ok = P(2, 8, 4, 8, 8, 1, 0, 1)
    assert fwd(ok, [None] + [fake] * 10) == 1 and b"required" in lib.sscan_last_error()
    assert lib.sscan_heads_workspace_size(ok, sb.SSCAN_OP_FWD) == 0
    long = P(1, 1 << 16, 4, 8, 8, 1, 0, 1)
    need = lib.sscan_heads_workspace_size(long, sb.SSCAN_OP_FWD)
    assert need > 0 and need % 256 == 0
    assert lib.sscan_heads_fwd(long, *([fake] * 11), fake, need - 1, None) == 3
    need = lib.sscan_heads_workspace_size(ok, sb.SSCAN_OP_BWD)
    assert lib.sscan_heads_bwd(ok, *([fake] * 19), fake, need - 1, None) == 3
    for name, i in (("dz", 7), ("dD", 6), ("ddelta_bias", 2)):   # the input left out, its gradient asked for
        args = [fake] * 19
        args[i] = None
        assert lib.sscan_heads_bwd(ok, *args, fake, need, None) == 1 and name.encode() in lib.sscan_last_error()
    assert lib.sscan_heads_step(ok, *([fake] * 10), None) == 1 and b"seqlen" in lib.sscan_last_error()


def test_reference_gradient_matches_differences():
    x = {k: R.d64(v) for k, v in case((2, 9, 4, 3, 5, 2), 2, "f32", "cpu").items()}
    dout = torch.randn(2, 9, 4, 3, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    R_check_differences("heads", x, dout)
