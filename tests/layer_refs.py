"""The layers around the scan in 64 bits on the CPU, token by token from their definitions, with
gradients by automatic differentiation: what the GPU tests compare with.  ``inputs`` draws them."""
import math

import numpy as np
import torch

# Half a rounding step relative to the value, by I/O type: what one rounding of a result costs.
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def d64(t):
    return None if t is None else t.detach().double().cpu()


def conv(u, weight, bias=None, state0=None, silu=True):
    """(out, state_last)"""
    b, L, D = u.shape
    K = weight.shape[1]
    win = state0 if state0 is not None else u.new_zeros(b, K - 1, D)
    full = torch.cat([win, u], 1)
    out = []
    for t in range(L):
        y = (full[:, t:t + K] * weight.t()).sum(1)
        y = y + bias if bias is not None else y
        out.append(y * torch.sigmoid(y) if silu else y)
    return (torch.stack(out, 1) if out else torch.zeros_like(u)), full[:, L:]


def gated(u, a_raw, i_raw, Lam, a_bias=None, i_bias=None, h0=None, rate=8.0):
    """(out, h_last)"""
    b, L, D = u.shape
    h = h0 if h0 is not None else u.new_zeros(b, D)
    out = []
    c = rate * torch.logaddexp(Lam, torch.zeros_like(Lam))
    for t in range(L):
        r = torch.sigmoid(a_raw[:, t] + (a_bias if a_bias is not None else 0))
        i = torch.sigmoid(i_raw[:, t] + (i_bias if i_bias is not None else 0))
        h = torch.exp(-c * r) * h + torch.sqrt(-torch.expm1(-2 * c * r)) * i * u[:, t]
        out.append(h)
    return (torch.stack(out, 1) if out else torch.zeros_like(u)), h


def heads(u, delta_raw, A, B, C, delta_bias=None, D_skip=None, z=None, h0=None, softplus=True):
    """(out, h_last)"""
    b, L, H, P = u.shape
    G, N = B.shape[2:]
    S = h0 if h0 is not None else u.new_zeros(b, H, P, N)
    out = []
    for t in range(L):
        dl = delta_raw[:, t] + (delta_bias if delta_bias is not None else 0)
        dl = torch.logaddexp(dl, torch.zeros_like(dl)) if softplus else dl
        q = dl * A
        # expm1(q) / A with its limit at A = 0
        w = torch.where(A == 0, dl, torch.expm1(q) / torch.where(A == 0, torch.ones_like(A), A))
        Bt, Ct = (x[:, t].repeat_interleave(H // G, 1) for x in (B, C))
        S = torch.exp(q)[..., None, None] * S + (w[..., None] * u[:, t])[..., None] * Bt[:, :, None]
        y = (S * Ct[:, :, None]).sum(-1)
        y = y + D_skip[:, None] * u[:, t] if D_skip is not None else y
        out.append(y * z[:, t] * torch.sigmoid(z[:, t]) if z is not None else y)
    return (torch.stack(out, 1) if out else torch.zeros_like(u)), S


FN = {"conv": conv, "gated": gated, "heads": heads}


def grads(op, x, dout, **kw):
    """d sum(out * dout) / d input for every tensor of the dict x, in 64 bits."""
    leaves = {k: d64(v).requires_grad_() for k, v in x.items() if v is not None}
    out, _ = FN[op](**leaves, **kw)
    got = torch.autograd.grad((out * d64(dout)).sum(), list(leaves.values()), allow_unused=True)
    return {k: torch.zeros_like(leaves[k]) if g is None else g for k, g in zip(leaves, got)}


def inputs(op, seed, io="f32", device="cpu", state=True, biases=True, **s):
    """Seeded inputs of one operator under its keyword names."""
    rng = np.random.default_rng(seed)
    dt = DTYPES[io]

    def normal(*shape, dtype=dt):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype).to(device)

    def uniform(lo, hi, *shape):
        return torch.from_numpy(rng.uniform(lo, hi, shape).astype(np.float32)).to(device)

    b, L = s["batch"], s["length"]
    if op == "conv":
        D, K = s["dim"], s["taps"]
        return {"u": normal(b, L, D), "weight": uniform(-0.5, 0.5, D, K),
                "bias": uniform(-0.5, 0.5, D) if biases else None,
                "state0": normal(b, K - 1, D) if state else None}
    if op == "gated":
        D = s["dim"]
        lam = [math.log(math.expm1(-math.log(v) / 8)) for v in rng.uniform(0.9, 0.999, D)]
        return {"u": normal(b, L, D), "a_raw": normal(b, L, D), "i_raw": normal(b, L, D),
                "Lam": torch.tensor(lam, dtype=torch.float32, device=device),
                "a_bias": uniform(-0.5, 0.5, D) if biases else None,
                "i_bias": uniform(-0.5, 0.5, D) if biases else None,
                "h0": normal(b, D, dtype=torch.float32) if state else None}
    H, P, N, G = s["heads"], s["headdim"], s["dstate"], s["groups"]
    dt_bias = np.log(np.expm1(np.exp(rng.uniform(math.log(1e-3), math.log(1e-1), H))))
    return {"u": normal(b, L, H, P), "delta_raw": normal(b, L, H),
            "A": -(torch.arange(H, dtype=torch.float32, device=device) % 16 + 1),
            "B": normal(b, L, G, N), "C": normal(b, L, G, N),
            "delta_bias": torch.from_numpy(dt_bias.astype(np.float32)).to(device) if biases else None,
            "D_skip": normal(H, dtype=torch.float32) if biases else None,
            "z": normal(b, L, H, P) if s.get("gate", True) else None,
            "h0": normal(b, H, P, N, dtype=torch.float32) if state else None}


def token(x, t):
    """One token of a dict of inputs: (batch, L, ...) tensors at step t; parameters as they are."""
    rows = {"u", "a_raw", "i_raw", "delta_raw", "B", "C", "z"}
    return {k: v[:, t].contiguous() if k in rows and v is not None else v for k, v in x.items()}


def off(got, ref):
    """max |got - ref| / max |ref|"""
    got, ref = d64(got), d64(ref)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    if ref.numel() == 0:
        return 0.0
    assert torch.isfinite(ref).all()
    top = float(ref.abs().max())
    err = float((got - ref).abs().max())
    return err / top if top > 0 else err


def shifted(t):
    """The same values one element past the start of their storage (no wide access possible)."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v
