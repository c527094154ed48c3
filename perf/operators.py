"""The layers around the selective scan that the package offers, as measured cases: the causal
depthwise convolution that feeds a scan (``conv``), the gated linear recurrence with one state per
channel (``gated``), and the multi-head linear recurrence with a matrix state (``heads``).  Each has
a forward pass, a training pass (forward and backward) and a one-token generation step.

``run`` computes them in elementary torch operations (fp32, rounded once at the end), or, where
``own`` is true, by the package's calls.  ``exact`` computes the same outputs in 64 bits, token by
token, from the operators' definitions.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_RATE = 8.0
_TAPS_BOUND = 0.5


# ---------------------------------------------------------------- cases

def listed():
    conv = dict(op="conv", taps=4, silu=True)
    heads = dict(op="heads", gate=True)
    return [
        # the input branch of the 130M-width layer, prefill
        dict(conv, name="conv_fwd_130m", kind="fwd", batch=8, length=2048, dim=1536, io="bf16", state=False),
        # its training pass, continued from a carried window; odd length, and a width off the vector size
        dict(conv, name="conv_train_odd_f32", kind="train", batch=3, length=1021, dim=1531, io="f32", state=True),
        # one generated token for 64 sequences at the 2.8B width
        dict(conv, name="conv_step_2.8b", kind="step", batch=64, length=1, dim=5120, io="bf16", state=True),
        # the recurrence at the 2.8B width: many channels, moderate length
        dict(op="gated", name="gated_fwd_2.8b", kind="fwd", batch=8, length=2048, dim=5120, io="bf16", state=False),
        # training at the 130M width
        dict(op="gated", name="gated_train_130m", kind="train", batch=8, length=2048, dim=1536, io="bf16", state=True),
        # one long sequence: few channels, the sequence itself has to be split
        dict(op="gated", name="gated_fwd_long", kind="fwd", batch=1, length=131072, dim=1536, io="bf16", state=True),
        # one generated token
        dict(op="gated", name="gated_step_2.8b", kind="step", batch=64, length=1, dim=5120, io="bf16", state=True),
        # the multi-head form of the 2.8B width with the scan's own 16 states
        dict(heads, name="heads_fwd_2.8b", kind="fwd", batch=8, length=2048, heads=80, headdim=64, dstate=16, groups=1,
             io="bf16", state=False),
        # a long sequence with a large state
        dict(heads, name="heads_fwd_long", kind="fwd", batch=1, length=65536, heads=24, headdim=64, dstate=128, groups=1,
             io="bf16", state=True),
        # training at the 130M width, heads sharing B and C
        dict(heads, name="heads_train_130m", kind="train", batch=8, length=2048, heads=24, headdim=64, dstate=64, groups=1,
             io="bf16", state=True),
        # fp32 training, ragged sizes, two groups
        dict(heads, name="heads_train_odd_f32", kind="train", batch=2, length=515, heads=6, headdim=40, dstate=24, groups=2,
             io="f32", state=True),
        # one generated token
        dict(heads, name="heads_step_2.8b", kind="step", batch=64, length=1, heads=80, headdim=64, dstate=16, groups=1,
             io="bf16", state=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "gated", "heads"])
    kind = rng.choice(["fwd", "fwd", "train", "train", "step"])
    io = rng.choice(["bf16", "bf16", "f32"])
    state = kind == "step" or rng.random() < 0.5
    length = 1 if kind == "step" else _log(rng, 1, 32768)
    batch = _log(rng, 1, 128) if kind == "step" else _log(rng, 1, 8)
    room = 8 * 2048 * 1536 // (batch * length)          # channels that keep the work within the listed cases'
    c = dict(op=op, kind=kind, batch=batch, length=length, io=io, state=state)
    if op != "heads":
        dim = _log(rng, 8, max(8, min(5120, room)))
        c["dim"] = dim if rng.random() < 0.4 else max(8, dim // 8 * 8)
        if op == "conv":
            c["taps"] = rng.randint(2, 4)
            c["silu"] = rng.random() < 0.8
        return c
    c["headdim"] = rng.choice([16, 32, 48, 64, 64, rng.randint(8, 64)])
    c["dstate"] = rng.choice([16, 32, 64, 128, rng.randint(4, 128)])
    c["groups"] = rng.choice([1, 1, 1, 2, 4])
    most = max(1, room // (c["headdim"] * c["groups"]))
    c["heads"] = c["groups"] * _log(rng, 1, max(1, min(80 // c["groups"], most)))
    c["gate"] = rng.random() < 0.7
    return c


def _fp(case):
    return {k: v for k, v in case.items() if k != "name"}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)
    dt = _DT[case["io"]]
    b, n = case["batch"], case["length"]
    step = case["kind"] == "step"

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32) * (hi - lo) + lo

    def rows(*tail):                                    # a (batch, L, ...) tensor, or one token of it
        return normal(b, *tail) if step else normal(b, n, *tail)

    s = {"case": _fp(case)}
    if case["op"] == "conv":
        d, k = case["dim"], case["taps"]
        s["u"] = rows(d)
        s["weight"] = uniform(-_TAPS_BOUND, _TAPS_BOUND, d, k)
        s["bias"] = uniform(-_TAPS_BOUND, _TAPS_BOUND, d)
        s["state"] = normal(b, k - 1, d) if case["state"] else None
    elif case["op"] == "gated":
        d = case["dim"]
        s["u"], s["a_raw"], s["i_raw"] = rows(d), rows(d), rows(d)
        # exp(-rate softplus(Lam)) uniform in [0.9, 0.999]: memories of ten to a thousand tokens
        s["Lam"] = torch.log(torch.expm1(-torch.log(uniform(0.9, 0.999, d)) / _RATE))
        s["a_bias"], s["i_bias"] = uniform(-0.5, 0.5, d), uniform(-0.5, 0.5, d)
        s["state"] = normal(b, d, dtype=torch.float32) if case["state"] else None
    else:
        h, p, st, g = case["heads"], case["headdim"], case["dstate"], case["groups"]
        s["u"], s["delta_raw"] = rows(h, p), rows(h)
        s["B"], s["C"] = rows(g, st), rows(g, st)
        s["z"] = rows(h, p) if case["gate"] else None
        s["A"] = -(torch.arange(h, device=dev, dtype=torch.float32) % 16 + 1)
        # softplus(bias) log-uniform in [1e-3, 1e-1], as the package's own workloads draw the step size
        s["delta_bias"] = torch.log(torch.expm1(torch.exp(uniform(math.log(1e-3), math.log(1e-1), h))))
        s["D_skip"] = normal(h, dtype=torch.float32)
        s["state"] = normal(b, h, p, st, dtype=torch.float32) if case["state"] else None
    s["dout"] = torch.randn(s["u"].shape, generator=gen, device=dev, dtype=torch.float32).to(dt) \
        if case["kind"] == "train" else None
    return s


def work(case):
    es = 2 if case["io"] == "bf16" else 4
    tok = case["batch"] * case["length"]
    train, step = case["kind"] == "train", case["kind"] == "step"
    if case["op"] == "heads":
        h, p, st, g = case["heads"], case["headdim"], case["dstate"], case["groups"]
        el = tok * h * p
        small = tok * (2 * g * st + h)
        one = (3 if case["gate"] else 2) * el + small            # u, z, out, B, C, delta
        by = one * es
        if train:                                                # + dout, du, dz, dB, dC, ddelta
            by += ((3 if case["gate"] else 2) * el + small) * es
        if case["state"]:
            by += 4 * case["batch"] * h * p * st * (3 if train else 2)
        return {"bytes": by, "flops": el * st * (18 if train else 6)}
    el = tok * case["dim"]
    if case["op"] == "conv":
        by = (4 if train else 2) * el * es
        if case["state"]:
            by += case["batch"] * (case["taps"] - 1) * case["dim"] * es * (3 if train else 2)
        return {"bytes": by, "flops": el * (6 * case["taps"] + 20 if train else 2 * case["taps"] + 6)}
    by = (8 if train else 4) * el * es
    if case["state"]:
        by += 4 * case["batch"] * case["dim"] * (3 if train else 2)
    return {"bytes": by, "flops": el * (60 if train else 20)}


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    return {"conv": _run_conv, "gated": _run_gated, "heads": _run_heads}[case["op"]](state, case)


def _run_conv(s, case):
    u, w, b, st, act, dt = s["u"], s["weight"], s["bias"], s["state"], case["silu"], s["u"].dtype
    if own:
        from selective_state_space_33_b200 import sscan_conv_bwd, sscan_conv_fwd, sscan_conv_step
        if case["kind"] == "step":
            return {"out": sscan_conv_step(u, w, st, b, silu=act), "state": st}
        out, last = sscan_conv_fwd(u, w, b, st, silu=act, return_last_state=True)
        r = {"out": out, "last": last}
        if case["kind"] == "train":
            r.update(sscan_conv_bwd(u, w, s["dout"], b, st, silu=act, want_dstate0=st is not None))
        return r
    k = case["taps"]
    if case["kind"] == "step":
        win = torch.cat([st, u[:, None]], 1)
        y = (win.float() * w.t()).sum(1) + b
        st.copy_(win[:, 1:])
        return {"out": _act(y, act).to(dt), "state": st}
    n = u.shape[1]
    head = st if st is not None else torch.zeros(u.shape[0], k - 1, u.shape[2], dtype=dt, device=u.device)
    full = torch.cat([head, u], 1)
    x = full.float()
    y = sum(x[:, j:j + n] * w[:, j] for j in range(k)) + b
    r = {"out": _act(y, act).to(dt), "last": full[:, n:].clone()}
    if case["kind"] == "train":
        dy = s["dout"].float() * (_dact(y) if act else 1.0)
        pad = torch.zeros_like(x[:, :k - 1])
        dyp = torch.cat([pad, dy, pad], 1)               # dx[j] = sum_k w[k] dy[j - k], j from the window's start
        dx = sum(dyp[:, k - 1 - j:k - 1 - j + n + k - 1] * w[:, j] for j in range(k))
        r["du"] = dx[:, k - 1:].to(dt)
        r["dweight"] = torch.stack([(x[:, j:j + n] * dy).sum((0, 1), dtype=torch.float64).float() for j in range(k)], 1)
        r["dbias"] = dy.sum((0, 1), dtype=torch.float64).float()
        if st is not None:
            r["dstate0"] = dx[:, :k - 1].to(dt)
    return r


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _act(y, act):
    return y * _sigmoid(y) if act else y


def _dact(y):
    s = _sigmoid(y)
    return s * (1 + y * (1 - s))


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20))))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h_{-1} = 0, by doubling: after each round every step holds
    the composition of twice as many steps."""
    n, d = b.shape[1], 1
    while d < n:
        b = torch.cat([b[:, :d], torch.addcmul(b[:, d:], a[:, d:], b[:, :-d])], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _run_gated(s, case):
    u, ar, ir, lam, ab, ib, st = (s[k] for k in ("u", "a_raw", "i_raw", "Lam", "a_bias", "i_bias", "state"))
    dt = u.dtype
    if own:
        from selective_state_space_33_b200 import sscan_gated_bwd, sscan_gated_fwd, sscan_gated_step
        if case["kind"] == "step":
            return {"out": sscan_gated_step(u, ar, ir, lam, st, ab, ib, rate=_RATE), "state": st}
        if case["kind"] == "fwd":
            out, last = sscan_gated_fwd(u, ar, ir, lam, ab, ib, st, rate=_RATE, return_last_state=True)
            return {"out": out, "last": last}
        out, last, saved = sscan_gated_fwd(u, ar, ir, lam, ab, ib, st, rate=_RATE, return_last_state=True,
                                           return_checkpoints=True)
        g = sscan_gated_bwd(u, ar, ir, lam, s["dout"], ab, ib, st, rate=_RATE, checkpoints=saved,
                            want_dh0=st is not None)
        return {"out": out, "last": last, **g}
    x = u.float()
    c = _RATE * _softplus(lam)
    r, i = _sigmoid(ar.float() + ab), _sigmoid(ir.float() + ib)
    sr = c * r
    a = torch.exp(-sr)
    m = torch.sqrt(-torch.expm1(-2 * sr))
    b = m * i * x
    if case["kind"] == "step":
        h = a * st + b
        st.copy_(h)
        return {"out": h.to(dt), "state": st}
    if st is not None:
        b = torch.cat([(b[:, 0] + a[:, 0] * st)[:, None], b[:, 1:]], 1)
    h = _scan(a, b)
    res = {"out": h.to(dt), "last": h[:, -1].clone()}
    if case["kind"] == "train":
        after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        g = _scan(after.flip(1), s["dout"].float().flip(1)).flip(1)
        first = (st if st is not None else torch.zeros_like(h[:, 0]))[:, None]
        prev = torch.cat([first, h[:, :-1]], 1)
        ds = -g * (a * prev - a * a / m * i * x)         # gradient with respect to s = -log a
        res["du"] = (g * m * i).to(dt)
        res["da_raw"] = (ds * sr * (1 - r)).to(dt)
        di = g * m * x * i * (1 - i)
        res["di_raw"] = di.to(dt)
        res["dLam"] = ((ds * r).sum((0, 1), dtype=torch.float64) * _RATE * _sigmoid(lam.double())).float()
        res["da_bias"] = (ds * sr * (1 - r)).sum((0, 1), dtype=torch.float64).float()
        res["di_bias"] = di.sum((0, 1), dtype=torch.float64).float()
        if st is not None:
            res["dh0"] = a[:, 0] * g[:, 0]
    return res


_Q = 64


def _run_heads(s, case):
    u, dr, A, B, C, bias, D, z, st, dt = (s["u"], s["delta_raw"], s["A"], s["B"], s["C"], s["delta_bias"], s["D_skip"],
                                          s["z"], s["state"], s["u"].dtype)
    if own:
        from selective_state_space_33_b200 import sscan_heads_bwd, sscan_heads_fwd, sscan_heads_step
        if case["kind"] == "step":
            return {"out": sscan_heads_step(u, dr, A, B, C, st, bias, D, z), "state": st}
        out, last = sscan_heads_fwd(u, dr, A, B, C, bias, D, z, st, return_last_state=True)
        r = {"out": out, "last": last}
        if case["kind"] == "train":
            r.update(sscan_heads_bwd(u, dr, A, B, C, s["dout"], bias, D, z, st, want_dh0=st is not None))
        return r
    h, p, ns, g = case["heads"], case["headdim"], case["dstate"], case["groups"]
    rep = h // g
    raw = dr.float() + bias
    dl = _softplus(raw)
    q = dl * A
    w = torch.expm1(q) / A
    if case["kind"] == "step":
        Bh, Ch = (t.float().repeat_interleave(rep, 1) for t in (B, C))
        S = torch.exp(q)[..., None, None] * st + (w[..., None] * u.float())[..., None] * Bh[:, :, None]
        y = (S * Ch[:, :, None]).sum(-1) + D[:, None] * u.float()
        st.copy_(S)
        return {"out": (y * _act(z.float(), True) if z is not None else y).to(dt), "state": st}
    b, n = u.shape[:2]
    nc = -(-n // _Q)

    def fold(t):                                         # (b, L, heads, ...) -> (b, chunks, heads, Q, ...), zero-padded
        t = t.float()
        if nc * _Q != n:
            t = torch.cat([t, torch.zeros(b, nc * _Q - n, *t.shape[2:], device=t.device)], 1)
        return t.reshape(b, nc, _Q, *t.shape[2:]).transpose(2, 3)

    def unfold(t):
        return t.transpose(2, 3).reshape(b, nc * _Q, *t.shape[2:3], *t.shape[4:])[:, :n]

    x, qc, wc = fold(u), fold(q), fold(w)
    Bc, Cc = (fold(t).repeat_interleave(rep, 2) for t in (B, C))
    cum = qc.cumsum(-1)
    e = torch.exp(cum)
    end = torch.exp(cum[..., -1:] - cum)                 # decay from each step to its chunk's end
    tri = torch.ones(_Q, _Q, dtype=torch.bool, device=u.device).tril()
    Lm = torch.exp(torch.where(tri, cum[..., :, None] - cum[..., None, :], -math.inf))
    G = Cc @ Bc.transpose(-1, -2)
    loc = (x * (end * wc)[..., None]).transpose(-1, -2) @ Bc
    dec = e[..., -1][..., None, None]
    if st is not None:
        loc = torch.cat([(loc[:, 0] + dec[:, 0] * st)[:, None], loc[:, 1:]], 1)
    S = _scan(dec, loc)                                  # the state after each chunk
    Sin = torch.cat([(st if st is not None else torch.zeros_like(S[:, 0]))[:, None], S[:, :-1]], 1)
    M = G * Lm * wc[..., None, :]
    CS = Cc @ Sin.transpose(-1, -2)
    y = unfold(M @ x + e[..., None] * CS) + D[:, None] * u.float()
    zf = z.float() if z is not None else None
    res = {"out": (y * _act(zf, True) if z is not None else y).to(dt), "last": S[:, -1].clone()}
    if case["kind"] != "train":
        return res
    do = s["dout"].float()
    if z is not None:
        res["dz"] = (do * y * _dact(zf)).to(dt)
        do = do * _act(zf, True)
    dy = fold(do)
    back = (dy * e[..., None]).transpose(-1, -2) @ Cc    # what each chunk adds to the adjoint of its entering state
    R = _scan(dec.flip(1), back.flip(1)).flip(1)         # adjoint of each chunk's entering state
    dS = torch.cat([R[:, 1:], torch.zeros_like(R[:, :1])], 1)
    H = dy @ x.transpose(-1, -2)
    GL, HL = G * Lm, H * Lm
    Sb = Bc @ dS.transpose(-1, -2)                       # (Q, P): dS B_s
    du = unfold((GL * wc[..., None, :]).transpose(-1, -2) @ dy + (end * wc)[..., None] * Sb) + D[:, None] * do
    HLw = HL * wc[..., None, :]
    dB = unfold(HLw.transpose(-1, -2) @ Cc + (end * wc)[..., None] * (x @ dS))
    dC = unfold(HLw @ Bc + e[..., None] * (dy @ Sin))
    pair = G * HL
    xs = end * (x * Sb).sum(-1)
    pw = pair * wc[..., None, :]
    dcum = pw.sum(-1) - pw.sum(-2) + e * (dy * CS).sum(-1) - xs * wc
    tail = (xs * wc).sum(-1) + (dec * dS * Sin).sum((-1, -2))
    dcum = torch.cat([dcum[..., :-1], dcum[..., -1:] + tail[..., None]], -1)
    dq = unfold(dcum.flip(-1).cumsum(-1).flip(-1)[..., None])[..., 0]
    dw = unfold((pair.sum(-2) + xs)[..., None])[..., 0]
    ddl = dq * A + dw * torch.exp(q)
    draw_ = ddl * _sigmoid(raw)
    # d w / d A = (q e^q - expm1(q)) / A^2, in 64 bits: the difference cancels near q = 0
    qd, Ad = q.double(), A.double()
    dA = (dq.double() * dl + dw.double() * (qd * torch.exp(qd) - torch.expm1(qd)) / Ad ** 2).sum((0, 1))
    res.update(du=du.to(dt), ddelta_raw=draw_.to(dt), dA=dA.float(),
               dB=dB.reshape(b, n, g, rep, ns).sum(3).to(dt), dC=dC.reshape(b, n, g, rep, ns).sum(3).to(dt),
               ddelta_bias=draw_.sum((0, 1), dtype=torch.float64).float(),
               dD=(do * u.float()).sum((0, 1, 3), dtype=torch.float64).float())
    if st is not None:
        res["dh0"] = R[:, 0].clone()
    return res


# ---------------------------------------------------------------- the definitions, token by token in 64 bits

def exact(case, seed):
    if case["length"] * case["batch"] > 200000 or (case["kind"] == "train" and case["length"] > 20000):
        return None
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()}
    if case["kind"] == "step":
        for k in ("u", "a_raw", "i_raw", "delta_raw", "B", "C", "z"):
            if d.get(k) is not None:
                d[k] = d[k].unsqueeze(1)
    r = {"conv": _exact_conv, "gated": _exact_gated, "heads": _exact_heads}[case["op"]](case, d)
    if case["kind"] == "step":
        return {"out": r["out"][:, 0], "state": r["last"]}
    return r


def _exact_conv(case, d):
    u, w, k = d["u"], d["weight"], case["taps"]
    b, n, c = u.shape
    win = d["state"] if d["state"] is not None else u.new_zeros(b, k - 1, c)
    x = torch.cat([win, u], 1)
    y = torch.einsum("blck,ck->blc", x.unfold(1, k, 1), w) + d["bias"]
    sg = torch.sigmoid(y)
    r = {"out": y * sg if case["silu"] else y, "last": x[:, x.shape[1] - (k - 1):]}
    if d["dout"] is not None:
        dy = d["dout"] * (sg + y * sg * (1 - sg)) if case["silu"] else d["dout"]
        dx = torch.zeros_like(x)
        for j in range(k):
            dx[:, j:j + n] += dy * w[:, j]
        r["du"], r["dbias"] = dx[:, k - 1:], dy.sum((0, 1))
        r["dweight"] = torch.einsum("blck,blc->ck", x.unfold(1, k, 1), dy)
        if d["state"] is not None:
            r["dstate0"] = dx[:, :k - 1]
    return r


def _exact_gated(case, d):
    u = d["u"]
    b, n, c = u.shape
    sp = torch.logaddexp(d["Lam"], torch.zeros_like(d["Lam"]))
    h = d["state"] if d["state"] is not None else u.new_zeros(b, c)
    h0, hs, cr = h, [], _RATE * sp
    la_all = -cr * torch.sigmoid(d["a_raw"] + d["a_bias"])
    b_all = torch.sqrt(-torch.expm1(2 * la_all)) * torch.sigmoid(d["i_raw"] + d["i_bias"]) * u
    a_all = torch.exp(la_all)
    for t in range(n):
        h = a_all[:, t] * h + b_all[:, t]
        hs.append(h)
    r = {"out": torch.stack(hs, 1), "last": h}
    if d["dout"] is not None:
        g = torch.zeros_like(h)
        du, da, di, dl = (torch.empty_like(u) for _ in range(4))
        for t in range(n - 1, -1, -1):
            g = g + d["dout"][:, t]
            rg, ig = torch.sigmoid(d["a_raw"][:, t] + d["a_bias"]), torch.sigmoid(d["i_raw"][:, t] + d["i_bias"])
            la = -cr * rg
            a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
            dla = g * a * (hs[t - 1] if t else h0) - g * ig * u[:, t] * a * a / m
            du[:, t], di[:, t] = g * m * ig, g * m * u[:, t] * ig * (1 - ig)
            da[:, t], dl[:, t] = -dla * cr * rg * (1 - rg), -dla * rg
            g = a * g
        r.update(du=du, da_raw=da, di_raw=di, da_bias=da.sum((0, 1)), di_bias=di.sum((0, 1)),
                 dLam=dl.sum((0, 1)) * _RATE * torch.sigmoid(d["Lam"]))
        if d["state"] is not None:
            r["dh0"] = g
    return r


def _exact_heads(case, d):
    u, B, C, A = d["u"], d["B"], d["C"], d["A"]
    b, n, h, p = u.shape
    ns, rep = case["dstate"], h // case["groups"]
    raw = d["delta_raw"] + d["delta_bias"]
    dl = torch.logaddexp(raw, torch.zeros_like(raw))
    ea, w = torch.exp(dl * A), torch.expm1(dl * A) / A
    S = d["state"] if d["state"] is not None else u.new_zeros(b, h, p, ns)

    def of(t, M):
        return M[:, t].repeat_interleave(rep, 1)[:, :, None]

    def step(t, S):
        return ea[:, t, :, None, None] * S + (w[:, t, :, None] * u[:, t])[..., None] * of(t, B)

    ys, kept, seg = [], [], 64
    for t in range(n):
        if t % seg == 0:
            kept.append(S if d["dout"] is not None else None)
        S = step(t, S)
        ys.append((S * of(t, C)).sum(-1) + d["D_skip"][:, None] * u[:, t])
    y = torch.stack(ys, 1)
    sg = torch.sigmoid(d["z"]) if d["z"] is not None else None
    r = {"out": y * d["z"] * sg if sg is not None else y, "last": S}
    if d["dout"] is None:
        return r
    do = d["dout"]
    if sg is not None:
        r["dz"] = do * y * (sg + d["z"] * sg * (1 - sg))
        do = do * d["z"] * sg
    g = torch.zeros_like(kept[0])
    du, dB, dC = torch.empty_like(u), torch.empty_like(B), torch.empty_like(C)
    dq, dw = torch.empty_like(raw), torch.empty_like(raw)
    for k in range(len(kept) - 1, -1, -1):
        t0, t1 = k * seg, min(n, (k + 1) * seg)
        hist = [kept[k]]
        for t in range(t0, t1):
            hist.append(step(t, hist[-1]))
        for t in range(t1 - 1, t0 - 1, -1):
            g = g + do[:, t][..., None] * of(t, C)
            dC[:, t] = (do[:, t][..., None] * hist[t - t0 + 1]).sum(2).view(b, -1, rep, ns).sum(2)
            gB, gx = (g * of(t, B)).sum(-1), (g * u[:, t][..., None]).sum(2)
            du[:, t] = w[:, t, :, None] * gB + d["D_skip"][:, None] * do[:, t]
            dB[:, t] = (w[:, t, :, None] * gx).view(b, -1, rep, ns).sum(2)
            dw[:, t] = (gB * u[:, t]).sum(-1)
            g = ea[:, t, :, None, None] * g
            dq[:, t] = (g * hist[t - t0]).sum((-1, -2))
    q = dl * A
    ddr = (dq * A + dw * torch.exp(q)) * torch.sigmoid(raw)
    r.update(du=du, dB=dB, dC=dC, ddelta_raw=ddr, ddelta_bias=ddr.sum((0, 1)),
             dA=(dq * dl + dw * (q * torch.exp(q) - torch.expm1(q)) / A ** 2).sum((0, 1)),
             dD=(do * u).sum((0, 1, 3)))
    if d["state"] is not None:
        r["dh0"] = g
    return r
