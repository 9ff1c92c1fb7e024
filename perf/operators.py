"""Cases and plain forms of the operators around the recurrent token mixers: rotary positions on
the queries and keys, the short causal convolution, the selective state space scan, and group
normalisation with an activation.

`run(state)` makes one pass of an operator: in its plain form (elementary torch operations) while
`own` is False, through the library's entry points while it is True.  `exact(case, seed)` gives
the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------- the cases --

def listed():
    return [
        # one new token of 64 requests at their own positions in long contexts: latency
        dict(name="rotary_decode", op="rotary", dtype="bf16", B=64, H=32, Hk=8, T=1, D=128, R=128, layout="half",
             positions="batch", span=131072, scaling="linear", back=False),
        # a prompt at the retention benchmark's head layout, queries and fewer shared keys
        dict(name="rotary_prompt", op="rotary", dtype="bf16", B=4, H=32, Hk=8, T=8192, D=128, R=128, layout="half",
             positions="start", span=4096, scaling="none", back=False),
        # the gradient, an odd length, half of the head rotated in neighbouring pairs
        dict(name="rotary_grad_odd", op="rotary", dtype="f16", B=8, H=16, Hk=16, T=1023, D=64, R=32,
             layout="interleaved", positions="batch", span=65536, scaling="ntk", back=True),
        # one new token of 64 requests through the convolution: latency
        dict(name="conv_step", op="conv_step", dtype="bf16", B=64, C=4096, W=4, bias=True, silu=True),
        # ragged prompts in one padded batch, an odd width that no vector load fits
        dict(name="conv_ragged", op="conv", dtype="f16", B=6, T=1501, C=1111, W=3, bias=True, silu=True, ragged=True,
             carried=True),
        # a training step's convolution gradient
        dict(name="conv_grad", op="conv_bwd", dtype="bf16", B=8, T=4096, C=2048, W=4, bias=True, silu=True,
             ragged=False, carried=False),
        # one new token of 64 requests through the scan: bound by its state's traffic
        dict(name="scan_step", op="scan_step", dtype="bf16", B=64, C=4096, G=1, N=16, gate=True),
        # a batch of prompts
        dict(name="scan_prompt", op="scan", dtype="bf16", B=8, T=4096, C=2048, G=1, N=16, gate=True, ragged=False,
             carried=False),
        # one long prompt, continued from a state, with few channels: the length has to be split
        dict(name="scan_long", op="scan", dtype="f16", B=1, T=16000, C=1000, G=2, N=16, gate=True, ragged=False,
             carried=True),
        # a training step's scan gradient
        dict(name="scan_grad", op="scan_bwd", dtype="bf16", B=4, T=2048, C=2048, G=1, N=16, gate=True, ragged=False,
             carried=False),
        # a 256 x 256 grid with 640 channels, normalised in 32 groups ahead of vision attention
        dict(name="norm_grid", op="norm", dtype="f16", B=2, T=65536, C=640, G=32, silu=True, affine=True),
        # the gradient of an odd grid in fp32
        dict(name="norm_grad_odd", op="norm_bwd", dtype="f32", B=3, T=4087, C=330, G=30, silu=True, affine=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "conv", "conv_bwd", "conv_step", "scan", "scan", "scan_bwd", "scan_bwd",
                     "scan_step", "norm", "norm", "norm_bwd"])
    c = dict(op=op, dtype=rng.choice(["f32", "f16", "bf16"]))
    if op == "rotary":
        c["D"] = rng.choice([32, 64, 80, 96, 128, 192, 256, 2 * rng.randint(8, 128)])
        c["R"] = rng.choice([c["D"], 2 * rng.randint(1, c["D"] // 2)])
        c["Hk"] = _log(rng, 1, 32)
        c["H"] = c["Hk"] * rng.choice([1, 2, 4])
        c["T"] = rng.choice([1, _log(rng, 2, 8192)])
        most = max(1, (1 << 27) // ((c["H"] + c["Hk"]) * c["T"] * c["D"]))
        c["B"] = _log(rng, 1, min(128, most))
        c.update(layout=rng.choice(["half", "interleaved"]), positions=rng.choice(["start", "shared", "batch"]),
                 span=_log(rng, 16, 1000000), scaling=rng.choice(["none", "linear", "ntk"]),
                 back=rng.random() < 0.4)
        return c
    if op in ("norm", "norm_bwd"):
        c["G"] = rng.choice([1, 2, 8, 16, 30, 32, 32])
        c["C"] = c["G"] * _log(rng, 2, 4096 // c["G"])
        c["T"] = rng.choice([1, _log(rng, 2, 65536)])
        most = max(1, (1 << 25) // (c["C"] * c["T"]))
        c["B"] = _log(rng, 1, min(8192 if c["T"] == 1 else 64, most))
        c.update(silu=rng.random() < 0.7, affine=rng.random() < 0.85)
        return c
    c["C"] = rng.choice([64, 256, 1024, 1536, 2048, _log(rng, 8, 4096)])
    if op in ("conv", "conv_bwd", "conv_step"):
        c.update(W=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.7, silu=rng.random() < 0.7)
    else:
        c["G"] = rng.choice([g for g in (1, 1, 1, 2, 4) if c["C"] % g == 0])
        c["N"] = rng.choice([16, 16, 16, 8, 32, rng.randint(1, 64)])
        c["gate"] = rng.random() < 0.6
    if op in ("conv_step", "scan_step"):
        c["B"] = _log(rng, 1, 128)
        return c
    c["T"] = _log(rng, 1, 8192)
    per = c["C"] * c["T"] * (c["N"] if "N" in c else 8)
    most = max(1, (1 << (29 if op == "scan" else 28)) // per)
    while most == 1 and c["C"] * c["T"] * c.get("N", 8) > (1 << 28):
        c["T"] //= 2
    c["B"] = _log(rng, 1, min(16, most))
    c.update(ragged=rng.random() < 0.3, carried=rng.random() < 0.4)
    return c


# ------------------------------------------------------------------------------ the inputs --

def _inputs(case, seed):
    """What a program holds before the call, without the output buffers."""
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    dt = DTYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = {}
    B = case["B"]
    if op == "rotary":
        H, Hk, T, D, R = (case[n] for n in ("H", "Hk", "T", "D", "R"))
        # queries and keys (the gradients of the rotated ones, for the backward)
        s["q"], s["k"] = normal(B, H, T, D), normal(B, Hk, T, D)
        i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
        base = 10000.0 * (8.0 ** (R / (R - 2.0)) if case["scaling"] == "ntk" and R > 2 else 1.0)
        f = base ** (-2.0 * i / R)
        s["freqs"] = (f / 8.0 if case["scaling"] == "linear" else f).float()
        s["magnitude"] = 1.0 if case["scaling"] == "none" else 1.125
        s["start"], s["positions"] = 0, None
        off = torch.randint(0, case["span"], (B, 1), generator=g, device="cuda")
        steps = torch.arange(T, device="cuda")
        if case["positions"] == "batch":
            s["positions"] = (off + steps).contiguous()
        elif case["positions"] == "shared":
            s["positions"] = (off[0] + 3 * steps).contiguous()
        else:
            s["start"] = case["span"]
        return s
    C = case["C"]
    if op in ("norm", "norm_bwd"):
        T, G = case["T"], case["G"]
        # activations with a mean and a spread of their own in every channel
        x = torch.randn((B, T, C), generator=g, device="cuda")
        s["x"] = (x * uniform(C, lo=0.5, hi=2.0) + normal(C, dtype=torch.float32)).to(dt)
        s["gamma"] = 1 + normal(C, scale=0.2, dtype=torch.float32) if case["affine"] else None
        s["beta"] = normal(C, scale=0.2, dtype=torch.float32) if case["affine"] else None
        if op == "norm_bwd":
            s["dy"] = normal(B, T, C)
            # the statistics that the forward pass handed out
            xg = s["x"].double().view(B, T, G, C // G)
            m = xg.mean((1, 3))
            v = (xg - m[:, None, :, None]).square().mean((1, 3))
            s["mean"], s["rstd"] = m.float(), (v + 1e-5).rsqrt().float()
        return s
    T = 1 if op.endswith("_step") else case["T"]
    tail = () if op.endswith("_step") else (T,)
    s["lengths"] = None
    if case.get("ragged"):
        n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = T
        s["lengths"] = n
    if op.startswith("conv"):
        W = case["W"]
        s["x"] = normal(B, *tail, C)
        s["w"] = uniform(C, W, lo=-1, hi=1) * W ** -0.5
        s["bias"] = uniform(C, lo=-0.5, hi=0.5) if case["bias"] else None
        s["state_in"] = normal(B, W - 1, C) if case.get("carried", True) else None
        if op == "conv_bwd":
            s["dy"] = normal(B, T, C)
            s["dstate_in"] = normal(B, W - 1, C) if case["carried"] else None
        return s
    G, N = case["G"], case["N"]
    s["x"] = normal(B, *tail, C)
    s["Bm"], s["Cm"] = normal(B, *tail, G, N), normal(B, *tail, G, N)
    # rates -1 .. -N with a spread, steps between 1e-3 and 1e-1 after the softplus
    s["A"] = -(torch.arange(1, N + 1, device="cuda") * uniform(C, N, lo=0.7, hi=1.4)).contiguous()
    step = torch.exp(uniform(C, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["dt"] = normal(B, *tail, C, scale=0.5)
    s["D"] = uniform(C, lo=0.5, hi=1.5)
    s["z"] = normal(B, *tail, C) if case["gate"] else None
    s["state_in"] = normal(B, C, N, dtype=torch.float32) if case.get("carried", True) else None
    if op == "scan_bwd":
        s["dy"] = normal(B, T, C)
        s["dstate_in"] = normal(B, C, N, dtype=torch.float32) if case["carried"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    e = torch.empty_like
    # the buffers that a program hands to the calls
    if op == "rotary":
        s["oq"], s["ok"] = e(s["q"]), e(s["k"])
    elif op == "norm":
        s["y"] = e(s["x"])
        s["mean"] = torch.empty((case["B"], case["G"]), device="cuda")
        s["rstd"] = e(s["mean"])
    elif op == "norm_bwd":
        s["dx"] = e(s["x"])
        s["dgamma"] = None if s["gamma"] is None else e(s["gamma"])
        s["dbeta"] = None if s["beta"] is None else e(s["beta"])
    elif op.startswith("conv"):
        if op == "conv_bwd":
            s["dx"], s["dw"] = e(s["x"]), e(s["w"])
            s["dbias"] = None if s["bias"] is None else e(s["bias"])
            s["dstate_out"] = None if s["state_in"] is None else e(s["state_in"])
        else:
            s["y"] = e(s["x"])
            s["state_out"] = torch.empty((case["B"], case["W"] - 1, case["C"]), dtype=s["x"].dtype, device="cuda")
    elif op == "scan_bwd":
        for n in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias"):
            s["d" + n] = e(s[n])
        s["dz"] = None if s["z"] is None else e(s["z"])
        s["dstate_out"] = None if s["state_in"] is None else e(s["state_in"])
    else:
        s["y"] = e(s["x"])
        s["state_out"] = torch.empty((case["B"], case["C"], case["N"]), device="cuda")
    s["case"] = case
    return s


# -------------------------------------------------------------------------- the plain forms --

def _f(t):
    return None if t is None else t.float()


def _sigmoid(t):
    return 1 / (1 + torch.exp(-t))


def _plain_rotary(s):
    c = s["case"]
    B, T, R, D = c["B"], c["T"], c["R"], c["D"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(s["start"], s["start"] + T, device="cuda")
    if pos.dim() == 1:
        pos = pos[None]
    # far positions: the angle in 64 bits
    ang = pos.double()[..., None] * s["freqs"].double()
    if c["back"]:
        ang = -ang
    cos = (torch.cos(ang) * s["magnitude"]).float()[:, None]
    sin = (torch.sin(ang) * s["magnitude"]).float()[:, None]
    out = []
    for t in (s["q"], s["k"]):
        x = t.float()
        y = x.clone()
        if c["layout"] == "half":
            a, b = x[..., :R // 2], x[..., R // 2:R]
            y[..., :R // 2] = a * cos - b * sin
            y[..., R // 2:R] = a * sin + b * cos
        else:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y[..., 0:R:2] = a * cos - b * sin
            y[..., 1:R:2] = a * sin + b * cos
        out.append(y.to(t.dtype))
    return out


def _valid(lengths, T):
    """[B, T, 1]: 1 for the tokens of each sequence, 0 behind them."""
    return (torch.arange(T, device="cuda")[None] < lengths[:, None]).float()[..., None]


def _extended(s, T):
    """The state's rows and the sequence's, tokens behind its end as zeros: [B, W - 1 + T, C]."""
    c = s["case"]
    x = s["x"].float().view(c["B"], T, c["C"])
    if s["lengths"] is not None:
        x = torch.where(_valid(s["lengths"], T) > 0, x, torch.zeros_like(x))
    st = s["state_in"]
    st = x.new_zeros(c["B"], c["W"] - 1, c["C"]) if st is None else st.float()
    return torch.cat([st, x], 1)


def _tail_rows(s, T):
    """Row numbers in the extended sequence of the state after the last token: [B, W - 1, C]."""
    c = s["case"]
    n = torch.full((c["B"],), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    rows = n[:, None] + torch.arange(c["W"] - 1, device="cuda")
    return rows[..., None].expand(c["B"], c["W"] - 1, c["C"])


def _plain_conv(s):
    c = s["case"]
    T = 1 if c["op"] == "conv_step" else c["T"]
    e = _extended(s, T)
    a = s["bias"] if s["bias"] is not None else torch.zeros(c["C"], device="cuda")
    for j in range(c["W"]):
        a = a + s["w"][:, j] * e[:, j:j + T]
    y = a * _sigmoid(a) if c["silu"] else a
    if s["lengths"] is not None:
        y = y * _valid(s["lengths"], T)
    st = torch.gather(e, 1, _tail_rows(s, T))
    return [y.view(s["x"].shape).to(s["x"].dtype), st.to(s["x"].dtype)]


def _plain_conv_bwd(s):
    c = s["case"]
    T, W = c["T"], c["W"]
    e = _extended(s, T)
    g = s["dy"].float()
    if c["silu"]:
        a = s["bias"] if s["bias"] is not None else torch.zeros(c["C"], device="cuda")
        for j in range(W):
            a = a + s["w"][:, j] * e[:, j:j + T]
        sg = _sigmoid(a)
        g = g * sg * (1 + a * (1 - sg))
    if s["lengths"] is not None:
        v = _valid(s["lengths"], T)
        g = torch.where(v > 0, g, torch.zeros_like(g))
    de = torch.zeros_like(e)
    for j in range(W):
        de[:, j:j + T] += s["w"][:, j] * g
    if s["dstate_in"] is not None:
        de.scatter_add_(1, _tail_rows(s, T), s["dstate_in"].float())
    dx = de[:, W - 1:]
    if s["lengths"] is not None:
        dx = torch.where(v > 0, dx, torch.zeros_like(dx))
    out = [dx.to(s["x"].dtype), torch.stack([(e[:, j:j + T] * g).sum((0, 1)) for j in range(W)], 1)]
    if s["bias"] is not None:
        out.append(g.sum((0, 1)))
    if s["state_in"] is not None:
        out.append(de[:, :W - 1].to(s["x"].dtype))
    return out


def _recurrence(a, u, first):
    """h_t = a_t h_{t-1} + u_t along dim 1 from h_{-1} = first (or 0): neighbouring spans joined, twice
    as long each time, in log2(T) passes over the whole tensors."""
    h, a, d = u.clone(), a.clone(), 1
    if first is not None:
        h[:, 0] += a[:, 0] * first
    while d < u.shape[1]:
        h0, a0 = h, a
        h = h0.clone()
        h[:, d:].addcmul_(a0[:, d:], h0[:, :-d])
        if 2 * d < u.shape[1]:
            a = a0.clone()
            a[:, d:] *= a0[:, :-d]
        d *= 2
    return h


def _plain_scan_parts(s, T):
    """The steps, the decays and the inputs of the recurrence, and the states after every token."""
    c = s["case"]
    B, C, G, N = c["B"], c["C"], c["G"], c["N"]
    x = s["x"].float().view(B, T, C)
    raw = s["dt"].float().view(B, T, C) + s["dt_bias"]
    # log(1 + e^r) = max(r, 0) + log1p(e^-|r|)
    step = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    if s["lengths"] is not None:
        step = step * _valid(s["lengths"], T)
    Bm = s["Bm"].float().view(B, T, G, 1, N)
    a = torch.exp(step[..., None] * s["A"])
    u = ((step * x).view(B, T, G, C // G, 1) * Bm).view(B, T, C, N)
    h = _recurrence(a, u, s["state_in"])
    return x, raw, step, a, u, h, h[:, -1]


def _plain_scan(s):
    c = s["case"]
    T = 1 if c["op"] == "scan_step" else c["T"]
    B, C, G, N = c["B"], c["C"], c["G"], c["N"]
    x, _, _, _, _, h, last = _plain_scan_parts(s, T)
    Cm = s["Cm"].float().view(B, T, G, 1, N)
    y = (h.view(B, T, G, C // G, N) * Cm).sum(-1).view(B, T, C) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float().view(B, T, C)
        y = y * z * _sigmoid(z)
    if s["lengths"] is not None:
        y = torch.where(_valid(s["lengths"], T) > 0, y, torch.zeros_like(y))
    return [y.view(s["x"].shape).to(s["x"].dtype), last.clone()]


def _plain_scan_bwd(s):
    c = s["case"]
    B, T, C, G, N = c["B"], c["T"], c["C"], c["G"], c["N"]
    x, raw, step, a, u, h, _ = _plain_scan_parts(s, T)
    Bm, Cm = s["Bm"].float().view(B, T, G, 1, N), s["Cm"].float().view(B, T, G, 1, N)
    hg = h.view(B, T, G, C // G, N)
    dy = s["dy"].float()
    if s["lengths"] is not None:
        dy = torch.where(_valid(s["lengths"], T) > 0, dy, torch.zeros_like(dy))
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sg = _sigmoid(z)
        y = (hg * Cm).sum(-1).view(B, T, C) + s["D"] * x
        out["dz"] = dy * y * sg * (1 + z * (1 - sg))
        dy = dy * z * sg
    dyg = dy.view(B, T, G, C // G, 1)
    out["dCm"] = (hg * dyg).sum(3)
    # lam_t = dy_t C_t + a_{t+1} lam_{t+1}, the gradient of the state after token t
    back = torch.ones_like(a)
    back[:, 1:] = a[:, 1:].flip(1)
    lam = _recurrence(back, (dyg * Cm).view(B, T, C, N).flip(1), s["dstate_in"]).flip(1)
    carry = a[:, 0] * lam[:, 0]
    lamg = lam.view(B, T, G, C // G, N)
    lb = (lamg * Bm).sum(-1).view(B, T, C)
    out["dBm"] = (lamg * (step * x).view(B, T, G, C // G, 1)).sum(3)
    out["dx"] = step * lb + dy * s["D"]
    out["dD"] = (dy * x).sum((0, 1))
    h -= u                                                     # a_t h_{t-1}
    h *= lam
    out["dA"] = (h * step[..., None]).sum((0, 1))
    h *= s["A"]
    ds = h.sum(-1) + x * lb
    ddt = ds * _sigmoid(raw)
    if s["lengths"] is not None:
        ddt = ddt * _valid(s["lengths"], T)
    out["ddt"] = ddt
    out["ddt_bias"] = ddt.sum((0, 1))
    names = ["dx", "ddt", "dA", "dBm", "dCm", "dD", "ddt_bias"] + (["dz"] if s["z"] is not None else [])
    r = [out[n].to(s[n[1:]].dtype) for n in names]
    if s["state_in"] is not None:
        r.append(carry)
    return r


def _plain_norm(s):
    c = s["case"]
    B, T, C, G = c["B"], c["T"], c["C"], c["G"]
    x = s["x"].float().view(B, T, G, C // G)
    m = x.mean((1, 3))
    d = x - m[:, None, :, None]
    r = 1 / torch.sqrt(d.square().mean((1, 3)) + 1e-5)
    a = (d * r[:, None, :, None]).view(B, T, C)
    if c["affine"]:
        a = a * s["gamma"] + s["beta"]
    y = a * _sigmoid(a) if c["silu"] else a
    return [y.to(s["x"].dtype), m, r]


def _plain_norm_bwd(s):
    c = s["case"]
    B, T, C, G = c["B"], c["T"], c["C"], c["G"]
    r = s["rstd"][:, None, :, None]
    xh = ((s["x"].float().view(B, T, G, C // G) - s["mean"][:, None, :, None]) * r).view(B, T, C)
    g = s["dy"].float()
    if c["silu"]:
        a = xh * s["gamma"] + s["beta"] if c["affine"] else xh
        sg = _sigmoid(a)
        g = g * sg * (1 + a * (1 - sg))
    out = []
    if c["affine"]:
        out = [(g * xh).sum((0, 1)), g.sum((0, 1))]
        g = g * s["gamma"]
    gg, xg = g.view(B, T, G, C // G), xh.view(B, T, G, C // G)
    m0 = gg.mean((1, 3), keepdim=True)
    m1 = (gg * xg).mean((1, 3), keepdim=True)
    dx = (r * (gg - m0 - xg * m1)).view(B, T, C)
    return [dx.to(s["x"].dtype)] + out


_PLAIN = {"rotary": _plain_rotary, "conv": _plain_conv, "conv_step": _plain_conv, "conv_bwd": _plain_conv_bwd,
          "scan": _plain_scan, "scan_step": _plain_scan, "scan_bwd": _plain_scan_bwd, "norm": _plain_norm,
          "norm_bwd": _plain_norm_bwd}


# ------------------------------------------------------------------------- the library's calls --

def _own(s):
    import linear_attention_attn_b200 as la
    c = s["case"]
    op = c["op"]
    act = "silu" if c.get("silu") else "none"
    if op == "rotary":
        f = la.la_rotary_bwd if c["back"] else la.la_rotary_fwd
        f(s["q"], s["k"], s["oq"], s["ok"], s["freqs"], positions=s["positions"], start=s["start"],
          layout=c["layout"], magnitude=s["magnitude"])
        return [s["oq"], s["ok"]]
    if op == "conv":
        la.la_short_conv_fwd(s["x"], s["w"], s["y"], bias=s["bias"], state_in=s["state_in"], state_out=s["state_out"],
                             lengths=s["lengths"], activation=act)
        return [s["y"], s["state_out"]]
    if op == "conv_step":
        la.la_short_conv_step(s["x"], s["w"], s["y"], s["state_in"], s["state_out"], bias=s["bias"], activation=act)
        return [s["y"], s["state_out"]]
    if op == "conv_bwd":
        la.la_short_conv_bwd(s["x"], s["w"], s["dy"], s["dx"], s["dw"], bias=s["bias"], dbias=s["dbias"],
                             state_in=s["state_in"], dstate_in=s["dstate_in"], dstate_out=s["dstate_out"],
                             lengths=s["lengths"], activation=act)
        return [s[n] for n in ("dx", "dw", "dbias", "dstate_out") if s[n] is not None]
    if op == "scan":
        la.la_selective_scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["y"], D=s["D"], z=s["z"],
                                 dt_bias=s["dt_bias"], state_in=s["state_in"], state_out=s["state_out"],
                                 lengths=s["lengths"])
        return [s["y"], s["state_out"]]
    if op == "scan_step":
        la.la_selective_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["y"], s["state_in"], s["state_out"],
                                  D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        return [s["y"], s["state_out"]]
    if op == "scan_bwd":
        la.la_selective_scan_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], s["dx"], s["ddt"], s["dA"],
                                 s["dBm"], s["dCm"], D=s["D"], dD=s["dD"], z=s["z"], dz=s["dz"],
                                 dt_bias=s["dt_bias"], ddt_bias=s["ddt_bias"], state_in=s["state_in"],
                                 dstate_in=s["dstate_in"], dstate_out=s["dstate_out"], lengths=s["lengths"])
        names = ("dx", "ddt", "dA", "dBm", "dCm", "dD", "ddt_bias", "dz", "dstate_out")
        return [s[n] for n in names if s[n] is not None]
    if op == "norm":
        la.la_group_norm_fwd(s["x"], s["y"], c["G"], gamma=s["gamma"], beta=s["beta"], eps=1e-5, activation=act,
                             mean=s["mean"], rstd=s["rstd"])
        return [s["y"], s["mean"], s["rstd"]]
    la.la_group_norm_bwd(s["x"], s["dy"], s["dx"], c["G"], s["mean"], s["rstd"], gamma=s["gamma"], beta=s["beta"],
                         dgamma=s["dgamma"], dbeta=s["dbeta"], activation=act)
    return [s[n] for n in ("dx", "dgamma", "dbeta") if s[n] is not None]


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- the definitions in 64 bits --

def _exact_rotary(c, s):
    T, R = c["T"], c["R"]
    pos = s["positions"]
    pos = torch.arange(T, device="cuda") + s["start"] if pos is None else pos
    ang = pos.double().reshape(-1, 1, T, 1) * s["freqs"].double()
    turn = torch.polar(torch.full_like(ang, s["magnitude"]), -ang if c["back"] else ang)
    out = []
    for t in (s["q"], s["k"]):
        r, keep = t[..., :R].double(), t[..., R:].double()
        # pairs (a, b) as complex numbers a + i b, turned by the angle
        pairs = r.unflatten(-1, (2, R // 2)).transpose(-1, -2) if c["layout"] == "half" else r.unflatten(-1, (R // 2, 2))
        p = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        p = p.transpose(-1, -2) if c["layout"] == "half" else p
        out.append(torch.cat([p.flatten(-2), keep], -1))
    return out


def _silu64(a):
    return a * torch.special.expit(a)


def _ends(s, B, T):
    return [T] * B if s["lengths"] is None else s["lengths"].tolist()


def _exact_conv(c, s, x, w, bias, state):
    """Each sequence by itself: the windows of its own rows, then the state after them."""
    B, W, C = c["B"], c["W"], c["C"]
    T = 1 if c["op"] == "conv_step" else c["T"]
    x = x.reshape(B, T, C)
    ys, sts = [], []
    for b, n in enumerate(_ends(s, B, T)):
        first = x.new_zeros(W - 1, C) if state is None else state[b]
        e = torch.cat([first, x[b, :n]])
        a = e.unfold(0, W, 1) if n else e.new_zeros(0, C, W)
        a = (a * w).sum(-1) + (0 if bias is None else bias)
        y = _silu64(a) if c["silu"] else a
        ys.append(torch.cat([y, y.new_zeros(T - n, C)]))
        sts.append(e[n:])
    return torch.stack(ys), torch.stack(sts)


def _exact_scan(c, s, p):
    """One token after the other."""
    B, C, G, N = c["B"], c["C"], c["G"], c["N"]
    T = 1 if c["op"] == "scan_step" else c["T"]
    x, raw = p["x"].reshape(B, T, C), p["dt"].reshape(B, T, C) + p["dt_bias"]
    Bm, Cm = p["Bm"].reshape(B, T, G, N), p["Cm"].reshape(B, T, G, N)
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    ends = torch.tensor(_ends(s, B, T), device="cuda")
    h = x.new_zeros(B, C, N) if p["state_in"] is None else p["state_in"]
    gate = [None] * T if p["z"] is None else _silu64(p["z"].reshape(B, T, C)).unbind(1)
    ys = []
    for t, (xt, d, bt, ct, zt) in enumerate(zip(x.unbind(1), step.unbind(1), Bm.unbind(1), Cm.unbind(1), gate)):
        live = (ends > t).view(B, 1)
        b = bt.repeat_interleave(C // G, 1)
        new = torch.exp(d[..., None] * p["A"]) * h + b * (d * xt)[..., None]
        h = new if s["lengths"] is None else torch.where(live[..., None], new, h)
        y = torch.einsum("bgcn,bgn->bgc", h.view(B, G, C // G, N), ct).reshape(B, C) + p["D"] * xt
        if zt is not None:
            y = y * zt
        ys.append(y if s["lengths"] is None else torch.where(live, y, torch.zeros_like(y)))
    return torch.stack(ys, 1), h


def _exact_norm(c, x, gamma, beta):
    B, T, C, G = c["B"], c["T"], c["C"], c["G"]
    rows = x.view(B, T, G, C // G).transpose(1, 2).reshape(B, G, -1)
    var, mean = torch.var_mean(rows, -1, correction=0)
    n = (rows - mean[..., None]) / torch.sqrt(var + 1e-5)[..., None]
    y = n.view(B, G, T, C // G).transpose(1, 2).reshape(B, T, C)
    if gamma is not None:
        y = y * gamma + beta
    return (_silu64(y) if c["silu"] else y), mean, 1 / torch.sqrt(var + 1e-5)


def _leaf(t):
    return None if t is None else t.double().clone().requires_grad_()


def exact(case, seed):
    c, op = case, case["op"]
    s = _inputs(case, seed)

    def d(n):
        return None if s[n] is None else s[n].double()
    if op == "rotary":
        return _exact_rotary(c, s)
    if op in ("conv", "conv_step"):
        y, st = _exact_conv(c, s, d("x"), d("w"), d("bias"), d("state_in"))
        return [y.view(s["x"].shape), st]
    if op == "norm":
        return list(_exact_norm(c, d("x"), d("gamma"), d("beta")))
    scan = ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "z", "state_in")
    if op in ("scan", "scan_step"):
        with torch.no_grad():
            y, h = _exact_scan(c, s, {n: d(n) for n in scan})
        return [y.view(s["x"].shape), h]
    # the gradients: by automatic differentiation of the definitions
    if op == "conv_bwd":
        p = {n: _leaf(s[n]) for n in ("x", "w", "bias", "state_in")}
        y, st = _exact_conv(c, s, p["x"], p["w"], p["bias"], p["state_in"])
        seeds = [d("dy")]
        outs = [y]
    elif op == "scan_bwd":
        # every token keeps some tensors of the state's size in 64 bits for the way back
        if 8 * 8 * c["B"] * c["T"] * c["C"] * c["N"] > 60e9 or c["T"] > 8192:
            return None
        p = {n: _leaf(s[n]) for n in scan}
        y, st = _exact_scan(c, s, p)
        seeds, outs = [d("dy")], [y]
    else:
        p = {n: _leaf(s[n]) for n in ("x", "gamma", "beta")}
        st = None
        seeds, outs = [d("dy")], [_exact_norm(c, p["x"], p["gamma"], p["beta"])[0]]
    if s.get("dstate_in") is not None:
        seeds.append(d("dstate_in"))
        outs.append(st)
    leaves = [p[n] for n in p if p[n] is not None]
    return list(torch.autograd.grad(outs, leaves, seeds))


# --------------------------------------------------------------------------------- the work --

def work(case):
    c, op = case, case["op"]
    es = 4 if c["dtype"] == "f32" else 2
    B = c["B"]
    if op == "rotary":
        n = B * (c["H"] + c["Hk"]) * c["T"]
        # every element in and out; two products and two sums (a pair: four and two) on the rotated part
        return {"bytes": 2 * es * n * c["D"], "flops": 3 * n * c["R"]}
    C = c["C"]
    if op in ("norm", "norm_bwd"):
        n = B * c["T"] * C
        par = 8 * C if c["affine"] else 0
        stats = 8 * B * c["G"]
        if op == "norm":
            return {"bytes": 2 * es * n + par + stats, "flops": (10 if c["silu"] else 5) * n}
        return {"bytes": 3 * es * n + 2 * par + stats, "flops": (22 if c["silu"] else 13) * n}
    T = 1 if op.endswith("_step") else c["T"]
    n = B * T * C
    if op.startswith("conv"):
        W = c["W"]
        st = B * (W - 1) * C * es
        par = 4 * C * (W + (1 if c["bias"] else 0))
        extra = 5 if c["silu"] else 0
        if op == "conv_bwd":
            return {"bytes": 3 * es * n + 2 * par + (3 * st if c["carried"] else 0),
                    "flops": n * (4 * W + (2 * W + 10 if c["silu"] else 0))}
        return {"bytes": 2 * es * n + par + st * (2 if c.get("carried", True) else 1), "flops": n * (2 * W + extra)}
    G, N = c["G"], c["N"]
    bc = 2 * B * T * G * N * es
    st = 4 * B * C * N
    par = 4 * C * (N + 2)
    gate = 1 if c["gate"] else 0
    if op == "scan_bwd":
        # x, dt, dy (z) in, dx, ddt (dz) out; an exponential, the state again, and its gradient's terms
        return {"bytes": (5 + 2 * gate) * es * n + 2 * bc + 2 * par + (3 * st if c["carried"] else 0),
                "flops": 20 * n * N}
    # an exponential, three products, two sums for each state and token
    return {"bytes": (3 + gate) * es * n + bc + par + st * (2 if c.get("carried", True) else 1),
            "flops": 6 * n * N}
