"""Parity of rotary positions, the short convolution, the selective scan and group normalisation with
their 64-bit definitions: types, layouts, odd sizes, padded batches, carried states, empty sequences.

Bounds: half a step of the storage type for the rounding of the result, plus counted fp32 roundings
(2^-24 each) of the sum of the magnitudes that meet in a result (tests/mixer_ref.close)."""
import math

import pytest
import torch

import linear_attention_attn_b200 as la
from tests import mixer_ref as ref
from tests.mixer_ref import DTYPES, close

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _dev():
    return torch.device("cuda", 0)


def _gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=_dev()) * scale).to(dtype)
    return normal


def _leaves(*ts):
    return [None if t is None else t.double().requires_grad_() for t in ts]


def _lengths(T, B):
    """Lengths of a padded batch: full, empty, one, outside the range on both sides."""
    vals = [T, 0, 1, T + 7, -2, T // 2 + 1][:B]
    return torch.tensor(vals + [max(1, T - 1)] * (B - len(vals)), dtype=torch.int32, device=_dev())


def _pad_nan(t, lengths):
    """The tensor with NaN behind every sequence's end, and with zeros there."""
    n = torch.tensor(ref.ends(lengths, t.shape[0], t.shape[1]), device=t.device)
    live = (torch.arange(t.shape[1], device=t.device)[None] < n[:, None]).view(t.shape[:2] + (1,) * (t.dim() - 2))
    return torch.where(live, t, torch.full_like(t, NAN)), torch.where(live, t, torch.zeros_like(t))


def _empties(*ts):
    """Result buffers holding NaN, so that what is not written shows."""
    return [torch.full_like(t, NAN) for t in ts]


# ---------------------------------------------------------------------------------- rotary --

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,H,Hk,T,D,R", [(2, 4, 2, 37, 64, 64), (3, 3, 1, 1, 128, 64), (1, 2, 2, 5, 66, 26),
                                          (2, 1, 3, 9, 7, 2), (1, 8, 8, 300, 80, 80), (64, 32, 8, 1, 128, 128)])
def test_rotary(dtype, layout, B, H, Hk, T, D, R):
    normal = _gen(1)
    q, k = normal(B, H, T, D, dtype=DTYPES[dtype]), normal(B, Hk, T, D, dtype=DTYPES[dtype])
    freqs = la.la_rotary_frequencies(R).to(_dev())
    pos = torch.randint(-50, 2 ** 31, (B, T), device=_dev())
    oq, ok = _empties(q, k)
    la.la_rotary_fwd(q, k, oq, ok, freqs, positions=pos, layout=layout, magnitude=1.25)
    for name, x, y in (("q", q, oq), ("k", k, ok)):
        want = ref.rotary(x.double(), pos.double(), freqs.double(), layout, 1.25)
        # the angle is off by pi 2^-24 (3.2 roundings) plus the sine's own 2, two products, a sum
        close(y, want, name, 12, 2.5 * x.abs().max().double())
        if R < D:
            assert torch.equal(y[..., R:], x[..., R:])
    # the gradient: of the same angles, by automatic differentiation
    dq, dk = _empties(q, k)
    la.la_rotary_bwd(q, k, dq, dk, freqs, positions=pos, layout=layout, magnitude=1.25)
    for name, x, y in (("dq", q, dq), ("dk", k, dk)):
        leaf = torch.zeros_like(x, dtype=torch.float64).requires_grad_()
        o = ref.rotary(leaf, pos.double(), freqs.double(), layout, 1.25)
        close(y, torch.autograd.grad(o, leaf, x.double())[0], name, 12, 2.5 * x.abs().max().double())


def test_rotary_positions_in_place_and_single_tensor():
    normal = _gen(2)
    q = normal(2, 3, 11, 32, dtype=torch.bfloat16)
    freqs = la.la_rotary_frequencies(32).to(_dev())
    steps = torch.arange(11, device=_dev()) + 100000
    outs = []
    for kw in (dict(start=100000), dict(positions=steps), dict(positions=steps.expand(2, 11).contiguous())):
        o, = _empties(q)
        la.la_rotary_fwd(q, None, o, None, freqs, **kw)
        outs.append(o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    same = q.clone()
    la.la_rotary_fwd(same, None, same, None, freqs, start=100000)
    assert torch.equal(same, outs[0])
    # an address that only an element divides
    for layout in ("half", "interleaved"):
        flat = torch.zeros(q.numel() + 1, dtype=q.dtype, device=_dev())
        odd = flat[1:].view_as(q)
        odd.copy_(q)
        a, b = _empties(q, q)
        la.la_rotary_fwd(odd, None, a, None, freqs, start=3, layout=layout)
        la.la_rotary_fwd(q, None, b, None, freqs, start=3, layout=layout)
        assert torch.equal(a, b)
    e = q[:, :, :0].contiguous()
    la.la_rotary_fwd(e, e.clone(), torch.empty_like(e), torch.empty_like(e), freqs)


# -------------------------------------------------------------------------------- short conv --

CONV = [("f32", 2, 37, 64, 4, "silu"), ("f16", 3, 16, 72, 3, "silu"), ("bf16", 2, 300, 130, 4, "silu"),
        ("bf16", 6, 33, 11, 2, "none"), ("f16", 1, 2, 40, 8, "silu"), ("f32", 4, 1, 5, 4, "none"),
        ("f32", 6, 50, 12, 7, "silu"), ("f16", 2, 700, 64, 5, "none"), ("bf16", 2, 90, 34, 8, "silu"), ("f32", 2, 90, 68, 8, "silu"), ("bf16", 2, 65, 24, 6, "silu")]


@pytest.mark.parametrize("dtype,B,T,C,W,act", CONV)
@pytest.mark.parametrize("padded,carried", [(False, False), (True, True), (False, True)])
def test_short_conv(dtype, B, T, C, W, act, padded, carried):
    normal = _gen(3)
    dt = DTYPES[dtype]
    x, dy = normal(B, T, C, dtype=dt), normal(B, T, C, dtype=dt)
    w, bias = normal(C, W, scale=0.5), normal(C)
    s, ds = (normal(B, W - 1, C, dtype=dt), normal(B, W - 1, C, dtype=dt)) if carried else (None, None)
    lengths = _lengths(T, B) if padded else None
    xp, x = _pad_nan(x, lengths)
    dyp, dy = _pad_nan(dy, lengths)
    y, so = torch.full_like(x, NAN), torch.full((B, W - 1, C), NAN, dtype=dt, device=_dev())
    la.la_short_conv_fwd(xp, w, y, bias=bias, state_in=s, state_out=so, lengths=lengths, activation=act)
    lx, lw, lb, ls = _leaves(x, w, bias, s)
    wy, ws = ref.conv(lx, lw, lb, ls, lengths, act)
    mag = W * w.abs().max().double() * x.abs().max().double() + bias.abs().max()
    if carried:
        mag = max(mag, W * w.abs().max().double() * s.abs().max().double() + bias.abs().max())
    # W products and sums; the sigmoid to a few 2^-22 and |s| roundings more
    close(y, wy.detach(), "y", 2 * W + 24, mag)
    assert torch.equal(so.double(), ws.detach())

    dx, = _empties(x)
    dw, db = _empties(w, bias)
    dso = torch.full((B, W - 1, C), NAN, dtype=dt, device=_dev())
    la.la_short_conv_bwd(xp, w, dyp, dx, dw, bias=bias, dbias=db, state_in=s, dstate_in=ds,
                         dstate_out=dso if carried else None, lengths=lengths, activation=act)
    leaves = [lx, lw, lb] + ([ls] if carried else [])
    outs, seeds = ([wy, ws], [dy.double(), ds.double()]) if carried else ([wy], [dy.double()])
    grads = torch.autograd.grad(outs, leaves, seeds)
    g = 1.1 * dy.abs().double()
    gm = W * w.abs().max().double() * g.max() + (ds.abs().max().double() if carried else 0)
    k = 4 * W + 64 + 4 * mag                      # act' to a few 2^-22, moving with |s| <= mag
    close(dx, grads[0], "dx", k, gm)
    xm = max(x.abs().max(), s.abs().max() if carried else 0).double()
    close(dw, grads[1], "dw", k + B * T, (g.sum((0, 1)) * xm)[:, None])
    close(db, grads[2], "dbias", k + B * T, g.sum((0, 1)))
    if carried:
        close(dso, grads[3], "dstate_out", k, gm)


def test_short_conv_segments_and_steps_make_the_whole():
    """A prompt in two parts and then single tokens, the state updated in place: the whole call's rows."""
    normal = _gen(4)
    B, T, C, W = 3, 40, 48, 4
    x = normal(B, T, C, dtype=torch.bfloat16)
    w, bias = normal(C, W), normal(C)
    whole, = _empties(x)
    la.la_short_conv_fwd(x, w, whole, bias=bias)
    st = torch.zeros(B, W - 1, C, dtype=x.dtype, device=_dev())
    parts = []
    for a, b in ((0, 2), (2, 33)):
        part = x[:, a:b].contiguous()
        y, = _empties(part)
        la.la_short_conv_fwd(part, w, y, bias=bias, state_in=st, state_out=st)
        parts.append(y)
    for t in range(33, T):
        tok = x[:, t].contiguous()
        y, = _empties(tok)
        la.la_short_conv_step(tok, w, y, st, bias=bias)
        parts.append(y[:, None])
    assert torch.equal(torch.cat(parts, 1), whole)
    assert torch.equal(st, x[:, T - W + 1:])


# ------------------------------------------------------------------------------ selective scan --

def _scan_case(dtype, B, T, C, G, N, gate, softplus, carried, padded, seed=5):
    normal = _gen(seed)
    dt = DTYPES[dtype]
    c = dict(x=normal(B, T, C, dtype=dt), dt=normal(B, T, C, dtype=dt, scale=0.7),
             A=-torch.exp(normal(C, N)), Bm=normal(B, T, G, N, dtype=dt), Cm=normal(B, T, G, N, dtype=dt),
             D=normal(C), z=normal(B, T, C, dtype=dt) if gate else None, dt_bias=normal(C, scale=0.5) - 1.5,
             state_in=normal(B, C, N) if carried else None)
    if not softplus:
        c["dt"] = c["dt"].abs() * 0.2
        c["dt_bias"] = None
    lengths = _lengths(T, B) if padded else None
    dy, dstate = normal(B, T, C, dtype=dt), normal(B, C, N) if carried else None
    fed = dict(c)
    for n in ("x", "dt", "Bm", "Cm", "z"):
        if c[n] is not None:
            fed[n], c[n] = _pad_nan(c[n], lengths)
    dyp, dy = _pad_nan(dy, lengths)
    return c, fed, lengths, dy, dyp, dstate


SCAN_ORDER = ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state_in")


def _scan_magnitudes(c, lengths, softplus, dy, dstate):
    """Sums of the magnitudes of the terms of y, the state and every gradient: the scan of absolute
    values, each factor's derivative replaced by its absolute value."""
    v = {n: None if c[n] is None else c[n].double() for n in SCAN_ORDER}
    leaf = {n: None if t is None else t.abs().requires_grad_() for n, t in v.items()}
    B, T, C = c["x"].shape
    G, N = c["Bm"].shape[2:]
    r = v["dt"] if v["dt_bias"] is None else v["dt"] + v["dt_bias"]
    d0 = torch.logaddexp(r, torch.zeros_like(r)) if softplus else r
    slope = torch.special.expit(r) if softplus else torch.ones_like(r)
    move = leaf["dt"] - leaf["dt"].detach()
    if leaf["dt_bias"] is not None:
        move = move + leaf["dt_bias"] - leaf["dt_bias"].detach()
    d = d0.abs() + slope * move
    gate = None
    if v["z"] is not None:
        sg = torch.special.expit(v["z"])
        gate = (v["z"] * sg).abs() + (sg * (1 + v["z"] * (1 - sg))).abs() * (leaf["z"] - leaf["z"].detach())
    ys, hs = [], []
    for b, n in enumerate(ref.ends(lengths, B, T)):
        h = v["x"].new_zeros(C, N) if leaf["state_in"] is None else leaf["state_in"][b]
        rows = []
        for t in range(n):
            Bt, Ct = (leaf[m][b, t].repeat_interleave(C // G, 0) for m in ("Bm", "Cm"))
            e = d[b, t, :, None] * leaf["A"]
            a = torch.exp(d0[b, t, :, None] * v["A"]) * (1 + e - e.detach())
            h = a * h + (d[b, t] * leaf["x"][b, t])[:, None] * Bt
            y = (h * Ct).sum(-1) + leaf["D"] * leaf["x"][b, t]
            rows.append(y if gate is None else y * gate[b, t])
        ys.append(torch.cat([torch.stack(rows) if rows else h.new_zeros(0, C), h.new_zeros(T - n, C)]))
        hs.append(h)
    y, h = torch.stack(ys), torch.stack(hs)
    leaves = [leaf[n] for n in SCAN_ORDER if leaf[n] is not None]
    outs, seeds = ([y, h], [dy.double().abs(), dstate.abs().double()]) if dstate is not None else ([y], [dy.double().abs()])
    grads = torch.autograd.grad(outs, leaves, seeds, allow_unused=True)
    names = [n for n in SCAN_ORDER if leaf[n] is not None]
    return y.detach(), h.detach(), {n: g for n, g in zip(names, grads)}


SCAN = [("f32", 2, 37, 40, 1, 16, True, True, False, False), ("bf16", 1, 300, 70, 2, 16, True, True, True, False),
        ("f16", 6, 50, 33, 3, 8, False, True, True, True), ("f32", 4, 1, 5, 1, 1, True, False, True, False),
        ("f32", 2, 17, 130, 1, 3, False, False, False, False), ("bf16", 2, 64, 24, 2, 33, True, True, True, True),
        ("f16", 3, 16, 20, 4, 64, True, True, False, True), ("f32", 1, 700, 9, 1, 16, True, True, True, False),
        ("f32", 6, 520, 10, 2, 5, True, True, True, True), ("bf16", 8, 40, 1200, 1, 16, True, True, False, False),
        ("f32", 2, 3, 300, 1, 4, True, True, False, False), ("bf16", 2, 15, 64, 64, 2, True, True, True, False)]


@pytest.mark.parametrize("dtype,B,T,C,G,N,gate,softplus,carried,padded", SCAN)
def test_selective_scan(dtype, B, T, C, G, N, gate, softplus, carried, padded):
    c, fed, lengths, dy, dyp, dstate = _scan_case(dtype, B, T, C, G, N, gate, softplus, carried, padded)
    y, so = torch.full_like(c["x"], NAN), torch.full((B, C, N), NAN, device=_dev())
    opt = dict(D=fed["D"], z=fed["z"], dt_bias=fed["dt_bias"], state_in=fed["state_in"], lengths=lengths,
               softplus=softplus)
    la.la_selective_scan_fwd(fed["x"], fed["dt"], fed["A"], fed["Bm"], fed["Cm"], y, state_out=so, **opt)
    leaves = dict(zip(SCAN_ORDER, _leaves(*(c[n] for n in SCAN_ORDER))))
    wy, wh = ref.scan(*(leaves[n] for n in SCAN_ORDER), lengths, softplus)
    ym, hm, gm = _scan_magnitudes(c, lengths, softplus, dy, dstate)
    # a step of the recurrence: the exponent's rounding (at most 8 in size where the state still
    # matters), the exponential's 2^-22, the step's own few, a product and a sum: 24 roundings
    k = 24 * T + 64
    close(y, wy.detach(), "y", k, ym)
    close(so, wh.detach(), "state_out", k, hm)

    got = {n: torch.full_like(c[n], NAN) for n in SCAN_ORDER if c[n] is not None}
    la.la_selective_scan_bwd(fed["x"], fed["dt"], fed["A"], fed["Bm"], fed["Cm"], dyp, got["x"], got["dt"], got["A"],
                             got["Bm"], got["Cm"], dD=got["D"], dz=got.get("z"), ddt_bias=got.get("dt_bias"),
                             dstate_in=dstate, dstate_out=got.get("state_in"), **opt)
    names = [n for n in SCAN_ORDER if leaves[n] is not None]
    outs, seeds = ([wy, wh], [dy.double(), dstate.double()]) if carried else ([wy], [dy.double()])
    grads = dict(zip(names, torch.autograd.grad(outs, [leaves[n] for n in names], seeds)))
    for n in names:
        # a product of a state and a state's gradient, each with the steps' roundings; then a sum over
        # the tokens or the group's channels
        close(got[n], grads[n], "d" + n, 2 * k + B * T + C, gm[n])


def test_selective_scan_gradient_against_differences():
    """fp32 directional derivatives of sum(y dy) + sum(state_out dstate) through the forward kernel."""
    c, _, _, dy, _, dstate = _scan_case("f32", 2, 40, 24, 2, 16, True, True, True, False, seed=6)

    def loss(p):
        y, so = torch.empty_like(p["x"]), torch.empty_like(p["state_in"])
        la.la_selective_scan_fwd(p["x"], p["dt"], p["A"], p["Bm"], p["Cm"], y, D=p["D"], z=p["z"],
                                 dt_bias=p["dt_bias"], state_in=p["state_in"], state_out=so)
        return float((y.double() * dy.double()).sum() + (so.double() * dstate.double()).sum())
    got = {n: torch.empty_like(c[n]) for n in SCAN_ORDER}
    la.la_selective_scan_bwd(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], dy, got["x"], got["dt"], got["A"], got["Bm"],
                             got["Cm"], D=c["D"], dD=got["D"], z=c["z"], dz=got["z"], dt_bias=c["dt_bias"],
                             ddt_bias=got["dt_bias"], state_in=c["state_in"], dstate_in=dstate,
                             dstate_out=got["state_in"])
    normal = _gen(7)
    eps = 2.0 ** -7
    size = sum(float((dy.double().abs().sum(), dstate.double().abs().sum())[i]) for i in (0, 1))
    for n in SCAN_ORDER:
        v = torch.sign(normal(*c[n].shape)) * c[n].abs().clamp(min=0.1)
        d = (loss({**c, n: c[n] + eps * v}) - loss({**c, n: c[n] - eps * v})) / (2 * eps)
        want = float((got[n].double() * v.double()).sum())
        # the second-order term of a relative move of 2^-7 is 2^-14 of the third derivative's size; the
        # loss carries 2^-24 a term, divided by eps
        tol = 2.0 ** -10 * float((got[n].double() * v.double()).abs().sum()) + 64 * 2.0 ** -24 * size / eps
        assert abs(d - want) <= tol, (n, d, want, tol)


def test_selective_scan_parts_and_steps_make_the_whole():
    """A prompt in two calls, then single tokens with the state in place, against one call."""
    B, T, C, N = 2, 330, 48, 16
    c, *_ = _scan_case("f32", B, T, C, 1, N, True, True, False, False, seed=8)
    whole, end = torch.empty_like(c["x"]), torch.empty(B, C, N, device=_dev())
    kw = dict(D=c["D"], dt_bias=c["dt_bias"])
    la.la_selective_scan_fwd(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], whole, z=c["z"], state_out=end, **kw)
    st = torch.zeros(B, C, N, device=_dev())
    parts = []
    for a, b in ((0, 301), (301, 320)):
        p = {n: c[n][:, a:b].contiguous() for n in ("x", "dt", "Bm", "Cm", "z")}
        y = torch.empty_like(p["x"])
        la.la_selective_scan_fwd(p["x"], p["dt"], c["A"], p["Bm"], p["Cm"], y, z=p["z"], state_in=st, state_out=st, **kw)
        parts.append(y)
    for t in range(320, T):
        p = {n: c[n][:, t].contiguous() for n in ("x", "dt", "Bm", "Cm", "z")}
        y = torch.empty_like(p["x"])
        la.la_selective_scan_step(p["x"], p["dt"], c["A"], p["Bm"], p["Cm"], y, st, z=p["z"], **kw)
        parts.append(y[:, None])
    ym, hm, _ = _scan_magnitudes({**c, "state_in": None}, None, True, c["x"], None)
    # both sides carry the recurrence's roundings (see test_selective_scan)
    close(torch.cat(parts, 1), whole.double(), "y", 2 * (24 * T + 64), ym)
    close(st, end.double(), "state", 2 * (24 * T + 64), hm)


@pytest.mark.parametrize("N", [1, 6, 16, 31, 64])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_selective_scan_step(dtype, N):
    B, C, G = 5, 66, 3
    c, *_ = _scan_case(dtype, B, 1, C, G, N, True, True, True, False, seed=9)
    one = {n: c[n][:, 0].contiguous() for n in ("x", "dt", "Bm", "Cm", "z")}
    y, so = torch.full_like(one["x"], NAN), torch.full((B, C, N), NAN, device=_dev())
    la.la_selective_scan_step(one["x"], one["dt"], c["A"], one["Bm"], one["Cm"], y, c["state_in"], so, D=c["D"],
                              z=one["z"], dt_bias=c["dt_bias"])
    wy, wh = ref.scan(*(None if c[n] is None else c[n].double() for n in SCAN_ORDER), None, True)
    ym, hm, _ = _scan_magnitudes(c, None, True, c["x"], None)
    close(y, wy[:, 0], "y", 24 + 64, ym[:, 0])
    close(so, wh, "state_out", 24 + 64, hm)


def test_scan_without_tokens_passes_states_on():
    x = torch.empty(2, 0, 8, device=_dev())
    bc = torch.empty(2, 0, 1, 4, device=_dev())
    A, st = -torch.ones(8, 4, device=_dev()), torch.randn(2, 8, 4, device=_dev())
    out = torch.full_like(st, NAN)
    la.la_selective_scan_fwd(x, x, A, bc, bc, torch.empty_like(x), state_in=st, state_out=out)
    assert torch.equal(out, st)
    la.la_selective_scan_fwd(x, x, A, bc, bc, torch.empty_like(x), state_out=out)
    assert torch.equal(out, torch.zeros_like(out))
    dA, dso = torch.full_like(A, NAN), torch.full_like(st, NAN)
    e = [torch.empty_like(t) for t in (x, x, bc, bc)]
    la.la_selective_scan_bwd(x, x, A, bc, bc, x, e[0], e[1], dA, e[2], e[3], dstate_in=st, dstate_out=dso)
    assert torch.equal(dA, torch.zeros_like(A)) and torch.equal(dso, st)


# ----------------------------------------------------------------------------------- group norm --

NORM = [("f32", 2, 37, 64, 8, "silu"), ("f16", 3, 300, 60, 30, "silu"), ("bf16", 2, 1000, 320, 32, "none"),
        ("bf16", 300, 1, 512, 8, "silu"), ("f32", 5, 1, 33, 11, "none"), ("f16", 2, 4099, 40, 4, "silu"),
        ("f32", 1, 17, 1290, 1, "silu"), ("bf16", 7, 1, 4096, 1, "silu"), ("f32", 3, 1, 4097, 1, "none"),
        ("f16", 2, 5, 2600, 2, "silu"), ("f32", 1, 2, 3, 3, "silu"), ("bf16", 4, 64, 256, 32, "silu"),
        ("f16", 40, 1, 9000, 3, "silu"), ("bf16", 3, 3, 30, 15, "none"), ("bf16", 1, 900, 6000, 6, "silu"),
        ("f16", 2, 500, 4100, 50, "silu"), ("f32", 2, 130, 8200, 1, "silu"), ("f16", 1, 70, 9225, 9, "none")]


@pytest.mark.parametrize("dtype,B,T,C,G,act", NORM)
@pytest.mark.parametrize("affine", [True, False])
def test_group_norm(dtype, B, T, C, G, act, affine):
    normal = _gen(10)
    dt = DTYPES[dtype]
    x, dy = (normal(B, T, C) * (0.5 + normal(C).abs()) + normal(C)).to(dt), normal(B, T, C, dtype=dt)
    ga, be = (1 + 0.2 * normal(C), 0.2 * normal(C)) if affine else (None, None)
    y, = _empties(x)
    mean, rstd = (torch.full((B, G), NAN, device=_dev()) for _ in range(2))
    la.la_group_norm_fwd(x, y, G, gamma=ga, beta=be, eps=1e-3, activation=act, mean=mean, rstd=rstd)
    lx, lga, lbe = _leaves(x, ga, be)
    wy, wm, wr = ref.norm(lx, lga, lbe, G, 1e-3, act)
    xm = x.abs().amax((1, 2)).double()
    # sums over 64 terms a thread at most before they are joined, means joined twice
    close(mean, wm.detach(), "mean", 100, xm[:, None])
    close(rstd, wr.detach(), "rstd", 200, (wr * (1 + wr * xm[:, None])).detach())
    xh = ref.norm(x.double(), None, None, G, 1e-3, "none")[0]
    gmax = 1.0 if ga is None else ga.abs().max().double()
    ch = C // G
    rs = wr.detach().repeat_interleave(ch, 1)[:, None]
    # (x - mean) rstd: 200 roundings of |x| rstd, of |xh|^2 through the variance
    unit = gmax * (rs * xm[:, None, None] * (1 + xh.abs())) + 1
    close(y, wy.detach(), "y", 250, unit)

    leaves = [lx] + ([lga, lbe] if affine else [])
    grads = torch.autograd.grad([wy], leaves, [dy.double()])
    dx, = _empties(x)
    dga, dbe = (torch.full((C,), NAN, device=_dev()) for _ in range(2)) if affine else (None, None)
    la.la_group_norm_bwd(x, dy, dx, G, mean, rstd, gamma=ga, beta=be, dgamma=dga, dbeta=dbe, activation=act)
    g = 1.1 * dy.abs().double()
    close(dx, grads[0], "dx", 400, rs * gmax * g.max() * (1 + xh.abs()) * unit.amax())
    if affine:
        close(dga, grads[1], "dgamma", 300 + B * T, (g * (xh.abs() + unit)).sum((0, 1)))
        close(dbe, grads[2], "dbeta", 300 + B * T, (g * unit).sum((0, 1)))


@pytest.mark.parametrize("T,C,G", [(1, 256, 4), (3000, 64, 8), (200, 32, 2)])
def test_group_norm_far_mean(T, C, G):
    """A mean 10^4 spreads away: sums of squares about zero would lose the spread altogether."""
    x = _gen(11)(2, T, C) + 10000
    y, = _empties(x)
    la.la_group_norm_fwd(x, y, G)
    want = ref.norm(x.double(), None, None, G, 1e-5, "none")[0]
    close(y, want, "y", 60, 10010.0 * 1.2 * (1 + want.abs().max()))


def test_group_norm_in_place_misaligned_and_empty():
    normal = _gen(12)
    for B, T, C, G in ((40, 1, 96, 4), (2, 600, 48, 6)):
        x, dy = normal(B, T, C, dtype=torch.float16), normal(B, T, C, dtype=torch.float16)
        a, m, r = torch.empty_like(x), torch.empty(B, G, device=_dev()), torch.empty(B, G, device=_dev())
        la.la_group_norm_fwd(x, a, G, activation="silu", mean=m, rstd=r)
        b = x.clone()
        la.la_group_norm_fwd(b, b, G, activation="silu")
        assert torch.equal(a, b)
        d1, d2 = torch.empty_like(x), dy.clone()
        la.la_group_norm_bwd(x, dy, d1, G, m, r, activation="silu")
        la.la_group_norm_bwd(x, d2, d2, G, m, r, activation="silu")
        assert torch.equal(d1, d2)
        flat = torch.zeros(x.numel() + 1, dtype=x.dtype, device=_dev())
        odd = flat[1:].view_as(x)
        odd.copy_(x)
        c, = _empties(x)
        la.la_group_norm_fwd(odd, c, G, activation="silu")
        close(c, a.double(), "misaligned", 400, 8.0)     # another access width sums in another order
    e = torch.empty(2, 0, 8, dtype=torch.float32, device=_dev())
    dg = torch.full((8,), NAN, device=_dev())
    m = torch.zeros(2, 2, device=_dev())
    la.la_group_norm_fwd(e, torch.empty_like(e), 2, mean=m)
    la.la_group_norm_bwd(e, e, torch.empty_like(e), 2, m, m, dgamma=dg)
    assert torch.equal(dg, torch.zeros_like(dg))
