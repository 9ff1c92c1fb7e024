"""Non-finite values, outlying rows, far positions, narrow accesses and wide rows of the operators around the
token mixers, against their 64-bit definitions."""
from fractions import Fraction

import pytest
import torch

import linear_attention_attn_b200 as la
from tests import mixer_ref as ref
from tests.mixer_ref import DTYPES, close

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def _dev():
    return torch.device("cuda", 0)


def _gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=_dev()) * scale).to(dtype)
    return normal


def _same_where_not_finite(got, want, name):
    """NaN and infinities exactly where the definition has them; returns the mask of the finite rest."""
    for kind, a, b in (("nan", torch.isnan(got), torch.isnan(want)), ("+inf", got == INF, want == INF),
                       ("-inf", got == -INF, want == -INF)):
        assert torch.equal(a, b), "%s: %d %s, %d expected" % (name, int(a.sum()), kind, int(b.sum()))
    return torch.isfinite(want)


# ----------------------------------------------------------------------------------- group norm --

# groups in registers, in tiles, in tiles of an odd width, wider than a block
@pytest.mark.parametrize("dtype,T,C,G", [("f32", 40, 16, 4), ("f32", 3000, 64, 8), ("bf16", 3000, 64, 8),
                                         ("f16", 4099, 33, 3), ("f32", 700, 8200, 1)])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("where", [0.0, 0.4, 1.0])
def test_group_norm_hands_non_finite_values_on(dtype, T, C, G, bad, where):
    """A NaN or an infinity anywhere in a group: mean as the sum has it, a NaN variance, NaN everywhere."""
    x = _gen(1)(2, T, C, dtype=DTYPES[dtype])
    x[1, int(where * (T - 1)), C // G // 2] = bad
    y, mean, rstd = torch.empty_like(x), torch.empty(2, G, device=_dev()), torch.empty(2, G, device=_dev())
    la.la_group_norm_fwd(x, y, G, mean=mean, rstd=rstd)
    wy, wm, wr = ref.norm(x.double(), None, None, G, 1e-5, "none")
    assert int(torch.isnan(wr).sum()) == 1 and int(torch.isnan(wy).sum()) == T * (C // G)
    for name, got, want in (("mean", mean, wm), ("rstd", rstd, wr), ("y", y, wy)):
        ok = _same_where_not_finite(got, want, name)
        close(got[ok], want[ok], name, 400, 8.0)


@pytest.mark.parametrize("C,G", [(257, 1), (511, 7)])
def test_group_norm_variance_behind_an_outlying_first_row(C, G):
    """First rows 10^4 spreads away from thousands of rows that one thread sums up: squares about them
    would leave the spread to rounding."""
    B, T = 296, 8192
    x = _gen(2)(B, T, C)
    x[:, 0] += 1e4
    y, mean, rstd = torch.empty_like(x), torch.empty(B, G, device=_dev()), torch.empty(B, G, device=_dev())
    la.la_group_norm_fwd(x, y, G, mean=mean, rstd=rstd)
    for b in (0, 17, B - 1):
        _, wm, wr = ref.norm(x[b:b + 1].double(), None, None, G, 1e-5, "none")
        # the bounds of the parity tests: 100 and 200 roundings
        xm = x[b].abs().max().double()
        close(mean[b:b + 1], wm, "mean", 100, xm)
        close(rstd[b:b + 1], wr, "rstd", 200, wr * (1 + wr * xm))


@pytest.mark.parametrize("dtype,B,C,G", [("f32", 9, 8192, 2), ("bf16", 5, 4095, 1), ("f16", 5, 4094, 1),
                                         ("f32", 3, 12285, 3), ("f32", 700, 2050, 1)])
def test_group_norm_gradient_of_wide_single_rows(dtype, B, C, G):
    """T = 1 with up to 16 vectors a thread."""
    normal = _gen(3)
    dt = DTYPES[dtype]
    x, dy = normal(B, 1, C, dtype=dt), normal(B, 1, C, dtype=dt)
    ga, be = 1 + 0.2 * normal(C), 0.2 * normal(C)
    y, mean, rstd = torch.empty_like(x), torch.empty(B, G, device=_dev()), torch.empty(B, G, device=_dev())
    la.la_group_norm_fwd(x, y, G, gamma=ga, beta=be, activation="silu", mean=mean, rstd=rstd)
    leaves = [t.double().requires_grad_() for t in (x, ga, be)]
    wy, _, wr = ref.norm(*leaves, G, 1e-5, "silu")
    grads = torch.autograd.grad(wy, leaves, dy.double())
    dx, dga, dbe = torch.full_like(x, NAN), torch.full_like(ga, NAN), torch.full_like(be, NAN)
    la.la_group_norm_bwd(x, dy, dx, G, mean, rstd, gamma=ga, beta=be, dgamma=dga, dbeta=dbe, activation="silu")
    # the bounds of the parity tests (400 and 300 + B T roundings)
    xh = ref.norm(x.double(), None, None, G, 1e-5, "none")[0]
    rs = wr.detach().repeat_interleave(C // G, 1)[:, None]
    unit = ga.abs().max().double() * (rs * x.abs().max().double() * (1 + xh.abs())) + 1
    g = 1.1 * dy.abs().double()
    close(dx, grads[0], "dx", 400, rs * ga.abs().max().double() * g.max() * (1 + xh.abs()) * unit.amax())
    close(dga, grads[1], "dgamma", 300 + B, (g * (xh.abs() + unit)).sum((0, 1)))
    close(dbe, grads[2], "dbeta", 300 + B, (g * unit).sum((0, 1)))


def _odd(t):
    """The same values at an address that only one element divides."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:].copy_(t.reshape(-1))
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,T,C,G", [(40, 1, 96, 4), (3, 1, 4096, 1), (2, 600, 48, 6), (2, 90, 2600, 2)])
def test_group_norm_gradient_at_addresses_of_one_element(dtype, B, T, C, G):
    normal = _gen(4)
    dt = DTYPES[dtype]
    x, dy = normal(B, T, C, dtype=dt), normal(B, T, C, dtype=dt)
    ga = 1 + 0.2 * normal(C)
    mean, rstd = torch.empty(B, G, device=_dev()), torch.empty(B, G, device=_dev())
    la.la_group_norm_fwd(x, torch.empty_like(x), G, gamma=ga, mean=mean, rstd=rstd)
    outs = []
    for f in (lambda t: t, _odd):
        dx, dga, dbe = f(torch.full_like(x, NAN)), f(torch.full_like(ga, NAN)), f(torch.full_like(ga, NAN))
        la.la_group_norm_bwd(f(x), f(dy), dx, G, f(mean), f(rstd), gamma=f(ga), dgamma=dga, dbeta=dbe)
        outs.append((dx, dga, dbe))
    # another access width sums in another order: the bounds of the parity tests on both sides
    (dx, dga, dbe), (dx2, dga2, dbe2) = outs
    close(dx2, dx.double(), "dx", 800 + 2.0 ** 24 * torch.finfo(dt).eps / 2, dx.abs().max().double() + 8)
    close(dga2, dga.double(), "dgamma", 600 + 2 * B * T, (dy.double().abs() * 6).sum((0, 1)))
    close(dbe2, dbe.double(), "dbeta", 600 + 2 * B * T, (dy.double().abs() * 2).sum((0, 1)))


# ------------------------------------------------------------------------------------- rotary --

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_angles_of_far_positions(layout):
    """Angles reduced exactly, as fractions, up to the positions that 64-bit numbers hold."""
    pos = [0, 1, -1, 2 ** 31 + 12345, 2 ** 35 + 1, -(2 ** 40) - 3, 2 ** 45 + 1, 2 ** 52 + 7, 2 ** 53, -(2 ** 53)]
    rates = torch.tensor([1.0, 0.7498942, 0.3, 1e-3, 1e-7, 3e-12])
    ang = [[float((Fraction(p) * Fraction(float(f)) / TWO_PI) % 1 * TWO_PI) for f in rates] for p in pos]
    ang = torch.tensor(ang, dtype=torch.float64, device=_dev())[None, None]
    q = _gen(6)(1, 2, len(pos), 12)
    o = torch.full_like(q, NAN)
    la.la_rotary_fwd(q, None, o, None, rates.to(_dev()), positions=torch.tensor(pos, device=_dev()), layout=layout)
    a, b = (q[..., :6], q[..., 6:]) if layout == "half" else (q[..., 0::2], q[..., 1::2])
    a, b = a.double(), b.double()
    u, v = a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()
    want = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    # the bound of the parity test: the angle off by pi 2^-24, the sine's own 2 roundings, two products, a sum
    close(o, want, "rotary", 12, 2.5 * q.abs().max().double())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_gradient_at_addresses_of_one_element(dtype, layout):
    normal = _gen(5)
    q, k = normal(2, 3, 7, 64, dtype=DTYPES[dtype]), normal(2, 1, 7, 64, dtype=DTYPES[dtype])
    freqs = la.la_rotary_frequencies(32).to(_dev())
    outs = []
    for f in (lambda t: t, _odd):
        dq, dk = f(torch.full_like(q, NAN)), f(torch.full_like(k, NAN))
        la.la_rotary_bwd(f(q), f(k), dq, dk, f(freqs), start=77, layout=layout, magnitude=1.5)
        outs.append((dq, dk))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------- convolution --

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 4, 7])
def test_short_conv_rows_behind_the_end_take_no_part(dtype, W):
    """An infinite last row (its gradient 0 behind it times infinity is no term of dw), and channels with
    infinite or NaN taps, whose rows behind the end still come out as zeros."""
    normal = _gen(7)
    dt = DTYPES[dtype]
    B, T, C = 4, 40, 12
    x, dy, w = normal(B, T, C, dtype=dt), normal(B, T, C, dtype=dt), normal(C, W)
    lengths = torch.tensor([T, 21, 0, 1], dtype=torch.int32, device=_dev())
    ends = lengths.tolist()
    s, ds = normal(B, W - 1, C, dtype=dt), normal(B, W - 1, C, dtype=dt)
    for b, n in enumerate(ends):
        x[b, n:], dy[b, n:] = NAN, NAN
        if n:
            x[b, n - 1, 3] = INF
    w[5, W - 1], w[6, 0], w[7, W // 2] = INF, NAN, -INF
    y = torch.full_like(x, NAN)
    la.la_short_conv_fwd(x, w, y, state_in=s, lengths=lengths, activation="none")
    dx, dw, dso = torch.full_like(x, NAN), torch.full_like(w, NAN), torch.full_like(s, NAN)
    la.la_short_conv_bwd(x, w, dy, dx, dw, state_in=s, dstate_in=ds, dstate_out=dso, lengths=lengths,
                         activation="none")
    # the formula, token by token
    wdw = torch.zeros(C, W, dtype=torch.float64, device=_dev())
    wdx = torch.zeros(B, T, C, dtype=torch.float64, device=_dev())
    wds = torch.zeros(B, W - 1, C, dtype=torch.float64, device=_dev())
    w64 = w.double()
    for b, n in enumerate(ends):
        e = torch.cat([s[b], x[b, :n]]).double()
        de = torch.zeros_like(e)
        for t in range(n):
            for j in range(W):
                wdw[:, j] += dy[b, t].double() * e[t + j]
                de[t + j] += dy[b, t].double() * w64[:, j]
        de[n:] += ds[b].double()
        wds[b], wdx[b, :n] = de[:W - 1], de[W - 1:]
        assert torch.equal(y[b, n:], torch.zeros_like(y[b, n:]))
    for name, got, want in (("dx", dx, wdx), ("dw", dw, wdw), ("dstate_out", dso, wds)):
        ok = _same_where_not_finite(got, want, name)
        close(got[ok], want[ok], name, 4 * W + 64 + B * T, 200.0)


# -------------------------------------------------------------------------------------- scan --

ORDER = ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state_in")


def _infinite_case(dtype, N, what, skip, gate, T=21, seed=8):
    """One channel in three meets an infinite x or dt in the middle; x, B, C and the state positive, so that
    the formula's sums are of one sign."""
    normal = _gen(seed)
    dt = DTYPES[dtype]
    B, C = 2, 12
    c = dict(x=normal(B, T, C, dtype=dt).abs(), dt=normal(B, T, C, dtype=dt, scale=0.5), A=-torch.exp(normal(C, N)),
             Bm=normal(B, T, 1, N, dtype=dt).abs() + 0.5, Cm=normal(B, T, 1, N, dtype=dt).abs() + 0.5,
             D=normal(C).abs() if skip else None, z=normal(B, T, C, dtype=dt).abs() if gate else None, dt_bias=None,
             state_in=normal(B, C, N).abs())
    c[what][:, 9, ::3] = INF
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 9, 16, 18, 33, 64])
@pytest.mark.parametrize("what", ["x", "dt"])
@pytest.mark.parametrize("skip,gate", [(False, True), (True, False)])
def test_selective_scan_infinities_meet_no_padding(dtype, N, what, skip, gate):
    """Infinite inputs give NaN only where the formula does, whatever the number of states."""
    c = _infinite_case(dtype, N, what, skip, gate)
    B, T, C = c["x"].shape
    leaves = {n: None if c[n] is None else c[n].double().requires_grad_() for n in ORDER}
    wy, wh = ref.scan(*(leaves[n] for n in ORDER), None, True)
    y, so = torch.full_like(c["x"], 7.0), torch.full_like(c["state_in"], 7.0)
    opt = dict(D=c["D"], z=c["z"], state_in=c["state_in"])
    la.la_selective_scan_fwd(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], y, state_out=so, **opt)
    assert not torch.isnan(wy).any() and torch.isinf(wy).any()
    for name, got, want in (("y", y, wy.detach()), ("state_out", so, wh.detach())):
        ok = _same_where_not_finite(got, want, name)
        close(got[ok], want[ok], name, 24 * T + 64)
    # the single token
    h, h2 = c["state_in"].double(), c["state_in"].clone()
    for t in (8, 9, 10):
        one = {n: c[n][:, t:t + 1].contiguous() for n in ("x", "dt", "Bm", "Cm", "z") if c[n] is not None}
        wy1, h = ref.scan(*(one[n].double() if n in one else None if c[n] is None else h if n == "state_in"
                            else c[n].double() for n in ORDER), None, True)
        tok = {n: v[:, 0].contiguous() for n, v in one.items()}
        y1 = torch.empty_like(tok["x"])
        la.la_selective_scan_step(tok["x"], tok["dt"], c["A"], tok["Bm"], tok["Cm"], y1, h2, D=c["D"], z=tok.get("z"))
        for name, got, want in (("step y", y1, wy1[:, 0]), ("step state", h2, h)):
            ok = _same_where_not_finite(got, want, name)
            close(got[ok], want[ok], name, 400)


def _formula_gradients(c, dy):
    """The gradients' formulas written out (automatic differentiation multiplies by zeros of its own)."""
    v = {n: None if t is None else t.double() for n, t in c.items()}
    x, A, z, D = v["x"], v["A"], v["z"], v["D"]
    B, T, C = x.shape
    r = v["dt"]
    d = torch.logaddexp(r, torch.zeros_like(r))
    sg = None if z is None else torch.special.expit(z)
    dy = dy.double()
    e = dy if z is None else dy * (z * sg)
    hs, h = [v["state_in"]], v["state_in"]
    for t in range(T):
        h = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * x[:, t])[..., None] * v["Bm"][:, t]
        hs.append(h)
    g = {n: torch.zeros_like(v[n]) for n in ORDER if v[n] is not None}
    w = torch.zeros_like(h)
    for t in reversed(range(T)):
        a = torch.exp(d[:, t, :, None] * A)
        lam = e[:, t, :, None] * v["Cm"][:, t] + w
        g["Cm"][:, t, 0] = (e[:, t, :, None] * hs[t + 1]).sum(1)
        g["Bm"][:, t, 0] = ((d[:, t] * x[:, t])[..., None] * lam).sum(1)
        q = (lam * v["Bm"][:, t]).sum(-1)
        w = a * lam
        p = w * hs[t]
        g["x"][:, t] = d[:, t] * q if D is None else d[:, t] * q + D * e[:, t]
        g["dt"][:, t] = (x[:, t] * q + (A * p).sum(-1)) * torch.special.expit(r[:, t])
        g["A"] += (d[:, t, :, None] * p).sum(0)
        if D is not None:
            g["D"] += (e[:, t] * x[:, t]).sum(0)
        if z is not None:
            y = (hs[t + 1] * v["Cm"][:, t]).sum(-1)
            y = y if D is None else y + D * x[:, t]
            g["z"][:, t] = dy[:, t] * y * (sg[:, t] * (1 + z[:, t] * (1 - sg[:, t])))
    g["state_in"] = w
    return g


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 9, 16, 18, 33, 64])
@pytest.mark.parametrize("skip,gate", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("T", [24, 21])
def test_selective_scan_gradient_of_infinities(T, N, skip, gate):
    """An infinite incoming gradient at one token of some channels, and an infinite x at the last one."""
    c = _infinite_case("f32", N, "x", skip, gate, T)
    c["x"] = torch.where(torch.isinf(c["x"]), torch.ones_like(c["x"]), c["x"])
    c["x"][:, -1, 1::3] = INF
    dy = _gen(9)(*c["x"].shape).abs()
    dy[:, 9, ::3] = INF
    got = {n: torch.full_like(c[n], 7.0) for n in ORDER if c[n] is not None}
    la.la_selective_scan_bwd(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], dy, got["x"], got["dt"], got["A"], got["Bm"],
                             got["Cm"], D=c["D"], dD=got.get("D"), z=c["z"], dz=got.get("z"),
                             state_in=c["state_in"], dstate_out=got["state_in"])
    want = _formula_gradients(c, dy)
    for n in got:
        ok = _same_where_not_finite(got[n], want[n], "d" + n)
        scale = want[n][ok].abs().max() if ok.any() else 1.0
        close(got[n][ok], want[n][ok], "d" + n, 2 * (24 * dy.shape[1] + 64) + dy.numel(), scale)


@pytest.mark.parametrize("T,d", [(2048, 2.0 ** -8), (64, 2.0 ** -2)])
def test_decays_are_not_off_to_one_side(T, d):
    """One state a channel that decays by exp(-d / 10) to exp(-d 1.38) at every token: averaged over channels, the
    decays are off by at most 1.2e-8, the bound that scan::decay2 states (the exponential unit's truncation alone
    measures 1.65e-8 at d = 1/4)."""
    C = 4096
    g = torch.Generator(device="cuda").manual_seed(10)
    A = -(torch.rand(C, 1, generator=g, device=_dev()) * 1.28 + 0.1)
    dt = torch.full((1, T, C), d, device=_dev())
    x, bc = torch.zeros(1, T, C, device=_dev()), torch.zeros(1, T, 1, 1, device=_dev())
    s = torch.ones(1, C, 1, device=_dev())
    so = torch.empty_like(s)
    la.la_selective_scan_fwd(x, dt, A, bc, bc, torch.empty_like(x), state_in=s, state_out=so, softplus=False)
    off = (so.double().log()[0, :, 0] - A.double()[:, 0] * d * T) / T
    # a channel's decay is also rounded, by up to 2^-25, the same way at every token, and so is the product with
    # its state, by chance: over 4096 channels that averages to 2^-25 / sqrt(3 4096) = 2.7e-10 and less
    assert abs(float(off.mean())) <= 1.2e-8, float(off.mean())
