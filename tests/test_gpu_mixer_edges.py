"""Non-finite values, outlying rows, far positions and narrow accesses of the operators around the
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
