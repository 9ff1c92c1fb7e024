"""The operators around the token mixers without a GPU: refusals before any CUDA call, workspace
sizes, the rotary frequencies, and the 64-bit definitions against differences."""
import ctypes
import math

import pytest
import torch

import linear_attention_attn_b200 as la
from tests import mixer_ref as ref

P = ctypes.c_void_p
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
MB = 1 << 24          # spacing of the made-up addresses: no two tensors of a call overlap


def _addr(names, **over):
    at = {n: (i + 1) * MB for i, n in enumerate(names)}
    at.update(over)
    return [at[n] for n in names], at


def _rotary(B=1, H=2, Hk=1, T=4, D=8, R=8, layout=0, dt=2, mag=1.0, per=0, back=False, **over):
    v, _ = _addr(["q", "k", "oq", "ok", "freqs", "pos"], **over)
    f = la.raw_lib().la_rotary_bwd if back else la.raw_lib().la_rotary_fwd
    return f(*v, per, 0, layout, mag, B, H, Hk, T, D, R, dt, None)


@pytest.mark.parametrize("back", [False, True])
def test_rotary_refusals(back):
    assert _rotary(back=back, B=0) == INVALID
    assert _rotary(back=back, H=0) == INVALID
    assert _rotary(back=back, Hk=0) == INVALID
    assert _rotary(back=back, T=-1) == INVALID
    assert _rotary(back=back, R=7) == INVALID
    assert _rotary(back=back, R=10) == INVALID
    assert _rotary(back=back, R=0) == INVALID
    assert _rotary(back=back, D=2048, R=8) == UNSUPPORTED
    assert _rotary(back=back, dt=5) == UNSUPPORTED
    assert _rotary(back=back, layout=2) == UNSUPPORTED
    assert _rotary(back=back, mag=math.nan) == INVALID
    assert _rotary(back=back, per=2) == INVALID
    assert _rotary(back=back, q=None) == INVALID
    assert _rotary(back=back, k=None) == INVALID          # ok without k
    assert _rotary(back=back, freqs=None) == INVALID
    assert _rotary(back=back, q=MB + 1) == ALIGNMENT
    assert _rotary(back=back, pos=6 * MB + 4) == ALIGNMENT
    assert _rotary(back=back, oq=MB + 2) == INVALID       # overlaps q without being q
    assert _rotary(back=back, ok=MB) == INVALID           # overlaps the other tensor
    assert _rotary(back=back, T=0, q=None, k=None, oq=None, ok=None) == 0


def _conv(T=4, B=1, C=8, W=4, act=1, dt=2, **over):
    v, _ = _addr(["x", "w", "bias", "si", "y", "so", "len"], **over)
    return la.raw_lib().la_short_conv_fwd(*v, act, B, T, C, W, dt, None)


def test_conv_refusals():
    assert _conv(W=1) == UNSUPPORTED
    assert _conv(W=9) == UNSUPPORTED
    assert _conv(act=2) == UNSUPPORTED
    assert _conv(dt=3) == UNSUPPORTED
    assert _conv(C=0) == INVALID
    assert _conv(T=-1) == INVALID
    assert _conv(C=(1 << 20) + 1) == UNSUPPORTED
    for n in ("x", "w", "y"):
        assert _conv(**{n: None}) == INVALID
    assert _conv(x=MB + 1) == ALIGNMENT
    assert _conv(w=2 * MB + 2) == ALIGNMENT
    assert _conv(len=7 * MB + 2) == ALIGNMENT
    assert _conv(y=MB) == INVALID                          # in place is not allowed
    assert _conv(so=4 * MB + 2) == INVALID                 # the state: the same buffer or another one
    lib = la.raw_lib()
    v, _ = _addr(["x", "w", "bias", "si", "y", "so"], si=None)
    assert lib.la_short_conv_step(*v, 1, 1, 8, 4, 2, None) == INVALID
    v, _ = _addr(["x", "w", "bias", "si", "y", "so"], so=None)
    assert lib.la_short_conv_step(*v, 1, 1, 8, 4, 2, None) == INVALID


def _conv_bwd(T=4, B=1, C=8, W=4, act=1, dt=2, ws=20 * MB, wsb=MB, **over):
    v, _ = _addr(["x", "w", "bias", "si", "dy", "dsi", "dx", "dw", "db", "dso", "len"], **over)
    return la.raw_lib().la_short_conv_bwd(*v, act, B, T, C, W, dt, ws, wsb, None)


def test_conv_bwd_refusals():
    assert _conv_bwd(ws=None) == WORKSPACE
    assert _conv_bwd(wsb=8) == WORKSPACE
    assert _conv_bwd(ws=20 * MB + 64) == ALIGNMENT
    assert _conv_bwd(ws=MB) == INVALID                     # the workspace over x
    assert _conv_bwd(dx=5 * MB) == INVALID                 # over dy
    assert _conv_bwd(dso=6 * MB) == INVALID                # over dstate_in
    assert _conv_bwd(dw=None) == INVALID
    assert la.raw_lib().la_last_error() == b"dw is NULL"


SCAN_IN = ["x", "dt", "A", "Bm", "Cm", "D", "z", "bias", "si"]


def _scan(B=1, T=4, C=8, G=1, N=16, dt=2, ws=None, wsb=0, **over):
    v, _ = _addr(SCAN_IN + ["y", "so", "len"], **over)
    return la.raw_lib().la_selective_scan_fwd(*v, 1, B, T, C, G, N, dt, ws, wsb, None)


def _scan_bwd(B=1, T=4, C=8, G=1, N=16, dt=2, ws=30 * MB, wsb=MB, **over):
    names = SCAN_IN + ["dy", "dsi", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dso", "len"]
    v, _ = _addr(names, **over)
    return la.raw_lib().la_selective_scan_bwd(*v, 1, B, T, C, G, N, dt, ws, wsb, None)


def test_scan_refusals():
    assert _scan(G=3) == INVALID
    assert _scan(G=0) == INVALID
    assert _scan(N=0) == UNSUPPORTED
    assert _scan(N=65) == UNSUPPORTED
    assert _scan(dt=9) == UNSUPPORTED
    assert _scan(x=None) == INVALID
    assert _scan(A=3 * MB + 2) == ALIGNMENT
    assert _scan(y=MB) == INVALID
    assert _scan(y=7 * MB) == INVALID                      # over z
    assert _scan(so=9 * MB + 4) == INVALID
    assert _scan(T=1000) == WORKSPACE                      # few channels, long: split into segments
    lib = la.raw_lib()
    v, _ = _addr(SCAN_IN + ["y", "so"], so=None)
    assert lib.la_selective_scan_step(*v, 1, 1, 8, 1, 16, 2, None) == INVALID


def test_scan_bwd_refusals():
    assert _scan_bwd(ws=None) == WORKSPACE
    assert _scan_bwd(wsb=256) == WORKSPACE
    assert _scan_bwd(dz=None) == INVALID
    assert _scan_bwd(z=None) == INVALID
    assert _scan_bwd(dx=10 * MB) == INVALID                # over dy
    assert _scan_bwd(dso=11 * MB) == INVALID               # over dstate_in
    assert _scan_bwd(dB=4 * MB) == INVALID                 # over Bm
    assert _scan_bwd(ddt=None) == INVALID


def _norm(B=1, T=4, C=8, G=2, eps=1e-5, act=1, dt=2, ws=20 * MB, wsb=MB, **over):
    v, _ = _addr(["x", "ga", "be", "y", "m", "r"], **over)
    return la.raw_lib().la_group_norm_fwd(*v, eps, act, B, T, C, G, dt, ws, wsb, None)


def test_norm_refusals():
    assert _norm(G=3) == INVALID
    assert _norm(eps=0.0) == INVALID
    assert _norm(eps=math.nan) == INVALID
    assert _norm(act=4) == UNSUPPORTED
    assert _norm(y=MB + 2) == INVALID
    assert _norm(y=None) == INVALID
    assert _norm(m=6 * MB) == INVALID                      # mean over rstd
    assert _norm(ws=None) == WORKSPACE
    v, _ = _addr(["x", "dy", "m", "r", "ga", "be", "dx", "dga", "dbe"])
    f = la.raw_lib().la_group_norm_bwd
    assert f(*v, 1, 1, 4, 8, 2, 2, None, 0, None) == WORKSPACE
    v[2] = None
    assert f(*v, 1, 1, 4, 8, 2, 2, 20 * MB, MB, None) == INVALID


def test_workspace_sizes():
    size = la.la_mixer_workspace_size
    for op, n in (("short_conv_bwd", 4), ("selective_scan_bwd", 16), ("group_norm_bwd", 1)):
        a = size(op, 2, 100, 64, 1, n, torch.bfloat16)
        assert a > 0 and a % 256 == 0
        assert size(op, 0, 100, 64, 1, n, torch.bfloat16) == 0
        assert size(op, 2, 0, 64, 1, n, torch.bfloat16) == 0
    assert size("selective_scan_fwd", 8, 4096, 2048, 1, 16, torch.bfloat16) == 0
    assert size("selective_scan_fwd", 1, 4096, 256, 1, 16, torch.bfloat16) > 0
    assert size("group_norm_fwd", 64, 1, 512, 8, 1, torch.bfloat16) == 0
    assert size("bidir_fwd", 8, 100, 64, 1, 1, torch.bfloat16) == 0
    assert la.la_workspace_size("group_norm_fwd", 8, 16, 64, 64, torch.float16) == 0


def test_rotary_frequencies():
    f = la.la_rotary_frequencies
    R = 64
    i = torch.arange(R // 2, dtype=torch.float64)
    plain = 10000.0 ** (-2 * i / R)
    assert torch.equal(f(R), plain.float())
    assert torch.equal(f(R, 500000.0), (500000.0 ** (-2 * i / R)).float())
    assert torch.equal(f(R, scaling="linear", factor=4.0), (plain / 4).float())
    ntk = f(R, scaling="ntk", factor=8.0).double()
    assert ntk[0] == 1 and abs(float(ntk[-1] * 8 / plain[-1]) - 1) < 1e-6
    parts = f(R, scaling="by_parts", factor=16.0, original_length=4096, beta_fast=32, beta_slow=1).double()
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], plain.float().double()[turns >= 32])
    assert torch.equal(parts[turns <= 1], (plain / 16).float().double()[turns <= 1])
    mid = (turns > 1) & (turns < 32)
    keep = (turns - 1) / 31
    want = plain * keep + plain / 16 * (1 - keep)
    assert mid.any() and ((parts / want - 1).abs()[mid] < 2.0 ** -23).all()
    for bad in (dict(base=0.0), dict(scaling="linear", factor=0.5), dict(scaling="by_parts", factor=2.0),
                dict(scaling="by_parts", factor=2.0, original_length=10, beta_fast=1, beta_slow=1)):
        with pytest.raises(la.LAError):
            f(R, **bad)
    with pytest.raises(la.LAError):
        f(2, scaling="ntk", factor=2.0)
    with pytest.raises(ValueError):
        f(7)
    with pytest.raises(ValueError):
        f(8, scaling="other")


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        la.la_group_norm_fwd(x, x.clone(), 2)
    with pytest.raises(ValueError):
        la.la_short_conv_fwd(x, torch.zeros(8, 4), x.clone())


def _leaf(*shape, seed=0, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale + shift).requires_grad_()


def test_definitions_against_differences():
    """The 64-bit definitions that the GPU tests differentiate: derivatives against differences."""
    lengths = torch.tensor([3, 0, 5], dtype=torch.int32)
    x, w, b, s = _leaf(3, 5, 2), _leaf(2, 3, seed=1), _leaf(2, seed=2), _leaf(3, 2, 2, seed=3)
    torch.autograd.gradcheck(lambda *a: ref.conv(*a, lengths, "silu"), (x, w, b, s))
    x, dt, A = _leaf(3, 5, 4), _leaf(3, 5, 4, seed=1), _leaf(4, 3, seed=2, scale=0.3, shift=-1)
    Bm, Cm, D, z = _leaf(3, 5, 2, 3, seed=3), _leaf(3, 5, 2, 3, seed=4), _leaf(4, seed=5), _leaf(3, 5, 4, seed=6)
    h = _leaf(3, 4, 3, seed=7)
    torch.autograd.gradcheck(lambda *a: ref.scan(*a, lengths, True), (x, dt, A, Bm, Cm, D, z, b.new_zeros(4), h))
    torch.autograd.gradcheck(lambda *a: ref.norm(*a, 2, 1e-3, "silu")[0], (x, _leaf(4, seed=8), _leaf(4, seed=9)))
    q = _leaf(1, 2, 3, 6)
    for lay in ("half", "interleaved"):
        torch.autograd.gradcheck(lambda t: ref.rotary(t, torch.tensor([[0., 7., 3.]], dtype=torch.float64),
                                                      torch.tensor([1.0, 0.1], dtype=torch.float64), lay, 1.5), (q,))
