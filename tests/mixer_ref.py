"""Definitions in 64 bits of the operators around the token mixers, and error bounds, for their tests.

Every function takes float64 tensors (any device) and is differentiable, so gradients come from
automatic differentiation of the definition."""
import math

import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rotary(x, pos, freqs, layout, magnitude):
    """x [B, H, T, D], pos [B, T] float64."""
    R = 2 * freqs.numel()
    ang = (pos[..., None] * freqs)[:, None]
    c, s = torch.cos(ang) * magnitude, torch.sin(ang) * magnitude
    if layout == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat([a * c - b * s, a * s + b * c, x[..., R:]], -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), x[..., R:]], -1)


def silu(t):
    return t * torch.special.expit(t)


def ends(lengths, B, T):
    return [T] * B if lengths is None else [n if 0 <= n <= T else (0 if n < 0 else T) for n in lengths.tolist()]


def conv(x, w, bias, state, lengths, act):
    """(y, state after the last token); x [B, T, C], state [B, W - 1, C] or None."""
    B, T, C = x.shape
    W = w.shape[1]
    ys, sts = [], []
    for b, n in enumerate(ends(lengths, B, T)):
        e = torch.cat([x.new_zeros(W - 1, C) if state is None else state[b], x[b, :n]])
        y = sum(w[:, j] * e[j:j + n] for j in range(W))
        y = y + (0 if bias is None else bias)
        ys.append(torch.cat([silu(y) if act == "silu" else y, x.new_zeros(T - n, C)]))
        sts.append(e[n:])
    return torch.stack(ys), torch.stack(sts)


def scan(x, dt, A, Bm, Cm, D, z, bias, state, lengths, softplus):
    """(y, state after the last token); x [B, T, C], Bm [B, T, G, N], state [B, C, N] or None."""
    B, T, C = x.shape
    G, N = Bm.shape[2:]
    r = dt if bias is None else dt + bias
    d = torch.logaddexp(r, torch.zeros_like(r)) if softplus else r
    ys, hs = [], []
    for b, n in enumerate(ends(lengths, B, T)):
        h = x.new_zeros(C, N) if state is None else state[b]
        rows = []
        for t in range(n):
            Bt, Ct = (m[b, t].repeat_interleave(C // G, 0) for m in (Bm, Cm))
            h = torch.exp(d[b, t, :, None] * A) * h + (d[b, t] * x[b, t])[:, None] * Bt
            y = (h * Ct).sum(-1)
            y = y if D is None else y + D * x[b, t]
            rows.append(y if z is None else y * silu(z[b, t]))
        ys.append(torch.cat([torch.stack(rows) if rows else x.new_zeros(0, C), x.new_zeros(T - n, C)]))
        hs.append(h)
    return torch.stack(ys), torch.stack(hs)


def norm(x, gamma, beta, G, eps, act):
    """(y, mean [B, G], rstd [B, G]); x [B, T, C]."""
    B, T, C = x.shape
    v = x.view(B, T, G, C // G)
    m = v.mean((1, 3))
    r = 1 / torch.sqrt((v - m[:, None, :, None]).square().mean((1, 3)) + eps)
    y = ((v - m[:, None, :, None]) * r[:, None, :, None]).reshape(B, T, C)
    y = y if gamma is None else y * gamma
    y = y if beta is None else y + beta
    return (silu(y) if act == "silu" else y), m, r


def close(got, want, name, roundings, scale=None):
    """|got - want| within half a step of the storage type plus `roundings` roundings of 2^-24 of
    `scale` (the sum of the magnitudes that meet in the element; default: the largest |want|)."""
    want = want.double()
    if want.numel() == 0:
        assert got.shape == want.shape
        return
    s = want.abs().max() if scale is None else scale
    fi = torch.finfo(got.dtype)
    tol = want.abs() * (fi.eps / 2) + roundings * 2.0 ** -24 * s + fi.tiny * fi.eps
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = int(torch.argmax((err - tol).nan_to_num(math.inf)))
        raise AssertionError("%s: %d of %d off; worst got %r want %r tol %r" % (
            name, int(bad.sum()), bad.numel(), float(got.flatten()[i]), float(want.flatten()[i]),
            float(tol.expand_as(want).flatten()[i])))
