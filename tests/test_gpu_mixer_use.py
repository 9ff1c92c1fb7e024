"""The operators around the token mixers as they are used: whole blocks for training and for serving,
captured and replayed, on other streams, next to each other, at offsets past 2^31, with steps and
positions at the ends of their ranges, and when a launch fails."""
import math
import threading

import pytest
import torch

import linear_attention_attn_b200 as la
from tests import mixer_ref as ref
from tests.mixer_ref import close

pytestmark = pytest.mark.gpu
NAN = float("nan")


def _dev():
    return torch.device("cuda", 0)


def _normal(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def f(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=_dev()) * scale).to(dtype)
    return f


# ------------------------------------------------------------------------------- whole blocks --

class StateSpaceBlock:
    """x -> short convolution (SiLU) -> selective scan (gated) -> group norm, and back: the calls that a
    program with its own projections makes."""

    def __init__(self, C, N, G, W, seed=21):
        n = _normal(seed)
        self.w, self.bias = n(C, W, scale=0.5), n(C, scale=0.2)
        self.A, self.D, self.dt_bias = -torch.exp(n(C, N)), n(C), n(C, scale=0.3) - 2
        self.gamma, self.beta = 1 + 0.1 * n(C), 0.1 * n(C)
        self.C, self.N, self.G, self.W = C, N, G, W

    def forward(self, x, dt, Bm, Cm, z, ws=None, stream=None, conv_state=None, state=None):
        u, y, o = (torch.empty_like(x) for _ in range(3))
        m, r = (torch.empty(x.shape[0], self.G, device=x.device) for _ in range(2))
        la.la_short_conv_fwd(x, self.w, u, bias=self.bias, state_out=conv_state, stream=stream)
        la.la_selective_scan_fwd(u, dt, self.A, Bm, Cm, y, D=self.D, z=z, dt_bias=self.dt_bias, state_out=state,
                                 workspace=ws, stream=stream)
        la.la_group_norm_fwd(y, o, self.G, gamma=self.gamma, beta=self.beta, mean=m, rstd=r, workspace=ws, stream=stream)
        return o, (x, dt, Bm, Cm, z, u, y, m, r)

    def backward(self, saved, do, ws=None, stream=None):
        x, dt, Bm, Cm, z, u, y, m, r = saved
        e = torch.empty_like
        g = {n: e(t) for n, t in (("y", y), ("u", u), ("dt", dt), ("Bm", Bm), ("Cm", Cm), ("z", z), ("x", x), ("A", self.A),
                                  ("D", self.D), ("dt_bias", self.dt_bias), ("w", self.w), ("bias", self.bias),
                                  ("gamma", self.gamma), ("beta", self.beta))}
        la.la_group_norm_bwd(y, do, g["y"], self.G, m, r, gamma=self.gamma, beta=self.beta, dgamma=g["gamma"],
                             dbeta=g["beta"], workspace=ws, stream=stream)
        la.la_selective_scan_bwd(u, dt, self.A, Bm, Cm, g["y"], g["u"], g["dt"], g["A"], g["Bm"], g["Cm"], D=self.D,
                                 dD=g["D"], z=z, dz=g["z"], dt_bias=self.dt_bias, ddt_bias=g["dt_bias"], workspace=ws,
                                 stream=stream)
        la.la_short_conv_bwd(x, self.w, g["u"], g["x"], g["w"], bias=self.bias, dbias=g["bias"], workspace=ws,
                             stream=stream)
        return g

    def inputs(self, B, T, dtype, seed=22):
        n = _normal(seed)
        return (n(B, T, self.C, dtype=dtype), n(B, T, self.C, dtype=dtype, scale=0.5), n(B, T, 1, self.N, dtype=dtype),
                n(B, T, 1, self.N, dtype=dtype), n(B, T, self.C, dtype=dtype))


def test_state_space_block_trains():
    """Values and every gradient of the chain in fp32 against the chained definitions in 64 bits."""
    blk = StateSpaceBlock(64, 16, 4, 4)
    ins = blk.inputs(2, 150, torch.float32)
    do = _normal(23)(2, 150, 64)
    o, saved = blk.forward(*ins)
    g = blk.backward(saved, do)
    L = {n: t.double().requires_grad_() for n, t in zip(("x", "dt", "Bm", "Cm", "z"), ins)}
    P = {n: getattr(blk, n).double().requires_grad_() for n in ("w", "bias", "A", "D", "dt_bias", "gamma", "beta")}
    u, _ = ref.conv(L["x"], P["w"], P["bias"], None, None, "silu")
    y, _ = ref.scan(u, L["dt"], P["A"], L["Bm"], L["Cm"], P["D"], L["z"], P["dt_bias"], None, None, True)
    want, _, _ = ref.norm(y, P["gamma"], P["beta"], 4, 1e-5, "none")
    names = list(L) + list(P)
    grads = torch.autograd.grad(want, list(L.values()) + list(P.values()), do.double())
    # 24 T + 64 roundings of the recurrence (see the parity tests) act on intermediate sums of up to a few
    # hundred times the result; 64 counts those sums' size
    close(o, want.detach(), "o", 64 * 64, want.abs().max().detach())
    for n, w in zip(names, grads):
        close(g[n], w, "d" + n, 64 * 256, w.abs().max())


def test_state_space_block_serves():
    """A prompt of ragged lengths, then single tokens with the states in place, against the whole
    sequences one by one."""
    blk = StateSpaceBlock(96, 16, 3, 4)
    B, T, new = 3, 40, 5
    x, dt, Bm, Cm, z = blk.inputs(B, T + new, torch.float32)
    lens = torch.tensor([40, 17, 2], dtype=torch.int32, device=_dev())
    cs, st = torch.empty(B, 3, 96, device=_dev()), torch.empty(B, 96, 16, device=_dev())
    p = [t[:, :T].contiguous() for t in (x, dt, Bm, Cm, z)]
    u, y = torch.empty_like(p[0]), torch.empty_like(p[0])
    la.la_short_conv_fwd(p[0], blk.w, u, bias=blk.bias, state_out=cs, lengths=lens)
    la.la_selective_scan_fwd(u, p[1], blk.A, p[2], p[3], y, D=blk.D, z=p[4], dt_bias=blk.dt_bias, state_out=st, lengths=lens)
    outs = []
    rows = torch.arange(B, device=_dev())
    for i in range(new):
        at = lens.long() + i                                # each request's next token
        tok = [t[rows, at].contiguous() for t in (x, dt, Bm, Cm, z)]
        ut, yt = torch.empty_like(tok[0]), torch.empty_like(tok[0])
        la.la_short_conv_step(tok[0], blk.w, ut, cs, bias=blk.bias)
        la.la_selective_scan_step(ut, tok[1], blk.A, tok[2], tok[3], yt, st, D=blk.D, z=tok[4], dt_bias=blk.dt_bias)
        outs.append(yt)
    for b in range(B):
        n = int(lens[b]) + new
        one = [t[b:b + 1, :n].contiguous() for t in (x, dt, Bm, Cm, z)]
        u, y = torch.empty_like(one[0]), torch.empty_like(one[0])
        la.la_short_conv_fwd(one[0], blk.w, u, bias=blk.bias)
        la.la_selective_scan_fwd(u, one[1], blk.A, one[2], one[3], y, D=blk.D, z=one[4], dt_bias=blk.dt_bias)
        got = torch.stack([o[b] for o in outs])
        # both sides carry the recurrence's roundings: 24 a token on sums of a few times the result
        close(got, y[0, n - new:].double(), "request %d" % b, 2 * (24 * n + 64) * 4)


def test_retention_with_rotary_and_group_norm():
    """Rotary queries and keys -> retention -> per-token group norm over the heads, one prompt against the
    same tokens decoded one at a time."""
    n = _normal(24)
    B, H, T, D = 2, 3, 20, 64
    q, k, v = (n(B, H, T, D, dtype=torch.bfloat16, scale=0.3) for _ in range(3))
    freqs = la.la_rotary_frequencies(D, scaling="ntk", factor=4.0).to(_dev())
    gamma = [0.9, 0.97, 1.0]
    rq, rk, o = (torch.empty_like(q) for _ in range(3))
    la.la_rotary_fwd(q, k, rq, rk, freqs, start=1000, layout="interleaved")
    la.la_chunk_decay_fwd(rq, rk, v, o, gamma)
    rows = o.transpose(1, 2).reshape(B * T, 1, H * D).contiguous()
    la.la_group_norm_fwd(rows, rows, H)
    st = torch.zeros(B, H, D, D, device=_dev())
    for t in range(T):
        tok = [x[:, :, t:t + 1].contiguous() for x in (q, k)]
        pos = torch.full((B, 1), 1000 + t, device=_dev())
        la.la_rotary_fwd(tok[0], tok[1], tok[0], tok[1], freqs, positions=pos, layout="interleaved")
        assert torch.equal(tok[0][:, :, 0], rq[:, :, t])
        ot = torch.empty(B, H, D, dtype=q.dtype, device=_dev())
        la.la_chunk_decay_step(tok[0].view(B, H, D), tok[1].view(B, H, D), v[:, :, t].contiguous(), ot, st, gamma)
        yt = ot.reshape(B, 1, H * D)
        la.la_group_norm_fwd(yt, yt, H)
        # two forms of retention, each rounded to bf16 (a step 2^-7 of the value) before the norm
        a, b = yt[:, 0].float(), rows.view(B, T, -1)[:, t].float()
        assert (a - b).abs().max() <= 4 * 2.0 ** -7 * b.abs().max()


# ------------------------------------------------------------------ graphs, streams, neighbours --

def _step_tensors(blk, B=2, T=400, dtype=torch.bfloat16, seed=25):
    return blk.inputs(B, T, dtype, seed), _normal(seed + 1)(B, T, blk.C, dtype=dtype)


def _flat(o, g):
    return [o] + [g[n] for n in sorted(g)]


def test_runs_are_bitwise_equal_on_any_stream():
    blk = StateSpaceBlock(80, 16, 4, 4)
    ins, do = _step_tensors(blk)
    o, saved = blk.forward(*ins)
    want = _flat(o, blk.backward(saved, do))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        # buffers are made on the current stream and used on the other: order both ways
        o, saved = blk.forward(*ins, stream=stream)
        g = blk.backward(saved, do, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(want, _flat(o, g)):
            assert torch.equal(a, b)


def test_graphs_replay_and_share_their_pool():
    """Two captured training steps from one memory pool, replayed in turn on new inputs, while an eager
    step of the same parameters has run before."""
    blk = StateSpaceBlock(48, 8, 4, 3)
    ins, do = _step_tensors(blk, T=300)
    eager = _flat(*(lambda o, s: (o, blk.backward(s, do)))(*blk.forward(*ins)))
    graphs, outs, holds = [], [], []
    pool = None
    for i in range(2):
        mine = [t.clone() for t in ins]
        holds.append(mine)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            o, s = blk.forward(*mine)
            outs.append(_flat(o, blk.backward(s, do)))
        pool = g.pool()
        graphs.append(g)
    for turn in range(2):
        for i in (0, 1):
            graphs[i].replay()
            torch.cuda.synchronize()
            for a, b in zip(eager, outs[i]):
                assert torch.equal(a, b)
    other = blk.inputs(2, 300, torch.bfloat16, 77)
    for m, t in zip(holds[1], other):
        m.copy_(t)
    graphs[1].replay()
    torch.cuda.synchronize()
    o, s = blk.forward(*other)
    for a, b in zip(_flat(o, blk.backward(s, do)), outs[1]):
        assert torch.equal(a, b)
    del graphs


def test_two_threads_on_two_streams():
    blk = StateSpaceBlock(64, 16, 4, 4)
    cases = [_step_tensors(blk, T=500, seed=s) for s in (31, 33)]
    want = []
    for ins, do in cases:
        o, s = blk.forward(*ins)
        want.append(_flat(o, blk.backward(s, do)))
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    o, s = blk.forward(*cases[i][0])
                    got[i] = _flat(o, blk.backward(s, cases[i][1]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:          # reported by the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in (0, 1):
        for a, b in zip(want[i], got[i]):
            assert torch.equal(a, b)


def test_workspace_is_checked_and_its_contents_do_not_matter():
    blk = StateSpaceBlock(32, 16, 2, 4)
    ins, do = _step_tensors(blk, B=1, T=300)
    need = max(la.la_mixer_workspace_size(op, 1, 300, 32, g, n, torch.bfloat16) for op, g, n in
               (("selective_scan_fwd", 1, 16), ("selective_scan_bwd", 1, 16), ("group_norm_fwd", 2, 1),
                ("group_norm_bwd", 2, 1), ("short_conv_bwd", 1, 4)))
    runs = []
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=_dev())
        o, s = blk.forward(*ins, ws=ws)
        runs.append(_flat(o, blk.backward(s, do, ws=ws)))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    with pytest.raises(la.LAError) as e:
        blk.backward(s, do, ws=torch.empty(256, dtype=torch.uint8, device=_dev()))
    assert e.value.status == 4


def test_a_failed_launch_is_reported_and_the_next_call_works():
    blk = StateSpaceBlock(32, 16, 2, 4)
    ins, do = _step_tensors(blk, B=1, T=300)
    o, s = blk.forward(*ins)
    want = _flat(o, blk.backward(s, do))
    try:
        for after in (0, 1):                    # either launch of the segmented scan
            la.la_debug_fail_launch(after + 1)  # the convolution's passes
            with pytest.raises(la.LAError) as e:
                blk.forward(*ins)
            assert e.value.status == 5 and "injected" in str(e.value)
    finally:
        la.la_debug_fail_launch(-1)
    o, s = blk.forward(*ins)
    for a, b in zip(want, _flat(o, blk.backward(s, do))):
        assert torch.equal(a, b)


def test_binding_refusals():
    x = torch.zeros(2, 4, 8, device=_dev())
    w, f = torch.zeros(8, 4, device=_dev()), torch.zeros(4, device=_dev())
    y = torch.empty_like(x)
    with pytest.raises(ValueError):
        la.la_short_conv_fwd(x, w, y.half())
    with pytest.raises(ValueError):
        la.la_short_conv_fwd(x, w[:, ::2], y)
    with pytest.raises(ValueError):
        la.la_short_conv_fwd(x, w, y, lengths=torch.zeros(2, dtype=torch.int64, device=_dev()))
    with pytest.raises(ValueError):
        la.la_short_conv_fwd(x.transpose(1, 2), w, y)
    with pytest.raises(ValueError):
        la.la_short_conv_fwd(x, w, y, activation="gelu")
    with pytest.raises(TypeError):
        la.la_group_norm_fwd(x.double(), y, 2)
    with pytest.raises(TypeError):
        la.la_group_norm_fwd(x, "y", 2)
    with pytest.raises(la.LAError):
        la.la_short_conv_fwd(x, w, x)                        # in place is refused
    with pytest.raises(la.LAError):
        la.la_group_norm_fwd(x, y, 3)
    q = torch.zeros(1, 2, 3, 8, device=_dev())
    with pytest.raises(ValueError):
        la.la_rotary_fwd(q, q.clone(), torch.empty_like(q), None, f)
    with pytest.raises(ValueError):
        la.la_rotary_fwd(q, None, torch.empty_like(q), None, f, positions=torch.zeros(2, dtype=torch.int64, device=_dev()))
    with pytest.raises(la.LAError):
        la.la_rotary_fwd(q, None, torch.empty_like(q), None, torch.zeros(5, device=_dev()))


# -------------------------------------------------------------------------- the ends of ranges --

def test_steps_of_minus_infinity_skip_tokens_exactly():
    """dt = -inf makes a step of 0: the token neither decays nor feeds the state, bit for bit."""
    n = _normal(40)
    B, T, C, N = 2, 21, 40, 16
    x, dt, Bm, Cm = n(B, T, C), n(B, T, C), n(B, T, 1, N), n(B, T, 1, N)
    A = -torch.exp(n(C, N))
    keep = torch.tensor([t % 3 != 1 for t in range(T)], device=_dev())
    masked = dt.clone()
    masked[:, ~keep] = -math.inf
    y, s, y2, s2 = torch.empty_like(x), torch.empty(B, C, N, device=_dev()), None, torch.empty(B, C, N, device=_dev())
    la.la_selective_scan_fwd(x, masked, A, Bm, Cm, y, state_out=s)
    part = [t[:, keep].contiguous() for t in (x, dt, Bm, Cm)]
    y2 = torch.empty_like(part[0])
    la.la_selective_scan_fwd(part[0], part[1], A, part[2], part[3], y2, state_out=s2)
    assert torch.equal(y[:, keep], y2) and torch.equal(s, s2)
    # and large steps forget everything before them
    big = dt.clone()
    big[:, 10] = 1e4
    la.la_selective_scan_fwd(x, big, A.clamp(max=-1.0), Bm, Cm, y)
    assert torch.isfinite(y).all()
    g = {k: torch.full_like(v, NAN) for k, v in dict(x=x, dt=dt, A=A, Bm=Bm, Cm=Cm).items()}
    la.la_selective_scan_bwd(x, masked, A, Bm, Cm, torch.ones_like(x), g["x"], g["dt"], g["A"], g["Bm"], g["Cm"])
    for t in g.values():
        assert torch.isfinite(t).all()
    assert torch.equal(g["dt"][:, ~keep], torch.zeros_like(g["dt"][:, ~keep]))


def test_infinite_and_nan_values_go_where_the_formula_sends_them():
    n = _normal(41)
    x = n(1, 40, 16)
    x[0, 20, 3] = NAN
    w, y = n(16, 4), torch.empty_like(x)
    la.la_short_conv_fwd(x, w, y, activation="none")
    bad = torch.isnan(y[0])
    assert bad[20:24, 3].all() and int(bad.sum()) == 4
    A, bc = -torch.ones(16, 4, device=_dev()), n(1, 40, 1, 4)
    la.la_selective_scan_fwd(x, n(1, 40, 16), A, bc, bc, y)
    bad = torch.isnan(y[0])
    assert bad[20:, 3].all() and int(bad.sum()) == 20
    la.la_group_norm_fwd(x, y, 4)
    bad = torch.isnan(y[0])
    assert bad[:, :4].all() and int(bad.sum()) == 160


def test_far_positions_keep_their_angle():
    q = _normal(42)(1, 1, 4, 8)
    freqs = torch.tensor([1.0, 0.3, 1e-3, 1e-7], device=_dev())
    pos = torch.tensor([0, 2 ** 31 + 12345, 2 ** 45 + 1, -(2 ** 40)], device=_dev())
    o = torch.empty_like(q)
    la.la_rotary_fwd(q, None, o, None, freqs, positions=pos)
    # 2^45 turns' worth of angle in 64 bits leaves 2^-53 2^45 2 pi = 0.025 of a radian at frequency 1; up
    # to 2^31 it is below fp32's own rounding
    turns = [[p * float(f) for f in freqs] for p in pos.tolist()]
    ang = torch.tensor(turns, dtype=torch.float64, device=_dev())[None, None]
    a, b = q[..., :4].double(), q[..., 4:].double()
    want = torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)
    close(o[:, :, :2], want[:, :, :2], "near", 16, 2.5 * q.abs().max().double())
    err = 2.0 ** -52 * 2 ** 45 * 2
    assert ((o[:, :, 2:].double() - want[:, :, 2:]).abs() <= (err + 1e-6) * 3 * q.abs().max()).all()


def test_offsets_past_two_to_the_31():
    """Tensors of 2^31 elements and more: the last rows against a small call that continues there."""
    C, N, tail = 4096, 16, 64
    T = (1 << 31) // C + 1000
    dev = _dev()
    g = torch.Generator(device="cuda").manual_seed(43)
    x = torch.empty(1, T, C, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    cut = T - tail
    end = x[:, cut:].contiguous()
    n = _normal(44)
    # convolution
    w = n(C, 4, scale=0.5)
    y, so = torch.empty_like(x), torch.empty(1, 3, C, dtype=x.dtype, device=dev)
    la.la_short_conv_fwd(x, w, y, state_out=so)
    y2 = torch.empty_like(end)
    first = x[:, cut - 3:cut].contiguous()
    la.la_short_conv_fwd(end, w, y2, state_in=first)
    assert torch.equal(y[:, cut:], y2) and torch.equal(so, x[:, T - 3:])
    dw = torch.empty_like(w)
    la.la_short_conv_bwd(x, w, x, y, dw)
    d2 = torch.empty_like(end)
    la.la_short_conv_bwd(end, w, end, d2, dw, state_in=first)
    assert torch.equal(y[:, cut:], d2)
    # rotary, the elements as two heads of 128
    heads = x.view(1, 2, T * C // 256, 128)
    f = la.la_rotary_frequencies(128).to(dev)
    ro = y.view(heads.shape)
    la.la_rotary_fwd(heads, None, ro, None, f)
    last = heads[:, :, -tail:].contiguous()
    r2 = torch.empty_like(last)
    la.la_rotary_fwd(last, None, r2, None, f, start=heads.shape[2] - tail)
    assert torch.equal(ro[:, :, -tail:], r2)
    del heads, last
    # scan
    A, dtb = -torch.exp(n(C, N)), n(C) - 2
    Bm, Cm = (n(1, T, 1, N, dtype=torch.bfloat16) for _ in range(2))
    st, st2 = torch.empty(1, C, N, device=dev), torch.empty(1, C, N, device=dev)
    la.la_selective_scan_fwd(x, x, A, Bm, Cm, y, z=x, dt_bias=dtb, state_out=st)
    head = x[:, :cut].contiguous()
    yh = torch.empty_like(head)
    la.la_selective_scan_fwd(head, head, A, Bm[:, :cut].contiguous(), Cm[:, :cut].contiguous(), yh, dt_bias=dtb,
                             state_out=st2)
    del head, yh
    Be, Ce = Bm[:, cut:].contiguous(), Cm[:, cut:].contiguous()
    s3 = st2.clone()
    la.la_selective_scan_fwd(end, end, A, Be, Ce, y2, z=end, dt_bias=dtb, state_in=st2, state_out=s3)
    # the two sides join their segments at other tokens: fp32 roundings of the last few hundred tokens
    close(y[:, cut:], y2.double(), "scan y", 1 << 12, y2.abs().max().double())
    close(st, s3.double(), "scan state", 1 << 12)
    dx, dd = y, torch.empty_like(x)
    gA, gB, gC = torch.empty_like(A), torch.empty_like(Bm), torch.empty_like(Cm)
    la.la_selective_scan_bwd(x, x, A, Bm, Cm, x, dx, dd, gA, gB, gC, dt_bias=dtb)
    ex, ed, eB, eC = torch.empty_like(end), torch.empty_like(end), torch.empty_like(Be), torch.empty_like(Ce)
    la.la_selective_scan_bwd(end, end, A, Be, Ce, end, ex, ed, gA, eB, eC, dt_bias=dtb, state_in=st2)
    for name, a, b in (("dx", dx[:, cut:], ex), ("ddt", dd[:, cut:], ed), ("dB", gB[:, cut:], eB), ("dC", gC[:, cut:], eC)):
        close(a, b.double(), name, 1 << 12, b.abs().max().double())
    del dd
    # group norm: the statistics and the last rows by chunks in 64 bits
    m, r = torch.empty(1, 32, device=dev), torch.empty(1, 32, device=dev)
    la.la_group_norm_fwd(x, y, 32, mean=m, rstd=r)
    s1 = torch.zeros(32, dtype=torch.float64, device=dev)
    s2 = torch.zeros_like(s1)
    for part in x[0].split(32768):
        v = part.double().view(-1, 32, 128)
        s1 += v.sum((0, 2))
        s2 += v.square().sum((0, 2))
    mu = s1 / (T * 128)
    rs = 1 / torch.sqrt(s2 / (T * 128) - mu ** 2 + 1e-5)
    close(m[0], mu, "mean", 200, 1.0)
    close(r[0], rs, "rstd", 400, 1.0)
    want = ((end[0].double().view(-1, 32, 128) - mu[:, None]) * rs[:, None]).view(1, tail, C)
    close(y[:, cut:], want, "norm y", 400, want.abs().max())
    la.la_group_norm_bwd(x, x, y, 32, m, r)
    # dy = x: m0 = mean(x), m1 = mean(x xh)
    m1 = (s2 / (T * 128) - mu ** 2) * rs
    xh = (end[0].double().view(-1, 32, 128) - mu[:, None]) * rs[:, None]
    wd = (rs[:, None] * (end[0].double().view(-1, 32, 128) - mu[:, None] - xh * m1[:, None])).view(1, tail, C)
    close(y[:, cut:], wd, "norm dx", 800, want.abs().max())


def _odd(t):
    """The same values at an address that only one element divides."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:].copy_(t.reshape(-1))
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_addresses_of_one_element_give_the_same_bits(dtype):
    """Narrow accesses change no sum's order in the convolution and the scan."""
    blk = StateSpaceBlock(64, 16, 4, 4)
    ins = blk.inputs(2, 90, dtype)
    x, dt, Bm, Cm, z = ins
    ox, odt, oB, oC, oz = (_odd(t) for t in ins)
    do = _normal(50)(2, 90, 64, dtype=dtype)
    y, y2 = torch.empty_like(x), _odd(torch.empty_like(x))
    la.la_short_conv_fwd(x, blk.w, y, bias=blk.bias)
    la.la_short_conv_fwd(ox, _odd(blk.w), y2, bias=_odd(blk.bias))
    assert torch.equal(y, y2)
    dw, dw2 = torch.empty_like(blk.w), torch.empty_like(blk.w)
    la.la_short_conv_bwd(x, blk.w, do, y, dw)
    la.la_short_conv_bwd(ox, blk.w, _odd(do), y2, dw2)
    assert torch.equal(y, y2) and torch.equal(dw, dw2)
    st, st2 = torch.empty(2, 64, 16, device=_dev()), _odd(torch.empty(2, 64, 16, device=_dev()))
    la.la_selective_scan_fwd(x, dt, blk.A, Bm, Cm, y, z=z, dt_bias=blk.dt_bias, state_out=st)
    la.la_selective_scan_fwd(ox, odt, _odd(blk.A), oB, oC, y2, z=oz, dt_bias=blk.dt_bias, state_out=st2)
    assert torch.equal(y, y2) and torch.equal(st, st2)
    g, g2 = ([torch.empty_like(t) for t in (x, dt, blk.A, Bm, Cm, z, st)] for _ in range(2))
    g2 = [_odd(t) for t in g2]
    la.la_selective_scan_bwd(x, dt, blk.A, Bm, Cm, do, g[0], g[1], g[2], g[3], g[4], z=z, dz=g[5], dt_bias=blk.dt_bias,
                             state_in=st, dstate_out=g[6])
    la.la_selective_scan_bwd(ox, odt, _odd(blk.A), oB, oC, _odd(do), g2[0], g2[1], g2[2], g2[3], g2[4], z=oz, dz=g2[5],
                             dt_bias=blk.dt_bias, state_in=st2, dstate_out=g2[6])
    for a, b in zip(g, g2):
        assert torch.equal(a, b)
    # one token
    tok = [t[:, 0].contiguous() for t in ins]
    o, o2 = torch.empty_like(tok[0]), _odd(torch.empty_like(tok[0]))
    s, s2 = st.clone(), _odd(st)
    la.la_selective_scan_step(tok[0], tok[1], blk.A, tok[2], tok[3], o, s, z=tok[4])
    t2 = [_odd(t) for t in tok]
    la.la_selective_scan_step(t2[0], t2[1], _odd(blk.A), t2[2], t2[3], o2, s2, z=t2[4])
    assert torch.equal(o, o2) and torch.equal(s, s2)
