"""The layer operators on the GPU against their fp64 definitions.

Every element is held to |got - want| <= u |want| + c 2^-24 M, where u = eps/2
of the output's type (one rounding; 0 for fp32, whose last rounding is in c),
M is the sum of the absolute values of the element's terms (oracle) and c
counts the fp32 roundings on the way:

  conv    W + 1 terms, SiLU's exponential and division (|p| <= 8 here: 2 + 1.2
          |p| and 2 units of 2^-23 each, twice for the derivative): c = 64;
          sums over tokens (dw, dbias) add at most 64 + 4 + 8 additions and
          one for each eighth block: c = 64 + 2 * 64
  scan    a step's factor is off by (3 |dt' A| + 4) units (argument, 2-ulp
          exponential) and its input by about 16 (softplus, products); errors
          add up over at most T steps: c = 64 + (7 + 3 X) T with X the largest |dt' A|;
          the backward pass goes through the recurrence twice, and sums over
          channels or tokens add at most another 64
  qk_norm a sum of at most 256 squares in 8 + 5 levels, root, division, an
          angle's sine (pi units of 2^-24 and 2 ulp), products: c = 64; backward
          twice that; dw sums over n rows in parts: c = 128 + rows / 16
"""
import math

import pytest
import torch

import delta_rule_linear_kla_b200 as K
from delta_rule_linear_kla_b200 import api
from helpers import Padded
from oracle import layer_ops as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24


def check(got, want, c, what=""):
    v, m = want
    assert got.shape == v.shape, (what, got.shape, v.shape)
    u = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    # 1e-37: results below fp32's normal range may be flushed
    bar = u * v.abs() + c * U * m * (1 + u) + 1e-37
    err = (got.double().cpu() - v).abs()
    bad = ~(err <= bar)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError((what, int(bad.sum()), at, float(got[at]), float(v[at]),
                              float((err / bar).nan_to_num(1e9).max())))


class Rand:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def n(self, *s, dt=torch.float32, scale=1.0):
        return (torch.randn(s, generator=self.g) * scale).to(dt)


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def wide(t, before, after):
    """t as the middle columns of a wider matrix (same values)."""
    lead = t.shape[:2]
    flat = t.reshape(*lead, -1)
    w = torch.full((*lead, before + flat.shape[-1] + after), float("nan"), dtype=t.dtype,
                   device=t.device)
    w[..., before:before + flat.shape[-1]] = flat
    return w[..., before:before + flat.shape[-1]].unflatten(-1, t.shape[2:])


# ------------------------------------------------------------- convolution

CONV = [  # B, T, D, W, dtype, silu, bias, state, lengths, wide
    (2, 1, 64, 4, "bf16", True, True, True, None, False),
    (1, 2, 7, 4, "fp32", True, False, True, None, False),
    (3, 3, 1, 2, "bf16", False, True, False, [3, 0, 1], False),
    (2, 5, 8, 4, "bf16", True, True, True, [2, 5], True),
    (2, 67, 40, 3, "fp32", True, True, True, [67, 1], True),
    (1, 300, 136, 4, "bf16", True, False, False, None, True),
    (3, 130, 33, 2, "fp32", False, True, True, [130, 64, 0], False),
    (1, 1037, 24, 4, "bf16", True, True, True, None, False),
    (2, 260, 100, 4, "bf16", True, True, True, [-3, 999], False),  # clamped to 0 and T
    (1, 9, 257, 4, "bf16", True, True, True, None, True),  # odd rows of a wide matrix
]


def conv_case(case, seed):
    B, T, D, W, dt, silu, bias, state, lengths, w_ = case
    r = Rand(seed)
    t = DT[dt]
    x, w = r.n(B, T, D, dt=t), r.n(D, W, scale=0.5)
    b = r.n(D) if bias else None
    s0 = r.n(B, W - 1, D, dt=t) if state else None
    gy, gs = r.n(B, T, D, dt=t), r.n(B, W - 1, D, dt=t) if state else None
    if lengths is not None:  # whatever lies behind a sequence's end is not read
        for i, n in enumerate(lengths):
            x[i, max(n, 0):] = float("nan")
            gy[i, max(n, 0):] = float("inf")
    return x, w, b, s0, gy, gs, None if lengths is None else torch.tensor(lengths,
                                                                          dtype=torch.int32)


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_forward(case):
    x, w, b, s0, _, _, n = conv_case(case, 10)
    B, T, D, W, dt, silu = case[:6]
    xg, wg, bg, sg, ng = gpu(x, w, b, s0, n)
    if case[9]:
        xg = wide(xg, 16, 8)
    y, sT = Padded((B, T, D), DT[dt], "cuda"), Padded((B, W - 1, D), DT[dt], "cuda")
    api.conv_fwd(xg, wg, bg, sg, silu=silu, lengths=ng, y=y.t, sT=sT.t)
    want = ref.conv(x, w, b, s0, silu, case[8])
    check(y.t, want["y"], 64, "y")
    assert torch.equal(sT.t.double().cpu(), want["sT"][0])  # copied, not computed
    assert y.intact() and sT.intact()


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_backward(case):
    x, w, b, s0, gy, gs, n = conv_case(case, 11)
    B, T, D, W, dt, silu = case[:6]
    xg, wg, bg, sg, ng, gyg, gsg = gpu(x, w, b, s0, n, gy, gs)
    if case[9]:
        xg = wide(xg, 8, 16)
    got = api.conv_bwd(xg, wg, gyg, bg, sg, gsg, silu=silu, lengths=ng)
    want = ref.conv_bwd(x, w, gy, b, s0, gs, silu, case[8])
    for k in ("dx", "ds0"):
        check(got[k], want[k], 64, k)
    for k in ("dw", "dbias"):
        if got[k] is not None:
            check(got[k], want[k], 192, k)
    again = api.conv_bwd(xg, wg, gyg, bg, sg, gsg, silu=silu, lengths=ng)
    assert all(got[k] is None or torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D,W", [(64, 4), (33, 3), (12, 2)])
def test_conv_steps_are_the_prompt(dt, D, W):
    """Token by token from the prompt's state: the same bits as the prompt."""
    r = Rand(12)
    x, w, b = gpu(r.n(3, 9, D, dt=DT[dt]), r.n(D, W), r.n(D))
    y, sT = api.conv_fwd(x, w, b)
    y0, s = api.conv_fwd(x[:, :4].contiguous(), w, b)
    rest = [api.conv_step(x[:, t], w, s, b) for t in range(4, 9)]  # x[:, t]: rows of a matrix
    assert torch.equal(torch.cat([y0, torch.stack(rest, 1)], 1), y)
    assert torch.equal(s, sT)


# -------------------------------------------------------------------- scan

SSM = [  # B, T, D, G, N, dtype, z, skip, bias, softplus, state, lengths, wide
    (1, 1, 8, 1, 16, "bf16", True, True, True, True, True, None, False),
    (2, 2, 5, 1, 8, "fp32", True, False, False, True, False, None, False),
    (2, 17, 24, 2, 16, "bf16", True, True, True, True, True, [17, 3], True),
    (1, 33, 130, 1, 32, "fp32", False, True, True, False, True, None, False),
    (3, 64, 12, 4, 64, "bf16", True, True, True, True, False, [64, 0, 31], False),
    (1, 95, 66, 1, 64, "fp32", True, False, True, True, True, None, True),
    (2, 100, 200, 1, 16, "fp32", True, True, True, True, True, [100, 49], False),
    (1, 130, 300, 2, 8, "bf16", True, True, False, True, True, None, True),
    (2, 8, 129, 1, 16, "bf16", True, True, True, True, True, None, False),  # 2 tiles and 1
    (2, 9, 65, 1, 8, "bf16", True, True, True, True, True, [9, 8], False),
    (1, 40, 6, 6, 16, "fp32", False, True, True, True, True, None, False),  # groups of one
    (1, 41, 33, 1, 32, "bf16", True, True, True, True, True, None, True),
    (1, 1300, 10, 1, 16, "fp32", True, True, True, True, True, None, False),   # segments
    (2, 1100, 6, 2, 8, "bf16", True, True, True, True, True, [1100, 700], False),
    (3, 1100, 6, 1, 16, "fp32", True, True, True, True, True, [90, 0, 641], False),  # segments
    # without a token
]


def ssm_case(case, seed):
    B, T, D, G, N, dt, z, skip, bias, softplus, state, lengths, _ = case
    r = Rand(seed)
    t = DT[dt]
    a = dict(u=r.n(B, T, D, dt=t), Bm=r.n(B, T, G, N, dt=t), Cm=r.n(B, T, G, N, dt=t),
             A=-torch.arange(1, N + 1).float() * torch.exp(r.n(D, N, scale=0.2)),
             D=r.n(D) if skip else None, z=r.n(B, T, D, dt=t) if z else None,
             # without the softplus the step itself has to stay positive: e^{-dt' N}
             # of a negative one leaves fp32's range within a few tokens
             dt_bias=None if not bias else r.n(D, scale=0.5) - 3 if softplus
             else 0.01 * r.n(D).abs(),
             h0=r.n(B, D, N) if state else None)
    a["dt"] = (r.n(B, T, D) - (0 if bias else 3)) if softplus \
        else 0.05 * torch.exp(r.n(B, T, D))
    a["dt"] = a["dt"].to(t)
    gy, gh = r.n(B, T, D, dt=t), r.n(B, D, N) if state else None
    if lengths is not None:
        for i, n in enumerate(lengths):
            for k in ("u", "dt", "Bm", "Cm", "z"):
                if a[k] is not None:
                    a[k][i, n:] = float("nan")
            gy[i, n:] = float("inf")
    X = 1.0
    raw = a["dt"].float() + (0 if a["dt_bias"] is None else a["dt_bias"])
    s = torch.nn.functional.softplus(raw) if softplus else raw
    X = float((s.nan_to_num(0.0).amax((0, 1))[:, None] * a["A"].abs()).max())
    c = 64 + (7 + 3 * X) * T
    return a, gy, gh, None if lengths is None else torch.tensor(lengths, dtype=torch.int32), c


def ssm_gpu(a, widen):
    g = {k: None if v is None else v.cuda() for k, v in a.items()}
    if widen:
        for k, (lo, hi) in {"u": (8, 8), "z": (24, 0), "Bm": (4, 12), "Cm": (16, 3)}.items():
            if g[k] is not None and k != "u":
                g[k] = wide(g[k], lo // 8 * 8, hi)
    return g


@pytest.mark.parametrize("case", SSM, ids=str)
def test_ssm_forward(case):
    a, _, _, n, c = ssm_case(case, 20)
    B, T, D, G, N, dt = case[:6]
    g = ssm_gpu(a, case[12])
    y, hT = Padded((B, T, D), DT[dt], "cuda"), Padded((B, D, N), torch.float32, "cuda")
    api.ssm_fwd(**g, softplus=case[9], lengths=None if n is None else n.cuda(), y=y.t, hT=hT.t)
    want = ref.ssm(**a, softplus=case[9], lengths=case[11])
    check(y.t, want["y"], c, "y")
    check(hT.t, want["hT"], c, "hT")
    assert y.intact() and hT.intact()
    if g["h0"] is not None:  # the state in place
        h = g["h0"].clone()
        y2, _ = api.ssm_fwd(**dict(g, h0=h), softplus=case[9],
                            lengths=None if n is None else n.cuda(), hT=h)
        assert torch.equal(y2, y.t) and torch.equal(h, hT.t)


@pytest.mark.parametrize("case", SSM, ids=str)
def test_ssm_backward(case):
    a, gy, gh, n, c = ssm_case(case, 21)
    g = ssm_gpu(a, case[12])
    kw = dict(softplus=case[9], lengths=None if n is None else n.cuda())
    args = (g["u"], g["dt"], g["A"], g["Bm"], g["Cm"], gy.cuda(), g["D"], g["z"], g["dt_bias"],
            g["h0"], None if gh is None else gh.cuda())
    got = api.ssm_bwd(*args, **kw)
    want = ref.ssm_bwd(a["u"], a["dt"], a["A"], a["Bm"], a["Cm"], gy, a["D"], a["z"],
                       a["dt_bias"], a["h0"], gh, case[9], case[11])
    for k, v in got.items():
        if v is not None:
            check(v, want[k], 2 * c + 128, k)
    again = api.ssm_bwd(*args, **kw)
    assert all(v is None or torch.equal(v, again[k]) for k, v in got.items())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D,G,N", [(5, 1, 8), (66, 2, 16), (130, 1, 64), (33, 1, 32)])
def test_ssm_steps_follow_the_prompt(dt, D, G, N):
    case = (3, 12, D, G, N, dt, True, True, True, True, True, None, False)
    a, _, _, _, c = ssm_case(case, 22)
    g = ssm_gpu(a, False)
    want = ref.ssm(**a)
    cut = {k: (v[:, :7].contiguous() if k in ("u", "dt", "Bm", "Cm", "z") else v)
           for k, v in g.items()}
    _, S = api.ssm_fwd(**cut)
    for t in range(7, 12):
        y = api.ssm_step(g["u"][:, t], g["dt"][:, t], g["A"], g["Bm"][:, t], g["Cm"][:, t], S,
                         g["D"], g["z"][:, t], g["dt_bias"])
        check(y, tuple(v[:, t] for v in want["y"]), c, t)
    check(S, want["hT"], c, "state")


def test_ssm_extreme_steps():
    """A step of 0 keeps the state to the bit, one so large that every decay
    is 0 leaves only the token's own input, and far-out raw steps pass the
    softplus without overflow."""
    B, T, D, N = 1, 40, 16, 16
    r = Rand(23)
    u, Bm, Cm, h0 = gpu(r.n(B, T, D), r.n(B, T, 1, N), r.n(B, T, 1, N), r.n(B, D, N))
    A = -torch.ones(D, N, device="cuda")
    dt = torch.full((B, T, D), -200.0, device="cuda")
    _, h = api.ssm_fwd(u, dt, A, Bm, Cm, h0=h0)
    assert torch.equal(h, h0)
    dt[:, -1] = 1000.0
    y, h = api.ssm_fwd(u, dt, A, Bm, Cm, h0=h0)
    own = 1000.0 * u[:, -1, :, None] * Bm[:, -1]
    assert torch.allclose(h, own, rtol=1e-6) and torch.isfinite(y).all()


def test_ssm_growth_leaves_zeros():
    """A growing channel (A > 0) whose states are still 0 when the growth of
    the segments before passes fp32's range (e^128 and more): the state is that
    of the late input, as without a cut.  The gradients of the last tokens and
    of C are finite too; earlier ones are not (the adjoint state itself passes
    e^1000 there)."""
    B, T, D, N = 1, 2000, 16, 8
    assert api.ssm_fwd_workspace_size(B, T, D, 1, N) > 0  # cut into segments
    u = torch.zeros(B, T, D, device="cuda")
    u[:, -3:] = 1.0
    dt = torch.ones((B, T, D), device="cuda")
    A = torch.ones(D, N, device="cuda")
    bc = torch.ones(B, T, 1, N, device="cuda")
    y, h = api.ssm_fwd(u, dt, A, bc, bc, softplus=False)
    want = sum(math.exp(i) for i in range(3))
    assert not y[:, :-3].any()
    assert torch.allclose(h, torch.full_like(h, want), rtol=1e-6)
    gy = torch.zeros_like(y)
    gy[:, -1] = 1.0
    g = api.ssm_bwd(u, dt, A, bc, bc, gy, softplus=False)
    du = [N * math.exp(i) for i in (2, 1, 0)]
    assert torch.allclose(g["du"][0, -3:, 0].cpu(), torch.tensor(du), rtol=1e-6)
    assert torch.allclose(g["dC"][0, -1], torch.full_like(g["dC"][0, -1], D * want), rtol=1e-6)
    assert not g["dC"][:, :-1].any()


@pytest.mark.parametrize("B,T,D,N,lens", [(2, 37, 70, 16, [37, 5]), (1, 2000, 16, 8, [1990])])
def test_ssm_states_without_memory(B, T, D, N, lens):
    """A = -inf (a decay of 0 after every step) is the A whose decay underflows:
    the places behind the last token keep the state, in both directions."""
    r = Rand(24)
    u, dt, z, gy = (r.n(B, T, D) for _ in range(4))
    A = -0.5 - r.n(D, N).abs()
    Bm, Cm = r.n(B, T, 1, N), r.n(B, T, 1, N)
    x = gpu(u, dt, A, Bm, Cm, gy, z)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = {}
    for a in (-1e30, -math.inf):
        x[2][::3, ::2] = a
        y, h = api.ssm_fwd(*x[:5], z=x[6], lengths=n)
        state = h.clone()
        one = api.ssm_step(x[0][:, 0], x[1][:, 0], x[2], x[3][:, 0], x[4][:, 0], state)
        grads = api.ssm_bwd(*x[:6], z=x[6], lengths=n)
        got[a] = dict(grads, y=y, h=h, one=one, state=state)
    for name, v in got[-1e30].items():
        if v is not None:
            assert v.isfinite().all(), name
            assert torch.equal(v, got[-math.inf][name]), name


# ------------------------------------------------------- norm and rotation

QK = [  # B, T, Hq, Hk, d, rot, dtype, norm, weight, interleaved, first position, wide
    (2, 1, 1, 1, 64, 64, "bf16", "l2", False, False, 5, False),
    (1, 7, 5, 1, 128, 64, "bf16", "rms", True, False, 0, True),
    (2, 33, 4, 2, 64, 64, "bf16", "rms", True, True, 100, True),
    (1, 50, 3, 3, 80, 40, "fp32", "rms", True, False, 1000000, False),
    (1, 50, 3, 3, 80, 36, "fp32", "l2", False, False, 131071, False),  # pairs across lanes
    (2, 20, 8, 4, 96, 0, "bf16", "l2", False, False, 0, False),
    (1, 19, 2, 2, 256, 256, "fp32", None, False, True, 3, False),
    (1, 200, 1, 0, 8, 8, "fp32", "rms", True, False, 0, False),
    (1, 3, 300, 7, 32, 6, "bf16", "l2", False, True, 9, False),
]


def qk_case(case, seed):
    B, T, Hq, Hk, d, rot, dt, norm, weight, inter, first, w_ = case
    r = Rand(seed)
    t = DT[dt]
    q, k = r.n(B, T, Hq, d, dt=t), r.n(B, T, Hk, d, dt=t)
    q[:, 0, 0] = 0  # a head of zeros stays zeros
    wq, wk = (r.n(d), r.n(d)) if weight else (None, None)
    f = 10000.0 ** (-torch.arange(rot // 2) * 2.0 / rot) if rot else None
    pos = (first + torch.arange(B * T).reshape(B, T) * 3).int()
    gq, gk = r.n(B, T, Hq, d, dt=t), r.n(B, T, Hk, d, dt=t)
    kw = dict(norm=norm, interleaved=inter, scale=1.25 if rot else 1.0)
    return q, k, wq, wk, f, pos, gq, gk, kw


@pytest.mark.parametrize("case", QK, ids=str)
def test_qk_norm(case):
    q, k, wq, wk, f, pos, gq, gk, kw = qk_case(case, 30)
    q_, k_, wqg, wkg, fg, pg, gqg, gkg = gpu(q, k, wq, wk, f, pos, gq, gk)
    if case[11]:
        q_, k_ = wide(q_, 8, 16), wide(k_, 0, 8)
    more = dict(wq=wqg, wk=wkg, positions=pg, inv_freq=fg, **kw)
    oq, ok = Padded(q.shape, q.dtype, "cuda"), Padded(k.shape, k.dtype, "cuda")
    api.qk_norm_fwd(q_, k_, oq=oq.t, ok=ok.t, **more)
    for got, x, w in ((oq, q, wq), (ok, k, wk)):
        check(got.t, ref.head_norm(x, w, pos, f, **kw), 64)
        assert got.intact()
    r = api.qk_norm_bwd(q_, k_, gqg, gkg, **more)
    for x, g, w, n in ((q, gq, wq, "q"), (k, gk, wk, "k")):
        want = ref.head_norm_bwd(x, g, w, pos, f, **kw)
        check(r["d" + n], want["dx"], 128, "d" + n)
        if w is not None:
            check(r["dw" + n], want["dw"], 128 + x[..., 0].numel() / 16, "dw" + n)


def test_qk_norm_positions():
    """No positions count from pos0, one row serves all sequences, and one
    token of each sequence is the prompt of length 1."""
    r = Rand(31)
    q, k = gpu(r.n(2, 9, 2, 64), r.n(2, 9, 1, 64))
    f = (10000.0 ** (-torch.arange(16) / 16.0)).cuda()
    pos = torch.arange(40, 49, dtype=torch.int32, device="cuda")
    a = api.qk_norm_fwd(q, k, inv_freq=f, pos0=40)
    b = api.qk_norm_fwd(q, k, inv_freq=f, positions=pos)
    c = api.qk_norm_fwd(q, k, inv_freq=f, positions=pos.expand(2, 9).contiguous())
    one = api.qk_norm_fwd(q[:, 3], k[:, 3], inv_freq=f, positions=pos[3:4].expand(2).contiguous())
    part = api.qk_norm_fwd(q[:, 2:5].contiguous(), k[:, 2:5].contiguous(), inv_freq=f,
                           positions=pos[2:5])  # not 16-byte aligned
    for i in range(2):
        assert torch.equal(a[i], b[i]) and torch.equal(a[i], c[i])
        assert torch.equal(one[i], a[i][:, 3]) and torch.equal(part[i], a[i][:, 2:5])
    with pytest.raises(ValueError, match="32 bits"):
        api.qk_norm_fwd(q, k, inv_freq=f, pos0=2**31 - 4)
    a = api.qk_norm_fwd(q, k, inv_freq=f, pos0=2**31 - 9)
    pos = (2**31 - 9 + torch.arange(9)).expand(2, 9)
    # the fp64 product of a 31-bit position and a 24-bit frequency is off by
    # 2^-53 of up to 2^31 radians, 2^-22: 4 units beside the c = 64
    check(a[0], ref.head_norm(q, None, pos, f), 68)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rot,interleaved", [(16, False), (12, False), (20, True)])
def test_channels_that_are_not_turned_stay(rot, interleaved, dt):
    """Without a norm, channels behind the rotation come out unchanged, in
    both directions: infinities and NaN too, and none reaches a neighbour."""
    r = Rand(32)
    q, g = r.n(2, 5, 3, 64, dt=DT[dt]), r.n(2, 5, 3, 64, dt=DT[dt])
    for x in (q, g):
        x[:, :, 0, rot], x[:, 1, :, rot + 3], x[0, 2, :, 40] = math.inf, -math.inf, math.nan
    q, g = gpu(q, g)
    f = (10000.0 ** (-torch.arange(rot // 2) * 2.0 / rot)).cuda()
    kw = dict(norm=None, inv_freq=f, interleaved=interleaved)
    out = api.qk_norm_fwd(q, q.clone(), **kw)
    grads = api.qk_norm_bwd(q, q.clone(), g, g.clone(), **kw)
    for got, x in ((out[0], q), (out[1], q), (grads["dq"], g), (grads["dk"], g)):
        assert torch.equal(got[..., rot:].nan_to_num(7.0), x[..., rot:].nan_to_num(7.0))
        assert torch.equal(got[..., rot:].isnan(), x[..., rot:].isnan())
        assert got[..., :rot].isfinite().all()


# ------------------------------------------------ gradients through autograd

def _differences(loss, leaves, seed, h=2.0 ** -6):
    """<gradient, direction> against the central difference of the fp32 loss:
    truncation about h^2 / 6 of the third derivative, rounding about 2^-24 /
    h of the loss's terms: 2e-3 of the scale covers both."""
    total = loss(leaves)
    grads = torch.autograd.grad(total, list(leaves.values()))
    r = torch.Generator(device="cuda").manual_seed(seed)
    for (name, x), g in zip(leaves.items(), grads):
        d = torch.randn(x.shape, generator=r, device="cuda")
        d = d / d.norm() * x.detach().norm().clamp(min=1.0)
        with torch.no_grad():
            up = loss(dict(leaves, **{name: x + h * d}))
            dn = loss(dict(leaves, **{name: x - h * d}))
        want, got = float(up - dn) / (2 * h), float((g * d).sum())
        scale = float((g.norm() * d.norm())) + 1e-3
        assert abs(got - want) <= 2e-3 * scale + 1e-4, (name, got, want, scale)


def test_layer_gradients_against_differences():
    """conv -> norm -> gated delta prefill's inputs, and conv -> scan, as
    layers: autograd's gradients agree with differences of the loss."""
    r = Rand(40)
    B, T, D, N = 2, 37, 64, 16
    leaf = lambda *s, scale=1.0: r.n(*s, scale=scale).cuda().requires_grad_(True)  # noqa: E731
    co = r.n(B, T, D).cuda()
    x = dict(x=leaf(B, T, D), w=leaf(D, 4, scale=0.5), b=leaf(D, scale=0.3),
             dt=leaf(B, T, D, scale=0.5), A=(-torch.rand(D, N).cuda() - 0.5).requires_grad_(True),
             Bm=leaf(B, T, 1, N), Cm=leaf(B, T, 1, N), Dw=leaf(D), z=leaf(B, T, D),
             bias=(leaf(D).detach() * 0.2 - 2).requires_grad_(True), h0=leaf(B, D, N))

    def scan_layer(v):
        u, _ = K.kla_conv(v["x"], v["w"], v["b"])
        y, h = K.kla_ssm(u, v["dt"], v["A"], v["Bm"], v["Cm"], v["Dw"], v["z"], v["bias"],
                         v["h0"])
        return (y * co).sum() / 8 + 0.1 * h.square().sum() / 8
    _differences(scan_layer, x, 41)

    H, d = 2, 32
    f = (100.0 ** (-torch.arange(8) / 8.0)).cuda()
    y = dict(q=leaf(B, T, H, d), k=leaf(B, T, 1, d), wq=leaf(d), wk=leaf(d))
    cq, ck = r.n(B, T, H, d).cuda(), r.n(B, T, 1, d).cuda()

    def norm_layer(v):
        oq, ok = K.kla_qk_norm(v["q"], v["k"], wq=v["wq"], wk=v["wk"], inv_freq=f, norm="rms")
        return ((oq * cq).sum() + (ok * ck).sum()) / 8
    _differences(norm_layer, y, 42)


def test_autograd_of_wide_and_unused_inputs():
    """A gradient reaches the matrix that x, z, B and C are columns of, and an
    output that nothing uses adds nothing."""
    r = Rand(43)
    B, T, D, N = 2, 19, 32, 8
    xz = r.n(B, T, 2 * D).cuda().requires_grad_(True)
    bc = r.n(B, T, 2 * N).cuda().requires_grad_(True)
    w, A = r.n(D, 4).cuda(), -torch.rand(D, N).cuda()
    dt = r.n(B, T, D).cuda()

    def run(cat):
        x, z = (xz[..., :D], xz[..., D:]) if not cat else (xz[..., :D].contiguous(),
                                                           xz[..., D:].contiguous())
        u, _ = K.kla_conv(x, w)
        Bm, Cm = bc[..., :N].unflatten(-1, (1, N)), bc[..., N:].unflatten(-1, (1, N))
        y, _ = K.kla_ssm(u, dt, A, Bm, Cm, z=z)
        return torch.autograd.grad(y.square().sum(), [xz, bc])
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b) and a.abs().sum() > 0


# ------------------------------------------------------- used together

@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_delta_layer_prompt_then_tokens(dt):
    """A gated delta layer: convolution and SiLU, L2 norm and rotation,
    recurrence.  The prompt of T tokens gives what a shorter prompt and then
    single tokens give (same conv bits; the recurrence within its bars)."""
    r = Rand(50)
    B, T, H, d, cut, W = 2, 70, 2, 64, 64, 4
    D = H * d
    t = DT[dt]
    x, w = gpu(r.n(B, T, 2 * D, dt=t), r.n(2 * D, W, scale=0.5))
    v, g, beta = gpu(r.n(B, T, H, d, dt=t), -torch.rand(B, T, H) * 0.1, torch.rand(B, T, H))
    f = (10000.0 ** (-torch.arange(16) / 16.0)).cuda()

    def prompt(n):
        c, s = api.conv_fwd(x[:, :n].contiguous(), w)
        q, k = api.qk_norm_fwd(c[..., :D].unflatten(-1, (H, d)), c[..., D:].unflatten(-1, (H, d)),
                               inv_freq=f)
        sl = lambda a: a[:, :n].contiguous()  # noqa: E731
        o, S = api.gdn_chunk_fwd(q, k, sl(v), sl(g), sl(beta))
        return o, S, s
    o_all, S_all, s_all = prompt(T)
    _, S, s = prompt(cut)
    for i in range(cut, T):
        c = api.conv_step(x[:, i], w, s)
        pos = torch.full((B,), i, dtype=torch.int32, device="cuda")
        q, k = api.qk_norm_fwd(c[:, :D].unflatten(-1, (H, d)), c[:, D:].unflatten(-1, (H, d)),
                               inv_freq=f, positions=pos)
        o = api.gdn_decode_step(q, k, v[:, i].contiguous(), g[:, i].contiguous(),
                                beta[:, i].contiguous(), S)
        bar = 1e-2 if dt == "bf16" else 1e-4
        assert (o.float() - o_all[:, i].float()).norm() <= 2 * bar * o_all[:, i].float().norm()
    assert torch.equal(s, s_all)
    assert (S - S_all).norm() <= 2 * bar * S_all.norm()


def test_streams_and_graphs():
    """On a stream of the caller's, and captured: two graphs of the same
    calls, replayed in turn on new inputs, give what plain calls give."""
    r = Rand(51)
    B, T, D, N = 1, 1200, 48, 16  # few channels: the scan is cut into segments
    assert api.ssm_fwd_workspace_size(B, T, D, 1, N) > 0
    w, A = r.n(D, 4).cuda(), -torch.rand(D, N).cuda()
    make = lambda: [r.n(B, T, D).cuda(), r.n(B, T, D).cuda() - 2, r.n(B, T, 1, N).cuda(),  # noqa: E731
                    r.n(B, T, 1, N).cuda(), r.n(B, T, D).cuda()]

    def calls(x, dt, Bm, Cm, gy, stream=None):
        u, _ = api.conv_fwd(x, w, stream=stream)
        y, h = api.ssm_fwd(u, dt, A, Bm, Cm, z=x, stream=stream)
        gr = api.ssm_bwd(u, dt, A, Bm, Cm, gy, z=x, stream=stream)
        gc = api.conv_bwd(x, w, gr["du"], stream=stream)
        q, k = api.qk_norm_fwd(u.view(B, T, 2, 24), gr["du"].view(B, T, 2, 24), stream=stream)
        return [u, y, h, q, k] + [gr[n] for n in ("du", "ddt", "dA", "dB", "dC", "dz")] \
            + [gc["dx"], gc["dw"]]
    ins = make()
    want = calls(*ins)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = calls(*ins, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        hold = [t.clone() for t in ins]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = calls(*hold)
        graphs.append((g, hold, out))
    for turn in range(4):
        new = make()
        g, hold, out = graphs[turn % 2]
        for h, n in zip(hold, new):
            h.copy_(n)
        g.replay()
        want = calls(*new)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), turn


def test_training_step_captured_while_an_eager_graph_lives():
    """Forward and backward captured through autograd replay the eager
    gradients, with an eager graph of the same parameters still alive.  The
    captured pass has leaves of its own (detached aliases of the parameters):
    autograd ties a leaf's gradient to the stream of the first graph that uses
    it, which a capture cannot wait for."""
    r = Rand(52)
    B, T, D, N = 2, 40, 32, 8
    x, dt, Bm, Cm, gy = gpu(r.n(B, T, D), r.n(B, T, D), r.n(B, T, 1, N), r.n(B, T, 1, N),
                            r.n(B, T, D))
    w = r.n(D, 4).cuda().requires_grad_(True)
    A = (-torch.rand(D, N).cuda()).requires_grad_(True)

    def grads(w, A):
        u, _ = K.kla_conv(x, w)
        q, _ = K.kla_qk_norm(u.view(B, T, 1, D), u.view(B, T, 1, D))
        y, _ = K.kla_ssm(q.view(B, T, D), dt, A, Bm, Cm)
        return torch.autograd.grad(y, [w, A], gy, retain_graph=True), y
    want, alive = grads(w, A)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        own = [p.detach().requires_grad_(True) for p in (w, A)]
        grads(*own)
    torch.cuda.current_stream().wait_stream(side)
    own = [p.detach().requires_grad_(True) for p in (w, A)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, _ = grads(*own)
    for _ in range(2):
        with torch.no_grad():
            w *= 0.5  # the aliases share the parameters' memory
        g.replay()
    torch.cuda.synchronize()
    assert alive.grad_fn is not None
    again, _ = grads(w, A)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert not torch.equal(got[0], want[0])


def test_empty_prompts():
    D, N = 16, 8
    x = torch.empty(2, 0, D, device="cuda")
    s0, h0 = torch.randn(2, 3, D, device="cuda"), torch.randn(2, D, N, device="cuda")
    w, A = torch.randn(D, 4, device="cuda"), -torch.rand(D, N, device="cuda")
    bc = torch.empty(2, 0, 1, N, device="cuda")
    y, s = api.conv_fwd(x, w, None, s0)
    assert y.shape == x.shape and torch.equal(s, s0)
    y, h = api.ssm_fwd(x, x, A, bc, bc, h0=h0)
    assert y.shape == x.shape and torch.equal(h, h0)
    _, h = api.ssm_fwd(x, x, A, bc, bc)
    assert not h.any()
    g = api.ssm_bwd(x, x, A, bc, bc, x, h0=h0, grad_hT=h0)
    assert not g["dA"].any() and torch.equal(g["dh0"], h0)
    g = api.conv_bwd(x, w, x, None, s0, s0)
    assert not g["dw"].any() and torch.equal(g["ds0"], s0)
    q = torch.empty(2, 0, 1, 64, device="cuda")
    w64 = torch.ones(64, device="cuda")
    r = api.qk_norm_bwd(q, q, q, q, wq=w64, norm="rms")
    assert not r["dwq"].any() and r["dq"].shape == q.shape


def test_offsets_past_32_bits():
    """More than 2^31 elements an activation: the last tokens are those of a
    short prompt that starts from what stands before them."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    T, D, N, tail = (1 << 20) + 100, 2048, 8, 300
    gen = torch.Generator(device="cuda").manual_seed(60)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x, w = mk(1, T, D), torch.randn(D, 4, generator=gen, device="cuda")
    assert x.numel() > 1 << 31
    cut = lambda a: a[:, -tail:].contiguous()  # noqa: E731
    y, sT = api.conv_fwd(x, w)
    s0 = x[:, -tail - 3:-tail].contiguous()
    yt, st = api.conv_fwd(cut(x), w, None, s0)
    assert torch.equal(y[:, -tail:], yt) and torch.equal(sT, st)
    del y
    g = api.conv_bwd(x, w, x)
    gt = api.conv_bwd(cut(x), w, cut(x), None, s0)
    assert torch.equal(g["dx"][:, -tail:], gt["dx"])
    del g
    # decays of e^-4 a token: 300 tokens before nothing is left
    A = torch.full((D, N), -8.0, device="cuda")
    dt = torch.full((1, T, D), 0.5, device="cuda", dtype=torch.bfloat16)
    bc = mk(1, T, 1, N)
    args = lambda f: (f(x), f(dt), A, f(bc), f(bc))  # noqa: E731
    y, h = api.ssm_fwd(*args(lambda a: a), softplus=False)
    yt, ht = api.ssm_fwd(*args(cut), softplus=False)
    assert torch.equal(y[:, -50:], yt[:, -50:]) and torch.equal(h, ht)
    del y
    g = api.ssm_bwd(*args(lambda a: a), x, softplus=False)
    gt = api.ssm_bwd(*args(cut), cut(x), softplus=False)
    for k in ("du", "ddt", "dB", "dC"):
        assert torch.equal(g[k][:, -50:], gt[k][:, -50:]), k
    del g, dt, bc
    q, k = x.view(1, T, 16, 128), x.view(1, T, 16, 128)[:, :, :1].contiguous()
    f = (10000.0 ** (-torch.arange(64) / 64.0)).cuda()
    oq, ok = api.qk_norm_fwd(q, k, inv_freq=f)
    tq, tk = api.qk_norm_fwd(cut(q), cut(k), inv_freq=f, pos0=T - tail)
    assert torch.equal(oq[:, -tail:], tq) and torch.equal(ok[:, -tail:], tk)
    del oq
    g = api.qk_norm_bwd(q, k, q, k, inv_freq=f)
    gt = api.qk_norm_bwd(cut(q), cut(k), cut(q), cut(k), inv_freq=f, pos0=T - tail)
    assert torch.equal(g["dq"][:, -tail:], gt["dq"])


def test_large_batch_of_single_tokens():
    """More sequences than a launch's y or z extent would take."""
    B, D, N = 70001, 8, 8
    r = Rand(53)
    x, w = gpu(r.n(B, D), r.n(D, 2))
    s = torch.zeros(B, 1, D, device="cuda")
    y = api.conv_step(x, w, s, silu=False)
    assert torch.equal(s[:, 0], x) and torch.allclose(y, x * w[:, 1])
    S = torch.zeros(B, D, N, device="cuda")
    bc = torch.ones(B, 1, N, device="cuda")
    A = -torch.ones(D, N, device="cuda")
    y = api.ssm_step(x, torch.ones_like(x), A, bc, bc, S, softplus=False)
    assert torch.equal(S, x[..., None].expand(B, D, N)) and torch.allclose(y, N * x)
    y, _ = api.ssm_fwd(x[:, None], torch.ones_like(x)[:, None], A, bc[:, None], bc[:, None],
                       softplus=False)
    assert torch.allclose(y[:, 0], N * x)
    q, _ = api.qk_norm_fwd(x[:, None], x[:, None], norm=None)
    assert torch.equal(q[:, 0], x)


def test_refusals_on_the_device():
    x = torch.zeros(2, 5, 64, device="cuda")
    w = torch.zeros(64, 4, device="cuda")
    with pytest.raises(ValueError, match="dtype|bfloat16|float32"):
        api.conv_fwd(x.half(), w)
    with pytest.raises(ValueError, match="w must"):
        api.conv_fwd(x, w[:32])
    with pytest.raises(ValueError, match="rows must not overlap"):
        api.conv_fwd(x[:, :1].expand(2, 5, 64), w)
    with pytest.raises(ValueError, match="lengths"):
        api.conv_fwd(x, w, lengths=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError, match="s0 must be contiguous"):
        api.conv_fwd(x, w, s0=torch.zeros(2, 64, 3, device="cuda").mT)
    with pytest.raises(K.KLAError):
        api.conv_fwd(x, torch.zeros(64, 5, device="cuda"))
    s = torch.zeros(2, 3, 64, device="cuda")
    with pytest.raises(K.KLAError):
        api.conv_fwd(x, w, s0=s, sT=s)
    A = torch.zeros(64, 12, device="cuda")
    bc = torch.zeros(2, 5, 1, 12, device="cuda")
    with pytest.raises(K.KLAError):
        api.ssm_fwd(x, x, A, bc, bc)
    with pytest.raises(ValueError, match="Cm must have shape"):
        api.ssm_fwd(x, x, A, bc, bc[:, :4])
    q = torch.zeros(2, 5, 2, 100, device="cuda")
    with pytest.raises(K.KLAError):
        api.qk_norm_fwd(q, q)
    with pytest.raises(ValueError, match="positions"):
        api.qk_norm_fwd(q, q, positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="norm must"):
        api.qk_norm_fwd(q, q, norm="max")
