"""The layer operators at the ends of their arguments' ranges, and layouts and cuts
beside the ones of test_layer_ops_gpu.py.  Bars are the ones of that file where
none is derived here."""
import math

import pytest
import torch

import delta_rule_linear_kla_b200 as K
from delta_rule_linear_kla_b200 import api
from oracle import layer_ops as ref
from test_layer_ops_gpu import DT, Rand, U, check, gpu, ssm_case, wide

pytestmark = pytest.mark.gpu


def _room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip("needs %d GB of device memory" % gigabytes)


def test_ssm_step_groups_past_32_bits():
    """A token whose rows of B and C have more than 2^31 elements (a group for
    every channel): the last channels come out as in a call of their own."""
    _room(48)
    D, N, tail = (1 << 28) + 64, 8, 4096
    gen = torch.Generator(device="cuda").manual_seed(70)
    mk = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    u, dt, Bm, Cm = mk(1, D), mk(1, D), mk(1, D, N), mk(1, D, N)
    assert Bm.numel() > 1 << 31
    A = torch.rand(D, N, generator=gen, device="cuda").neg_()
    S = torch.rand(1, D, N, generator=gen, device="cuda")
    cut = [t[:, -tail:].clone() for t in (u, dt, Bm, Cm, S)]
    y = api.ssm_step(u, dt, A, Bm, Cm, S)
    want = api.ssm_step(cut[0], cut[1], A[-tail:].contiguous(), cut[2], cut[3], cut[4])
    assert torch.equal(y[:, -tail:], want) and torch.equal(S[:, -tail:], cut[4])


NOEPS = [  # B, T, Hq, Hk, d: heads or tokens that do not fill a block
    (1, 7, 5, 1, 128), (2, 5, 1, 1, 64), (1, 1, 3, 2, 80), (3, 41, 2, 0, 8), (1, 301, 17, 3, 32),
]


@pytest.mark.parametrize("eps", [0.0, 1e-40])  # 1e-40: below fp32's normal range
@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("case", NOEPS, ids=str)
def test_qk_norm_without_eps(case, norm, eps):
    """No eps: the row places of a block that hold no row add nothing to the
    weights' gradients (a row of zeros there would be 0 / 0).  Bars as for the
    other norms: c = 64, 128 backward, and a unit for every 16 rows of dw."""
    B, T, Hq, Hk, d = case
    r = Rand(71)
    q, k, gq, gk = (r.n(B, T, h, d) for h in (Hq, Hk, Hq, Hk))
    w = r.n(d)
    qg, kg, gqg, gkg, wg = gpu(q, k, gq, gk, w)
    kw = dict(norm=norm, eps=eps)
    out = api.qk_norm_fwd(qg, kg, wq=wg, wk=wg, **kw)
    got = api.qk_norm_bwd(qg, kg, gqg, gkg, wq=wg, wk=wg, **kw)
    for i, (n, x, g) in enumerate((("q", q, gq), ("k", k, gk))):
        check(out[i], ref.head_norm(x, w, **kw), 64, n)
        want = ref.head_norm_bwd(x, g, w, **kw)
        check(got["d" + n], want["dx"], 128, "d" + n)
        check(got["dw" + n], want["dw"], 128 + x[..., 0].numel() / 16, "dw" + n)


def _given_as(y, other, tail):
    """Gradients of `tail` for y whole and for y behind `other` in one tensor:
    the gradient then is a contiguous view that starts at any element."""
    c = torch.arange(y.numel(), device=y.device).to(y.dtype).reshape(y.shape) / y.numel() - 0.5
    whole = torch.autograd.grad(y, tail, c, retain_graph=True)
    flat = torch.cat([other.flatten(), y.flatten()])
    behind = torch.autograd.grad(flat, tail, torch.cat([torch.zeros_like(other).flatten(),
                                                        c.flatten()]), retain_graph=True)
    return zip(whole, behind)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_gradients_that_start_at_any_element(dt):
    """Autograd hands the backward pass of a concatenation's part a view: the
    same bits as for a gradient of its own memory."""
    r = Rand(72)
    t = DT[dt]
    leaf = lambda *s: r.n(*s, dt=t).cuda().requires_grad_(True)  # noqa: E731
    odd = torch.zeros(5, device="cuda", dtype=t)
    odd32 = torch.zeros(5, device="cuda")
    D, N = 3, 8
    x, w = leaf(1, 7, D), r.n(D, 4).cuda().requires_grad_(True)
    y, sT = K.kla_conv(x, w)
    bc, A = leaf(1, 7, 1, N), (-torch.rand(D, N).cuda()).requires_grad_(True)
    o, hT = K.kla_ssm(x, x, A, bc, bc)
    q = leaf(1, 7, 2, 8)
    nq, nk = K.kla_qk_norm(q, q)
    for out, other, to in ((y, odd, [x, w]), (sT, odd, [x]), (o, odd, [x, A, bc]),
                           (hT, odd32, [x, A, bc]), (nq, odd, [q]), (nk, odd, [q])):
        for a, b in _given_as(out, other, to):
            assert torch.equal(a, b) and a.abs().sum() > 0


def test_prefill_gradients_that_start_at_any_element():
    r = Rand(73)
    q, k, v = (r.n(1, 65, 1, 64, dt=torch.bfloat16).cuda().requires_grad_(True) for _ in range(3))
    g, eta = -0.1 * torch.rand(1, 65, 1, device="cuda"), torch.rand(1, 65, 1, device="cuda")
    o, hT = K.kla_prefill(q, k, v, g, eta)
    for out, to in ((o, [q, k, v]), (hT, [k, v])):
        for a, b in _given_as(out, torch.zeros(5, device="cuda", dtype=out.dtype), to):
            assert torch.equal(a, b) and a.abs().sum() > 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_of_fp32_rows(interleaved):
    """The cosine and sine that fp32 rows are turned by, read off rows of one 1
    and zeros, over 10^5 angles up to 10^6 radians.  In units of 2^-24: the
    angle, a multiple of pi in [-1, 1], rounded to fp32 turns by pi 2^-25 at
    most (1.6); sine and cosine within 1 ulp of values up to 1 (1), and the
    products with 1 and 0 add nothing: 2.6, and 0.1 for what is of second
    order and the fp64 angle (10^6 2^-53)."""
    T, d = 8000, 32
    f = torch.linspace(1e-3, 1.0, d // 2)
    pos = (torch.arange(T) * 125).int()
    x = torch.zeros(1, T, 1, d)
    x[..., (slice(0, d, 2) if interleaved else slice(0, d // 2))] = 1.0
    kw = dict(norm=None, interleaved=interleaved)
    got, _ = api.qk_norm_fwd(x.cuda(), x.cuda(), inv_freq=f.cuda(), positions=pos.cuda(), **kw)
    want, _ = ref.head_norm(x, None, pos[None], f, **kw)
    assert float((got.double().cpu() - want).abs().max()) <= 2.7 * U


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_qk_norm_of_tiny_rows_without_eps(dt):
    """Rows of entries near 5e-21 without an eps: their squares and the sum of
    them (3e-39) lie below fp32's normal range, where a square is off by 2^-150
    at most and a sum of 128 by 2^-142 in all, 2^-14 of the sum; half of that
    in the norm, 2^-15 of the result.  Backward twice that, and for dw."""
    r = Rand(74)
    d = 128
    q = ((r.n(2, 9, 2, d).sign() * (4e-21 + 2e-21 * torch.rand(2, 9, 2, d)))).to(DT[dt])
    g, w = r.n(2, 9, 2, d, dt=DT[dt]), r.n(d)
    qg, gg, wg = gpu(q, g, w)
    kw = dict(norm="l2", eps=0.0)
    out, _ = api.qk_norm_fwd(qg, qg.clone(), wq=wg, **kw)
    got = api.qk_norm_bwd(qg, qg.clone(), gg, gg.clone(), wq=wg, **kw)
    c = 2.0 ** 9  # 2^-15 in units of 2^-24
    check(out, ref.head_norm(q, w, **kw), c, "out")
    want = ref.head_norm_bwd(q, g, w, **kw)
    check(got["dq"], want["dx"], 2 * c, "dq")
    check(got["dwq"], want["dw"], 2 * c, "dwq")


@pytest.mark.parametrize("late", [False, True])  # the steps in the first or the second segment
@pytest.mark.parametrize("sign,start", [(1.0, 1e-20), (-1.0, 1e30)])
def test_ssm_segment_factors_past_fp32(sign, start, late):
    """A segment whose states grow (or decay) by e^96 = 2^138 as a whole, from
    a start that keeps every state inside fp32, forward and backward.  Bars of
    the other scans: c = 64 + (7 + 3 X) T, X = 0.75."""
    B, T, D, N = 1, 256, 16, 8
    assert api.ssm_fwd_workspace_size(B, T, D, 1, N) > 0  # cut into two segments
    r = Rand(75)
    dt = torch.zeros(B, T, D)
    dt[:, 128:] += 0.75 * late
    dt[:, :128] += 0.75 * (not late)
    u, A = torch.zeros(B, T, D), torch.full((D, N), sign)
    Bm, Cm = r.n(B, T, 1, N), r.n(B, T, 1, N)
    h0 = start * (1 + torch.rand(B, D, N))
    # the adjoint state makes the same way from the other end
    gy, gh = torch.zeros(B, T, D), (1e-12 if sign > 0 else 1.0) * (1 + torch.rand(B, D, N))
    c = 64 + (7 + 3 * 0.75) * T
    a = dict(u=u, dt=dt, A=A, Bm=Bm, Cm=Cm, h0=h0)
    x = {k: v.cuda() for k, v in a.items()}
    y, h = api.ssm_fwd(**x, softplus=False)
    want = ref.ssm(**a, softplus=False)
    check(y, want["y"], c, "y")
    check(h, want["hT"], c, "hT")
    got = api.ssm_bwd(x["u"], x["dt"], x["A"], x["Bm"], x["Cm"], gy.cuda(), h0=x["h0"],
                      grad_hT=gh.cuda(), softplus=False)
    want = ref.ssm_bwd(u, dt, A, Bm, Cm, gy, h0=h0, ghT=gh, softplus=False)
    for k, v in got.items():
        if v is not None:
            check(v, want[k], 2 * c + 128, k)


def test_ssm_long_memories():
    """Decays of memories of 300 to 3000 tokens (exponents of -0.0027 to -0.0004 to
    the base 2, mean error of the hardware's exponential 0.5e-8): over all
    states the mean error of a decay is smaller than that, for the prompt, its
    backward pass and the token.  Roundings have no mean: 2e-8 a decay over 4e6
    of them leaves 1e-11."""
    r = Rand(79)
    B, T, D, N = 4, 2048, 64, 8
    A = -0.1 * torch.exp(0.3 * r.n(D, N).clamp(-1.5, 1.5))
    dt = 0.0073 * torch.exp(0.3 * r.n(B, T, D).clamp(-1.5, 1.5))
    x = (dt.amin() * A.abs().amin(), dt.amax() * A.abs().amax())
    assert 2.5e-4 < x[0] * math.log2(math.e) and x[1] * math.log2(math.e) < 2.7e-3
    Ag, dg = gpu(A, dt)
    zero, bc = torch.zeros(B, T, D, device="cuda"), torch.zeros(B, T, 1, N, device="cuda")
    one = torch.ones(B, D, N, device="cuda")
    want = (dg.double().sum(1)[..., None] * Ag.double())
    _, h = api.ssm_fwd(zero, dg, Ag, bc, bc, h0=one, softplus=False)
    g = api.ssm_bwd(zero, dg, Ag, bc, bc, zero, h0=one, grad_hT=one, softplus=False)
    for got in (h, g["dh0"]):
        off = float(((got.double().log() - want) / T).mean())
        assert abs(off) < 0.5e-8, off
    S, n = torch.ones(B * 16, D, N, device="cuda"), T // 16
    d = dg.view(B, 16, n, D).flatten(0, 1)
    for t in range(n):
        api.ssm_step(zero[0, :64], d[:, t], Ag, bc[0, :64], bc[0, :64], S, softplus=False)
    off = float(((S.double().log() - d.double().sum(1)[..., None] * Ag.double()) / n).mean())
    assert abs(off) < 0.5e-8, off


def test_convolution_of_2_32_single_channels():
    """More than 2^32 channels of one token, taken one by one (an odd channel
    count): prompt and token are those of the same rows alone."""
    _room(56)
    B, D, W = (1 << 20) + 300, 4097, 2
    assert B * D > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(76)
    x = torch.randn(B, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    s = torch.randn(B, 1, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    w, b = torch.randn(D, W, generator=gen, device="cuda"), torch.randn(D, device="cuda")
    edge = ((1 << 32) - 256) // D  # sequences that 32 bits of threads count
    some = [slice(0, 2), slice(edge - 2, edge + 2), slice(B - 2, B)]
    n = torch.ones(B, dtype=torch.int32, device="cuda")
    n[edge + 1] = n[1] = 0
    y, sT = api.conv_fwd(x[:, None], w, b, s, lengths=n)
    for i in some:
        yi, si = api.conv_fwd(x[i, None].clone(), w, b, s[i].clone(), lengths=n[i].clone())
        assert torch.equal(y[i], yi) and torch.equal(sT[i], si)
    del y, sT
    old = [s[i].clone() for i in some]
    y = api.conv_step(x, w, s, b)
    for i, o in zip(some, old):
        assert torch.equal(y[i], api.conv_step(x[i].clone(), w, o, b))
        assert torch.equal(s[i], o)
    assert torch.equal(s[:, 0], x)


BEHIND = [(20, 11), (20, 0), (9, 8), (300, 130)]  # T, tokens that exist


@pytest.mark.parametrize("T,n", BEHIND)
def test_conv_places_behind_the_last_token(T, n):
    """Gradients of tokens that do not exist are zeros, whatever the taps."""
    r = Rand(77)
    x, gy, w = gpu(r.n(1, T, 12), r.n(1, T, 12), r.n(12, 4))
    w[3, 0], w[5, 3], w[7, 1] = math.inf, math.nan, -math.inf
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = api.conv_bwd(x, w, gy, lengths=lens)
    assert not got["dx"][:, n:].any()


@pytest.mark.parametrize("T,n", BEHIND)
def test_ssm_places_behind_the_last_token(T, n):
    """Gradients of tokens that do not exist are zeros, whatever the states,
    their gradients and A."""
    r = Rand(78)
    B, D, N = 1, 12, 8
    x, gy, dt, A, bc, gh, h0 = gpu(r.n(B, T, D), r.n(B, T, D), r.n(B, T, D), -torch.rand(D, N),
                                   r.n(B, T, 1, N), r.n(B, D, N), r.n(B, D, N))
    gh[0, 3, 2], gh[0, 5, 1], h0[0, 6, 3], A[7, 4] = math.inf, math.nan, -math.inf, math.nan
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = api.ssm_bwd(x, dt, A, bc, bc, gy, z=x, h0=h0, grad_hT=gh, lengths=lens)
    for k in ("du", "ddt", "dB", "dC", "dz"):
        assert not got[k][:, n:].any(), k


def test_arguments_that_are_no_tensors():
    x = torch.zeros(2, 5, 64, device="cuda")
    with pytest.raises(ValueError, match="w must be"):
        api.conv_fwd(x, torch.zeros(64, 0, device="cuda"))
    q = x.view(2, 5, 1, 64)
    with pytest.raises(ValueError, match="positions must be a CUDA tensor"):
        api.qk_norm_fwd(q, q, positions=[0, 1, 2, 3, 4])
    with pytest.raises(ValueError, match="inv_freq must be a CUDA tensor"):
        api.qk_norm_bwd(q, q, q, q, inv_freq=[1.0, 0.5])


# B, T, D, G, N, dtype, z, skip, bias, softplus, state, lengths, -, columns before and behind u, dt
WIDE = [
    ((2, 70, 24, 1, 16, "bf16", True, True, True, True, True, [70, 33], 0), (8, 4), (4, 12)),
    ((2, 41, 24, 2, 8, "fp32", True, True, True, True, True, None, 0), (4, 4), (3, 2)),
    ((1, 67, 130, 1, 32, "bf16", False, True, True, True, False, None, 0), (5, 1), (1, 1)),
    ((1, 33, 20, 1, 64, "fp32", True, False, True, True, True, [20], 0), (3, 2), (8, 0)),
    ((1, 700, 64, 1, 16, "bf16", True, True, True, True, True, None, 0), (8, 8), (16, 0)),  # cut
]


@pytest.mark.parametrize("case,pu,pd", WIDE, ids=str)
def test_ssm_rows_of_wider_matrices(case, pu, pd):
    """u and dt as columns of wider matrices, NaN around them."""
    _against_definition(case, lambda g: dict(g, u=wide(g["u"], *pu), dt=wide(g["dt"], *pd)))


# cut into segments, with several blocks of channels a group and wide states
CUT = [
    (1, 700, 70, 1, 32, "fp32", True, True, True, True, True, None, 0),
    (2, 600, 40, 1, 64, "bf16", True, True, True, True, True, [600, 290], 0),
    (1, 520, 72, 2, 64, "fp32", False, True, True, True, False, None, 0),
    (1, 530, 300, 1, 16, "bf16", True, True, True, True, True, [400], 0),
    (1, 515, 270, 2, 8, "fp32", True, True, True, True, True, None, 0),
]


@pytest.mark.parametrize("case", CUT, ids=str)
def test_ssm_cut_sequences(case):
    B, T, D, G, N = case[:5]
    assert api.ssm_fwd_workspace_size(B, T, D, G, N) > 0
    _against_definition(case, lambda g: g)


def _against_definition(case, lay):
    a, gy, gh, n, c = ssm_case(case, 78)
    g = lay({k: None if v is None else v.cuda() for k, v in a.items()})
    kw = dict(softplus=case[9], lengths=None if n is None else n.cuda())
    y, hT = api.ssm_fwd(**g, **kw)
    want = ref.ssm(**a, softplus=case[9], lengths=case[11])
    check(y, want["y"], c, "y")
    check(hT, want["hT"], c, "hT")
    got = api.ssm_bwd(g["u"], g["dt"], g["A"], g["Bm"], g["Cm"], gy.cuda(), g["D"], g["z"],
                      g["dt_bias"], g["h0"], None if gh is None else gh.cuda(), **kw)
    want = ref.ssm_bwd(a["u"], a["dt"], a["A"], a["Bm"], a["Cm"], gy, a["D"], a["z"],
                       a["dt_bias"], a["h0"], gh, case[9], case[11])
    for k, v in got.items():
        if v is not None:
            check(v, want[k], 2 * c + 128, k)
