"""The layer operators without a GPU: pins of their fp64 definitions
(closed forms, differences, splits of a sequence) and the argument checks of
the C ABI and of the binding."""
import math

import pytest
import torch

from delta_rule_linear_kla_b200 import _native, api, kla_conv, kla_qk_norm, kla_ssm
from delta_rule_linear_kla_b200 import build as kbuild
from oracle import layer_ops as ref

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 1 << 24  # fake, 16-byte-aligned device addresses: never dereferenced here


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _native.lib()


def rnd(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, dtype=torch.float64)


def diff_check(fwd, grads, args, outs, seed, skip=()):
    """<gradients, direction> against a central difference of the loss
    sum <output, fixed cotangent>.  fp64 with step 1e-5: the difference is off
    by about step^2 and 1e-16 / step, far below the 1e-7 bar."""
    r = rnd(seed)
    for name, x in args.items():
        if x is None or name in skip:
            continue
        d = r(*x.shape)

        def loss(e):
            o = fwd(**dict(args, **{name: x + e * d}))
            return sum((o[k][0] * c).sum() for k, c in outs.items())
        want = float((loss(1e-5) - loss(-1e-5)) / 2e-5)
        got = float((grads[name] * d).sum())
        assert abs(got - want) <= 1e-7 * max(1.0, abs(want)), (name, got, want)


@pytest.mark.parametrize("silu,lengths", [(True, None), (False, [5, 0, 2])])
def test_conv_definition(silu, lengths):
    r = rnd(1)
    B, T, D, W = 3, 5, 2, 4
    x, w, b, s0 = r(B, T, D), r(D, W), r(D), r(B, W - 1, D)
    gy, gs = r(B, T, D), r(B, W - 1, D)
    o = ref.conv(x, w, b, s0, silu, lengths)
    p = torch.nn.functional.conv1d(torch.cat([s0, x], 1).mT, w[:, None], b, groups=D).mT
    for i in range(B):
        n = T if lengths is None else lengths[i]
        want = p[i, :n] * torch.sigmoid(p[i, :n]) if silu else p[i, :n]
        assert torch.allclose(o["y"][0][i, :n], want, atol=1e-12)
        assert not o["y"][0][i, n:].any()
    g = ref.conv_bwd(x, w, gy, b, s0, gs, silu, lengths)
    diff_check(lambda x, w, bias, s0: ref.conv(x, w, bias, s0, silu, lengths),
               {"x": g["dx"][0], "w": g["dw"][0], "bias": g["dbias"][0], "s0": g["ds0"][0]},
               dict(x=x, w=w, bias=b, s0=s0), {"y": gy, "sT": gs}, 2)
    if lengths is None:  # a prompt cut in two
        one = ref.conv(x[:, :2], w, b, s0, silu)
        two = ref.conv(x[:, 2:], w, b, one["sT"][0], silu)
        assert torch.equal(torch.cat([one["y"][0], two["y"][0]], 1), o["y"][0])
        assert torch.equal(two["sT"][0], o["sT"][0])


@pytest.mark.parametrize("softplus,lengths", [(True, None), (False, [4, 0])])
def test_ssm_definition(softplus, lengths):
    r = rnd(3)
    B, T, D, G, N = 2, 4, 4, 2, 3
    a = dict(u=r(B, T, D), dt=r(B, T, D) * 0.3 + 0.2, A=-r(D, N).abs(), Bm=r(B, T, G, N),
             Cm=r(B, T, G, N), D=r(D), z=r(B, T, D), dt_bias=0.1 * r(D), h0=r(B, D, N))
    gy, gh = r(B, T, D), r(B, D, N)
    f = lambda **k: ref.ssm(**k, softplus=softplus, lengths=lengths)  # noqa: E731
    g = ref.ssm_bwd(a["u"], a["dt"], a["A"], a["Bm"], a["Cm"], gy, a["D"], a["z"], a["dt_bias"],
                    a["h0"], gh, softplus, lengths)
    names = {"u": "du", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "z": "dz",
             "dt_bias": "ddt_bias", "h0": "dh0"}
    diff_check(f, {k: g[n][0] for k, n in names.items()}, a, {"y": gy, "hT": gh}, 4)
    if lengths is None:  # a prompt cut in two
        cut = lambda s: {k: (v[:, s] if k in ("u", "dt", "Bm", "Cm", "z") else v)  # noqa: E731
                         for k, v in a.items()}
        one = f(**cut(slice(0, 1)))
        two = f(**dict(cut(slice(1, 4)), h0=one["hT"][0]))
        full = f(**a)
        assert torch.allclose(torch.cat([one["y"][0], two["y"][0]], 1), full["y"][0], atol=1e-12)
        assert torch.allclose(two["hT"][0], full["hT"][0], atol=1e-12)


def test_ssm_definition_closed_form():
    """One state, constant step s and input: h_t = x (1 - a^t) / (1 - a), x =
    s u B, a = e^{s A}."""
    T, s, A0 = 6, 0.25, -2.0
    one = torch.ones(1, T, 1, dtype=torch.float64)
    o = ref.ssm(3 * one, s * one, torch.full((1, 1), A0), 0.5 * one[..., None],
                2 * one[..., None], softplus=False)
    a, x = math.exp(s * A0), s * 3 * 0.5
    want = [2 * x * (1 - a ** (t + 1)) / (1 - a) for t in range(T)]
    assert torch.allclose(o["y"][0].flatten(), torch.tensor(want, dtype=torch.float64))


@pytest.mark.parametrize("norm", [None, "l2", "rms"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm_definition(norm, interleaved):
    r = rnd(5)
    x, w, g = r(2, 3, 2, 8), r(8), r(2, 3, 2, 8)
    pos = torch.tensor([[0, 5, 7], [100, 3, 2]])
    f = torch.tensor([1.0, 0.3, 0.01])
    kw = dict(positions=pos, inv_freq=f, norm=norm, eps=1e-3, interleaved=interleaved, scale=1.2)
    fwd = lambda x, w: {"o": ref.head_norm(x, w, **kw)}  # noqa: E731
    b = ref.head_norm_bwd(x, g, w, **kw)
    diff_check(fwd, {"x": b["dx"][0], "w": b["dw"][0]}, dict(x=x, w=w), {"o": g}, 6)
    # the rotation keeps lengths up to the scale, and position 0 turns nothing
    o = ref.head_norm(x, w, **kw)[0]
    v = ref.head_norm(x, w, norm=norm, eps=1e-3)[0]
    assert torch.allclose(o[..., :6].norm(dim=-1), 1.2 * v[..., :6].norm(dim=-1))
    assert torch.allclose(o[0, 0, :, :6], 1.2 * v[0, 0, :, :6])
    assert torch.equal(o[..., 6:], v[..., 6:])


# ---------------------------------------------------------------- refusals

def test_conv_refusals(lib):
    def fwd(x=A, ldx=64, w=2 * A, bias=None, s0=None, lens=None, y=4 * A, sT=None, B=2, T=16,
            D=64, W=4, dtype=0):
        return lib.kla_conv_fwd(x, ldx, w, bias, s0, lens, y, sT, B, T, D, W, 1, dtype, None)
    assert fwd(x=None) == INVALID
    assert fwd(w=None) == INVALID
    assert fwd(y=None) == INVALID
    assert fwd(y=A) == INVALID                    # over x
    assert fwd(x=A + 1) == fwd(y=4 * A + 8) == INVALID   # misaligned
    assert fwd(ldx=63) == INVALID                 # rows overlap
    assert fwd(s0=6 * A, sT=6 * A) == INVALID     # the state in place
    assert fwd(B=0) == fwd(T=-1) == fwd(D=0) == fwd(W=0) == fwd(dtype=2) == INVALID
    assert fwd(B=2**31 - 1, T=2**30, D=2**20, ldx=2**20) == INVALID  # 2^81 elements
    assert fwd(W=1) == fwd(W=5) == UNSUPPORTED
    assert fwd(B=1, T=2**30 + 1, D=1, ldx=1) == UNSUPPORTED
    assert fwd(B=1, T=1, D=2**31 - 1, ldx=2**31 - 1) == UNSUPPORTED
    # a written buffer between the first and the last row of a wide matrix
    assert fwd(ldx=1 << 20, y=A + (1 << 21)) == INVALID
    need = lib.kla_conv_bwd_workspace_size(2, 16, 64, 4)
    assert need > 0 and lib.kla_conv_bwd_workspace_size(2, 0, 64, 4) == 0

    def bwd(gy=3 * A, dx=4 * A, dw=5 * A, ws=7 * A, wsb=need, ds0=None, T=16):
        return lib.kla_conv_bwd(A, 64, 2 * A, None, None, None, gy, None, dx, dw, None, ds0, 2,
                                T, 64, 4, 1, 0, ws, wsb, None)
    assert bwd(gy=None) == bwd(dx=None) == bwd(dw=None) == bwd(ws=None) == INVALID
    assert bwd(wsb=need - 1) == INVALID
    assert bwd(dx=3 * A) == bwd(ws=4 * A) == bwd(ds0=5 * A) == INVALID
    step = lambda s=4 * A, y=5 * A, W=4: lib.kla_conv_step(  # noqa: E731
        A, 64, 2 * A, None, s, y, 2, 64, W, 1, 0, None)
    assert step(s=None) == step(y=None) == step(y=4 * A) == step(s=A) == INVALID
    assert step(W=7) == UNSUPPORTED


def test_ssm_refusals(lib):
    def fwd(u=A, dt=2 * A, Am=3 * A, Bm=4 * A, Cm=5 * A, z=None, h0=None, y=7 * A, hT=None,
            B=2, T=16, D=64, G=1, N=16, ldu=64, ldb=16, ldz=64, dtype=0, ws=None, wsb=0):
        return lib.kla_ssm_fwd(u, dt, Am, Bm, Cm, None, z, None, h0, None, y, hT, B, T, D, G, N,
                               ldu, 64, ldb, 16, ldz, 1, dtype, ws, wsb, None)
    assert fwd(u=None) == fwd(dt=None) == fwd(Am=None) == fwd(y=None) == INVALID
    assert fwd(y=A) == fwd(hT=3 * A) == INVALID
    assert fwd(h0=8 * A, hT=8 * A + 64) == INVALID   # partly over the start state
    assert fwd(ldu=63) == fwd(ldb=15) == fwd(z=6 * A, ldz=8) == INVALID
    assert fwd(D=65, ldu=65, G=2) == INVALID         # groups of unequal size
    assert fwd(N=12) == fwd(N=128, ldb=128) == UNSUPPORTED
    assert fwd(u=A + 1) == fwd(Am=3 * A + 4) == fwd(dtype=3) == fwd(G=0) == fwd(T=-2) == INVALID
    assert lib.kla_ssm_fwd_workspace_size(8, 4096, 2048, 1, 16) == 0   # enough channels
    need = lib.kla_ssm_fwd_workspace_size(1, 4096, 64, 1, 16)          # cut into segments
    assert need > 0
    assert fwd(B=1, T=4096) == INVALID               # no workspace
    assert fwd(B=1, T=4096, ws=9 * A, wsb=need - 1) == INVALID
    assert fwd(B=1, T=4096, ws=A, wsb=need) == INVALID   # workspace over u
    nb = lib.kla_ssm_bwd_workspace_size(2, 16, 64, 1, 16)
    assert nb >= 2 * 64 * 16 * 4

    def bwd(z=None, dz=None, dA=12 * A, dB=13 * A, ws=20 * A, wsb=nb, gy=9 * A, du=10 * A):
        return lib.kla_ssm_bwd(A, 2 * A, 3 * A, 4 * A, 5 * A, None, z, None, None, None, gy,
                               None, du, 11 * A, dA, dB, 14 * A, None, dz, None, None, 2, 16, 64,
                               1, 16, 64, 64, 16, 16, 64, 1, 0, ws, wsb, None)
    assert bwd(gy=None) == bwd(du=None) == bwd(dA=None) == bwd(dB=None) == bwd(ws=None) == INVALID
    assert bwd(wsb=nb - 1) == INVALID
    assert bwd(z=6 * A) == INVALID                   # a gate without its gradient
    assert bwd(du=9 * A) == bwd(dB=10 * A) == bwd(ws=A) == INVALID
    step = lambda S=6 * A, y=7 * A, N=16: lib.kla_ssm_step(  # noqa: E731
        A, 2 * A, 3 * A, 4 * A, 5 * A, None, None, None, S, y, 2, 64, 1, N, 64, 64, N, N, 64, 1,
        0, None)
    assert step(S=None) == step(y=None) == step(S=A) == step(y=6 * A) == INVALID
    assert step(N=24) == UNSUPPORTED
    assert lib.kla_ssm_bwd_workspace_size(1, 1, 2**30 + 1, 1, 16) == 0   # too many channels


def test_qk_norm_refusals(lib):
    def fwd(q=A, k=2 * A, ldq=256, ldk=128, pos=None, ps=0, f=3 * A, rot=64, norm=1, eps=1e-6,
            scale=1.0, oq=5 * A, ok=6 * A, B=2, T=8, Hq=2, Hk=1, d=128, dtype=0):
        return lib.kla_qk_norm_fwd(q, k, ldq, ldk, None, None, pos, ps, 0, f, rot, 0, scale,
                                   norm, eps, oq, ok, B, T, Hq, Hk, d, dtype, None)
    assert fwd(q=None) == fwd(ok=None) == fwd(f=None) == INVALID
    assert fwd(oq=A) == fwd(ok=5 * A) == INVALID
    assert fwd(ldq=255) == fwd(rot=130) == fwd(rot=63) == fwd(norm=3) == fwd(eps=-1.0) == INVALID
    assert fwd(eps=float("nan")) == fwd(scale=float("inf")) == fwd(Hq=0, Hk=0) == INVALID
    assert fwd(pos=4 * A, ps=7) == INVALID           # rows of positions overlap
    assert fwd(pos=4 * A + 2, ps=8) == fwd(f=3 * A + 1) == fwd(q=A + 8) == INVALID  # misaligned
    assert fwd(d=100, ldq=200, ldk=104, rot=0) == UNSUPPORTED
    assert fwd(d=264, ldq=528, ldk=264) == UNSUPPORTED
    assert fwd(ldq=260) == UNSUPPORTED               # rows not 16-byte multiples apart
    assert fwd(T=0) == OK
    need = lib.kla_qk_norm_bwd_workspace_size(2, 8, 2, 1, 128, 64)
    assert need > 0

    def bwd(gq=7 * A, dq=8 * A, dw=10 * A, ws=11 * A, wsb=need):
        return lib.kla_qk_norm_bwd(A, 2 * A, 256, 128, 3 * A, None, None, 0, 0, 4 * A, 64, 0,
                                   1.0, 2, 1e-6, gq, 9 * A, dq, 12 * A, dw, None, 2, 8, 2, 1,
                                   128, 0, ws, wsb, None)
    assert bwd(gq=None) == bwd(dq=None) == bwd(ws=None) == bwd(wsb=need - 4) == INVALID
    assert bwd(dq=7 * A) == bwd(dw=8 * A) == bwd(ws=A) == INVALID


X = torch.zeros(2, 5, 64)
H = torch.zeros(2, 5, 2, 64)
W4, P, BC = torch.zeros(64, 4), torch.zeros(64, 16), torch.zeros(2, 5, 1, 16)
HOST_CALLS = {
    "conv_fwd": lambda: api.conv_fwd(X, W4),
    "conv_bwd": lambda: api.conv_bwd(X, W4, X),
    "conv_step": lambda: api.conv_step(X[:, 0], W4, torch.zeros(2, 3, 64)),
    "ssm_fwd": lambda: api.ssm_fwd(X, X, P, BC, BC),
    "ssm_bwd": lambda: api.ssm_bwd(X, X, P, BC, BC, X),
    "ssm_step": lambda: api.ssm_step(X[:, 0], X[:, 0], P, BC[:, 0], BC[:, 0],
                                     torch.zeros(2, 64, 16)),
    "qk_norm_fwd": lambda: api.qk_norm_fwd(H, H),
    "qk_norm_bwd": lambda: api.qk_norm_bwd(H, H, H, H),
    "kla_conv": lambda: kla_conv(X, W4),
    "kla_ssm": lambda: kla_ssm(X, X, P, BC, BC),
    "kla_qk_norm": lambda: kla_qk_norm(H, H),
}


@pytest.mark.parametrize("name", sorted(HOST_CALLS))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="CUDA"):
        HOST_CALLS[name]()


@pytest.mark.parametrize("make,lead,want", [
    (lambda: torch.zeros(2, 5, 8), (2, 5), 8),
    (lambda: torch.zeros(2, 5, 24)[..., 8:16], (2, 5), 24),
    (lambda: torch.zeros(2, 1, 24)[..., :8], (2, 1), 24),
    (lambda: torch.zeros(1, 5, 24)[..., :8], (1, 5), 24),
    (lambda: torch.zeros(5, 24)[:, :8], (5,), 24),
    (lambda: torch.zeros(7, 9, 8)[:2, :5], (2, 5), None),      # uneven rows
    (lambda: torch.zeros(2, 5, 16)[..., ::2], (2, 5), None),   # strided elements
    (lambda: torch.zeros(2, 1, 8).expand(2, 5, 8), (2, 5), None),  # broadcast rows
    (lambda: torch.zeros(5, 2, 8).transpose(0, 1), (2, 5), None),
])
def test_row_pitch(make, lead, want, monkeypatch):
    t = make()
    dev = torch.device("cuda", 0)  # nothing here touches a device
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    if want is None:
        with pytest.raises(ValueError):
            api._rows(t, "t", torch.float32, lead, (8,), dev)
    else:
        assert api._rows(t, "t", torch.float32, lead, (8,), dev) == want
