"""fp64 definitions of the layer operators (test infrastructure only): the
short causal convolution, the selective state space scan and the norm and
rotation of queries and keys, token by token, with their adjoints written out.

Every function returns a dict name -> (value, magnitude): the magnitude is the
same sum with every term's absolute value, the scale that the rounding errors
of any evaluation order are relative to.
"""
import torch


def f64(x):
    return None if x is None else x.detach().cpu().double()


def _lens(lengths, B, T):
    if lengths is None:
        return [T] * B
    return [max(0, min(T, int(n))) for n in lengths]


def _silu(p):
    """value, derivative, bound of the derivative's terms."""
    s = torch.sigmoid(p)
    return p * s, s * (1 + p * (1 - s)), s * (1 + p.abs() * (1 - s))


# ------------------------------------------------------------ convolution

def _conv_rows(x, s0, W):
    B, T, D = x.shape
    head = x.new_zeros(B, W - 1, D) if s0 is None else s0
    return torch.cat([head, x], 1)


def conv(x, w, bias=None, s0=None, silu=True, lengths=None):
    """y and sT of the prompt (a sequence's rows behind its length are zero
    and not read)."""
    x, w, bias, s0 = map(f64, (x, w, bias, s0))
    B, T, D = x.shape
    W = w.shape[1]
    rows = _conv_rows(x, s0, W)
    y, my = torch.zeros(B, T, D).double(), torch.zeros(B, T, D).double()
    sT = torch.zeros(B, W - 1, D).double()
    for b, n in enumerate(_lens(lengths, B, T)):
        for t in range(n):
            p = sum(w[:, j] * rows[b, t + j] for j in range(W))
            m = sum(w[:, j].abs() * rows[b, t + j].abs() for j in range(W))
            if bias is not None:
                p, m = p + bias, m + bias.abs()
            y[b, t], my[b, t] = (_silu(p)[0] if silu else p), m
        sT[b] = rows[b, n:n + W - 1]
    return {"y": (y, my), "sT": (sT, sT.abs())}


def conv_bwd(x, w, gy, bias=None, s0=None, gs=None, silu=True, lengths=None):
    x, w, gy, bias, s0, gs = map(f64, (x, w, gy, bias, s0, gs))
    B, T, D = x.shape
    W = w.shape[1]
    rows = _conv_rows(x, s0, W)
    z = lambda *s: torch.zeros(*s).double()  # noqa: E731
    dr, mr = z(B, T + W - 1, D), z(B, T + W - 1, D)
    dw, mw, db, mb = z(D, W), z(D, W), z(D), z(D)
    for b, n in enumerate(_lens(lengths, B, T)):
        for t in range(n):
            dp, mp = gy[b, t], gy[b, t].abs()
            if silu:
                p = sum(w[:, j] * rows[b, t + j] for j in range(W))
                m = sum(w[:, j].abs() * rows[b, t + j].abs() for j in range(W))
                if bias is not None:
                    p, m = p + bias, m + bias.abs()
                _, d1, m1 = _silu(p)
                dp, mp = dp * d1, mp * (m1 + m)
            for j in range(W):
                dr[b, t + j] += w[:, j] * dp
                mr[b, t + j] += w[:, j].abs() * mp
                dw[:, j] += dp * rows[b, t + j]
                mw[:, j] += mp * rows[b, t + j].abs()
            db += dp
            mb += mp
        if gs is not None:
            dr[b, n:n + W - 1] += gs[b]
            mr[b, n:n + W - 1] += gs[b].abs()
    return {"dx": (dr[:, W - 1:], mr[:, W - 1:]), "dw": (dw, mw), "dbias": (db, mb),
            "ds0": (dr[:, :W - 1], mr[:, :W - 1])}


# ------------------------------------------------------------------- scan

def _ssm_setup(u, dt, A, Bm, Cm, D, z, dt_bias, softplus):
    u, dt, A, Bm, Cm, D, z, dt_bias = map(f64, (u, dt, A, Bm, Cm, D, z, dt_bias))
    Dn = u.shape[-1]
    G = Bm.shape[-2]
    at = torch.arange(Dn) // (Dn // G)
    raw = dt if dt_bias is None else dt + dt_bias
    st = torch.logaddexp(raw, torch.zeros(()).double()) if softplus else raw
    D = torch.zeros(Dn).double() if D is None else D
    return u, st, raw, A, Bm, Cm, D, z, at


def ssm(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, softplus=True, lengths=None):
    u, st, _, A, Bm, Cm, D, z, at = _ssm_setup(u, dt, A, Bm, Cm, D, z, dt_bias, softplus)
    B, T, Dn = u.shape
    N = A.shape[1]
    y, my = torch.zeros(B, T, Dn).double(), torch.zeros(B, T, Dn).double()
    hT, mT = torch.zeros(B, Dn, N).double(), torch.zeros(B, Dn, N).double()
    for b, n in enumerate(_lens(lengths, B, T)):
        h = torch.zeros(Dn, N).double() if h0 is None else f64(h0)[b].clone()
        m = h.abs()
        for t in range(n):
            a = torch.exp(st[b, t][:, None] * A)
            x = (st[b, t] * u[b, t])[:, None] * Bm[b, t][at]
            h, m = a * h + x, a * m + x.abs()
            C = Cm[b, t][at]
            v, mv = (h * C).sum(-1) + D * u[b, t], (m * C.abs()).sum(-1) + (D * u[b, t]).abs()
            if z is not None:
                gate = _silu(z[b, t])[0]
                v, mv = v * gate, mv * gate.abs()
            y[b, t], my[b, t] = v, mv
        hT[b], mT[b] = h, m
    return {"y": (y, my), "hT": (hT, mT)}


def ssm_bwd(u, dt, A, Bm, Cm, gy, D=None, z=None, dt_bias=None, h0=None, ghT=None,
            softplus=True, lengths=None):
    u, st, raw, A, Bm, Cm, D, z, at = _ssm_setup(u, dt, A, Bm, Cm, D, z, dt_bias, softplus)
    gy, ghT = f64(gy), f64(ghT)
    B, T, Dn = u.shape
    N, G = A.shape[1], Bm.shape[-2]
    names = {"du": (B, T, Dn), "ddt": (B, T, Dn), "dA": (Dn, N), "dB": (B, T, G, N),
             "dC": (B, T, G, N), "dD": (Dn,), "dz": (B, T, Dn), "ddt_bias": (Dn,),
             "dh0": (B, Dn, N)}
    v = {k: torch.zeros(s).double() for k, s in names.items()}
    m = {k: torch.zeros(s).double() for k, s in names.items()}
    for b, n in enumerate(_lens(lengths, B, T)):
        h = torch.zeros(Dn, N).double() if h0 is None else f64(h0)[b].clone()
        hs, ms = [h], [h.abs()]
        for t in range(n):
            a = torch.exp(st[b, t][:, None] * A)
            x = (st[b, t] * u[b, t])[:, None] * Bm[b, t][at]
            hs.append(a * hs[-1] + x)
            ms.append(a * ms[-1] + x.abs())
        e = torch.zeros(Dn, N).double() if ghT is None else ghT[b].clone()
        me = e.abs()
        for t in range(n - 1, -1, -1):
            g = gy[b, t]
            Bt, Ct, s = Bm[b, t][at], Cm[b, t][at], st[b, t]
            y0 = (hs[t + 1] * Ct).sum(-1) + D * u[b, t]
            my0 = (ms[t + 1] * Ct.abs()).sum(-1) + (D * u[b, t]).abs()
            if z is not None:
                val, d1, m1 = _silu(z[b, t])
                v["dz"][b, t], m["dz"][b, t] = g * y0 * d1, g.abs() * my0 * m1
                g = g * val
            dh, mh = e + Ct * g[:, None], me + Ct.abs() * g.abs()[:, None]
            a = torch.exp(s[:, None] * A)
            for sign, to, H, dH in ((1, v, hs, dh), (0, m, ms, mh)):
                ab = (lambda q: q) if sign else (lambda q: q.abs())
                E = a * dH
                fed = (dH * ab(Bt)).sum(-1)
                to["dC"][b, t].index_add_(0, at, H[t + 1] * ab(g)[:, None])
                to["dB"][b, t].index_add_(0, at, dH * ab(s * u[b, t])[:, None])
                to["du"][b, t] = ab(D * g) + ab(s) * fed
                ds = ab(u[b, t]) * fed + (ab(A) * H[t] * E).sum(-1)
                if softplus:
                    ds = ds * torch.sigmoid(raw[b, t])
                to["ddt"][b, t] = ds
                to["ddt_bias"] += ds
                to["dD"] += ab(g * u[b, t])
                to["dA"] += ab(s)[:, None] * H[t] * E
                if sign:
                    e = E
                else:
                    me = E
        v["dh0"][b], m["dh0"][b] = e, me
    return {k: (v[k], m[k]) for k in names}


# --------------------------------------------------- norm and rotation

def _angles(positions, inv_freq):
    ang = positions.double()[..., None] * f64(inv_freq)
    return torch.cos(ang)[:, :, None], torch.sin(ang)[:, :, None]


def _turn(x, cs, interleaved, sign, scale):
    """x rotated, and the magnitude of each output's terms."""
    if cs is None:
        return x, x.abs()
    c, s = cs[0] * scale, cs[1] * scale * sign
    r = 2 * c.shape[-1]
    out, mag = x.clone(), x.abs().clone()
    i = slice(0, r, 2) if interleaved else slice(0, r // 2)
    j = slice(1, r, 2) if interleaved else slice(r // 2, r)
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    mag[..., i] = mag[..., j] = (a.abs() + b.abs()) * abs(scale)
    return out, mag


def _unit(x, norm, eps):
    if norm is None:
        return x, torch.ones_like(x[..., :1])
    q = (x * x).sum(-1, keepdim=True)
    r = 1 / torch.sqrt((q if norm == "l2" else q / x.shape[-1]) + eps)
    return x * r, r


def head_norm(x, w=None, positions=None, inv_freq=None, norm="l2", eps=1e-6,
              interleaved=False, scale=1.0):
    """One of q, k: [B, T, H, d] with positions [B, T]."""
    x, w = f64(x), f64(w)
    cs = None if inv_freq is None else _angles(positions, inv_freq)
    n, _ = _unit(x, norm, eps)
    return _turn(n if w is None else n * w, cs, interleaved, 1.0, scale)


def head_norm_bwd(x, g, w=None, positions=None, inv_freq=None, norm="l2", eps=1e-6,
                  interleaved=False, scale=1.0):
    x, w, g = f64(x), f64(w), f64(g)
    cs = None if inv_freq is None else _angles(positions, inv_freq)
    g, mg = _turn(g, cs, interleaved, -1.0, scale)
    n, r = _unit(x, norm, eps)
    dw, mw = (g * n).sum((0, 1, 2)), (mg * n.abs()).sum((0, 1, 2))
    if w is not None:
        g, mg = g * w, mg * w.abs()
    if norm is None:
        return {"dx": (g, mg), "dw": (dw, mw)}
    m = x.shape[-1] if norm == "rms" else 1
    along, mal = (g * n).sum(-1, keepdim=True) / m, (mg * n.abs()).sum(-1, keepdim=True) / m
    return {"dx": (r * (g - n * along), r * (mg + n.abs() * mal)), "dw": (dw, mw)}
