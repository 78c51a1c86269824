"""Cases of the layer operators beside the delta-rule recurrence: the short
causal convolution, the selective state space scan and the per-head norm of
queries and keys with the rotation by position.  Each has its prompt form,
its backward pass and its form for single tokens.

``own`` false computes them in plain torch operations, true through
delta_rule_linear_kla_b200."""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the projected channels of a 0.4B-scale layer (q and k of 8 heads of
        # 128) over a batch of prompts, before the recurrence
        dict(name="conv_prompt_4k", op="conv", B=8, T=4096, D=2048, W=4, dtype="bf16", silu=True,
             bias=False, state=False, ragged=False),
        # a few padded prompts of uneven lengths that continue earlier ones, odd
        # channel count, no activation
        dict(name="conv_ragged_fp32", op="conv", B=3, T=1999, D=1001, W=3, dtype="fp32",
             silu=False, bias=True, state=True, ragged=True),
        # training at the 8192-token, 32 heads of 64 shape
        dict(name="conv_train_8k", op="conv_bwd", B=4, T=8192, D=2048, W=4, dtype="bf16",
             silu=True, bias=True, state=False, ragged=False),
        # one new token for each of 64 sequences
        dict(name="conv_step_b64", op="conv_step", B=64, D=2048, W=4, dtype="bf16", silu=True,
             bias=True),
        # a batch of prompts through a state space layer; the largest case
        dict(name="ssm_prompt_4k", op="ssm", B=8, T=4096, D=2048, G=1, N=16, dtype="bf16",
             z=True, skip=True, softplus=True, state=False, ragged=False),
        # one long prompt of odd size, two groups of inputs, a wider state,
        # continued from an earlier part
        dict(name="ssm_long_fp32", op="ssm", B=1, T=8191, D=1000, G=2, N=32, dtype="fp32",
             z=False, skip=True, softplus=True, state=True, ragged=True),
        # training
        dict(name="ssm_train_4k", op="ssm_bwd", B=2, T=4096, D=2048, G=1, N=16, dtype="bf16",
             z=True, skip=True, softplus=True, state=False, ragged=False),
        # one new token for each of 64 sequences
        dict(name="ssm_step_b64", op="ssm_step", B=64, D=2048, G=1, N=16, dtype="bf16", z=True,
             skip=True, softplus=True),
        # queries and keys of the 4096-token layer
        dict(name="qk_prompt_4k", op="qk", B=8, T=4096, Hq=8, Hk=8, d=128, rot=64, dtype="bf16",
             norm="l2", weight=False, interleaved=False, far=0),
        # training, fewer key heads than query heads, learned weights, the
        # whole head rotated in pairs
        dict(name="qk_train_8k", op="qk_bwd", B=4, T=8192, Hq=32, Hk=8, d=64, rot=64,
             dtype="bf16", norm="rms", weight=True, interleaved=True, far=0),
        # odd sizes at far positions
        dict(name="qk_odd_fp32", op="qk", B=2, T=777, Hq=5, Hk=1, d=80, rot=40, dtype="fp32",
             norm="rms", weight=True, interleaved=False, far=1000000),
        # one new token for each of 64 sequences behind a 32768-token prefix
        dict(name="qk_step_b64", op="qk", B=64, T=1, Hq=16, Hk=16, d=128, rot=128, dtype="bf16",
             norm="l2", weight=False, interleaved=False, far=32768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "conv_step", "ssm", "ssm", "ssm_bwd", "ssm_bwd",
                     "ssm_step", "qk", "qk", "qk_bwd"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("conv"):
        c.update(B=_log(rng, 1, 128), D=_log(rng, 40, 8192), W=rng.choice([2, 3, 4, 4]),
                 silu=rng.random() < 0.8, bias=flip())
        if flip():
            c["D"] = max(8, c["D"] // 8 * 8)
        if op != "conv_step":
            most = 1 << 25
            c["B"] = min(c["B"], 16)
            c.update(T=_log(rng, 1, min(65536, most // (c["B"] * c["D"]))), state=flip(),
                     ragged=flip())
    elif op.startswith("ssm"):
        c.update(B=_log(rng, 1, 128), G=rng.choice([1, 1, 1, 2, 4]),
                 N=rng.choice([8, 16, 16, 32, 64]), z=rng.random() < 0.7, skip=flip(),
                 softplus=rng.random() < 0.8)
        c["D"] = max(8, _log(rng, 64, 4096) // c["G"]) * c["G"]
        if op != "ssm_step":
            most = (1 << 28) if op == "ssm" else (1 << 27)
            c["B"] = min(c["B"], 8)
            c.update(T=_log(rng, 1, min(8192, most // (c["B"] * c["D"] * c["N"]))),
                     state=flip(), ragged=flip())
    else:
        c.update(B=_log(rng, 1, 64), Hk=rng.choice([1, 2, 3, 4, 8, 16]),
                 d=rng.choice([32, 64, 64, 80, 96, 128, 128, 256]),
                 norm=rng.choice(["l2", "rms", "none"]), interleaved=flip(),
                 far=rng.choice([0, 0, 5000, 1000000]))
        c["Hq"] = c["Hk"] * rng.choice([1, 1, 2, 4])
        c["rot"] = rng.choice([0, c["d"], c["d"] // 2, 8, 24]) if c["norm"] != "none" \
            else rng.choice([c["d"], c["d"] // 2])
        c["weight"] = c["norm"] == "rms" and flip()
        most = 1 << 25
        c["T"] = 1 if rng.random() < 0.2 else _log(
            rng, 1, min(16384, most // (c["B"] * (c["Hq"] + c["Hk"]) * c["d"])))
    return c


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    op, B = case["op"], case["B"]
    T = case.get("T", 1)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def rand(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case)
    if case.get("ragged"):
        n = torch.randint(max(1, T // 3), T + 1, (B,), generator=g, device="cuda")
        s["lengths"] = n.to(torch.int32)
    else:
        s["lengths"] = None
    if op.startswith("conv"):
        D, W = case["D"], case["W"]
        r = 1.0 / math.sqrt(W)
        s["w"] = rand(-r, r, D, W)
        s["b"] = rand(-r, r, D) if case["bias"] else None
        if op == "conv_step":
            s["x"], s["s0"] = randn(B, D).to(dt), randn(B, W - 1, D).to(dt)
            return s
        s["x"] = randn(B, T, D).to(dt)
        s["s0"] = randn(B, W - 1, D).to(dt) if case["state"] else None
        if op == "conv_bwd":
            s["gy"] = randn(B, T, D).to(dt)
            s["gs"] = randn(B, W - 1, D).to(dt) if case["state"] else None
    elif op.startswith("ssm"):
        D, G, N = case["D"], case["G"], case["N"]
        tok = (B,) if op == "ssm_step" else (B, T)
        u = randn(*tok, D)
        s["u"] = (u * torch.sigmoid(u)).to(dt)
        # step sizes spread over 1e-3 .. 1e-1, as such layers are initialised
        step = torch.exp(rand(math.log(1e-3), math.log(1e-1), D))
        if case["softplus"]:
            s["bias"] = step + torch.log(-torch.expm1(-step))
            s["dt"] = (0.5 * randn(*tok, D)).to(dt)
        else:
            s["bias"] = None
            s["dt"] = (step * torch.exp(0.5 * randn(*tok, D))).to(dt)
        s["A"] = -torch.arange(1, N + 1, device="cuda").float() * torch.exp(0.1 * randn(D, N))
        # B and C are neighbouring columns of one projection, as are u's source and z
        bc = randn(*tok, 2 * G * N).to(dt)
        s["Bm"] = bc[..., :G * N].unflatten(-1, (G, N))
        s["Cm"] = bc[..., G * N:].unflatten(-1, (G, N))
        s["z"] = randn(*tok, 2 * D).to(dt)[..., D:] if case["z"] else None
        if case["z"] and D % 8:
            s["z"] = s["z"].contiguous()
        s["skip_w"] = randn(D) if case["skip"] else None
        if op == "ssm_step":
            s["S"] = randn(B, D, N)
            return s
        s["h0"] = randn(B, D, N) if case["state"] else None
        if op == "ssm_bwd":
            s["gy"] = randn(B, T, D).to(dt)
            s["gh"] = randn(B, D, N) if case["state"] else None
    else:
        Hq, Hk, d, rot = case["Hq"], case["Hk"], case["d"], case["rot"]
        scale = torch.exp(rand(math.log(0.25), math.log(4.0), B, T, 1, 1))
        s["q"] = randn(B, T, Hq, d).to(dt)
        s["k"] = (scale * randn(B, T, Hk, d)).to(dt)
        s["wq"] = 1 + 0.1 * randn(d) if case["weight"] else None
        s["wk"] = 1 + 0.1 * randn(d) if case["weight"] else None
        s["inv_freq"] = s["pos"] = None
        if rot:
            # frequencies stretched eightfold beyond the trained length
            i = torch.arange(rot // 2, device="cuda").double()
            s["inv_freq"] = (10000.0 ** (-2 * i / rot) / (8.0 if case["far"] else 1.0)).float()
            first = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
            s["pos"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
        if op == "qk_bwd":
            s["gq"], s["gk"] = randn(B, T, Hq, d).to(dt), randn(B, T, Hk, d).to(dt)
    return s


# ---------------------------------------------------------------- the passes

def run(state):
    return _framework(state) if own else _PLAIN[state["op"]](state)


def _framework(s):
    from delta_rule_linear_kla_b200 import api
    op = s["op"]
    if op == "conv":
        return api.conv_fwd(s["x"], s["w"], s["b"], s["s0"], silu=s["silu"],
                            lengths=s["lengths"])
    if op == "conv_bwd":
        return api.conv_bwd(s["x"], s["w"], s["gy"], s["b"], s["s0"], s["gs"], silu=s["silu"],
                            lengths=s["lengths"], need_s0=s["state"])
    if op == "conv_step":
        return api.conv_step(s["x"], s["w"], s["s0"], s["b"], silu=s["silu"]), s["s0"]
    if op == "ssm":
        return api.ssm_fwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["skip_w"], s["z"],
                           s["bias"], s["h0"], softplus=s["softplus"], lengths=s["lengths"])
    if op == "ssm_bwd":
        return api.ssm_bwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["gy"], s["skip_w"],
                           s["z"], s["bias"], s["h0"], s["gh"], softplus=s["softplus"],
                           lengths=s["lengths"], need_h0=s["state"])
    if op == "ssm_step":
        return api.ssm_step(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["S"], s["skip_w"],
                            s["z"], s["bias"], softplus=s["softplus"]), s["S"]
    kw = dict(wq=s["wq"], wk=s["wk"], positions=s["pos"], inv_freq=s["inv_freq"],
              norm=None if s["norm"] == "none" else s["norm"], interleaved=s["interleaved"])
    if op == "qk":
        return api.qk_norm_fwd(s["q"], s["k"], **kw)
    return api.qk_norm_bwd(s["q"], s["k"], s["gq"], s["gk"], **kw)


EPS = 1e-6  # the calls' default


def _live(s, T):
    """[B, T, 1] truth values: the tokens before each sequence's length."""
    if s["lengths"] is None:
        return None
    return (torch.arange(T, device="cuda")[None, :] < s["lengths"][:, None])[..., None]


def _keep(live, x):
    return x if live is None else torch.where(live, x, torch.zeros((), device=x.device,
                                                                   dtype=x.dtype))


def _conv_inputs(s):
    x, W = s["x"], s["W"]
    B, T, D = x.shape
    s0 = s["s0"] if s["s0"] is not None else x.new_zeros(B, W - 1, D)
    return torch.cat([s0, x], 1)  # [B, T + W - 1, D]


def _last_rows(s, T, W):
    """Rows of the padded input that the final state holds."""
    n = s["lengths"] if s["lengths"] is not None else torch.full((s["B"],), T, device="cuda")
    return n[:, None].long() + torch.arange(W - 1, device="cuda")


def _plain_conv(s):
    xp = _conv_inputs(s)
    T, W = s["T"], s["W"]
    p = (xp.float().unfold(1, W, 1) * s["w"]).sum(-1)
    if s["b"] is not None:
        p = p + s["b"]
    y = p * torch.sigmoid(p) if s["silu"] else p
    y = _keep(_live(s, T), y).to(xp.dtype)
    at = _last_rows(s, T, W)[..., None].expand(-1, -1, s["D"])
    return y, xp.gather(1, at)


def _plain_conv_bwd(s):
    xp = _conv_inputs(s)
    T, W, D = s["T"], s["W"], s["D"]
    dt = xp.dtype
    win = xp.float().unfold(1, W, 1)  # [B, T, D, W]
    dp = s["gy"].float()
    if s["silu"]:
        p = (win * s["w"]).sum(-1)
        if s["b"] is not None:
            p = p + s["b"]
        sg = torch.sigmoid(p)
        dp = dp * sg * (1 + p * (1 - sg))
    dp = _keep(_live(s, T), dp)
    dw = (dp[..., None] * _keep(None if s["lengths"] is None else _live(s, T)[..., None], win)
          ).sum((0, 1))
    pad = torch.nn.functional.pad(dp, (0, 0, W - 1, W - 1))
    dxp = (pad.unfold(1, W, 1) * s["w"].flip(1)).sum(-1)  # [B, T + W - 1, D]
    if s["gs"] is not None:
        at = _last_rows(s, T, W)[..., None].expand(-1, -1, D)
        dxp = dxp.scatter_add(1, at, s["gs"].float())
    return {"dx": dxp[:, W - 1:].to(dt), "dw": dw, "dbias": dp.sum((0, 1)) if s["bias"] else None,
            "ds0": dxp[:, :W - 1].to(dt) if s["state"] else None}


def _plain_conv_step(s):
    x, st = s["x"], s["s0"]
    win = torch.cat([st, x[:, None]], 1)
    p = (win.float() * s["w"].t()).sum(1)
    if s["b"] is not None:
        p = p + s["b"]
    y = (p * torch.sigmoid(p) if s["silu"] else p).to(x.dtype)
    st.copy_(win[:, 1:])
    return y, st


def _scan(a, b, h0):
    """h[t] = a[t] h[t-1] + b[t] along dim 1, h[-1] = h0 (None = 0): 64 tokens
    at a time, one token of every such block at once, then block by block."""
    B, T = a.shape[:2]
    L = 64
    n = -(-T // L)
    if n * L != T:
        more = a.new_zeros(B, n * L - T, *a.shape[2:])
        a, b = torch.cat([a, more + 1], 1), torch.cat([b, more], 1)
    a = a.reshape(B, n, L, *a.shape[2:]).clone()
    b = b.reshape(B, n, L, *b.shape[2:]).clone()
    for i in range(1, L):
        b[:, :, i] += a[:, :, i] * b[:, :, i - 1]
        a[:, :, i] *= a[:, :, i - 1]
    start = torch.zeros_like(b[:, :, 0])
    if h0 is not None:
        start[:, 0] = h0
    for j in range(1, n):
        start[:, j] = a[:, j - 1, -1] * start[:, j - 1] + b[:, j - 1, -1]
    b += a * start[:, :, None]
    return b.reshape(B, n * L, *b.shape[3:])[:, :T]


def _ssm_terms(s):
    """Everything by groups: channels [.., G, D/G], states [.., G, D/G, N]."""
    G, D, N = s["G"], s["D"], s["N"]
    T = s["T"]
    live = _live(s, T)
    live4 = None if live is None else live[..., None]
    grp = lambda x: _keep(live4, x.float().unflatten(-1, (G, D // G)))  # noqa: E731
    u, raw = grp(s["u"]), grp(s["dt"])
    if s["bias"] is not None:
        raw = raw + s["bias"].view(G, D // G)
    step = raw
    if s["softplus"]:
        step = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20))))
    step = _keep(live4, step)
    Bm = _keep(live4, s["Bm"].float())[:, :, :, None]
    Cm = _keep(live4, s["Cm"].float())[:, :, :, None]
    A = s["A"].view(G, D // G, N)
    a = torch.exp(step[..., None] * A)
    h0 = None if s["h0"] is None else s["h0"].view(-1, G, D // G, N)
    h = _scan(a, (step * u)[..., None] * Bm, h0)
    pre = (h * Cm).sum(-1)
    if s["skip_w"] is not None:
        pre = pre + s["skip_w"].view(G, D // G) * u
    z = None if s["z"] is None else grp(s["z"])
    return live4, u, raw, step, Bm, Cm, A, a, h0, h, pre, z


def _plain_ssm(s):
    live, u, raw, step, Bm, Cm, A, a, h0, h, y, z = _ssm_terms(s)
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return _keep(live, y).flatten(2).to(s["u"].dtype), h[:, -1].flatten(1, 2).clone()


def _plain_ssm_bwd(s):
    live, u, raw, step, Bm, Cm, A, a, h0, h, pre, z = _ssm_terms(s)
    dt = s["u"].dtype
    D, N, G = s["D"], s["N"], s["G"]
    g = _keep(live, s["gy"].float().unflatten(-1, (G, D // G)))
    out = {"dz": None, "dD": None, "ddt_bias": None, "dh0": None}
    if z is not None:
        sg = torch.sigmoid(z)
        out["dz"] = (g * pre * sg * (1 + z * (1 - sg))).flatten(2).to(dt)
        g = g * z * sg
    du = torch.zeros_like(u)
    if s["skip_w"] is not None:
        out["dD"] = (g * u).sum((0, 1)).flatten()
        du = g * s["skip_w"].view(G, D // G)
    # dh[t] = C[t] g[t] + a[t+1] dh[t+1], from the last token back
    nxt = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1)
    gh = None if s["gh"] is None else s["gh"].view(-1, G, D // G, N)
    dh = _scan(nxt, (g[..., None] * Cm).flip(1), gh).flip(1)
    prev = torch.cat([torch.zeros_like(h[:, :1]) if h0 is None else h0[:, None], h[:, :-1]], 1)
    out["dC"] = (h * g[..., None]).sum(3).to(dt)
    out["dB"] = _keep(live, (dh * (step * u)[..., None]).sum(3)).to(dt)
    if live is not None:
        out["dC"] = _keep(live, out["dC"])
    fed = (dh * Bm).sum(-1)
    decay = dh * prev * a
    ddt = fed * u + (decay * A).sum(-1)
    out["dA"] = (decay * step[..., None]).sum((0, 1)).flatten(0, 1)
    if s["softplus"]:
        ddt = ddt * torch.sigmoid(raw)
    ddt = _keep(live, ddt)
    out["du"] = _keep(live, du + fed * step).flatten(2).to(dt)
    out["ddt"] = ddt.flatten(2).to(dt)
    if s["bias"] is not None:
        out["ddt_bias"] = ddt.sum((0, 1)).flatten()
    if s["state"]:
        out["dh0"] = (a[:, 0] * dh[:, 0]).flatten(1, 2)
    return out


def _plain_ssm_step(s):
    G, D, N = s["G"], s["D"], s["N"]
    u, step = s["u"].float(), s["dt"].float()
    if s["bias"] is not None:
        step = step + s["bias"]
    if s["softplus"]:
        step = torch.where(step > 20, step, torch.log1p(torch.exp(step.clamp(max=20))))
    wide = lambda m: m.float()[:, :, None].expand(-1, -1, D // G, -1).flatten(1, 2)  # noqa: E731
    S = s["S"]
    S.copy_(torch.exp(step[..., None] * s["A"]) * S + (step * u)[..., None] * wide(s["Bm"]))
    y = (S * wide(s["Cm"])).sum(-1)
    if s["skip_w"] is not None:
        y = y + s["skip_w"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(s["u"].dtype), S


def _angles(s):
    """cos and sin [B, T, 1, rot/2] from angles in 64 bits."""
    if s["inv_freq"] is None:
        return None
    ang = s["pos"].double()[..., None] * s["inv_freq"].double()
    return torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]


def _turn(x, cs, interleaved, back=False):
    if cs is None:
        return x
    c, n = cs
    if back:
        n = -n
    r = 2 * c.shape[-1]
    head, rest = x[..., :r], x[..., r:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = head[..., :r // 2], head[..., r // 2:]
        head = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([head, rest], -1)


def _inverse_norm(x, norm):
    if norm == "none":
        return None
    ss = x.square()
    return torch.rsqrt((ss.sum(-1, keepdim=True) if norm == "l2"
                        else ss.mean(-1, keepdim=True)) + EPS)


def _plain_qk(s):
    cs = _angles(s)

    def one(x, w):
        dt, x = x.dtype, x.float()
        r = _inverse_norm(x, s["norm"])
        x = x if r is None else x * r
        x = x if w is None else x * w
        return _turn(x, cs, s["interleaved"]).to(dt)

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _plain_qk_bwd(s):
    cs = _angles(s)

    def one(x, w, g):
        dt, x = x.dtype, x.float()
        g = _turn(g.float(), cs, s["interleaved"], back=True)
        r = _inverse_norm(x, s["norm"])
        if r is None:
            return g.to(dt), None
        unit = x * r
        dw = None if w is None else (g * unit).sum((0, 1, 2))
        g = g if w is None else g * w
        along = (g * unit).sum(-1, keepdim=True)
        if s["norm"] == "rms":
            along = along / x.shape[-1]
        return (r * (g - unit * along)).to(dt), dw

    dq, dwq = one(s["q"], s["wq"], s["gq"])
    dk, dwk = one(s["k"], s["wk"], s["gk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


_PLAIN = {"conv": _plain_conv, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
          "ssm": _plain_ssm, "ssm_bwd": _plain_ssm_bwd, "ssm_step": _plain_ssm_step,
          "qk": _plain_qk, "qk_bwd": _plain_qk_bwd}


# ---------------------------------------------------------------- the bounds

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op, B = case["op"], case["B"]
    T = case.get("T", 1)
    if op.startswith("conv"):
        n, W, D = B * T * case["D"], case["W"], case["D"]
        par = 4 * D * (W + case["bias"])
        act = 4 if case["silu"] else 0
        if op == "conv_step":
            return {"bytes": es * (2 * n + 2 * (W - 1) * n) + par, "flops": n * (2 * W + act)}
        st = es * B * (W - 1) * D
        if op == "conv":
            return {"bytes": es * 2 * n + par + st * (1 + case["state"]),
                    "flops": n * (2 * W + act)}
        return {"bytes": es * 3 * n + 2 * par + 3 * st * case["state"],
                "flops": n * (6 * W + 2 * act)}
    if op.startswith("ssm"):
        D, G, N = case["D"], case["G"], case["N"]
        n, bc = B * T * D, 2 * B * T * G * N
        par = 4 * D * (N + case["skip"] + case["softplus"])
        st = 4 * B * D * N
        if op == "ssm_step":
            return {"bytes": es * (n * (3 + case["z"]) + bc) + par + 2 * st, "flops": n * N * 7}
        if op == "ssm":
            return {"bytes": es * (n * (3 + case["z"]) + bc) + par + st * (1 + case["state"]),
                    "flops": n * N * 7}
        return {"bytes": es * (n * (5 + 2 * case["z"]) + 2 * bc) + 2 * par
                + 3 * st * case["state"], "flops": n * N * 22}
    d = case["d"]
    n = B * T * (case["Hq"] + case["Hk"]) * d
    pos = (4 * B * T + 2 * case["rot"]) if case["rot"] else 0
    par = 8 * d * case["weight"]
    if op == "qk":
        return {"bytes": es * 2 * n + pos + par, "flops": n * 6}
    return {"bytes": es * 3 * n + pos + 2 * par, "flops": n * 14}


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "conv_bwd": _exact_conv, "conv_step": _exact_conv,
            "ssm": _exact_ssm, "ssm_bwd": _exact_ssm, "ssm_step": _exact_ssm,
            "qk": _exact_qk, "qk_bwd": _exact_qk}[case["op"]](s)


def _leaf(x):
    return None if x is None else x.double().detach().requires_grad_(True)


def _grads(pairs, leaves):
    """Gradients of the sum of <output, given> by differentiation of the
    definition itself."""
    total = sum((o * g.double()).sum() for o, g in pairs if g is not None)
    names = [k for k, v in leaves.items() if v is not None]
    got = torch.autograd.grad(total, [leaves[k] for k in names], allow_unused=True)
    return {k: (torch.zeros_like(leaves[k]) if v is None else v) for k, v in zip(names, got)}


def _exact_conv(s):
    """Token by token sums over the taps, one row of the input at a time."""
    W = s["W"]
    step, bwd = s["op"] == "conv_step", s["op"] == "conv_bwd"
    x = s["x"][:, None] if step else s["x"]
    B, T, D = x.shape
    x, w, b, s0 = _leaf(x), _leaf(s["w"]), _leaf(s["b"]), _leaf(s["s0"])
    rows = torch.cat([x.new_zeros(B, W - 1, D) if s0 is None else s0, x], 1)
    p = sum(rows[:, j:j + T] * w[:, j] for j in range(W))
    p = p if b is None else p + b
    y = p / (1 + torch.exp(-p)) if s["silu"] else p
    n = s["lengths"].tolist() if s["lengths"] is not None else [T] * B
    y = torch.stack([torch.cat([y[i, :m], torch.zeros_like(y[i, m:])]) for i, m in enumerate(n)])
    last = torch.stack([rows[i, m:m + W - 1] for i, m in enumerate(n)])
    if not bwd:
        return (y[:, 0] if step else y).detach(), last.detach()
    g = _grads([(y, s["gy"]), (last, s["gs"])], {"dx": x, "dw": w, "dbias": b, "ds0": s0})
    return {k: g.get(k) for k in ("dx", "dw", "dbias", "ds0")}


def _exact_ssm(s):
    """The recurrence itself, token by token; its gradients by
    differentiating it."""
    step1, bwd = s["op"] == "ssm_step", s["op"] == "ssm_bwd"
    tok = (lambda x: None if x is None else x[:, None]) if step1 else (lambda x: x)
    G, D, N, B = s["G"], s["D"], s["N"], s["B"]
    T = s.get("T", 1)
    names = ("u", "dt", "Bm", "Cm", "z")
    L = {k: _leaf(tok(s[k])) for k in names}
    L["A"], L["D"], L["dt_bias"] = _leaf(s["A"]), _leaf(s["skip_w"]), _leaf(s["bias"])
    L["h0"] = _leaf(s["S"] if step1 else s["h0"])
    n = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, device="cuda")
    h = L["u"].new_zeros(B, D, N) if L["h0"] is None else L["h0"]
    which = torch.arange(D, device="cuda") // (D // G)
    ys = []
    with torch.set_grad_enabled(bwd):
        for t in range(T):
            live = (t < n)[:, None]
            delta = L["dt"][:, t]
            if L["dt_bias"] is not None:
                delta = delta + L["dt_bias"]
            if s["softplus"]:
                delta = delta.clamp(min=0) + torch.log1p(torch.exp(-delta.abs()))
            u = L["u"][:, t]
            new = torch.exp(delta[:, :, None] * L["A"]) * h \
                + (delta * u)[:, :, None] * L["Bm"][:, t][:, which]
            h = torch.where(live[:, :, None], new, h)
            y = (h * L["Cm"][:, t][:, which]).sum(-1)
            if L["D"] is not None:
                y = y + L["D"] * u
            if L["z"] is not None:
                z = L["z"][:, t]
                y = y * z / (1 + torch.exp(-z))
            ys.append(torch.where(live, y, torch.zeros_like(y)))
        y = torch.stack(ys, 1)
    if not bwd:
        return (y[:, 0] if step1 else y).detach(), h.detach()
    g = _grads([(y, s["gy"]), (h, s["gh"])], L)
    at = {"du": "u", "ddt": "dt", "dB": "Bm", "dC": "Cm", "dz": "z", "dA": "A", "dD": "D",
          "ddt_bias": "dt_bias", "dh0": "h0"}
    return {k: g.get(v) for k, v in at.items()}


def _exact_qk(s):
    """Each pair of channels as a complex number turned by e^{i angle}."""
    bwd = s["op"] == "qk_bwd"
    L = {"dq": _leaf(s["q"]), "dk": _leaf(s["k"]), "dwq": _leaf(s["wq"]), "dwk": _leaf(s["wk"])}

    def one(x, w):
        if s["norm"] != "none":
            sq = (x * x).sum(-1, keepdim=True)
            x = x / torch.sqrt((sq if s["norm"] == "l2" else sq / x.shape[-1]) + EPS)
        x = x if w is None else x * w
        if s["inv_freq"] is None:
            return x
        r = 2 * s["inv_freq"].numel()
        ang = (s["pos"].double()[:, :, None] * s["inv_freq"].double())[:, :, None]
        turn = torch.polar(torch.ones_like(ang), ang)
        pair = x[..., :r].unflatten(-1, (r // 2, 2) if s["interleaved"] else (2, r // 2))
        pair = pair if s["interleaved"] else pair.transpose(-1, -2)
        out = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        out = out if s["interleaved"] else out.transpose(-1, -2)
        return torch.cat([out.flatten(-2), x[..., r:]], -1)

    oq, ok = one(L["dq"], L["dwq"]), one(L["dk"], L["dwk"])
    if not bwd:
        return oq.detach(), ok.detach()
    g = _grads([(oq, s["gq"]), (ok, s["gk"])], L)
    return {k: g.get(k) for k in L}
