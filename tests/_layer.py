"""Plain 64-bit forms of the state space layer's calls, token by token, and what rounding may leave.

An output is a sum of products of the inputs.  `allowed` bounds its error by the sum of the magnitudes of its terms
(the same plain form run on magnitudes): every term goes through at most ROUNDINGS roundings of 32 bits (the step
and its exponential some ten, a decay's exponent, whose error e^G turns into at most |G| e^G 2^-24 < 2^-24 a
rounding, the factors' splits, the additions of up to 64 + 128 terms in blocks of 16, one scaling a chunk), 64 in all.  A bf16
output adds half a step of bf16, 2^-8 of its value, and its products hold 16 bits: 2^-16 of the terms' sum.
"""
import torch

F64 = torch.float64
ROUNDINGS = 64.0


def allowed(ref, terms, dtype):
    if dtype == torch.bfloat16:
        return 2.0 ** -8 * ref.abs() + (2.0 ** -16 + ROUNDINGS * 2.0 ** -24) * terms + 1e-30
    return 2.0 ** -24 * ref.abs() + ROUNDINGS * 2.0 ** -24 * terms + 1e-30


def check(name, got, ref, terms):
    got64 = got.detach().cpu().to(F64)
    assert got64.shape == ref.shape, (name, got64.shape, ref.shape)
    over = (got64 - ref).abs() / allowed(ref, terms, got.dtype)
    assert bool(torch.isfinite(got64).all()), name
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} times what rounding allows"


def wide(x):
    return None if x is None else x.detach().cpu().to(F64)


# ---- short convolution ---------------------------------------------------------------------------

def silu(c):
    return c / (1.0 + torch.exp(-c))


def conv(x, w, b, offs, state, activation=True):
    """Outputs, the sums c before the activation, final histories [n, dim, 3]."""
    out, cs = torch.zeros_like(x), torch.zeros_like(x)
    n = len(offs) - 1
    last = torch.zeros(n, x.shape[1], 3, dtype=x.dtype)
    for i in range(n):
        first = torch.zeros(3, x.shape[1], dtype=x.dtype) if state is None else state[i].T
        seq = torch.cat([first, x[offs[i]:offs[i + 1]]])
        L = offs[i + 1] - offs[i]
        c = sum(seq[j:j + L] * w[:, j] for j in range(4)) + (0.0 if b is None else b)
        cs[offs[i]:offs[i + 1]] = c
        out[offs[i]:offs[i + 1]] = silu(c) if activation else c
        last[i] = seq[-3:].T
    return out, cs, last


def conv_bwd(dc, x, w, offs, state, dlast):
    """Gradients from those of the sums c: dx, dw, db, dstate."""
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(x.shape[1], dtype=x.dtype)
    n = len(offs) - 1
    dst = torch.zeros(n, x.shape[1], 3, dtype=x.dtype)
    for i in range(n):
        first = torch.zeros(3, x.shape[1], dtype=x.dtype) if state is None else state[i].T
        a, L = offs[i], offs[i + 1] - offs[i]
        seq = torch.cat([first, x[a:a + L]])
        d = torch.zeros_like(seq)
        for j in range(4):
            d[j:j + L] += dc[a:a + L] * w[:, j]
            dw[:, j] += (dc[a:a + L] * seq[j:j + L]).sum(0)
        if dlast is not None:
            d[-3:] += dlast[i].T
        db += dc[a:a + L].sum(0)
        dx[a:a + L] = d[3:]
        dst[i] = d[:3].T
    return dx, dw, db, dst


def silu_slope(c):
    s = 1.0 / (1.0 + torch.exp(-c))
    return s * (1.0 + c * (1.0 - s))


# ---- selective scan --------------------------------------------------------------------------------

def gates(a, A_log, dt_bias):
    z = a + (0.0 if dt_bias is None else dt_bias)
    dt = z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))
    return z, dt, torch.exp(-torch.exp(A_log) * dt)


def ssm(x, B, C, dt, alpha, D, offs, S0):
    """y [T, H, P] and the final states: the recurrence token by token."""
    H, P, rep, N = x.shape[1], x.shape[2], x.shape[1] // B.shape[1], B.shape[2]
    y, n = torch.zeros_like(x), len(offs) - 1
    last = torch.zeros(n, H, P, N, dtype=x.dtype)
    for i in range(n):
        S = torch.zeros(H, P, N, dtype=x.dtype) if S0 is None else S0[i].clone()
        for t in range(offs[i], offs[i + 1]):
            S = alpha[t][:, None, None] * S + (dt[t][:, None] * x[t])[:, :, None] * B[t].repeat_interleave(rep, 0)[:, None, :]
            y[t] = (S * C[t].repeat_interleave(rep, 0)[:, None, :]).sum(-1)
            if D is not None:
                y[t] += D[:, None] * x[t]
        last[i] = S
    return y, last


def ssm_bwd(dy, x, B, C, dt, alpha, D, offs, S0, dlast):
    """The adjoint token by token: dx, dB, dC, ddt, dlog (of the log decays), dD [T, H], dS0."""
    H, P, G, N = x.shape[1], x.shape[2], B.shape[1], B.shape[2]
    rep, n = H // G, len(offs) - 1
    dx, dB, dC = torch.zeros_like(x), torch.zeros_like(B), torch.zeros_like(C)
    ddt, dlog = torch.zeros_like(dt), torch.zeros_like(dt)
    dS0 = torch.zeros(n, H, P, N, dtype=x.dtype)
    for i in range(n):
        S = torch.zeros(H, P, N, dtype=x.dtype) if S0 is None else S0[i].clone()
        before = []
        for t in range(offs[i], offs[i + 1]):
            before.append(S)
            S = alpha[t][:, None, None] * S + (dt[t][:, None] * x[t])[:, :, None] * B[t].repeat_interleave(rep, 0)[:, None, :]
        dS = torch.zeros_like(S) if dlast is None else dlast[i].clone()
        for t in range(offs[i + 1] - 1, offs[i] - 1, -1):
            Bt, Ct = B[t].repeat_interleave(rep, 0)[:, None, :], C[t].repeat_interleave(rep, 0)[:, None, :]
            dC[t] = (dy[t][:, :, None] * S).sum(1).reshape(G, rep, N).sum(1)
            dS = dS + dy[t][:, :, None] * Ct
            u = (dS * Bt).sum(-1)
            dx[t] = dt[t][:, None] * u
            ddt[t] = (u * x[t]).sum(-1)
            dB[t] = (dt[t][:, None, None] * x[t][:, :, None] * dS).sum(1).reshape(G, rep, N).sum(1)
            S = before.pop()
            dlog[t] = alpha[t] * (dS * S).sum((-1, -2))
            dS = alpha[t][:, None, None] * dS
        dS0[i] = dS
    dD = (dy * x).sum(-1)
    if D is not None:
        dx = dx + D[:, None] * dy
    return dx, dB, dC, ddt, dlog, dD, dS0


def scan_grads(dy, x, B, C, a, A_log, dt_bias, D, offs, S0, dlast):
    """The gradients of gdn_ssm_chunk_bwd, and the sums of their terms' magnitudes."""
    z, dt, alpha = gates(a, A_log, dt_bias)
    rate = torch.exp(A_log)
    inside = torch.zeros_like(dt)
    for i in range(len(offs) - 1):
        inside[offs[i]:offs[i + 1]] = 1.0
    slope = inside / (1.0 + torch.exp(-z))

    def finish(core, sign):
        dx, dB, dC, ddt, dlog, dD, dS0 = core
        da = (ddt - sign * rate * dlog) * slope
        return dict(dx=dx * inside[..., None], dB=dB, dC=dC, da=da, dA_log=(-sign * rate * dt * dlog).sum(0),
                    ddt_bias=da.sum(0), dD=(dD * inside).sum(0), dinitial_state=dS0)

    def mag(t):
        return None if t is None else t.abs()

    core = ssm_bwd(dy, x, B, C, dt, alpha, D, offs, S0, dlast)
    core_abs = ssm_bwd(mag(dy), mag(x), mag(B), mag(C), dt, alpha, mag(D), offs, mag(S0), mag(dlast))
    return finish(core, 1.0), finish(core_abs, -1.0)


# ---- norm and rotation -------------------------------------------------------------------------------

def rotate(m, cos, sin, interleaved):
    p = cos.shape[-1]
    out = m.clone()
    c, s = cos[:, None], sin[:, None]
    u = m[..., 0:2 * p:2] if interleaved else m[..., :p]
    v = m[..., 1:2 * p:2] if interleaved else m[..., p:2 * p]
    a, b = u * c - v * s, v * c + u * s
    if interleaved:
        out[..., 0:2 * p:2], out[..., 1:2 * p:2] = a, b
    else:
        out[..., :p], out[..., p:2 * p] = a, b
    return out


def norm_factor(x, l2, eps):
    ss = x.square().sum(-1, keepdim=True)
    return ((ss if l2 else ss / x.shape[-1]) + eps) ** -0.5


def qk(x, w, cos, sin, l2, eps, interleaved):
    m = x * norm_factor(x, l2, eps) * (1.0 if w is None else w)
    return rotate(m, cos, sin, interleaved), rotate(m.abs(), cos.abs(), -sin.abs(), interleaved).abs() + \
        rotate(m.abs(), cos.abs(), sin.abs(), interleaved).abs()


def qk_bwd(dout, x, w, cos, sin, l2, eps, interleaved):
    """dx, dw and the sums of magnitudes."""
    def mags(t):
        return (rotate(t.abs(), cos.abs(), -sin.abs(), interleaved).abs() +
                rotate(t.abs(), cos.abs(), sin.abs(), interleaved).abs())
    dm, adm = rotate(dout, cos, -sin, interleaved), mags(dout)
    r = norm_factor(x, l2, eps)
    n, inv = x * r, 1.0 if l2 else 1.0 / x.shape[-1]
    wt = 1.0 if w is None else w
    dn, adn = dm * wt, adm * abs(wt)
    dx = r * (dn - n * (dn * n).sum(-1, keepdim=True) * inv)
    adx = r * (adn + n.abs() * (adn * n.abs()).sum(-1, keepdim=True) * inv)
    return dx, (dm * n).sum((0, 1)), adx, (adm * n.abs()).sum((0, 1))
