"""Plain fp64 forms of the training operators, for the tests: each is its forward definition written out
in torch on the CPU, differentiated by autograd."""
from __future__ import annotations

import math

import numpy as np
import torch

F64 = torch.float64
# A fp32 output: the longest chain of roundings behind one value is a sum of 128 or 64 products at each of
# some eight products in a row, whose errors add like sqrt(8 * 128) half steps of 2^-24 (2e-6) where
# nothing cancels; ten times that leaves room for the cancellation in the row dots.
TOL_F32 = 2e-5
# A bf16 output is rounded once: at most half a step, 2^-8 of each value, and the fp32 error before it.
TOL_BF16 = 2.0 ** -8 + TOL_F32


def tol_of(t):
    return TOL_BF16 if t.dtype == torch.bfloat16 else TOL_F32


def rel_l2(x, ref):
    """||x - ref|| / ||ref||, and 0 where both are zero.  A reference below 2^-150 counts as zero: half the
    smallest fp32 (and bf16) magnitude, 2^-149 (2^-133), is its nearest representable neighbour's border."""
    x, ref = x.detach().cpu().to(F64), ref.detach().cpu().to(F64)
    ref = torch.where(ref.abs() < 2.0 ** -150, torch.zeros_like(ref), ref)
    assert x.shape == ref.shape, (x.shape, ref.shape)
    assert torch.isfinite(x).all()
    off, norm = float((x - ref).norm()), float(ref.norm())
    return off / norm if norm else (math.inf if off else 0.0)


def delta_forward(q, k, v, g, beta, cu, S0, scale, use_l2):
    """The recurrence token by token; q, k [T, Hk, d], v [T, H, d], g, beta [T, H], S0 [n, H, d, d]."""
    H, rep = v.shape[1], v.shape[1] // q.shape[1]
    if use_l2:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    q, k = (q * scale).repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    out, final = [], []
    for n in range(len(cu) - 1):
        S = S0[n]
        for t in range(cu[n], cu[n + 1]):
            S = S * g[t].exp()[:, None, None]
            u = beta[t][:, None] * (v[t] - (S @ k[t][:, :, None])[..., 0])
            S = S + u[:, :, None] * k[t][:, None, :]
            out.append((S @ q[t][:, :, None])[..., 0])
        final.append(S)
    y = torch.stack(out) if out else v.new_zeros((0, H, v.shape[-1]))
    return y, torch.stack(final)


def delta_inputs(lengths, H, Hk, d, dtype, seed, a_mean=-1.0, carried=True, lead=0, behind=0):
    """Seeded inputs of one packed batch, on the CPU; `lead` and `behind` tokens belong to no sequence."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    T, n = sum(lengths) + lead + behind, len(lengths)
    A = torch.exp(torch.rand(H, generator=gen) * math.log(8.0))
    inp = dict(q=rn(T, Hk, d).to(dtype), k=rn(T, Hk, d).to(dtype), v=rn(T, H, d).to(dtype),
               g=-A * torch.nn.functional.softplus(rn(T, H) + a_mean), beta=torch.sigmoid(rn(T, H)),
               dout=rn(T, H, d).to(dtype), initial_state=rn(n, H, d, d) * 0.1 if carried else None,
               dfinal_state=rn(n, H, d, d) * 0.1 if carried else None)
    inp["cu"] = [lead + int(x) for x in np.concatenate([[0], np.cumsum(lengths)])]
    return inp


def delta_grads(inp, scale=None, use_l2=True):
    """fp64 gradients of the inputs of delta_inputs: dq, dk, dv, dg, dbeta, dinitial_state."""
    d, n, H = inp["q"].shape[-1], len(inp["cu"]) - 1, inp["v"].shape[1]
    scale = d ** -0.5 if scale is None else scale
    S0 = inp["initial_state"]
    S0 = torch.zeros(n, H, d, d) if S0 is None else S0
    leaves = [x.to(F64).clone().requires_grad_() for x in (inp["q"], inp["k"], inp["v"], inp["g"], inp["beta"], S0)]
    y, S = delta_forward(*leaves[:5], inp["cu"], leaves[5], scale, use_l2)
    dS = inp["dfinal_state"]
    dS = torch.zeros_like(S) if dS is None else dS.to(F64)
    dy = inp["dout"].to(F64)[inp["cu"][0]:inp["cu"][-1]]
    got = torch.autograd.grad((y * dy).sum() + (S * dS).sum(), leaves, allow_unused=True)
    got = [torch.zeros_like(x) if gr is None else gr for gr, x in zip(got, leaves)]
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dinitial_state"), got))


# Half a step of an operand of a product that is kept in 22 bits.
EPS = 2.0 ** -23


def _delta_chunks(q, k, v, g, beta, dy, S, dS, scale, rounded):
    """Gradients of one sequence in the chunk form, in fp64 and by heads: q (scaled), k [H, T, d] and v, dy
    alike, g, beta [H, T], S, dS [H, d, d].  Returns those of q, k (as they are here), v, g and beta; rounded(x, s)
    is x with a relative error of s EPS."""
    C, T = 64, q.shape[1]

    def mul(A, B):
        # the operands' roundings, and the accumulator's: it is cut off at each of 3 inner / 16 steps (the terms
        # hi hi, hi lo and lo hi of 16 products), by half an EPS on average of a partial sum that grows to the
        # product, together 3 inner / 64 of it
        return rounded(rounded(A, 1.0) @ rounded(B, 1.0), 3 * A.shape[-1] / 64)

    def fade(x, far, low=None):
        # by e^far: 2 EPS in the exponential, |far| / 2 EPS in its argument (|far| 2^-24)
        f = far.exp() if low is None else far.masked_fill(~low, 0.0).exp() * low
        return x * rounded(f, torch.sqrt(4 + far ** 2 / 4))

    def dot(A, B):
        return rounded(A * B, 1.0).sum(-1)

    chunks, res = [], [torch.zeros_like(x) for x in (q, k, v, g, beta)]
    for c in range(0, T, C):
        i = slice(c, min(c + C, T))
        K, Q, V, Y, be, G = k[:, i], q[:, i], v[:, i], dy[:, i], beta[:, i, None], g[:, i].clamp(min=-128).cumsum(1)
        n = G.shape[1]
        low = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        far, to_end, G = G[:, :, None] - G[:, None], (G[:, -1:] - G)[..., None], G[..., None]
        A = be * fade(mul(K, K.mT), far, low.tril(-1))
        eye = torch.eye(n, dtype=F64, device=q.device).expand_as(A)
        X = rounded(torch.linalg.solve_triangular(eye + rounded(A, 1.0), eye, upper=False), 1.0)
        W, P = mul(X, be * fade(K, G)), fade(mul(Q, K.mT), far, low)
        U = mul(X, be * V) - mul(W, S.mT)
        chunks.append((i, K, Q, V, Y, be, G, far, to_end, low, X, W, P, U, S))
        S = fade(S, G[:, -1:]) + mul(fade(U, to_end).mT, K)
    for i, K, Q, V, Y, be, G, far, to_end, low, X, W, P, U, S in reversed(chunks):
        E = fade(mul(K, dS.mT), to_end)
        dR = mul(X.mT, mul(P.mT, Y) + E)
        dP, Z = fade(mul(Y, U.mT), far, low), -fade(mul(dR, U.mT), far, low.tril(-1))
        dQ, F = fade(mul(Y, S), G) + mul(dP, K), mul(Z, K) - fade(mul(dR, S), G)
        Hd, rest = fade(mul(U, dS), to_end), mul(dP.mT, Q) + mul(Z.mT, be * K)
        later, hk = dot(dQ, Q) + be[..., 0] * dot(F, K) - dot(rest, K), dot(Hd, K)
        carried = fade(dot(S, dS).sum(-1)[:, None], G[:, -1])
        dg = later.flip(1).cumsum(1).flip(1) + hk.cumsum(1) - hk + carried
        for x, y in zip(res, (dQ, be * F + Hd + rest, be * dR, dg, dot(dR, V) + dot(F, K))):
            x[:, i] = y
        dS = fade(dS, G[:, -1:]) + mul(Y.mT, fade(Q, G) - mul(P, W)) - mul(E.mT, W)
    return res


def delta_errors(inp, scale=None, use_l2=True, samples=32, device="cpu"):
    """Standard deviations of the errors of delta_grads' gradients token by token when the chunk form is rounded as
    _delta_chunks says, from random roundings of that size (in fp64; cancellations and errors that many terms
    share are then counted as they are): dq, dk [T, Hk] and dv [T, H] (a vector's 2-norm), dg and dbeta [T, H]."""
    (T, Hk, d), H, cu = inp["q"].shape, inp["v"].shape[1], inp["cu"]
    scale = d ** -0.5 if scale is None else scale
    q, k, v, g, beta, dy = (inp[x].to(device, F64) for x in ("q", "k", "v", "g", "beta", "dout"))
    rep = lambda x: x.repeat_interleave(H // Hk, 1)  # noqa: E731
    rq, rk = (torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6) if use_l2 else torch.ones_like(x[..., :1]) for x in (q, k))
    heads = [x.transpose(0, 1) for x in (rep(q * rq) * scale, rep(k * rk), v, g, beta, dy)]
    gen = torch.Generator(device=device).manual_seed(0)
    noisy = lambda x, s: x * (1 + s * EPS * torch.randn(x.shape, generator=gen, dtype=F64, device=device))  # noqa: E731
    out = {x: torch.zeros(T, Hk if x in ("dq", "dk") else H, dtype=F64) for x in ("dq", "dk", "dv", "dg", "dbeta")}
    for n in range(len(cu) - 1):
        i = slice(cu[n], cu[n + 1])
        states = [torch.zeros(H, d, d, dtype=F64, device=device) if inp[x] is None else inp[x][n].to(device, F64)
                  for x in ("initial_state", "dfinal_state")]

        def grads(count, rounded):  # [count, heads, tokens, ...]
            many = [x.repeat(count, *[1] * (x.dim() - 1)) for x in [x[:, i] for x in heads] + states]
            got = [x.reshape(count, H, *x.shape[1:]) for x in _delta_chunks(*many, scale, rounded)]
            for x, r in ((0, scale * rq), (1, rk)):
                got[x] = got[x].reshape(count, Hk, H // Hk, -1, d).sum(2) * r[i].transpose(0, 1)
            return got

        for x, many, one in zip(out, grads(samples, noisy), grads(1, lambda x, s: x)):
            square = ((many - one) ** 2).mean(0)
            out[x][i] = (square.sum(-1) if square.dim() == 3 else square).sqrt().transpose(0, 1).cpu()
    return out


def norm_forward(y, z, w, b, eps, rms):
    """The output norm over the last dimension of y [rows, groups, size] (w, b broadcast) with its SiLU."""
    if rms:
        m = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
    else:
        c = y - y.mean(-1, keepdim=True)
        m = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    m = m if w is None else m * w
    m = m if b is None else m + b
    t = m if z is None else z
    return (1.0 if z is None else m) * t * torch.sigmoid(t)


def norm_grads(dout, y, z, w, b, eps, rms):
    """fp64 gradients (dy, dz, dw, db), None where the input is."""
    leaves = [None if x is None else x.to(F64).clone().requires_grad_() for x in (y, z, w, b)]
    out = norm_forward(*leaves, eps, rms)
    got = iter(torch.autograd.grad(out, [x for x in leaves if x is not None], dout.to(F64)))
    return [None if x is None else next(got) for x in leaves]


def decay_grads(a, A_log, dt_bias, b, dg, dbeta):
    """fp64 gradients (da, dA_log, ddt_bias, db), None where the input is."""
    leaves = [None if x is None else x.to(F64).clone().requires_grad_() for x in (a, A_log, dt_bias, b)]
    x = leaves[0] if dt_bias is None else leaves[0] + leaves[2]
    g = -leaves[1].exp() * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    loss = (g * dg.to(F64)).sum()
    if b is not None:
        loss = loss + (torch.sigmoid(leaves[3]) * dbeta.to(F64)).sum()
    got = iter(torch.autograd.grad(loss, [x for x in leaves if x is not None]))
    return [None if x is None else next(got) for x in leaves]
