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


def delta_errors(inp, scale=None, use_l2=True):
    """Standard deviations, in units of EPS, of the gradients of delta_grads token by token, from the chunk form
    with its roundings: first-order propagation of variances in fp64.  dq, dk [T, Hk] and dv [T, H] (a vector's
    2-norm), dg and dbeta [T, H].  A token's gradient may be far smaller than the terms that it is the sum of, and
    its error goes by them.  What is rounded:
      a product's operands, to EPS of each element;
      its accumulator, cut off at each of 3 inner / 16 steps (the terms hi hi, hi lo, lo hi of 16 products), by
      half an EPS on average of a partial sum that grows to the product: together 3 inner / 64 of it;
      a decay e^-x, by 2 EPS in the exponential and by x / 2 EPS in its argument (x 2^-24)."""
    (T, Hk, d), H, cu = inp["q"].shape, inp["v"].shape[1], inp["cu"]
    scale = d ** -0.5 if scale is None else scale
    q, k, v, g, beta, dy = (inp[x].to(F64) for x in ("q", "k", "v", "g", "beta", "dout"))
    rep = lambda x: x.repeat_interleave(H // Hk, 1)  # noqa: E731
    rq, rk = (rep(torch.rsqrt((x * x).sum(-1) + 1e-6) if use_l2 else torch.ones(T, Hk, dtype=F64)) for x in (q, k))
    q, k = rep(q) * rq[..., None] * scale, rep(k) * rk[..., None]
    out = {x: torch.zeros(T, H, dtype=F64) for x in ("dq", "dk", "dv", "dg", "dbeta")}

    def mul(A, B):  # (values, variances) of a product of two such pairs
        (a, va), (b, vb) = A, B
        c = a @ b
        return c, va @ b ** 2 + a ** 2 @ vb + 2 * a ** 2 @ b ** 2 + (3 * a.shape[1] / 64 * c) ** 2

    exact = lambda x: (x, torch.zeros_like(x))  # noqa: E731
    add = lambda A, B, s=1.0: (A[0] + s * B[0], A[1] + B[1])  # noqa: E731
    by = lambda f, A: (f * A[0], f ** 2 * A[1])  # noqa: E731
    # by a decay
    fade = lambda f, A, x: (f * A[0], f ** 2 * (A[1] + (4 + x ** 2 / 4) * A[0] ** 2))  # noqa: E731
    t = lambda A: (A[0].T, A[1].T)  # noqa: E731
    dot = lambda A, B: (A[0] * B[0], A[1] * B[0] ** 2 + A[0] ** 2 * (B[1] + 2 * B[0] ** 2))  # noqa: E731
    for n in range(len(cu) - 1):
        for h in range(H):
            S = exact(torch.zeros(d, d, dtype=F64) if inp["initial_state"] is None else inp["initial_state"][n, h].to(F64))
            chunks = []
            for c in range(cu[n], cu[n + 1], 64):
                i = slice(c, min(c + 64, cu[n + 1]))
                K, Q, V, Y, be, G = exact(k[i, h]), exact(q[i, h]), exact(v[i, h]), exact(dy[i, h]), beta[i, h], g[i, h]
                G = G.clamp(min=-128).cumsum(0)
                far, x, to_end = G[:, None] - G[None], G[:, None], (G[-1] - G)[:, None]
                D, b, tail = far.exp().tril(), x.exp(), to_end.exp()
                A = fade((be[:, None] * D).tril(-1), mul(K, t(K)), far)
                X = torch.linalg.solve_triangular(torch.eye(len(be), dtype=F64) + A[0], torch.eye(len(be), dtype=F64), upper=False)
                X = X, X ** 2 @ (A[1] + A[0] ** 2) @ X ** 2 + X ** 2
                W, Pm = mul(X, fade(be[:, None] * b, K, x)), fade(D, mul(Q, t(K)), far)
                U = add(mul(X, by(be[:, None], V)), mul(W, t(S)), -1.0)
                chunks.append((i, K, Q, V, Y, be, D, b, tail, X, W, Pm, U, S, far, x, to_end))
                S = add(fade(b[-1], S, x[-1]), mul(t(fade(tail, U, to_end)), K))
            dS = exact(torch.zeros(d, d, dtype=F64) if inp["dfinal_state"] is None else inp["dfinal_state"][n, h].to(F64))
            for i, K, Q, V, Y, be, D, b, tail, X, W, Pm, U, S, far, x, to_end in reversed(chunks):
                E = fade(tail, mul(K, t(dS)), to_end)
                dR = mul(t(X), add(mul(t(Pm), Y), E))
                dP, Z = fade(D, mul(Y, t(U)), far), fade(-D.tril(-1), mul(dR, t(U)), far)
                dQ, F = add(fade(b, mul(Y, S), x), mul(dP, K)), add(mul(Z, K), fade(b, mul(dR, S), x), -1.0)
                Hd, rest = fade(tail, mul(U, dS), to_end), add(mul(t(dP), Q), mul(t(Z), by(be[:, None], K)))
                dK = add(by(be[:, None], F), add(Hd, rest))
                later = add(add(dot(dQ, Q), dot(by(be[:, None], F), K)), dot(rest, K))[1].sum(-1)
                out["dq"][i, h] = (scale * rq[i, h]) ** 2 * dQ[1].sum(-1)
                out["dk"][i, h] = rk[i, h] ** 2 * dK[1].sum(-1)
                out["dv"][i, h] = be ** 2 * dR[1].sum(-1)
                out["dbeta"][i, h] = (dot(dR, V)[1] + dot(F, K)[1]).sum(-1)
                hk = dot(Hd, K)[1].sum(-1)
                out["dg"][i, h] = later.flip(0).cumsum(0).flip(0) + hk.cumsum(0) - hk + b[-1] ** 2 * dot(S, dS)[1].sum()
                dS = add(add(fade(b[-1], dS, x[-1]), mul(t(Y), add(fade(b, Q, x), mul(Pm, W), -1.0))), mul(t(E), W), -1.0)
    for x in ("dq", "dk"):
        out[x] = out[x].reshape(T, Hk, H // Hk).sum(-1)
    return {x: y.sqrt() for x, y in out.items()}


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
