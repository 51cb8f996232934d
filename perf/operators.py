"""The operators of the training form, as cases to be measured: inputs, one pass, and the work of it.

A layer that is trained needs the gradients of what its forward pass calls.  Four operators:

  chunk_bwd        gdn_chunk_bwd: the gradients of the gated delta rule (gdn_chunk_fwd without gate and
                   convolution) with respect to q, k, v, g, beta and the initial state.
  rmsnorm_bwd      gdn_gate_rmsnorm_silu_bwd: the gradients of the gated output norm.
  groupnorm_fwd,   gdn_gate_groupnorm_silu and gdn_gate_groupnorm_silu_bwd: the output norm taken as a
  groupnorm_bwd    group norm over the heads (mean and variance of each head's channels, channels last),
                   with an affine map per channel and a SiLU, of the gate z or of the result itself.
  decay_bwd        gdn_decay_from_logits_bwd: the gradients of the gate preparation.

A case is a dict of plain values; `prepare` draws its inputs on the GPU from a seed, `run` is one pass
(the plain form in torch where `own` is false, this package's call where it is true), `exact` the same
outputs in 64 bits.  Sizes are those of the package's own workloads (synthetic.py) and tests, and
ragged ones beside them.
"""
import math

import torch

own = False

CHUNK = 64
BF16, F32 = "bf16", "f32"


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the smallest call: one short sequence in fp32 (the tiny workload's sizes), launch-bound
        dict(name="delta tiny f32", op="chunk_bwd", lengths="256", H=2, Hk=2, d=64, dtype=F32, a_mean=-1.0,
             carried=False),
        # a training step on the prefill workload's sizes
        dict(name="delta prefill", op="chunk_bwd", lengths="4096,4096", H=16, Hk=16, d=128, dtype=BF16,
             a_mean=-1.0, carried=False),
        # packed documents of very different lengths, grouped query/key heads, states carried in and out
        # (a longer document cut into pieces), head size 64
        dict(name="delta packed gva d64", op="chunk_bwd", lengths="1,37,513,2048,64,1333,700", H=8, Hk=2, d=64,
             dtype=BF16, a_mean=-1.0, carried=True),
        # long-context training: one sequence, 32 heads, decays close to 1 (the long workload's draw)
        dict(name="delta long", op="chunk_bwd", lengths="16384", H=32, Hk=32, d=128, dtype=BF16, a_mean=-4.0,
             carried=True),
        # the output gate's gradient after the prefill workload (bf16 activations) ...
        dict(name="rms bwd prefill", op="rmsnorm_bwd", rows=8192, heads=16, d=128, dtype=BF16, weight=True),
        # ... and on a short fp32 batch of d = 64 heads with an odd number of rows
        dict(name="rms bwd short f32", op="rmsnorm_bwd", rows=257, heads=3, d=64, dtype=F32, weight=True),
        # the group norm over heads: a training or prefill pass, gated
        dict(name="group fwd prefill", op="groupnorm_fwd", rows=8192, heads=16, d=128, dtype=BF16, gated=True),
        # one decode step of a few sequences, activation on the norm itself: latency
        dict(name="group fwd decode", op="groupnorm_fwd", rows=5, heads=16, d=64, dtype=F32, gated=False),
        dict(name="group bwd prefill", op="groupnorm_bwd", rows=8192, heads=16, d=128, dtype=BF16, gated=True),
        # groups whose size is no power of two, activation on the norm itself, fp32, ragged rows
        dict(name="group bwd odd f32", op="groupnorm_bwd", rows=1777, heads=12, d=80, dtype=F32, gated=False),
        # gate preparation of a long batch, and of a short one
        dict(name="decay bwd long", op="decay_bwd", rows=131072, heads=32),
        dict(name="decay bwd tiny", op="decay_bwd", rows=513, heads=6),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk_bwd", "chunk_bwd", "rmsnorm_bwd", "groupnorm_fwd", "groupnorm_bwd", "decay_bwd"])
    if op == "chunk_bwd":
        d = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8])
        H = Hk * rng.choice([1, 1, 2, 4])
        n = rng.choice([1, 1, 2, 3, 6])
        lengths = [_log_int(rng, 1, min(4096, 16384 // n)) for _ in range(n)]
        dtype = rng.choice([BF16, BF16, F32])
        return dict(op=op, lengths=",".join(map(str, lengths)), H=H, Hk=Hk, d=d, dtype=dtype,
                    a_mean=rng.choice([-1.0, -4.0]), carried=rng.random() < 0.5)
    if op == "decay_bwd":
        return dict(op=op, rows=_log_int(rng, 1, 131072), heads=rng.randint(1, 32))
    rows, heads = _log_int(rng, 1, 8192), rng.randint(1, 16)
    dtype = rng.choice([BF16, F32])
    if op == "rmsnorm_bwd":
        return dict(op=op, rows=rows, heads=heads, d=rng.choice([32, 64, 96, 128]), dtype=dtype,
                    weight=rng.random() < 0.7)
    return dict(op=op, rows=rows, heads=heads, d=rng.choice([64, 128, rng.randint(8, 128)]), dtype=dtype,
                gated=rng.random() < 0.6)


def _dt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    op = case["op"]
    s = dict(case=case, op=op)
    if op == "chunk_bwd":
        dt, H, Hk, d = _dt(case), case["H"], case["Hk"], case["d"]
        lengths = _lengths(case)
        T, n = sum(lengths), len(lengths)
        offs = [0]
        for L in lengths:
            offs.append(offs[-1] + L)
        s.update(q=randn(T, Hk, d).to(dt), k=randn(T, Hk, d).to(dt), v=randn(T, H, d).to(dt))
        A = torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(8.0))
        s.update(g=-A * torch.nn.functional.softplus(randn(T, H) + case["a_mean"]),
                 beta=torch.sigmoid(randn(T, H)), dout=randn(T, H, d).to(dt),
                 initial_state=randn(n, H, d, d) * 0.02 if case["carried"] else None,
                 dfinal_state=randn(n, H, d, d) * 0.05 if case["carried"] else None,
                 cu_seqlens=torch.tensor(offs, dtype=torch.int32, device=dev) if n > 1 else None)
        # where each sequence's tokens lie in the batch padded to whole chunks (the plain form's view)
        P = -(-max(lengths) // CHUNK) * CHUNK
        pos = torch.arange(P, device=dev)
        ln = torch.tensor(lengths, device=dev)[:, None]
        st = torch.tensor(offs[:-1], device=dev)[:, None]
        s["valid"] = pos[None, :] < ln
        s["index"] = torch.where(s["valid"], st + pos[None, :], torch.zeros_like(st))
    elif op == "decay_bwd":
        T, H = case["rows"], case["heads"]
        s.update(a=randn(T, H) - 1.0, A_log=torch.rand(H, generator=gen, device=dev) * math.log(8.0),
                 dt_bias=randn(H) * 0.5, b=randn(T, H), dg=randn(T, H), dbeta=randn(T, H))
    else:
        dt, rows, heads, d = _dt(case), case["rows"], case["heads"], case["d"]
        s.update(y=(randn(rows, heads, d) * 0.5).to(dt), eps=1e-6)
        if op == "rmsnorm_bwd":
            s.update(z=randn(rows, heads, d), weight=1.0 + 0.1 * randn(d) if case["weight"] else None,
                     dout=randn(rows, heads, d).to(dt))
        else:
            s.update(z=randn(rows, heads, d) if case["gated"] else None, weight=1.0 + 0.1 * randn(heads, d),
                     bias=0.1 * randn(heads, d))
            if op == "groupnorm_bwd":
                s.update(dout=randn(rows, heads, d).to(dt))
    return s


def run(s):
    return (_own if own else _plain)[s["op"]](s)


# ---- this package's calls -----------------------------------------------------------------------

def _own_chunk_bwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    dq, dk, dv, dg, dbeta, dS0 = gdn.gdn_chunk_bwd(
        s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], cu_seqlens=s["cu_seqlens"],
        initial_state=s["initial_state"], dfinal_state=s["dfinal_state"])
    out = dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta)
    if s["initial_state"] is not None:
        out["dinitial_state"] = dS0
    return out


def _own_rmsnorm_bwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    dy, dz, dw = gdn.gdn_gate_rmsnorm_silu_bwd(s["dout"], s["y"], s["z"], s["weight"], eps=s["eps"])
    return dict(dy=dy, dz=dz) if s["weight"] is None else dict(dy=dy, dz=dz, dweight=dw)


def _own_groupnorm_fwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    return dict(out=gdn.gdn_gate_groupnorm_silu(s["y"], s["z"], s["weight"], s["bias"], eps=s["eps"]))


def _own_groupnorm_bwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    dy, dz, dw, db = gdn.gdn_gate_groupnorm_silu_bwd(s["dout"], s["y"], s["z"], s["weight"], s["bias"],
                                                     eps=s["eps"])
    out = dict(dy=dy, dweight=dw, dbias=db)
    if s["z"] is not None:
        out["dz"] = dz
    return out


def _own_decay_bwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    da, dA_log, ddt_bias, db = gdn.gdn_decay_from_logits_bwd(s["a"], s["A_log"], s["dt_bias"], s["b"], s["dg"],
                                                             s["dbeta"])
    return dict(da=da, dA_log=dA_log, ddt_bias=ddt_bias, db=db)


_own = dict(chunk_bwd=_own_chunk_bwd, rmsnorm_bwd=_own_rmsnorm_bwd, groupnorm_fwd=_own_groupnorm_fwd,
            groupnorm_bwd=_own_groupnorm_bwd, decay_bwd=_own_decay_bwd)


# ---- plain forms: elementary torch operations in 32 bits -------------------------------------

def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower triangular A [..., C, C], by doubling the inverted diagonal blocks:
    X <- X - X A_off X with A_off the blocks that join two neighbours."""
    C = A.shape[-1]
    i = torch.arange(C, device=A.device)
    X = torch.eye(C, device=A.device, dtype=A.dtype).expand_as(A)
    size = 1
    while size < C:
        joins = (i[:, None] // (2 * size) == i[None, :] // (2 * size)) & (i[:, None] // size > i[None, :] // size)
        X = X - X @ (A * joins) @ X
        size *= 2
    return X


def _plain_chunk_fwd(q, k, v, g, beta, S):
    """The chunked form on whole chunks: q, k, v [n, H, N, C, d], g, beta [n, H, N, C], S [n, H, d, d].
    Returns the outputs and the final states."""
    d, C = q.shape[-1], CHUNK
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6) * (1.0 / math.sqrt(d))
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    G = g.cumsum(-1)
    i = torch.arange(C, device=q.device)
    low = i[:, None] >= i[None, :]
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, 0.0)) * low
    kk = k @ k.transpose(-1, -2)
    X = _unit_lower_inverse(beta[..., None] * kk * decay * (i[:, None] > i[None, :]))
    W = X @ (k * (beta * G.exp())[..., None])
    U0 = X @ (v * beta[..., None])
    att = (q @ k.transpose(-1, -2)) * decay
    qd, kd, last = q * G.exp()[..., None], k * torch.exp(G[..., -1:] - G)[..., None], G[..., -1].exp()
    out = []
    for W_c, U_c, att_c, qd_c, kd_c, last_c in zip(W.unbind(2), U0.unbind(2), att.unbind(2), qd.unbind(2),
                                                   kd.unbind(2), last.unbind(2)):
        St = S.transpose(-1, -2)
        U = U_c - W_c @ St
        out.append(qd_c @ St + att_c @ U)
        S = S * last_c[..., None, None] + U.transpose(-1, -2) @ kd_c
    return torch.stack(out, 2), S


def _plain_chunk_bwd(s):
    case = s["case"]
    n, (H, Hk, d) = s["valid"].shape[0], (case["H"], case["Hk"], case["d"])
    idx, valid = s["index"], s["valid"]
    with torch.enable_grad():
        q, k, v, g, beta = (s[x].float().requires_grad_() for x in ("q", "k", "v", "g", "beta"))
        S0 = s["initial_state"]
        S0 = torch.zeros(n, H, d, d, device=q.device) if S0 is None else S0.detach().clone()
        S0.requires_grad_()

        def chunks(x):  # [T, h, ...] -> [n, h, N, C, ...], zeros past a sequence's end
            x = x[idx] * valid.view(valid.shape + (1,) * (x.dim() - 1))
            x = x.transpose(1, 2)
            return x.reshape(x.shape[0], x.shape[1], -1, CHUNK, *x.shape[3:])

        rep = H // Hk
        out, S = _plain_chunk_fwd(chunks(q).repeat_interleave(rep, 1), chunks(k).repeat_interleave(rep, 1),
                                  chunks(v), chunks(g), chunks(beta), S0)
        dout = chunks(s["dout"].float())
        dS = s["dfinal_state"]
        dS = torch.zeros_like(S) if dS is None else dS
        dq, dk, dv, dg, db, dS0 = torch.autograd.grad((out, S), (q, k, v, g, beta, S0), (dout, dS))
    dt = s["q"].dtype
    res = dict(dq=dq.to(dt), dk=dk.to(dt), dv=dv.to(dt), dg=dg, dbeta=db)
    if s["initial_state"] is not None:
        res["dinitial_state"] = dS0
    return res


def _silu_and_slope(z):
    sg = torch.sigmoid(z)
    return z * sg, sg * (1.0 + z * (1.0 - sg))


def _plain_rmsnorm_bwd(s):
    y, z, do = s["y"].float(), s["z"], s["dout"].float()
    w = 1.0 if s["weight"] is None else s["weight"]
    r = torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"])
    n = y * r
    act, slope = _silu_and_slope(z)
    dm = do * act
    dn = dm * w
    dy = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    res = dict(dy=dy.to(s["y"].dtype), dz=do * n * w * slope)
    if s["weight"] is not None:
        res["dweight"] = (dm * n).sum((0, 1))
    return res


def _normalised(y, eps):
    mu = y.mean(-1, keepdim=True)
    c = y - mu
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + eps)
    return c * r, r


def _plain_groupnorm_fwd(s):
    n, _ = _normalised(s["y"].float(), s["eps"])
    m = n * s["weight"] + s["bias"]
    out = m * torch.sigmoid(m) if s["z"] is None else m * s["z"] * torch.sigmoid(s["z"])
    return dict(out=out.to(s["y"].dtype))


def _plain_groupnorm_bwd(s):
    n, r = _normalised(s["y"].float(), s["eps"])
    do, z = s["dout"].float(), s["z"]
    m = n * s["weight"] + s["bias"]
    act, slope = _silu_and_slope(m if z is None else z)
    dm = do * (slope if z is None else act)
    dn = dm * s["weight"]
    dy = r * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    res = dict(dy=dy.to(s["y"].dtype), dweight=(dm * n).sum(0), dbias=dm.sum(0))
    if z is not None:
        res["dz"] = do * m * slope
    return res


def _plain_decay_bwd(s):
    x = s["a"] + s["dt_bias"]
    A = s["A_log"].exp()
    sp = torch.where(x > 20.0, x, torch.log1p(torch.exp(x.clamp(max=20.0))))
    beta = torch.sigmoid(s["b"])
    da = -s["dg"] * A * torch.sigmoid(x)
    return dict(da=da, dA_log=-(s["dg"] * sp).sum(0) * A, ddt_bias=da.sum(0), db=s["dbeta"] * beta * (1.0 - beta))


_plain = dict(chunk_bwd=_plain_chunk_bwd, rmsnorm_bwd=_plain_rmsnorm_bwd, groupnorm_fwd=_plain_groupnorm_fwd,
              groupnorm_bwd=_plain_groupnorm_bwd, decay_bwd=_plain_decay_bwd)


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "chunk_bwd":
        T, n = sum(_lengths(case)), len(_lengths(case))
        H, Hk, d, e = case["H"], case["Hk"], case["d"], 2 if case["dtype"] == BF16 else 4
        moved = e * T * d * (4 * Hk + 3 * H)          # q, k, dq, dk; v, dout, dv
        moved += 4 * 4 * T * H                        # g, beta and their gradients
        if case["carried"]:
            moved += 3 * 4 * n * H * d * d            # initial state, dfinal in; dinitial out
        # per token and head, d x d products: S k, u k^T again; dy q^T, S^T dy, dS k, dS^T u, S^T du, du k^T
        return dict(bytes=moved, flops=8 * 2 * T * H * d * d)
    if op == "decay_bwd":
        n = case["rows"] * case["heads"]
        return dict(bytes=4 * (6 * n + 4 * case["heads"]), flops=20 * n)
    n, c, e = case["rows"] * case["heads"] * case["d"], case["heads"] * case["d"], 2 if case["dtype"] == BF16 else 4
    if op == "rmsnorm_bwd":                           # dout, y, z in; dy, dz out
        return dict(bytes=n * (3 * e + 8) + (8 * case["d"] if case["weight"] else 0), flops=25 * n)
    gate = 4 if case["gated"] else 0
    if op == "groupnorm_fwd":
        return dict(bytes=n * (2 * e + gate) + 8 * c, flops=15 * n)
    return dict(bytes=n * (3 * e + 2 * gate) + 16 * c, flops=30 * n)


# ---- the same outputs in 64 bits, from the definitions ------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact[case["op"]](s)


def _exact_chunk_bwd(s):
    """The recurrence token by token, and its adjoint token by token backwards.
      P = alpha S, u = beta (v - P k), S' = P + u k^T, y = S' q."""
    case = s["case"]
    lengths = _lengths(case)
    n, H, Hk, d, Tm = len(lengths), case["H"], case["Hk"], case["d"], max(lengths)
    dev, f64 = s["q"].device, torch.float64
    rep = H // Hk
    idx, valid = s["index"][:, :Tm], s["valid"][:, :Tm]

    def padded(x):                                    # [T, h, ...] -> [Tm, n, h, ...]
        x = x.to(f64)[idx] * valid.view(n, Tm, *([1] * (x.dim() - 1)))
        return x.transpose(0, 1)

    qr, kr = padded(s["q"]).repeat_interleave(rep, 2), padded(s["k"]).repeat_interleave(rep, 2)
    v, g, b, dy = padded(s["v"]), padded(s["g"]), padded(s["beta"]), padded(s["dout"])
    rq, rk = ((x.square().sum(-1, keepdim=True) + 1e-6) ** -0.5 for x in (qr, kr))
    sc = d ** -0.5
    q, k, alpha = qr * rq * sc, kr * rk, g.exp()

    def step(S, t):
        P = S * alpha[t][..., None, None]
        e = v[t] - torch.einsum("nhij,nhj->nhi", P, k[t])
        return P, e, P + (b[t][..., None] * e)[..., :, None] * k[t][..., None, :]

    S = torch.zeros(n, H, d, d, dtype=f64, device=dev) if s["initial_state"] is None else s["initial_state"].to(f64)
    kept = []
    for t in range(Tm):                               # one state kept in 64
        if t % CHUNK == 0:
            kept.append(S)
        S = step(S, t)[2]
    dS = torch.zeros_like(S) if s["dfinal_state"] is None else s["dfinal_state"].to(f64)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(b)
    for c in range(len(kept) - 1, -1, -1):
        trail, S = [], kept[c]
        for t in range(c * CHUNK, min(Tm, (c + 1) * CHUNK)):
            P, e, S = step(S, t)
            trail.append((t, P, e, S))
        for t, P, e, S in reversed(trail):
            dq[t] = torch.einsum("nhij,nhi->nhj", S, dy[t])
            dS = dS + dy[t][..., :, None] * q[t][..., None, :]
            du = torch.einsum("nhij,nhj->nhi", dS, k[t])
            bt = b[t][..., None]
            db[t] = (du * e).sum(-1)
            dv[t] = bt * du
            dk[t] = torch.einsum("nhij,nhi->nhj", dS, bt * e) - torch.einsum("nhij,nhi->nhj", P, bt * du)
            dS = dS - (bt * du)[..., :, None] * k[t][..., None, :]
            dg[t] = (dS * P).sum((-1, -2))
            dS = dS * alpha[t][..., None, None]
    xq, xk = qr * rq, kr * rk
    dqr = rq * sc * (dq - xq * (xq * dq).sum(-1, keepdim=True))
    dkr = rk * (dk - xk * (xk * dk).sum(-1, keepdim=True))
    dqr, dkr = (x.reshape(Tm, n, Hk, rep, d).sum(3) for x in (dqr, dkr))

    def packed(x):
        x = x.transpose(0, 1)
        return torch.cat([x[i, :L] for i, L in enumerate(lengths)])

    out = dict(dq=packed(dqr), dk=packed(dkr), dv=packed(dv), dg=packed(dg), dbeta=packed(db))
    if s["initial_state"] is not None:
        out["dinitial_state"] = dS
    return out


def _exact_norm(s):
    """The gated norm by its definition, differentiated in 64 bits."""
    op, f64 = s["op"], torch.float64
    y, z, w, b = (None if s.get(x) is None else s[x].to(f64).requires_grad_() for x in ("y", "z", "weight", "bias"))
    if op == "rmsnorm_bwd":
        m = y / (y.square().mean(-1, keepdim=True) + s["eps"]).sqrt()
        m = m if w is None else m * w
    else:
        mu = y.mean(-1, keepdim=True)
        var = (y - mu).square().mean(-1, keepdim=True)
        m = (y - mu) / (var + s["eps"]).sqrt() * w + b
    t = m if z is None else z
    out = (m if z is not None else 1.0) * (t / (1.0 + torch.exp(-t)))
    if op == "groupnorm_fwd":
        return dict(out=out.detach())
    names = [x for x, t in (("dy", y), ("dz", z), ("dweight", w), ("dbias", b)) if t is not None]
    grads = torch.autograd.grad(out, [t for t in (y, z, w, b) if t is not None], s["dout"].to(f64))
    return dict(zip(names, grads))


def _exact_decay_bwd(s):
    a, A_log, dt, b = (s[x].double().requires_grad_() for x in ("a", "A_log", "dt_bias", "b"))
    x = a + dt
    g = -A_log.exp() * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    beta = 1.0 / (1.0 + torch.exp(-b))
    da, dA, ddt, db = torch.autograd.grad((g, beta), (a, A_log, dt, b), (s["dg"].double(), s["dbeta"].double()))
    return dict(da=da, dA_log=dA, ddt_bias=ddt, db=db)


_exact = dict(chunk_bwd=_exact_chunk_bwd, rmsnorm_bwd=_exact_norm, groupnorm_fwd=_exact_norm,
              groupnorm_bwd=_exact_norm, decay_bwd=_exact_decay_bwd)
