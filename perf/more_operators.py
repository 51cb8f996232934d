"""A state space layer beside the delta rule, and what prepares queries and keys, as cases to be measured.

Three operators, each for whole prompts, for the tokens that follow and for training:

  short_conv   gdn_short_conv_fwd, gdn_short_conv_step, gdn_short_conv_bwd: the causal depthwise convolution
               with four taps (and SiLU) that the inputs of a recurrence come out of, as a call of its own.
  ssm          gdn_ssm_chunk_fwd, gdn_ssm_step, gdn_ssm_chunk_bwd: the selective state space scan.  Per head a
               state S [head size, state size] with one decay per token and head,
                   S_t = exp(-exp(A_log) dt_t) S_{t-1} + dt_t x_t B_t^T,   y_t = S_t C_t + D x_t,
                   dt_t = softplus(a_t + dt_bias);  heads share B and C in groups.
  qk_norm_rope gdn_qk_norm_rope, gdn_qk_norm_rope_bwd: queries and keys normalised per head (RMS with a weight,
               or to length one) and rotated by their position, in one pass.

A case is a dict of plain values; `prepare` draws its inputs on the GPU from a seed, `run` is one pass (the
plain form in torch where `own` is false, this package's call where it is true), `exact` the same outputs in
64 bits.  x, B and C are slices of one tensor (what the convolution leaves), q and k slices of a mixed
projection: rows with a stride, as a layer has them.
"""
import math

import torch

own = False

CHUNK = 64
TAPS = 4
BF16, F32 = "bf16", "f32"


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the convolution of a prefill batch: 64 heads of 64 channels, B and C of one group of 128
        dict(name="conv prefill", op="conv_fwd", lengths="4096,4096", dim=4352, dtype=BF16, bias=True, carried=False),
        # one token for a handful of sequences of a small fp32 layer: latency
        dict(name="conv token few", op="conv_step", N=5, T=1, slots=9, dim=384, dtype=F32, bias=False),
        # training on packed documents of odd lengths, histories carried in and their gradients out
        dict(name="conv train packed", op="conv_bwd", lengths="1,2,777,2048,3,1301", dim=2304, dtype=BF16, bias=True,
             carried=True),
        # the smallest prompt: one short sequence, two fp32 heads
        dict(name="ssm tiny f32", op="ssm_fwd", lengths="200", H=2, G=1, P=64, N=64, dtype=F32, carried=False),
        # prefill of two long prompts
        dict(name="ssm prefill", op="ssm_fwd", lengths="4096,4096", H=64, G=1, P=64, N=128, dtype=BF16, carried=False),
        # a packed batch of very different prompts, heads of 128, three groups, states carried on
        dict(name="ssm packed odd", op="ssm_fwd", lengths="1,37,513,3001,64,1333,700", H=12, G=3, P=128, N=64,
             dtype=BF16, carried=True),
        # a serving batch: one token for each of 256 sequences, states in a pool
        dict(name="ssm token batch", op="ssm_step", N=256, T=1, slots=300, H=32, G=1, P=64, N_state=128, dtype=BF16),
        # a few sequences, four tokens each (drafted tokens): latency
        dict(name="ssm tokens few", op="ssm_step", N=3, T=4, slots=8, H=8, G=2, P=64, N_state=128, dtype=BF16),
        # a training step on two long sequences
        dict(name="ssm train", op="ssm_bwd", lengths="4096,4096", H=32, G=2, P=64, N=128, dtype=BF16, carried=False),
        # training in fp32 on short packed sequences, states carried
        dict(name="ssm train odd f32", op="ssm_bwd", lengths="65,1,300,127", H=6, G=2, P=64, N=64, dtype=F32,
             carried=True),
        # queries and keys of a prefill batch, grouped heads, half of each head rotated
        dict(name="qk prefill", op="qk_fwd", T=8192, Hq=16, Hk=4, d=128, rot=64, norm="rms", interleaved=False,
             dtype=BF16),
        # their gradients, heads normalised to length one, pairs of neighbours rotated, odd number of tokens
        dict(name="qk train odd", op="qk_bwd", T=3001, Hq=16, Hk=16, d=64, rot=64, norm="l2", interleaved=True,
             dtype=BF16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_step", "conv_bwd", "ssm_fwd", "ssm_fwd", "ssm_step", "ssm_bwd", "ssm_bwd",
                     "qk_fwd", "qk_bwd"])
    dtype = rng.choice([BF16, BF16, F32])
    n = rng.choice([1, 1, 2, 3, 6])
    lengths = ",".join(str(_log_int(rng, 1, 6144 // n)) for _ in range(n))
    if op in ("conv_fwd", "conv_bwd"):
        return dict(op=op, lengths=lengths, dim=8 * _log_int(rng, 4, 320), dtype=dtype, bias=rng.random() < 0.5,
                    carried=rng.random() < 0.5)
    if op in ("conv_step", "ssm_step"):
        N, T = _log_int(rng, 1, 200), rng.choice([1, 1, 2, 3, 4])
        slots = N + rng.randint(0, 20)
        if op == "conv_step":
            return dict(op=op, N=N, T=T, slots=slots, dim=8 * _log_int(rng, 4, 640), dtype=dtype,
                        bias=rng.random() < 0.5)
        G = rng.choice([1, 1, 2, 3])
        return dict(op=op, N=N, T=T, slots=slots, H=G * rng.randint(1, 8), G=G, P=rng.choice([64, 128]),
                    N_state=rng.choice([64, 128]), dtype=dtype)
    if op in ("ssm_fwd", "ssm_bwd"):
        G = rng.choice([1, 1, 2, 3])
        return dict(op=op, lengths=lengths, H=G * rng.randint(1, 8), G=G, P=rng.choice([64, 128]),
                    N=rng.choice([64, 128]), dtype=dtype, carried=rng.random() < 0.5)
    Hk, d = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 96, 128, 256])
    return dict(op=op, T=_log_int(rng, 1, 6144), Hq=Hk * rng.choice([1, 2, 3]), Hk=Hk, d=d,
                rot=rng.choice([d, d, d // 2, d // 4]), norm=rng.choice(["rms", "l2"]),
                interleaved=rng.random() < 0.4, dtype=dtype)


def _dt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def _offsets(lengths):
    offs = [0]
    for L in lengths:
        offs.append(offs[-1] + L)
    return offs


MAX_POSITION = 32768


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32)

    op, dt = case["op"], _dt(case)
    s = dict(case=case, op=op)
    if op in ("conv_fwd", "conv_bwd", "ssm_fwd", "ssm_bwd"):
        lengths = _lengths(case)
        offs, n, T = _offsets(lengths), len(lengths), sum(lengths)
        s["cu_seqlens"] = torch.tensor(offs, dtype=torch.int32, device=dev) if n > 1 else None
    if op.endswith("_step"):
        slots = torch.randperm(case["slots"], generator=gen, device=dev)[:case["N"]]
        s["slots"], s["state_indices"] = slots, slots.int()

    if op.startswith("conv"):
        dim = case["dim"]
        s.update(weight=randn(dim, TAPS) * 0.5, bias=0.1 * randn(dim) if case["bias"] else None)
        if op == "conv_step":
            s.update(x=randn(case["N"], case["T"], dim).to(dt), state=randn(case["slots"], dim, TAPS - 1))
            return s
        # a layer's input projection: the convolved channels lie beside the gate's
        s["x"] = randn(T, dim + 512).to(dt)[:, 512:]
        s["state"] = randn(n, dim, TAPS - 1) if case["carried"] else None
        if op == "conv_bwd":
            s.update(dout=randn(T, dim).to(dt), dstate_out=randn(n, dim, TAPS - 1) if case["carried"] else None)
        # rows of the batch in which each sequence's tokens follow the three rows of its history (the plain form)
        seq = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(lengths, device=dev), output_size=T)
        ends = torch.tensor(offs[1:], device=dev) + 3 * torch.arange(1, n + 1, device=dev)
        back = torch.arange(-(TAPS - 1), 0, device=dev)
        s["rows"] = torch.arange(T, device=dev) + 3 * (seq + 1)
        s["history"] = (torch.tensor(offs[:-1], device=dev) + 3 * torch.arange(1, n + 1, device=dev))[:, None] + back
        s["last"] = ends[:, None] + back
        return s

    if op.startswith("ssm"):
        H, G, P = case["H"], case["G"], case["P"]
        Ns = case["N_state"] if op == "ssm_step" else case["N"]
        rows = (case["N"], case["T"]) if op == "ssm_step" else (T,)
        mixed = randn(*rows, H * P + 2 * G * Ns)
        mixed = (mixed * torch.sigmoid(mixed)).to(dt)      # what the convolution and its SiLU leave
        x, B, C = mixed.split([H * P, G * Ns, G * Ns], -1)
        s.update(x=x.unflatten(-1, (H, P)), B=B.unflatten(-1, (G, Ns)), C=C.unflatten(-1, (G, Ns)))
        # steps of 0.001 to 0.1 and decay rates of 1 to 16, the usual start of such a layer
        dt0 = torch.exp(math.log(1e-3) + rand(H) * math.log(1e2))
        s.update(a=randn(*rows, H), dt_bias=dt0 + torch.log(-torch.expm1(-dt0)), A_log=torch.log(1.0 + 15.0 * rand(H)),
                 D=1.0 + 0.1 * randn(H))
        if op == "ssm_step":
            s["state"] = randn(case["slots"], H, P, Ns)
            return s
        s["initial_state"] = randn(n, H, P, Ns) if case["carried"] else None
        if op == "ssm_bwd":
            s.update(dout=randn(T, H, P).to(dt), dfinal_state=randn(n, H, P, Ns) * 0.1 if case["carried"] else None)
        # where each sequence's tokens lie in the batch padded to whole chunks (the plain form's view)
        pos = torch.arange(-(-max(lengths) // CHUNK) * CHUNK, device=dev)
        st = torch.tensor(offs[:-1], device=dev)[:, None]
        s["valid"] = pos[None, :] < torch.tensor(lengths, device=dev)[:, None]
        s["index"] = torch.where(s["valid"], st + pos[None, :], torch.zeros_like(st))
        return s

    T, Hq, Hk, d, rot = case["T"], case["Hq"], case["Hk"], case["d"], case["rot"]
    mixed = randn(T, Hq + 2 * Hk, d).to(dt)                # queries, keys and values of one projection
    s.update(q=mixed[:, :Hq], k=mixed[:, Hq:Hq + Hk], eps=1e-6)
    s.update(q_weight=1.0 + 0.1 * randn(d) if case["norm"] == "rms" else None,
             k_weight=1.0 + 0.1 * randn(d) if case["norm"] == "rms" else None)
    # cosines and sines of every position, and a packed batch's positions: runs that start anywhere
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    angle = torch.arange(MAX_POSITION, device=dev, dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float()
    starts = torch.randint(0, MAX_POSITION - T, (4,), generator=gen, device=dev)
    t = torch.arange(T, device=dev)
    s["positions"] = (starts[t * 4 // T] + t).int()
    if op == "qk_bwd":
        s.update(dq_out=randn(T, Hq, d).to(dt), dk_out=randn(T, Hk, d).to(dt))
    return s


def run(s):
    return (_own if own else _plain)[s["op"]](s)


# ---- this package's calls -----------------------------------------------------------------------

def _own_conv_fwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    out, state = gdn.gdn_short_conv_fwd(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu_seqlens"],
                                        conv_state=s["state"])
    return dict(out=out, state=state)


def _own_conv_step(s):
    import gated_deltanet_recurrence_gb300 as gdn
    out = gdn.gdn_short_conv_step(s["x"], s["weight"], s["state"], s["bias"], state_indices=s["state_indices"])
    return dict(out=out, state=s["state"])


def _own_conv_bwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    dx, dw, db, ds = gdn.gdn_short_conv_bwd(s["dout"], s["x"], s["weight"], s["bias"], cu_seqlens=s["cu_seqlens"],
                                            conv_state=s["state"], dconv_state_out=s["dstate_out"])
    return {k: v for k, v in dict(dx=dx, dweight=dw, dbias=db, dstate=ds).items() if v is not None}


def _own_ssm_fwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    out, state = gdn.gdn_ssm_chunk_fwd(s["x"], s["B"], s["C"], s["a"], s["A_log"], dt_bias=s["dt_bias"], D=s["D"],
                                       cu_seqlens=s["cu_seqlens"], initial_state=s["initial_state"])
    return dict(out=out, state=state)


def _own_ssm_step(s):
    import gated_deltanet_recurrence_gb300 as gdn
    out = gdn.gdn_ssm_step(s["x"], s["B"], s["C"], s["a"], s["A_log"], s["state"], dt_bias=s["dt_bias"], D=s["D"],
                           state_indices=s["state_indices"])
    return dict(out=out, state=s["state"])


_SSM_GRADS = ("dx", "dB", "dC", "da", "dA_log", "ddt_bias", "dD", "dinitial_state")


def _own_ssm_bwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    grads = gdn.gdn_ssm_chunk_bwd(s["dout"], s["x"], s["B"], s["C"], s["a"], s["A_log"], dt_bias=s["dt_bias"],
                                  D=s["D"], cu_seqlens=s["cu_seqlens"], initial_state=s["initial_state"],
                                  dfinal_state=s["dfinal_state"])
    return {k: v for k, v in zip(_SSM_GRADS, grads) if v is not None}


def _qk_args(s):
    import gated_deltanet_recurrence_gb300 as gdn
    return dict(positions=s["positions"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                norm=gdn.GDN_NORM_RMS if s["case"]["norm"] == "rms" else gdn.GDN_NORM_L2,
                interleaved=s["case"]["interleaved"])


def _own_qk_fwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    q, k = gdn.gdn_qk_norm_rope(s["q"], s["k"], s["cos_sin"], **_qk_args(s))
    return dict(q=q, k=k)


def _own_qk_bwd(s):
    import gated_deltanet_recurrence_gb300 as gdn
    dq, dk, dwq, dwk = gdn.gdn_qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["cos_sin"], **_qk_args(s))
    return {k: v for k, v in dict(dq=dq, dk=dk, dq_weight=dwq, dk_weight=dwk).items() if v is not None}


_own = dict(conv_fwd=_own_conv_fwd, conv_step=_own_conv_step, conv_bwd=_own_conv_bwd, ssm_fwd=_own_ssm_fwd,
            ssm_step=_own_ssm_step, ssm_bwd=_own_ssm_bwd, qk_fwd=_own_qk_fwd, qk_bwd=_own_qk_bwd)


# ---- plain forms: elementary torch operations in 32 bits -------------------------------------

def _with_history(s):
    """The inputs in fp32, each sequence's tokens behind the three rows of its history."""
    n, dim = s["history"].shape[0], s["case"]["dim"]
    xp = torch.zeros(s["x"].shape[0] + 3 * n, dim, device=s["x"].device)
    xp[s["rows"]] = s["x"].float()
    if s["state"] is not None:
        xp[s["history"]] = s["state"].transpose(1, 2)
    return xp


def _convolved(s, xp):
    w, r = s["weight"], s["rows"]
    c = xp[r - 3] * w[:, 0] + xp[r - 2] * w[:, 1] + xp[r - 1] * w[:, 2] + xp[r] * w[:, 3]
    return c if s["bias"] is None else c + s["bias"]


def _plain_conv_fwd(s):
    xp = _with_history(s)
    c = _convolved(s, xp)
    return dict(out=(c * torch.sigmoid(c)).to(s["x"].dtype), state=xp[s["last"]].transpose(1, 2).contiguous())


def _plain_conv_step(s):
    T = s["case"]["T"]
    h = torch.cat([s["state"][s["slots"]].transpose(1, 2), s["x"].float()], 1)     # [N, 3 + T, dim]
    w = s["weight"]
    c = h[:, :T] * w[:, 0] + h[:, 1:T + 1] * w[:, 1] + h[:, 2:T + 2] * w[:, 2] + h[:, 3:] * w[:, 3]
    c = c if s["bias"] is None else c + s["bias"]
    s["state"][s["slots"]] = h[:, T:].transpose(1, 2)
    return dict(out=(c * torch.sigmoid(c)).to(s["x"].dtype), state=s["state"])


def _plain_conv_bwd(s):
    xp, r, w = _with_history(s), s["rows"], s["weight"]
    c = _convolved(s, xp)
    sg = torch.sigmoid(c)
    dc = s["dout"].float() * sg * (1.0 + c * (1.0 - sg))
    dxp = torch.zeros_like(xp)
    dxp[r - 3] += dc * w[:, 0]
    dxp[r - 2] += dc * w[:, 1]
    dxp[r - 1] += dc * w[:, 2]
    dxp[r] += dc * w[:, 3]
    if s["dstate_out"] is not None:
        dxp[s["last"]] += s["dstate_out"].transpose(1, 2)
    res = dict(dx=dxp[r].to(s["x"].dtype), dweight=torch.stack(
        [(dc * xp[r - 3]).sum(0), (dc * xp[r - 2]).sum(0), (dc * xp[r - 1]).sum(0), (dc * xp[r]).sum(0)], -1))
    if s["bias"] is not None:
        res["dbias"] = dc.sum(0)
    if s["state"] is not None:
        res["dstate"] = dxp[s["history"]].transpose(1, 2).contiguous()
    return res


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(x.clamp(max=20.0))))


def _decays(G):
    """exp(G_i - G_j) for j <= i, else 0: G are running sums in 64 bits, their differences lose nothing."""
    i = torch.arange(G.shape[-1], device=G.device)
    low = i[:, None] >= i[None, :]
    return torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, 0.0).float()) * low


def _plain_ssm_chunks(x, B, C, g, dt, S0):
    """The chunked form on whole chunks: x [n, H, M, K, P], B, C [n, H, M, K, N], g, dt [n, H, M, K], S0
    [n, H, P, N].  Returns the outputs and the final states."""
    n, H, M, K, P = x.shape
    N = B.shape[-1]
    G = g.double().cumsum(-1)
    v = x * dt[..., None]
    inner = ((C @ B.transpose(-1, -2)) * _decays(G)) @ v
    left = torch.exp((G[..., -1:] - G).float())
    U = (v * left[..., None]).transpose(-1, -2) @ B                                # what each chunk adds [n, H, M, P, N]
    # states at the chunks' starts and at the end: all former chunks' sums, decayed
    total = torch.cat([torch.zeros_like(G[..., :1, -1]), G[..., -1].cumsum(-1)], -1)
    U = torch.cat([S0[:, :, None], U], 2).reshape(n, H, M + 1, P * N)
    S = (_decays(total) @ U).reshape(n, H, M + 1, P, N)
    y = inner + (C * torch.exp(G.float())[..., None]) @ S[:, :, :-1].transpose(-1, -2)
    return y, S[:, :, -1]


def _plain_ssm(s, x, B, C, a, A_log, dt_bias, D, S0):
    idx, valid, case = s["index"], s["valid"], s["case"]
    dt = _softplus(a + dt_bias)
    g = -torch.exp(A_log) * dt

    def chunks(t):  # [T, h, ...] -> [n, h, M, K, ...], zeros past a sequence's end
        t = t[idx] * valid.view(valid.shape + (1,) * (t.dim() - 1))
        t = t.transpose(1, 2)
        return t.reshape(t.shape[0], t.shape[1], -1, CHUNK, *t.shape[3:])

    rep = case["H"] // case["G"]
    y, S = _plain_ssm_chunks(chunks(x), chunks(B).repeat_interleave(rep, 1), chunks(C).repeat_interleave(rep, 1),
                             chunks(g), chunks(dt), S0)
    y = y.flatten(2, 3).transpose(1, 2)[valid]                                     # [T, H, P], in order
    return y + D[:, None] * x, S


def _ssm_leaves(s):
    n, case = s["valid"].shape[0], s["case"]
    S0 = s["initial_state"]
    if S0 is None:
        S0 = torch.zeros(n, case["H"], case["P"], case["N"], device=s["x"].device)
    return [s[k].float() for k in ("x", "B", "C", "a", "A_log", "dt_bias", "D")] + [S0]


def _plain_ssm_fwd(s):
    y, S = _plain_ssm(s, *_ssm_leaves(s))
    return dict(out=y.to(s["x"].dtype), state=S)


def _plain_ssm_bwd(s):
    with torch.enable_grad():
        leaves = [t.detach().clone().requires_grad_() for t in _ssm_leaves(s)]
        y, S = _plain_ssm(s, *leaves)
        dS = torch.zeros_like(S) if s["dfinal_state"] is None else s["dfinal_state"]
        grads = torch.autograd.grad((y, S), leaves, (s["dout"].float(), dS))
    res = dict(zip(_SSM_GRADS, grads))
    res.update({k: res[k].to(s["x"].dtype) for k in ("dx", "dB", "dC")})
    if s["initial_state"] is None:
        del res["dinitial_state"]
    return res


def _plain_ssm_step(s):
    case, T = s["case"], s["case"]["T"]
    rep = case["H"] // case["G"]
    x, a = s["x"].float(), s["a"] + s["dt_bias"]
    B, C = (s[k].float().repeat_interleave(rep, 2) for k in ("B", "C"))            # [N, T, H, state]
    dt = _softplus(a)
    G = (-torch.exp(s["A_log"]) * dt).double().cumsum(1).transpose(1, 2)           # [N, H, T]
    S = s["state"][s["slots"]]
    v = x * dt[..., None]
    xt, Bt, Ct = (t.transpose(1, 2) for t in (v, B, C))                            # [N, H, T, ...]
    y = ((Ct @ Bt.transpose(-1, -2)) * _decays(G)) @ xt
    y = y + (Ct @ S.transpose(-1, -2)) * torch.exp(G.float())[..., None]
    left = torch.exp((G[..., -1:] - G).float())
    S = S * torch.exp(G[..., -1].float())[..., None, None] + (xt * left[..., None]).transpose(-1, -2) @ Bt
    s["state"][s["slots"]] = S
    out = y.transpose(1, 2) + s["D"][:, None] * x
    return dict(out=out.to(s["x"].dtype), state=s["state"])


def _rotated(x, cos, sin, interleaved):
    """x [T, h, d] with its first dimensions rotated in pairs; cos, sin [T, pairs]."""
    m = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        u, v = x[..., 0:2 * m:2], x[..., 1:2 * m:2]
        r = torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2)
    else:
        u, v = x[..., :m], x[..., m:2 * m]
        r = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
    return torch.cat([r, x[..., 2 * m:]], -1)


def _norm_scale(x, s):
    ss = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((ss / x.shape[-1] if s["case"]["norm"] == "rms" else ss) + s["eps"])


def _plain_qk_fwd(s):
    cos, sin = s["cos_sin"][s["positions"].long()].chunk(2, -1)
    q, k = s["q"].float(), s["k"].float()
    nq, nk = q * _norm_scale(q, s), k * _norm_scale(k, s)
    if s["q_weight"] is not None:
        nq, nk = nq * s["q_weight"], nk * s["k_weight"]
    il, dt = s["case"]["interleaved"], s["q"].dtype
    return dict(q=_rotated(nq, cos, sin, il).to(dt), k=_rotated(nk, cos, sin, il).to(dt))


def _plain_qk_grad(s, x, w, dout, cos, sin):
    dm = _rotated(dout.float(), cos, -sin, s["case"]["interleaved"])               # the rotation back
    x = x.float()
    r = _norm_scale(x, s)
    n = x * r
    dn = dm if w is None else dm * w
    dot = (dn * n).sum(-1, keepdim=True)
    dx = r * (dn - n * (dot / x.shape[-1] if s["case"]["norm"] == "rms" else dot))
    return dx.to(dout.dtype), None if w is None else (dm * n).sum((0, 1))


def _plain_qk_bwd(s):
    cos, sin = s["cos_sin"][s["positions"].long()].chunk(2, -1)
    dq, dwq = _plain_qk_grad(s, s["q"], s["q_weight"], s["dq_out"], cos, sin)
    dk, dwk = _plain_qk_grad(s, s["k"], s["k_weight"], s["dk_out"], cos, sin)
    return {k: v for k, v in dict(dq=dq, dk=dk, dq_weight=dwq, dk_weight=dwk).items() if v is not None}


_plain = dict(conv_fwd=_plain_conv_fwd, conv_step=_plain_conv_step, conv_bwd=_plain_conv_bwd, ssm_fwd=_plain_ssm_fwd,
              ssm_step=_plain_ssm_step, ssm_bwd=_plain_ssm_bwd, qk_fwd=_plain_qk_fwd, qk_bwd=_plain_qk_bwd)


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    op, e = case["op"], 2 if case["dtype"] == BF16 else 4
    if op.startswith("conv"):
        dim = case["dim"]
        if op == "conv_step":
            n = case["N"] * case["T"] * dim                # x in, out; the histories in and out
            return dict(bytes=2 * e * n + 24 * case["N"] * dim + 16 * dim, flops=12 * n)
        L = _lengths(case)
        n, state = sum(L) * dim, 12 * len(L) * dim
        if op == "conv_fwd":                               # x in, out; the final history, and the first if given
            return dict(bytes=2 * e * n + state * (2 if case["carried"] else 1) + 20 * dim, flops=12 * n)
        return dict(bytes=3 * e * n + (3 * state if case["carried"] else 0) + 40 * dim, flops=32 * n)
    if op.startswith("ssm"):
        H, G, P = case["H"], case["G"], case["P"]
        if op == "ssm_step":
            N, rows, seqs = case["N_state"], case["N"] * case["T"], case["N"]
            moved = e * rows * (2 * H * P + 2 * G * N) + 4 * rows * H + 8 * seqs * H * P * N
            return dict(bytes=moved, flops=5 * rows * H * P * N)
        L, N = _lengths(case), case["N"]
        T, state = sum(L), 4 * len(L) * H * P * N
        if op == "ssm_fwd":                                # x, B, C, a in; y and the final states out
            moved = e * T * (2 * H * P + 2 * G * N) + 4 * T * H + state * (2 if case["carried"] else 1)
            # per token and head: the state's update and its product with C
            return dict(bytes=moved, flops=4 * T * H * P * N)
        moved = e * T * (3 * H * P + 4 * G * N) + 8 * T * H + (3 * state if case["carried"] else 0)
        # the states again, their gradients' update, and the products with x, B, C and dout
        return dict(bytes=moved, flops=12 * T * H * P * N)
    T, d, h = case["T"], case["d"], case["Hq"] + case["Hk"]
    table = 4 * T * case["rot"] + 4 * T
    if op == "qk_fwd":
        return dict(bytes=2 * e * T * h * d + table, flops=10 * T * h * d)
    return dict(bytes=3 * e * T * h * d + table, flops=20 * T * h * d)


# ---- the same outputs in 64 bits, from the definitions ------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact[case["op"]](s)


def _exact_conv(s):
    """Sequence by sequence, in 64 bits; the gradients by differentiation."""
    f64, op = torch.float64, s["op"]
    lengths = _lengths(s["case"])
    x, w, b, st = (None if s[k] is None else s[k].to(f64).requires_grad_() for k in ("x", "weight", "bias", "state"))
    outs, lasts = [], []
    for n, part in enumerate(x.split(lengths)):
        first = torch.zeros(3, x.shape[1], dtype=f64, device=x.device) if st is None else st[n].T
        seq = torch.cat([first, part])
        c = sum(seq[j:j + part.shape[0]] * w[:, j] for j in range(TAPS))
        c = c if b is None else c + b
        outs.append(c / (1.0 + torch.exp(-c)))
        lasts.append(seq[-3:].T)
    out, last = torch.cat(outs), torch.stack(lasts)
    if op == "conv_fwd":
        return dict(out=out.detach(), state=last.detach())
    loss = (out * s["dout"].to(f64)).sum()
    if s["dstate_out"] is not None:
        loss = loss + (last * s["dstate_out"].to(f64)).sum()
    leaves = {k: t for k, t in dict(dx=x, dweight=w, dbias=b, dstate=st).items() if t is not None}
    return dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))


def _exact_conv_step(s):
    f64 = torch.float64
    pool, w, sl = s["state"].to(f64), s["weight"].to(f64), s["slots"]
    outs = []
    for t in range(s["case"]["T"]):
        h = torch.cat([pool[sl], s["x"][:, t].to(f64)[..., None]], -1)
        c = (h * w).sum(-1) + (0.0 if s["bias"] is None else s["bias"].to(f64))
        outs.append(c / (1.0 + torch.exp(-c)))
        pool[sl] = h[..., 1:]
    return dict(out=torch.stack(outs, 1), state=pool)


def _exact_gates(a, A_log, dt_bias):
    z = a + dt_bias
    dt = z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))
    return dt, torch.exp(-torch.exp(A_log) * dt)


def _exact_ssm_step(s):
    f64, case = torch.float64, s["case"]
    rep = case["H"] // case["G"]
    S, D = s["state"].to(f64), s["D"].to(f64)
    dt, alpha = _exact_gates(s["a"].to(f64), s["A_log"].to(f64), s["dt_bias"].to(f64))
    cur, outs = S[s["slots"]], []
    for t in range(case["T"]):
        x, B, C = s["x"][:, t].to(f64), *(s[k][:, t].to(f64).repeat_interleave(rep, 1) for k in ("B", "C"))
        cur = cur * alpha[:, t, :, None, None] + (dt[:, t, :, None] * x)[..., None] * B[..., None, :]
        outs.append((cur * C[..., None, :]).sum(-1) + D[:, None] * x)
    S[s["slots"]] = cur
    return dict(out=torch.stack(outs, 1), state=S)


def _exact_ssm(s):
    """The recurrence token by token, and its adjoint token by token backwards."""
    case, f64 = s["case"], torch.float64
    lengths, H, G, P, N = _lengths(case), case["H"], case["G"], case["P"], case["N"]
    n, Tm, rep = len(lengths), max(lengths), H // G
    idx, valid, dev = s["index"][:, :Tm], s["valid"][:, :Tm], s["x"].device

    def padded(t):                                         # [T, h, ...] -> [Tm, n, h, ...]
        t = t.to(f64)[idx] * valid.view(n, Tm, *([1] * (t.dim() - 1)))
        return t.transpose(0, 1)

    def packed(t):
        t = t.transpose(0, 1)
        return torch.cat([t[i, :L] for i, L in enumerate(lengths)])

    A_log, dt_bias, D = (s[k].to(f64) for k in ("A_log", "dt_bias", "D"))
    dt_all, alpha_all = _exact_gates(s["a"].to(f64), A_log, dt_bias)
    x, B, C, dt = padded(s["x"]), padded(s["B"]), padded(s["C"]), padded(dt_all)
    alpha = padded(alpha_all) + (~valid).T[:, :, None]     # a padding token leaves the state as it is

    def wide(t):                                           # groups -> heads
        return t.repeat_interleave(rep, 1)

    def step(S, t):
        return S * alpha[t][..., None, None] + (dt[t][..., None] * x[t])[..., None] * wide(B[t])[..., None, :]

    S = torch.zeros(n, H, P, N, dtype=f64, device=dev) if s["initial_state"] is None else s["initial_state"].to(f64)
    kept, ys = [], []
    for t in range(Tm):
        if t % CHUNK == 0:
            kept.append(S)
        S = step(S, t)
        if s["op"] == "ssm_fwd":
            ys.append((S @ wide(C[t])[..., None])[..., 0])
    if s["op"] == "ssm_fwd":
        return dict(out=packed(torch.stack(ys) + D[:, None] * x), state=S)

    dy = padded(s["dout"])
    dS = torch.zeros_like(S) if s["dfinal_state"] is None else s["dfinal_state"].to(f64)
    dx, dB, dC, ddt, dlog = (torch.zeros_like(t) for t in (x, B, C, dt, dt))
    for c in range(len(kept) - 1, -1, -1):
        trail, S = [], kept[c]
        for t in range(c * CHUNK, min(Tm, (c + 1) * CHUNK)):
            before, S = S, step(S, t)
            trail.append((t, before, S))
        for t, before, S in reversed(trail):
            dC[t] = (dy[t][..., None, :] @ S)[..., 0, :].reshape(n, G, rep, N).sum(2)
            dS = dS + dy[t][..., None] * wide(C[t])[..., None, :]
            u = (dS @ wide(B[t])[..., None])[..., 0]
            dx[t] = dt[t][..., None] * u
            ddt[t] = (u * x[t]).sum(-1)
            dB[t] = ((dt[t][..., None] * x[t])[..., None, :] @ dS)[..., 0, :].reshape(n, G, rep, N).sum(2)
            dlog[t] = (dS * before).sum((-1, -2)) * alpha[t]
            dS = dS * alpha[t][..., None, None]
    dx = dx + D[:, None] * dy
    rate = torch.exp(A_log)
    z = padded(s["a"]) + dt_bias
    da = (ddt - rate * dlog) / (1.0 + torch.exp(-z)) * valid.T[:, :, None]
    dlog = dlog * valid.T[:, :, None]
    out = dict(dx=packed(dx), dB=packed(dB), dC=packed(dC), da=packed(da), dA_log=(-rate * dt * dlog).sum((0, 1)),
               ddt_bias=da.sum((0, 1)), dD=(dy * x).sum((0, 1, 3)))
    if s["initial_state"] is not None:
        out["dinitial_state"] = dS
    return out


def _exact_qk(s):
    """Norm and rotation by their definitions (the rotation as a product of complex numbers)."""
    f64, case = torch.float64, s["case"]
    d, rot = case["d"], case["rot"]
    table = s["cos_sin"].to(f64)[s["positions"].long()]
    turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]

    def one(x, w):
        x = x.to(f64).requires_grad_()
        w = None if w is None else w.to(f64).requires_grad_()
        ss = x.square().sum(-1, keepdim=True)
        m = x / ((ss / d if case["norm"] == "rms" else ss) + s["eps"]).sqrt()
        m = m if w is None else m * w
        pairs = m[..., :rot].unflatten(-1, (rot // 2, 2) if case["interleaved"] else (2, rot // 2))
        pairs = pairs if case["interleaved"] else pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return x, w, torch.cat([z.flatten(-2), m[..., rot:]], -1)

    res = {}
    for name in ("q", "k"):
        x, w, out = one(s[name], s[name + "_weight"])
        if s["op"] == "qk_fwd":
            res[name] = out.detach()
            continue
        grads = torch.autograd.grad(out, [x] if w is None else [x, w], s[f"d{name}_out"].to(f64))
        res["d" + name] = grads[0]
        if w is not None:
            res[f"d{name}_weight"] = grads[1]
    return res if s["op"] == "qk_fwd" else {k: res[k] for k in ("dq", "dk", "dq_weight", "dk_weight") if k in res}


_exact = dict(conv_fwd=_exact_conv, conv_bwd=_exact_conv, conv_step=_exact_conv_step, ssm_fwd=_exact_ssm,
              ssm_bwd=_exact_ssm, ssm_step=_exact_ssm_step, qk_fwd=_exact_qk, qk_bwd=_exact_qk)
