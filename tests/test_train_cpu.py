"""CPU checks of the training entry points: refusals before any CUDA call, the binding's own checks,
and the plain fp64 forms the GPU tests compare with against finite differences."""
import ctypes

import pytest
import torch

import gated_deltanet_recurrence_gb300 as gdn
from tests import _train

P, Q4, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), None
ARG, DTYPE, WORKSPACE, UNSUPPORTED = -1, -2, -4, -7
CUDA_ONLY = "must be CUDA tensors"


def call(name, **kw):
    """Calls a library function with valid stand-in arguments, changed by kw; every call below must end
    in a refusal or have nothing to do."""
    args = {
        "gdn_chunk_bwd": dict(q=P, k=P, v=P, g=P, beta=P, cu=NUL, num_seqs=1, total_T=64, H=2, Hk=2, dk=128, dv=128,
                              dt=0, decay=0, scale=0.0, l2=1, S0=NUL, dout=P, odt=0, dSf=NUL, dq=P, dkk=P, dvv=P,
                              dg=P, dbeta=P, dS0=NUL, ws=P, wsb=0, stream=NUL),
        "gdn_gate_rmsnorm_silu_bwd": dict(dout=P, odt=0, y=P, dt=0, z=P, w=NUL, eps=1e-6, dy=P, dz=P, dw=NUL,
                                          rows=4, d=64, ws=NUL, wsb=0, stream=NUL),
        "gdn_gate_groupnorm_silu": dict(y=P, dt=0, z=NUL, w=NUL, b=NUL, eps=1e-6, out=P, odt=0, rows=4, groups=2,
                                        size=64, stream=NUL),
        "gdn_gate_groupnorm_silu_bwd": dict(dout=P, odt=0, y=P, dt=0, z=NUL, w=NUL, b=NUL, eps=1e-6, dy=P, dz=NUL,
                                            dw=NUL, db=NUL, rows=4, groups=2, size=64, ws=NUL, wsb=0, stream=NUL),
        "gdn_decay_from_logits_bwd": dict(a=P, A=P, bias=NUL, b=NUL, dg=P, dbeta=NUL, da=P, dA=NUL, ddt=NUL, db=NUL,
                                          T=8, H=4, ws=NUL, wsb=0, stream=NUL),
    }[name]
    assert set(kw) <= set(args)
    args.update(kw)
    return getattr(gdn.lib(), name)(*args.values())


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=2)), (DTYPE, dict(odt=-1)), (ARG, dict(num_seqs=0)), (ARG, dict(total_T=-1)), (ARG, dict(H=0)),
    (ARG, dict(H=3, Hk=2)), (ARG, dict(decay=2)), (UNSUPPORTED, dict(decay=1)), (UNSUPPORTED, dict(dk=96, dv=96)),
    (UNSUPPORTED, dict(dv=64)), (ARG, dict(total_T=65, num_seqs=2)), (ARG, dict(q=NUL)), (ARG, dict(dout=NUL)),
    (ARG, dict(dkk=NUL)), (ARG, dict(dbeta=NUL)), (ARG, dict(v=Q4)), (ARG, dict(dS0=Q4)), (ARG, dict(dSf=Q4)),
    (WORKSPACE, dict()), (WORKSPACE, dict(ws=NUL, wsb=1 << 40)), (WORKSPACE, dict(ws=ctypes.c_void_p(0x10010), wsb=1 << 40)),
    (ARG, dict(num_seqs=1 << 20, H=1 << 12, Hk=1 << 12, total_T=0)), (ARG, dict(total_T=1 << 30, H=4, Hk=4)),
    (0, dict(total_T=0, wsb=1 << 40))])
def test_chunk_bwd_refusals(status, kw):
    assert call("gdn_chunk_bwd", **kw) == status


def test_chunk_bwd_workspace_size():
    L = gdn.lib()
    size = L.gdn_chunk_bwd_workspace_size
    need = size(2, 8192, 16, 16, 128, 128)
    assert need > 0 and size(2, 8192, 16, 4, 128, 128) > need         # grouped heads: per-head gradients
    assert call("gdn_chunk_bwd", num_seqs=2, total_T=8192, H=16, Hk=16, wsb=need - 1) == WORKSPACE
    for bad in ((0, 64, 2, 2, 128, 128), (1, -1, 2, 2, 128, 128), (1, 64, 2, 3, 128, 128), (1, 64, 2, 2, 96, 96)):
        assert size(*bad) == 0


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=2)), (ARG, dict(num_seqs=0)), (ARG, dict(total_T=-1)), (ARG, dict(H=3)), (UNSUPPORTED, dict(dk=96, dv=96)),
    (ARG, dict(dv_=Q4)), (ARG, dict(dg=Q4)), (ARG, dict(total_T=1 << 30, H=4, Hk=4)), (0, dict(cu=NUL)), (0, dict(total_T=0)),
    (0, dict(dq=NUL, dk_=NUL, dv_=NUL, dg=NUL, dbeta=NUL))])
def test_zero_outside_refusals(status, kw):
    args = dict(cu=P, num_seqs=1, total_T=64, H=2, Hk=2, dk=128, dv=128, dt=0, dq=P, dk_=P, dv_=P, dg=P, dbeta=P, stream=NUL)
    assert set(kw) <= set(args)
    assert gdn.lib().gdn_chunk_bwd_zero_outside(*{**args, **kw}.values()) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(odt=3)), (DTYPE, dict(dt=-1)), (ARG, dict(d=100)), (ARG, dict(d=2048)), (ARG, dict(d=0)),
    (ARG, dict(rows=-1)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=float("nan"))), (ARG, dict(z=NUL)), (ARG, dict(dz=NUL)),
    (ARG, dict(y=NUL)), (ARG, dict(dout=Q4)), (WORKSPACE, dict(dw=P)), (WORKSPACE, dict(dw=P, ws=P, wsb=8)),
    (ARG, dict(rows=1 << 50)), (0, dict(rows=0))])
def test_rmsnorm_bwd_refusals(status, kw):
    assert call("gdn_gate_rmsnorm_silu_bwd", **kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dt=3)), (ARG, dict(size=0)), (ARG, dict(size=1025)), (ARG, dict(groups=0)),
    (ARG, dict(groups=1 << 20, size=2)), (ARG, dict(rows=-1)), (ARG, dict(eps=-1.0)), (ARG, dict(y=NUL)),
    (ARG, dict(y=Q4)), (0, dict(rows=0))])
def test_groupnorm_refusals(status, kw):
    assert call("gdn_gate_groupnorm_silu", **kw) == status
    assert call("gdn_gate_groupnorm_silu_bwd", **kw) == status


@pytest.mark.parametrize("status,kw", [
    (ARG, dict(z=P)), (ARG, dict(dz=P)), (ARG, dict(dy=NUL)), (WORKSPACE, dict(dw=P)), (WORKSPACE, dict(db=P, ws=Q4, wsb=1 << 30)),
    (DTYPE, dict(odt=7)), (ARG, dict(db=Q4))])
def test_groupnorm_bwd_refusals(status, kw):
    assert call("gdn_gate_groupnorm_silu_bwd", **kw) == status


@pytest.mark.parametrize("status,kw", [
    (ARG, dict(T=-1)), (ARG, dict(H=0)), (ARG, dict(a=NUL)), (ARG, dict(A=NUL)), (ARG, dict(dg=NUL)), (ARG, dict(da=NUL)),
    (ARG, dict(b=P)), (ARG, dict(b=P, dbeta=P)), (ARG, dict(db=P)), (ARG, dict(da=Q4)), (WORKSPACE, dict(dA=P)),
    (WORKSPACE, dict(ddt=P, ws=P, wsb=4)), (ARG, dict(T=1 << 50)), (0, dict(T=0))])
def test_decay_bwd_refusals(status, kw):
    assert call("gdn_decay_from_logits_bwd", **kw) == status


def test_workspace_sizes_of_refused_sizes_are_zero():
    L = gdn.lib()
    assert L.gdn_gate_bwd_workspace_size(10, 2, 64) > 0
    assert L.gdn_gate_bwd_workspace_size(-1, 2, 64) == 0 and L.gdn_gate_bwd_workspace_size(10, 2, 2048) == 0
    assert L.gdn_decay_bwd_workspace_size(10, 4) > 0
    assert L.gdn_decay_bwd_workspace_size(-1, 4) == 0 and L.gdn_decay_bwd_workspace_size(10, 0) == 0


# ---- the binding's checks ------------------------------------------------------------------------------

def _chunk_args():
    inp = _train.delta_inputs([70, 1], 4, 2, 64, torch.bfloat16, seed=1)
    kw = dict(cu_seqlens=torch.tensor(inp["cu"], dtype=torch.int32), initial_state=inp["initial_state"],
              dfinal_state=inp["dfinal_state"])
    return [inp[x] for x in ("q", "k", "v", "g", "beta", "dout")], kw


def test_consistent_calls_stop_at_the_cuda_check():
    args, kw = _chunk_args()
    y, c = torch.zeros(6, 4, 64), torch.zeros(4, 64)
    a = torch.zeros(10, 4)
    for f in (lambda: gdn.gdn_chunk_bwd(*args, **kw), lambda: gdn.gdn_gate_rmsnorm_silu_bwd(y, y, y, c[0]),
              lambda: gdn.gdn_gate_groupnorm_silu(y, y, c, c), lambda: gdn.gdn_gate_groupnorm_silu_bwd(y, y, y, c, c),
              lambda: gdn.gdn_decay_from_logits_bwd(a, a[0], a[0], a, a, a)):
        with pytest.raises(ValueError, match=CUDA_ONLY):
            f()


def test_undersized_and_mistyped_tensors_are_refused_by_name():
    args, kw = _chunk_args()
    for i, name in enumerate(("k", "v", "g", "beta", "dout")):
        short = list(args)
        short[i + 1] = short[i + 1][:-1]
        with pytest.raises(ValueError, match=f"{name} holds"):
            gdn.gdn_chunk_bwd(*short, **kw)
    for name, t in (("dq", args[0][:-1]), ("dg", args[3][:-1]), ("dinitial_state", kw["dfinal_state"][:1])):
        with pytest.raises(ValueError, match=f"{name} holds"):
            gdn.gdn_chunk_bwd(*args, **kw, **{name: t})
    with pytest.raises(TypeError, match="dq, dk, dv"):
        gdn.gdn_chunk_bwd(*args, **kw, dv=args[2].float())
    with pytest.raises(ValueError, match="one decay per head"):
        gdn.gdn_chunk_bwd(args[0], args[1], args[2], torch.zeros(71, 4, 64), args[4], args[5], **kw)
    y, c, a = torch.zeros(6, 4, 64), torch.zeros(4, 64), torch.zeros(10, 4)
    with pytest.raises(ValueError, match="dout holds"):
        gdn.gdn_gate_rmsnorm_silu_bwd(y[:5], y, y)
    with pytest.raises(TypeError, match="dy must have"):
        gdn.gdn_gate_rmsnorm_silu_bwd(y, y, y, dy=y.bfloat16())
    with pytest.raises(ValueError, match="weight holds"):
        gdn.gdn_gate_groupnorm_silu(y, None, c[:3])
    with pytest.raises(TypeError, match="z must be float32"):
        gdn.gdn_gate_groupnorm_silu_bwd(y, y, y.bfloat16())
    with pytest.raises(ValueError, match="dg holds"):
        gdn.gdn_decay_from_logits_bwd(a, a[0], None, None, a[:9], None)
    with pytest.raises(ValueError, match="given together"):
        gdn.gdn_decay_from_logits_bwd(a, a[0], None, a, a, None)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """With stand-ins for a stream and for a tensor on the GPU: made current, such a stream would leave the call on
    its own device's current stream, unordered with the given one."""
    from contextlib import nullcontext

    from gated_deltanet_recurrence_gb300 import _binding

    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)

    class OnGpu(torch.Tensor):
        is_cuda, device = True, torch.device("cuda", 0)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    ran = []
    call = _binding._on_stream(lambda t: ran.append(t))
    t = torch.zeros(1).as_subclass(OnGpu)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(t, stream=Stream(1))
    assert not ran
    call(t, stream=Stream(0))
    assert len(ran) == 1


# ---- the yardstick against differences ---------------------------------------------------------------

def _difference(f, x, direction, h=1e-6):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("use_l2", [True, False])
def test_plain_delta_gradients_match_differences(use_l2):
    """A directional derivative by central differences of step 1e-6 in fp64: truncation of order 1e-12
    and rounding of order 1e-16 / 1e-6 leave about 1e-9 of the value."""
    inp = _train.delta_inputs([9, 4], 2, 1, 64, torch.float64, seed=3)
    inp = {x: t.double() if isinstance(t, torch.Tensor) else t for x, t in inp.items()}
    ref = _train.delta_grads(inp, use_l2=use_l2, scale=0.3)

    def loss(**kw):
        i = dict(inp, **kw)
        y, S = _train.delta_forward(i["q"], i["k"], i["v"], i["g"], i["beta"], i["cu"], i["initial_state"], 0.3, use_l2)
        return float((y * i["dout"]).sum() + (S * i["dfinal_state"]).sum())

    gen = torch.Generator().manual_seed(4)
    for x in ("q", "k", "v", "g", "beta", "initial_state"):
        u = torch.randn(inp[x].shape, generator=gen, dtype=torch.float64)
        if x in ("q", "k") and not use_l2:
            u = u * 0.05
        num = _difference(lambda t: loss(**{x: t}), inp[x], u)
        ana = float((ref["d" + x] * u).sum())
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), (x, num, ana)


@pytest.mark.parametrize("use_l2", [True, False])
def test_plain_chunk_form_gives_the_gradients_of_the_recurrence(use_l2):
    """The form whose roundings give the token-wise tolerances; its normalised q's and k's gradients go through
    the norm here."""
    inp = _train.delta_inputs([150], 2, 2, 64, torch.float64, seed=5)
    if not use_l2:
        inp["q"], inp["k"] = inp["q"] / 8, inp["k"] / 8
    ref = _train.delta_grads(inp, use_l2=use_l2, scale=0.3)
    leaves = [inp[x].double().clone().requires_grad_() for x in ("q", "k")]
    q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) if use_l2 else x for x in leaves)
    v, g, beta, dy = (inp[x].double().transpose(0, 1) for x in ("v", "g", "beta", "dout"))
    got = _train._delta_chunks((0.3 * q).detach().transpose(0, 1), k.detach().transpose(0, 1), v, g, beta, dy,
                               inp["initial_state"][0].double(), inp["dfinal_state"][0].double(), 0.3, lambda x, s: x)
    dq, dk, dv, dg, dbeta = (x.transpose(0, 1) for x in got)
    dq, dk = torch.autograd.grad((0.3 * q, k), leaves, (dq, dk))
    for name, x in zip(("dq", "dk", "dv", "dg", "dbeta"), (dq, dk, dv, dg, dbeta)):
        assert _train.rel_l2(x, ref[name]) <= 1e-10, (name, _train.rel_l2(x, ref[name]))


@pytest.mark.parametrize("rms,gated", [(True, True), (False, True), (False, False)])
def test_plain_norm_gradients_match_differences(rms, gated):
    gen = torch.Generator().manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    y, w, do = rn(3, 2, 10), rn(2, 10), rn(3, 2, 10)
    z, b = rn(3, 2, 10) if gated else None, None if rms else rn(2, 10)
    args = [y, z, w, b]
    ref = _train.norm_grads(do, y, z, w, b, 1e-6, rms)
    for i, t in enumerate(args):
        if t is None:
            continue
        u = rn(*t.shape)
        f = lambda s: float((_train.norm_forward(*(args[:i] + [s] + args[i + 1:]), 1e-6, rms) * do).sum())  # noqa: E731
        num, ana = _difference(f, t, u), float((ref[i] * u).sum())
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), (i, num, ana)
