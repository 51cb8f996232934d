"""CPU checks of the state space layer's calls: refusals before any CUDA call, the binding's own checks, and the plain
64-bit forms the GPU tests compare with against finite differences and each other."""
import ctypes

import pytest
import torch

import gated_deltanet_recurrence_gb300 as gdn
from tests import _layer

P, Q4, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), None
ODD = ctypes.c_void_p(0x10002)
ARG, DTYPE, WORKSPACE, UNSUPPORTED, OK = -1, -2, -4, -7, 0
CUDA_ONLY = "must be CUDA tensors"
F64 = torch.float64

CONV = dict(x=P, xs=64, w=P, b=NUL, cu=NUL, n=1, T=8, dim=64, dt=0, silu=1, sin=NUL, sout=NUL, out=P, stream=NUL)
STEP = dict(x=P, xs=64, w=P, b=NUL, pool=P, slots=4, idx=NUL, N=4, T=1, dim=64, dt=0, silu=1, out=P, stream=NUL)
CONVB = dict(dout=P, x=P, xs=64, w=P, b=NUL, cu=NUL, n=1, T=8, dim=64, dt=0, silu=1, sin=NUL, dsout=NUL, dx=P, dw=P,
             db=NUL, dsin=NUL, zero=0, ws=P, wsb=0, stream=NUL)
SSM = dict(x=P, xs=128, B=P, Bs=64, C=P, Cs=64, a=P, A=P, bias=NUL, D=NUL, cu=NUL, n=1, T=8, H=2, G=1, P=64, N=64, dt=0,
           S0=NUL, Sf=NUL, out=P, ws=P, wsb=0, stream=NUL)
SSTEP = dict(x=P, xs=128, B=P, Bs=64, C=P, Cs=64, a=P, A=P, bias=NUL, D=NUL, pool=P, slots=4, idx=NUL, n=4, T=1, H=2, G=1,
             P=64, N=64, dt=0, out=P, stream=NUL)
SSMB = dict(dout=P, x=P, xs=128, B=P, Bs=64, C=P, Cs=64, a=P, A=P, bias=NUL, D=NUL, cu=NUL, n=1, T=8, H=2, G=1, P=64, N=64,
            dt=0, S0=NUL, dSf=NUL, dx=P, dB=P, dC=P, da=P, dA=NUL, db=NUL, dD=NUL, dS0=NUL, zero=0, ws=P, wsb=0, stream=NUL)
QK = dict(q=P, qs=128, k=P, ks=64, cs=P, pos=P, most=16, qw=NUL, kw=NUL, norm=0, eps=1e-6, il=0, T=8, H=2, Hk=1, d=64, rot=32,
          dt=0, qo=P, qos=128, ko=P, kos=64, stream=NUL)
QKB = dict(dqo=P, dko=P, q=P, qs=128, k=P, ks=64, cs=P, pos=P, most=16, qw=NUL, kw=NUL, norm=0, eps=1e-6, il=0, T=8, H=2,
           Hk=1, d=64, rot=32, dt=0, dq=P, dqs=128, dk=P, dks=64, dqw=NUL, dkw=NUL, ws=P, wsb=0, stream=NUL)
CALLS = dict(gdn_short_conv_fwd=CONV, gdn_short_conv_step=STEP, gdn_short_conv_bwd=CONVB, gdn_ssm_chunk_fwd=SSM,
             gdn_ssm_step=SSTEP, gdn_ssm_chunk_bwd=SSMB, gdn_qk_norm_rope=QK, gdn_qk_norm_rope_bwd=QKB)

REFUSED = [(n, s, kw) for n, cases in {
    "gdn_short_conv_fwd": [
        (DTYPE, dict(dt=2)), (ARG, dict(n=0)), (ARG, dict(T=-1)), (ARG, dict(T=9, n=2)), (ARG, dict(dim=0)),
        (UNSUPPORTED, dict(dim=60, xs=64)), (ARG, dict(xs=56)), (ARG, dict(xs=68)), (ARG, dict(x=NUL)), (ARG, dict(x=Q4)),
        (ARG, dict(w=NUL)), (ARG, dict(b=Q4)), (ARG, dict(out=NUL)), (ARG, dict(out=Q4)), (ARG, dict(sout=Q4)),
        (OK, dict(T=0))],
    "gdn_short_conv_step": [
        (DTYPE, dict(dt=-1)), (ARG, dict(N=-1)), (ARG, dict(T=0)), (ARG, dict(slots=0)), (ARG, dict(slots=3)),
        (UNSUPPORTED, dict(dim=4)), (ARG, dict(xs=60)), (ARG, dict(pool=NUL)), (ARG, dict(pool=Q4)), (ARG, dict(x=NUL)),
        (ARG, dict(out=NUL)), (OK, dict(N=0))],
    "gdn_short_conv_bwd": [
        (DTYPE, dict(dt=9)), (ARG, dict(n=-1)), (ARG, dict(T=9, n=2)), (UNSUPPORTED, dict(dim=60)), (ARG, dict(xs=8)),
        (ARG, dict(dout=NUL)), (ARG, dict(x=NUL)), (ARG, dict(dx=NUL)), (ARG, dict(w=NUL)), (ARG, dict(dw=Q4)),
        (WORKSPACE, dict()), (WORKSPACE, dict(ws=NUL, wsb=1 << 30)), (WORKSPACE, dict(ws=Q4, wsb=1 << 30)),
        (OK, dict(T=0, dw=NUL))],
    "gdn_ssm_chunk_fwd": [
        (DTYPE, dict(dt=2)), (ARG, dict(n=0)), (ARG, dict(T=9, n=2)), (ARG, dict(H=0)), (ARG, dict(G=0)),
        (ARG, dict(H=3, G=2, xs=192, Bs=128, Cs=128)), (UNSUPPORTED, dict(P=96)), (UNSUPPORTED, dict(N=256)),
        (ARG, dict(xs=120)), (ARG, dict(xs=132)), (ARG, dict(Bs=32)), (ARG, dict(Cs=68)), (ARG, dict(x=NUL)),
        (ARG, dict(B=NUL)), (ARG, dict(C=Q4)), (ARG, dict(a=NUL)), (ARG, dict(A=NUL)), (ARG, dict(out=NUL)),
        (ARG, dict(D=ODD)), (ARG, dict(H=20000, xs=20000 * 64)), (WORKSPACE, dict()), (WORKSPACE, dict(ws=NUL, wsb=1 << 40)),
        (WORKSPACE, dict(ws=ctypes.c_void_p(0x10010), wsb=1 << 40)), (OK, dict(T=0))],
    "gdn_ssm_step": [
        (DTYPE, dict(dt=2)), (ARG, dict(n=-1)), (ARG, dict(T=0)), (ARG, dict(slots=3)), (ARG, dict(H=2, G=3)),
        (UNSUPPORTED, dict(P=32)), (UNSUPPORTED, dict(N=16)), (ARG, dict(xs=64)), (ARG, dict(pool=NUL)), (ARG, dict(pool=Q4)),
        (ARG, dict(a=NUL)), (ARG, dict(out=Q4)), (OK, dict(n=0))],
    "gdn_ssm_chunk_bwd": [
        (DTYPE, dict(dt=2)), (ARG, dict(n=0)), (ARG, dict(H=3, G=2, xs=192, Bs=128, Cs=128)), (UNSUPPORTED, dict(P=8)),
        (ARG, dict(xs=100)), (ARG, dict(dout=NUL)), (ARG, dict(dx=NUL)), (ARG, dict(dB=NUL)), (ARG, dict(dC=Q4)),
        (ARG, dict(da=NUL)), (ARG, dict(dA=ODD)), (WORKSPACE, dict()), (WORKSPACE, dict(ws=NUL, wsb=1 << 40)),
        (WORKSPACE, dict(ws=ctypes.c_void_p(0x10010), wsb=1 << 40))],
    "gdn_qk_norm_rope": [
        (DTYPE, dict(dt=2)), (ARG, dict(T=-1)), (ARG, dict(H=0)), (ARG, dict(Hk=-1)), (UNSUPPORTED, dict(d=60, rot=4, qs=120)),
        (UNSUPPORTED, dict(d=512, qs=1024, ks=512)), (ARG, dict(rot=33)), (ARG, dict(rot=66)), (ARG, dict(eps=-1.0)),
        (ARG, dict(norm=2)), (ARG, dict(qs=120)), (ARG, dict(ks=68)), (ARG, dict(kos=8)), (ARG, dict(q=NUL)), (ARG, dict(k=Q4)),
        (ARG, dict(cs=NUL)), (ARG, dict(pos=NUL, most=7)), (ARG, dict(qo=NUL)), (ARG, dict(ko=NUL)), (OK, dict(T=0))],
    "gdn_qk_norm_rope_bwd": [
        (DTYPE, dict(dt=2)), (ARG, dict(H=0)), (ARG, dict(rot=1)), (ARG, dict(dqs=64)), (ARG, dict(dqo=NUL)), (ARG, dict(dko=NUL)),
        (ARG, dict(dq=NUL)), (ARG, dict(dk=Q4)), (ARG, dict(Hk=0, dkw=P)), (WORKSPACE, dict(dqw=P)),
        (WORKSPACE, dict(dqw=P, ws=NUL, wsb=1 << 30)), (OK, dict(T=0))],
}.items() for s, kw in cases]


@pytest.mark.parametrize("name,status,kw", REFUSED)
def test_refusals(name, status, kw):
    args = dict(CALLS[name])
    assert set(kw) <= set(args)
    args.update(kw)
    assert getattr(gdn.lib(), name)(*args.values()) == status


def test_workspace_sizes():
    L = gdn.lib()
    assert L.gdn_ssm_chunk_fwd_workspace_size(1, 64, 2, 1, 64, 64, 0) > 0
    assert L.gdn_ssm_chunk_fwd_workspace_size(1, 64, 2, 1, 64, 64, 1) == 0  # one kernel, nothing between kernels
    for bad in ((0, 64, 2, 1, 64, 64, 1), (1, -1, 2, 1, 64, 64, 1), (1, 64, 3, 2, 64, 64, 1), (1, 64, 2, 1, 32, 64, 1),
                (1, 64, 2, 1, 64, 64, 5)):
        assert L.gdn_ssm_chunk_fwd_workspace_size(*bad) == 0
        assert L.gdn_ssm_chunk_bwd_workspace_size(*bad) == 0
    assert L.gdn_ssm_chunk_bwd_workspace_size(3, 700, 4, 2, 128, 128, 0) > 0
    assert L.gdn_short_conv_bwd_workspace_size(1, 100, 64) > 0 and L.gdn_short_conv_bwd_workspace_size(1, 100, 60) == 0
    assert L.gdn_qk_norm_rope_bwd_workspace_size(10, 2, 1, 64) > 0 and L.gdn_qk_norm_rope_bwd_workspace_size(10, 2, 1, 60) == 0


# ---- the binding's checks ------------------------------------------------------------------------------

def _conv():
    return (torch.zeros(10, 64), torch.zeros(64, 4)), dict(bias=torch.zeros(64), conv_state=torch.zeros(1, 64, 3),
                                                            conv_state_out=torch.zeros(1, 64, 3), out=torch.zeros(10, 64))


def _ssm():
    return ([torch.zeros(10, 2, 64), torch.zeros(10, 1, 64), torch.zeros(10, 1, 64), torch.zeros(10, 2), torch.zeros(2)],
            dict(dt_bias=torch.zeros(2), D=torch.zeros(2), initial_state=torch.zeros(1, 2, 64, 64),
                 final_state=torch.zeros(1, 2, 64, 64), out=torch.zeros(10, 2, 64)))


def test_consistent_calls_reach_the_device_check():
    a, kw = _conv()
    with pytest.raises(ValueError, match=CUDA_ONLY):
        gdn.gdn_short_conv_fwd(*a, **kw)
    with pytest.raises(ValueError, match=CUDA_ONLY):
        gdn.gdn_short_conv_step(a[0], a[1], torch.zeros(10, 64, 3))
    with pytest.raises(ValueError, match=CUDA_ONLY):
        gdn.gdn_short_conv_bwd(a[0], *a)
    s, kw = _ssm()
    with pytest.raises(ValueError, match=CUDA_ONLY):
        gdn.gdn_ssm_chunk_fwd(*s, **kw)
    with pytest.raises(ValueError, match=CUDA_ONLY):
        gdn.gdn_ssm_chunk_bwd(s[0], *s)
    with pytest.raises(ValueError, match=CUDA_ONLY):
        gdn.gdn_ssm_step(*s, torch.zeros(10, 2, 64, 64))
    q, k = torch.zeros(5, 2, 64), torch.zeros(5, 1, 64)
    with pytest.raises(ValueError, match=CUDA_ONLY):
        gdn.gdn_qk_norm_rope(q, k, torch.zeros(5, 64))
    with pytest.raises(ValueError, match=CUDA_ONLY):
        gdn.gdn_qk_norm_rope_bwd(q, k, q, k, torch.zeros(5, 64))


@pytest.mark.parametrize("name", ["bias", "conv_state", "conv_state_out", "out"])
def test_undersized_conv_tensors_are_refused(name):
    a, kw = _conv()
    kw[name] = kw[name].flatten()[:-1]
    with pytest.raises(ValueError, match=f"{name} holds"):
        gdn.gdn_short_conv_fwd(*a, **kw)


@pytest.mark.parametrize("name", ["dt_bias", "D", "initial_state", "final_state", "out"])
def test_undersized_scan_tensors_are_refused(name):
    a, kw = _ssm()
    kw[name] = kw[name].flatten()[:-1]
    with pytest.raises(ValueError, match=f"{name} holds"):
        gdn.gdn_ssm_chunk_fwd(*a, **kw)


def test_shapes_types_and_strides_are_checked():
    s, _ = _ssm()
    with pytest.raises(ValueError, match="C is"):
        gdn.gdn_ssm_chunk_fwd(s[0], s[1], torch.zeros(10, 1, 128), s[3], s[4])
    with pytest.raises(TypeError, match="B must have"):
        gdn.gdn_ssm_chunk_fwd(s[0], s[1].bfloat16(), *s[2:])
    with pytest.raises(ValueError, match="rows of a token"):
        gdn.gdn_ssm_chunk_fwd(torch.zeros(10, 64, 2).transpose(1, 2), *s[1:])
    with pytest.raises(TypeError, match="a must be float32"):
        gdn.gdn_ssm_chunk_fwd(*s[:3], s[3].bfloat16(), s[4])
    with pytest.raises(ValueError, match="one stride apart"):
        gdn.gdn_short_conv_step(torch.zeros(4, 3, 2, 64)[:, :, 0].transpose(0, 1), torch.zeros(64, 4), torch.zeros(9, 64, 3))
    with pytest.raises(TypeError, match="int32"):
        gdn.gdn_short_conv_fwd(torch.zeros(4, 64), torch.zeros(64, 4), cu_seqlens=torch.tensor([0, 4]))
    with pytest.raises(TypeError, match="int32"):
        gdn.gdn_qk_norm_rope(torch.zeros(4, 1, 64), None, torch.zeros(4, 64), positions=torch.arange(4))
    with pytest.raises(TypeError, match="unsupported dtype"):
        gdn.gdn_short_conv_fwd(torch.zeros(4, 64).half(), torch.zeros(64, 4))


# ---- the plain forms ------------------------------------------------------------------------------------

def _diff(f, inputs, grads, h=1e-6):
    """Central differences in a random direction of each input, against its gradient."""
    gen = torch.Generator().manual_seed(7)
    for i, g in enumerate(grads):
        if inputs[i] is None:
            continue
        u = torch.randn(inputs[i].shape, generator=gen, dtype=F64)
        ends = [f(*inputs[:i], inputs[i] + s * h * u, *inputs[i + 1:]) for s in (1, -1)]
        num, ana = (ends[0] - ends[1]) / (2 * h), (g * u).sum()
        # the differences' own error: h^2 of the third derivative and 2^-53 / h of the value
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana.item()), (g * u).abs().sum().item()), (i, num, ana)


def test_plain_conv_gradients_against_differences():
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    offs, dim = [0, 1, 1, 4, 9], 3
    x, w, b, st, dy, dl = r(9, dim), r(dim, 4), r(dim), r(4, dim, 3), r(9, dim), r(4, dim, 3)

    def f(x, w, b, st):
        out, _, last = _layer.conv(x, w, b, offs, st)
        return (out * dy).sum() + (last * dl).sum()

    _, c, _ = _layer.conv(x, w, b, offs, st)
    _diff(f, (x, w, b, st), _layer.conv_bwd(dy * _layer.silu_slope(c), x, w, offs, st, dl))


def test_plain_scan_gradients_against_differences():
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    offs, H, G, Pd, N = [0, 3, 3, 8], 4, 2, 3, 5
    x, B, C, a, A, bias, D, S0 = r(8, H, Pd), r(8, G, N), r(8, G, N), r(8, H), r(H) * 0.3, r(H), r(H), r(3, H, Pd, N)
    dy, dl = r(8, H, Pd), r(3, H, Pd, N)

    def f(x, B, C, a, A, bias, D, S0):
        _, dt, alpha = _layer.gates(a, A, bias)
        y, last = _layer.ssm(x, B, C, dt, alpha, D, offs, S0)
        return (y * dy).sum() + (last * dl).sum()

    g, _ = _layer.scan_grads(dy, x, B, C, a, A, bias, D, offs, S0, dl)
    _diff(f, (x, B, C, a, A, bias, D, S0),
          [g[k] for k in ("dx", "dB", "dC", "da", "dA_log", "ddt_bias", "dD", "dinitial_state")])


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_rotation_gradients_against_differences(l2, interleaved):
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    x, w, dy, ang = r(5, 2, 8), r(8), r(5, 2, 8), r(5, 3)
    cos, sin = ang.cos(), ang.sin()

    def f(x, w):
        return (_layer.qk(x, w, cos, sin, l2, 1e-2, interleaved)[0] * dy).sum()

    _diff(f, (x, w), _layer.qk_bwd(dy, x, w, cos, sin, l2, 1e-2, interleaved)[:2])
    # turning a vector keeps its length
    out = _layer.rotate(x, cos, sin, interleaved)
    assert torch.allclose(out.square().sum(-1), x.square().sum(-1), rtol=1e-12)


def test_plain_scan_continues_where_it_stopped():
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    x, B, C, dt, alpha = r(9, 2, 3), r(9, 1, 4), r(9, 1, 4), r(9, 2).abs(), torch.rand(9, 2, generator=gen, dtype=F64)
    y, last = _layer.ssm(x, B, C, dt, alpha, None, [0, 9], None)
    y1, mid = _layer.ssm(x[:4], B[:4], C[:4], dt[:4], alpha[:4], None, [0, 4], None)
    y2, end = _layer.ssm(x[4:], B[4:], C[4:], dt[4:], alpha[4:], None, [0, 5], mid)
    assert torch.allclose(torch.cat([y1, y2]), y) and torch.allclose(end, last)
