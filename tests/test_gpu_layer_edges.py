"""Ends of the state space layer's calls: eps = 0, and parameters that are no numbers."""
import pytest
import torch

import gated_deltanet_recurrence_gb300 as gdn
from tests import _layer
from tests._layer import check, wide
from tests.test_gpu_layer import ARG_ERROR, BF, F32, angles, clean_error_word, dev, qk_inputs, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("T,H,H_k,d,rot,interleaved,dtype", [
    (1, 1, 1, 64, 32, False, F32), (7, 3, 1, 64, 64, True, BF), (33, 2, 2, 128, 64, False, BF), (5, 2, 1, 96, 24, False, F32),
    (6, 1, 2, 8, 4, False, F32), (9, 2, 0, 256, 256, False, F32), (2501, 4, 1, 64, 64, False, BF)])
def test_rotation_gradients_without_eps(T, H, H_k, d, rot, interleaved, l2, dtype):
    """No head of a row is zero; places without a row (tokens rounded up to whole warps, a position outside the table)
    add nothing to the weights' gradients."""
    for outside in (None, T // 2):
        q, k, table, pos, w, r = qk_inputs(T, H, H_k, d, rot, True, dtype, seed=T + d)
        if outside is not None:
            pos[outside] = 300
        kw = dict(positions=pos, q_weight=w[0], k_weight=w[1] if H_k else None, eps=0.0, interleaved=interleaved,
                  norm=gdn.GDN_NORM_L2 if l2 else gdn.GDN_NORM_RMS)
        douts = dev(r(T, H, d), dtype), dev(r(T, H_k, d), dtype) if H_k else None
        outs = gdn.gdn_qk_norm_rope(q, k, table, **kw)
        grads = gdn.gdn_qk_norm_rope_bwd(*douts, q, k, table, **kw)
        torch.cuda.synchronize()
        assert gdn.gdn_get_device_error() == (0 if outside is None else ARG_ERROR)
        rows = torch.tensor([t for t in range(T) if t != outside], dtype=torch.long)
        cos, sin = angles(table, pos[rows.cuda()], rot, len(rows))
        for i, x in enumerate((q, k)):
            if x is None:
                continue
            X, DO, wt = wide(x)[rows], wide(douts[i])[rows], wide(w[i])
            ref, terms = _layer.qk(X, wt, cos, sin, l2, 0.0, interleaved)
            check("rotated", outs[i][rows.cuda()], ref, terms)
            ref = _layer.qk_bwd(DO, X, wt, cos, sin, l2, 0.0, interleaved)
            check("dx", grads[i][rows.cuda()], ref[0], ref[2])
            check("dw", grads[2 + i], ref[1], 2 * ref[3])  # up to 128 additions one by one, as rows are many


@pytest.mark.parametrize("name", ["A_log", "dt_bias", "D"])
@pytest.mark.parametrize("dtype,T", [(F32, 150), (BF, 150), (F32, 2000), (BF, 2000)])  # 2000: in segments
def test_a_parameter_that_is_no_number_reaches_its_heads_outputs_and_no_others(name, dtype, T):
    """As in the definition, and as token by token: exp(NaN) S is no number, whatever S."""
    H = 2
    offs, _, s, S0, r = scan_inputs([T], 0, H, 1, 64, 64, dtype, True, True, seed=T)
    dout = dev(r(T, H, 64), dtype)
    good = *gdn.gdn_ssm_chunk_fwd(**s, initial_state=S0), *gdn.gdn_ssm_chunk_bwd(dout, **s, initial_state=S0)
    s[name] = s[name].clone()
    s[name][1] = float("nan")
    out, last, dx, dB, dC, da, *sums, dS0 = *gdn.gdn_ssm_chunk_fwd(**s, initial_state=S0), \
        *gdn.gdn_ssm_chunk_bwd(dout, **s, initial_state=S0)
    pool = S0.clone()
    n = 70
    step = gdn.gdn_ssm_step(*(s[k][:n][None].contiguous() for k in ("x", "B", "C", "a")), s["A_log"], pool,
                            dt_bias=s["dt_bias"], D=s["D"])[0]
    assert bool(torch.isnan(step[:, 1]).all()) and bool(torch.isnan(out[:, 1]).all())
    assert bool(torch.isnan(dx[:, 1]).all())
    if name != "D":
        assert bool(torch.isnan(pool[0, 1]).all()) and bool(torch.isnan(last[0, 1]).all())
        assert bool(torch.isnan(da[:, 1]).all()) and bool(torch.isnan(dS0[0, 1]).all())
        assert bool(torch.isnan(sums[0][1])) and bool(torch.isnan(dB).all()) and bool(torch.isnan(dC).all())
    for a, b in zip((out, dx, da), (good[0], good[2], good[5])):
        assert torch.equal(a[:, 0], b[:, 0])
    for a, b in zip((last, dS0), (good[1], good[9])):
        assert torch.equal(a[:, 0], b[:, 0])
    for a, b in zip(sums, good[6:9]):
        assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("P,N,H,G", [(64, 128, 2, 1), (128, 64, 4, 2), (64, 64, 1, 1)])
def test_gradients_of_B_and_C_are_rounded_once(P, N, H, G):
    """Sequences of one token whose x and dout have one channel each: dC = sum over heads of E B with E = dt dout x, dB =
    sum of E C, whose few roundings (the step's six, two products', one addition a head, three planes' sum, a cut of the
    tensor cores counted twice: at most 32 of 2^-24) move a bf16 output only next to a border of two values."""
    n = 300
    gen = torch.Generator().manual_seed(P + N + H)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, dout = torch.zeros(n, H, P), torch.zeros(n, H, P)
    x[:, :, 5], dout[:, :, 5] = r(n, H).abs() + 0.5, r(n, H).abs() + 0.5  # no cancellation between heads
    x, dout, B, C, a, A_log = x.to(BF), dout.to(BF), r(n, G, N).to(BF), r(n, G, N).to(BF), r(n, H), r(H)
    grads = gdn.gdn_ssm_chunk_bwd(*(dev(t) for t in (dout, x, B, C, a, A_log)), num_seqs=n)
    dt = torch.log1p(a.double().exp())
    E = (dt * dout[:, :, 5].double() * x[:, :, 5].double()).unflatten(1, (G, H // G)).sum(-1)[..., None]
    for got, ref in ((grads[1], E * C.double()), (grads[2], E * B.double())):
        # half the distance of two bf16 values at ref
        half = torch.exp2(torch.floor(torch.log2(ref.abs())) - 8)
        over = (got.cpu().double() - ref).abs() - half
        assert (over / ref.abs()).max().item() <= 32 * 2.0 ** -24
