"""The state space layer's calls at sizes where their launch rules choose other plans than for small ones: long runs of
tokens and rings that go round more than once (convolution), several heads a set, sets across the border of q and k and
blocks that walk on (norm and rotation), several heads a block (gradients and outputs of the scan); malformed offsets of
bf16 calls; the same bits again.  Against the plain 64-bit forms of tests/_layer.py, with its bounds."""
import pytest
import torch

import gated_deltanet_recurrence_gb300 as gdn
from tests import _layer
from tests._layer import F64, check, wide
from tests.test_gpu_layer import (  # noqa: F401
    BF, CU_ERROR, F32, check_grads, clean_error_word, cu, dev, draw, offsets, qk_inputs, angles, scan_inputs, scan_reference)

pytestmark = pytest.mark.gpu


# ---- short convolution: long runs --------------------------------------------------------------------

def packed_lengths(total):
    """A few odd lengths, some shorter than the taps, one of what is left."""
    lengths = [1, 0, 333, 2, 517, 3]
    return lengths + [total - sum(lengths)]


CONV_CASES = [  # tokens, channels, dtype: runs of 20 and 44 tokens (forward, gradients), 39 and 86, 66 and 98 (two rounds)
    (2100, 4352, BF), (2100, 4352, F32), (4100, 4352, F32), (14100, 4352, BF),
]


@pytest.mark.parametrize("total,dim,dtype", CONV_CASES)
def test_short_conv_with_long_runs(total, dim, dtype):
    """Channels are independent: the 64-bit form takes some of them."""
    lengths, r = packed_lengths(total), draw(total)
    offs = offsets(lengths, first=2)
    T = offs[-1] + 3
    x = dev(r(T, dim + 16), dtype)[:, 8:8 + dim]
    w, b, st = dev(r(dim, 4, scale=0.5)), dev(r(dim)), dev(r(len(lengths), dim, 3))
    dout, dlast = dev(r(T, dim), dtype), dev(r(len(lengths), dim, 3))
    out = torch.full((T, dim), 7.0, dtype=dtype, device="cuda")
    gdn.gdn_short_conv_fwd(x, w, b, cu_seqlens=cu(offs), conv_state=st, out=out)
    last = gdn.gdn_short_conv_fwd(x, w, b, cu_seqlens=cu(offs), conv_state=st)[1]
    assert bool((out[:2] == 7.0).all()) and bool((out[offs[-1]:] == 7.0).all())
    dx, dw, db, ds = gdn.gdn_short_conv_bwd(dout, x, w, b, cu_seqlens=cu(offs), conv_state=st, dconv_state_out=dlast)
    gen = torch.Generator().manual_seed(1)
    some = torch.cat([torch.arange(8), torch.randint(8, dim - 8, (32,), generator=gen), torch.arange(dim - 8, dim)])
    at = some.cuda()
    X, W, Bb, S, DO, DL = (wide(t) for t in (x[:, at], w[at], b[at], st[:, at], dout[:, at], dlast[:, at]))
    ref, c, ref_last = _layer.conv(X, W, Bb, offs, S)
    cmag = _layer.conv(X.abs(), W.abs(), Bb.abs(), offs, S.abs(), False)[0]
    n = slice(offs[0], offs[-1])
    check("out", out[n, at], ref[n], 2 * cmag[n])
    assert torch.equal(last[:, at].cpu().to(F64), ref_last)
    inside = torch.zeros(T, 1, dtype=F64)
    inside[n] = 1
    ref = _layer.conv_bwd(DO * inside * _layer.silu_slope(c), X, W, offs, S, DL)
    terms = _layer.conv_bwd(DO.abs() * inside * (1.1 + cmag), X.abs(), W.abs(), offs, S.abs(), DL.abs())
    check("dx", dx[:, at], ref[0], terms[0])
    # a run's up to 98 tokens, eight runs and at most 36 blocks are added one by one: three times 64 roundings
    check("dweight", dw[at], ref[1], 3 * terms[1])
    check("dbias", db[at], ref[2], 3 * terms[2])
    check("dstate", ds[:, at], ref[3], terms[3])


# ---- norm and rotation: several heads a set ------------------------------------------------------------

QK_CASES = [  # T, H, H_k, d, rot, l2, interleaved, weights, dtype
    # five heads a set, the last of q's 16 with k's 4
    (1201, 16, 4, 128, 64, False, False, True, BF), (1201, 16, 4, 128, 128, True, True, False, F32),
    # all 20 heads a set: five groups of four rows (ten of two backwards)
    (2501, 16, 4, 128, 128, False, False, True, BF), (2501, 16, 4, 96, 24, True, False, True, F32),
    # more than the 608 blocks that walk on, with sets without a row at the end
    (19461, 2, 1, 64, 64, False, False, True, BF), (4907, 2, 1, 256, 128, True, True, True, F32),
]


@pytest.mark.parametrize("T,H,H_k,d,rot,l2,interleaved,weights,dtype", QK_CASES)
def test_qk_norm_rope_with_several_heads_a_set(T, H, H_k, d, rot, l2, interleaved, weights, dtype):
    q, k, table, pos, w, r = qk_inputs(T, H, H_k, d, rot, weights, dtype, seed=T)
    kw = dict(positions=pos, q_weight=w[0], k_weight=w[1], norm=gdn.GDN_NORM_L2 if l2 else gdn.GDN_NORM_RMS, eps=1e-5,
              interleaved=interleaved)
    outs = gdn.gdn_qk_norm_rope(q, k, table, **kw)
    cos, sin = angles(table, pos, rot, T)
    douts = dev(r(T, H, d), dtype), dev(r(T, H_k, d), dtype)
    grads = gdn.gdn_qk_norm_rope_bwd(*douts, q, k, table, **kw)
    for i, x in enumerate((q, k)):
        ref, terms = _layer.qk(wide(x), wide(w[i]), cos, sin, l2, 1e-5, interleaved)
        check("rotated", outs[i], ref, terms)
        ref = _layer.qk_bwd(wide(douts[i]), wide(x), wide(w[i]), cos, sin, l2, 1e-5, interleaved)
        check("dx", grads[i], ref[0], ref[2])
        if weights:  # a thread's up to 32 rows, 32 sets, 20 rows of the table and 32 ranges one by one: two times 64
            check("dw", grads[2 + i], ref[1], 2 * ref[3])


# ---- scan: several heads a block ------------------------------------------------------------------------

def many_lengths(n, seed):
    """n short sequences, some empty, and two of more than two chunks."""
    gen = torch.Generator().manual_seed(seed)
    lengths = torch.randint(0, 12, (n,), generator=gen).tolist()
    lengths[n // 3], lengths[n // 2] = 300, 263
    return lengths


MANY_CASES = [  # sequences, H, G, P, N, dtype: chunks enough that a block takes 6, 8, 4, 3, 4 and 4 heads
    (110, 6, 1, 64, 128, BF), (130, 8, 1, 64, 64, BF), (160, 8, 2, 128, 64, BF), (80, 9, 1, 128, 128, BF),
    (320, 4, 1, 64, 64, F32), (170, 8, 1, 128, 64, F32),
]


@pytest.mark.parametrize("n,H,G,P,N,dtype", MANY_CASES)
def test_scan_with_several_heads_a_block(n, H, G, P, N, dtype):
    lengths = many_lengths(n, seed=n)
    offs, T, s, S0, r = scan_inputs(lengths, 5, H, G, P, N, dtype, True, True, seed=n, first=3)
    out = torch.full((T, H, P), 7.0, dtype=dtype, device="cuda")
    args = dict(cu_seqlens=cu(offs), initial_state=S0)
    got, last = gdn.gdn_ssm_chunk_fwd(**s, **args, out=out)
    (ref, ref_last), (terms, terms_last) = scan_reference(s, offs, S0)
    rows = slice(offs[0], offs[-1])
    check("out", got[rows], ref[rows], terms[rows])
    check("state", last, ref_last, terms_last)
    assert bool((got[:3] == 7.0).all()) and bool((got[offs[-1]:] == 7.0).all())
    dout, dlast = dev(r(T, H, P), dtype), dev(r(n, H, P, N))
    grads = gdn.gdn_ssm_chunk_bwd(dout, **s, **args, dfinal_state=dlast)
    check_grads(grads, dout, s, offs, S0, dlast, dtype)
    for _ in range(3):
        for a, b in zip(grads, gdn.gdn_ssm_chunk_bwd(dout, **s, **args, dfinal_state=dlast)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_of_a_training_batch_gives_the_same_bits_again(dtype):
    """Two sequences of 4096 tokens, 32 heads in two groups: 16 heads a block."""
    r = draw(71)
    T, H, G, P, N = 8192, 32, 2, 64, 128
    x, B, C = dev(r(T, H * P + 2 * G * N), dtype).split([H * P, G * N, G * N], -1)
    s = dict(x=x.unflatten(-1, (H, P)), B=B.unflatten(-1, (G, N)), C=C.unflatten(-1, (G, N)), a=dev(r(T, H) - 2),
             A_log=dev(r(H)), dt_bias=dev(r(H)), D=dev(r(H)), cu_seqlens=cu([0, 4096, 8192]))
    dout = dev(r(T, H, P), dtype)
    first = gdn.gdn_ssm_chunk_fwd(**s), gdn.gdn_ssm_chunk_bwd(dout, **s)
    for i in range(20):
        again = gdn.gdn_ssm_chunk_fwd(**s), gdn.gdn_ssm_chunk_bwd(dout, **s)
        for a, b in zip((*first[0], *first[1]), (*again[0], *again[1])):
            assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("offs,H", [([0, 900, 800, 3000], 1), ([-1, 900, 1000, 3000], 1), ([0, 900, 1000, 3001], 2),
                                    ([0, 40, 30, 200], 2), ([0, 40, 50, 201], 9)])
def test_malformed_offsets_of_bf16_calls_write_nothing(offs, H):
    """3000 tokens: in segments."""
    T = 200 if offs[-1] < 300 else 3000
    L = gdn.lib()
    assert (L.gdn_ssm_chunk_fwd_workspace_size(3, T, H, 1, 64, 64, 1) > 0) == (T == 3000)
    _, _, s, _, r = scan_inputs([T], 0, H, 1, 64, 64, BF, False, True, seed=14)
    bad, S0 = torch.tensor(offs, dtype=torch.int32, device="cuda"), dev(r(3, H, 64, 64))
    full = lambda *sh, dt=F32: torch.full(sh, 5.0, dtype=dt, device="cuda")  # noqa: E731
    outs = dict(out=full(T, H, 64, dt=BF), final_state=full(3, H, 64, 64))
    gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=bad, initial_state=S0, **outs)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == CU_ERROR
    grads = dict(dx=full(T, H, 64, dt=BF), dB=full(T, 1, 64, dt=BF), dC=full(T, 1, 64, dt=BF), da=full(T, H),
                 dinitial_state=full(3, H, 64, 64))
    gdn.gdn_ssm_chunk_bwd(full(T, H, 64, dt=BF), **s, cu_seqlens=bad, initial_state=S0, **grads)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == CU_ERROR
    x, w = dev(r(T, 64), BF), dev(r(64, 4))
    conv = dict(out=full(T, 64, dt=BF), conv_state_out=full(3, 64, 3))
    gdn.gdn_short_conv_fwd(x, w, cu_seqlens=bad, **conv)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == CU_ERROR
    cgrads = dict(dx=full(T, 64, dt=BF), dconv_state=full(3, 64, 3))
    gdn.gdn_short_conv_bwd(x, x, w, cu_seqlens=bad, **cgrads)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == CU_ERROR
    for name, t in {**outs, **grads, **conv, **cgrads}.items():
        assert bool((t == 5.0).all()), name
