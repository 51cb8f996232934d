"""The state space layer's calls on the GPU against their plain 64-bit forms, token by token (tests/_layer.py has them,
and what rounding may leave): prompts, tokens and gradients of the short convolution and of the selective scan, the
norm with the rotation; the ends where they can go wrong; and a layer that runs them together."""
import pytest
import torch

import gated_deltanet_recurrence_gb300 as gdn
from tests import _layer
from tests._layer import F64, check, wide

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CU_ERROR, ARG_ERROR = -3, -1


@pytest.fixture(autouse=True)
def clean_error_word():
    gdn.gdn_get_device_error()
    yield
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == 0


def offsets(lengths, first=0):
    offs = [first]
    for n in lengths:
        offs.append(offs[-1] + n)
    return offs


def cu(offs):
    return torch.tensor(offs, dtype=torch.int32, device="cuda")


def draw(seed):
    gen = torch.Generator().manual_seed(seed)
    return lambda *s, scale=1.0: torch.randn(*s, generator=gen) * scale


def dev(t, dtype=None):
    return None if t is None else t.to("cuda", dtype)


# ---- short convolution ---------------------------------------------------------------------------

CONV_CASES = [  # lengths, tokens behind the last sequence, dim, dtype, bias, state, silu
    ([1], 0, 8, F32, True, True, True), ([2], 0, 64, BF, False, False, True), ([3, 0, 5], 0, 40, F32, True, True, False),
    ([4, 1, 2, 3, 61], 7, 128, BF, True, True, True), ([130, 64, 0, 0, 1], 3, 2056, F32, False, True, True),
    ([300], 0, 4352, BF, True, False, True), ([1] * 70 + [0] * 5 + [9], 0, 24, BF, True, True, True),
]


def conv_inputs(lengths, tail, dim, dtype, bias, state, seed=0, first=0):
    r = draw(seed)
    offs = offsets(lengths, first)
    T = offs[-1] + tail
    x = dev(r(T, dim + 16), dtype)[:, 8:8 + dim]     # a slice of a wider tensor
    w, b = dev(r(dim, 4, scale=0.5)), dev(r(dim)) if bias else None
    return offs, T, x, w, b, dev(r(len(lengths), dim, 3)) if state else None, r


@pytest.mark.parametrize("lengths,tail,dim,dtype,bias,state,silu", CONV_CASES)
def test_short_conv(lengths, tail, dim, dtype, bias, state, silu):
    offs, T, x, w, b, st, _ = conv_inputs(lengths, tail, dim, dtype, bias, state, seed=dim)
    out = torch.full((T, dim), 7.0, dtype=dtype, device="cuda")
    got, last = gdn.gdn_short_conv_fwd(x, w, b, cu_seqlens=cu(offs), conv_state=st, silu=silu, out=out)
    ref, _, ref_last = _layer.conv(wide(x), wide(w), wide(b), offs, wide(st), silu)
    terms = _layer.conv(wide(x).abs(), wide(w).abs(), None if b is None else wide(b).abs(), offs,
                        None if st is None else wide(st).abs(), False)[0]
    n = offs[-1]
    check("out", got[:n], ref[:n], 2 * terms[:n])
    assert bool((got[n:] == 7.0).all())               # rows behind the last sequence stay as they were
    assert torch.equal(last.cpu().to(F64), ref_last)


def test_short_conv_equal_lengths_in_place_history_and_empty_batch():
    _, T, x, w, b, st, _ = conv_inputs([8, 8, 8], 0, 64, F32, True, True, seed=5)
    ref, last = gdn.gdn_short_conv_fwd(x, w, b, cu_seqlens=cu([0, 8, 16, 24]), conv_state=st)
    keep = st.clone()
    out, same = gdn.gdn_short_conv_fwd(x, w, b, num_seqs=3, conv_state=keep, conv_state_out=keep)
    assert torch.equal(out, ref) and torch.equal(keep, last) and same is keep
    out, last = gdn.gdn_short_conv_fwd(x[:0], w, b, num_seqs=3, conv_state=st)
    assert out.shape == (0, 64) and torch.equal(last, st)


@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("dim,dtype", [(8, F32), (136, BF), (2048, BF)])
def test_short_conv_step_continues_a_prompt(T, dim, dtype):
    """The tokens after a prompt give what the whole prompt would have given."""
    N = 5
    offs, total, x, w, b, st, r = conv_inputs([9] * N, 0, dim, dtype, True, True, seed=T)
    whole, last = gdn.gdn_short_conv_fwd(x, w, b, num_seqs=N, conv_state=st)
    seqs = x.unflatten(0, (N, 9))
    _, mid = gdn.gdn_short_conv_fwd(seqs[:, :9 - T].reshape(-1, dim), w, b, num_seqs=N, conv_state=st)
    pool = torch.full((9, dim, 3), 5.0, device="cuda")
    idx = [7, 0, 3, 8, 1]
    pool[idx] = mid
    tail = seqs[:, 9 - T:].contiguous()
    out = gdn.gdn_short_conv_step(tail, w, pool, b, state_indices=torch.tensor(idx, dtype=torch.int32, device="cuda"))
    assert torch.equal(out, whole.unflatten(0, (N, 9))[:, 9 - T:])
    assert torch.equal(pool[idx], last)
    assert bool((pool[[2, 4, 5, 6]] == 5.0).all())


def test_step_calls_skip_negative_and_catch_large_slots():
    r = draw(3)
    x, w, pool = dev(r(3, 1, 64)), dev(r(64, 4)), dev(r(4, 64, 3))
    before, out = pool.clone(), torch.full((3, 1, 64), 9.0, device="cuda")
    gdn.gdn_short_conv_step(x, w, pool, state_indices=torch.tensor([2, -1, 4], dtype=torch.int32, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == ARG_ERROR
    assert bool((out[1:] == 9.0).all()) and torch.equal(pool[[0, 1, 3]], before[[0, 1, 3]]) and not torch.equal(pool[2], before[2])
    st = dev(r(4, 2, 64, 64))
    before, out = st.clone(), torch.full((3, 1, 2, 64), 9.0, device="cuda")
    gdn.gdn_ssm_step(dev(r(3, 1, 2, 64)), dev(r(3, 1, 1, 64)), dev(r(3, 1, 1, 64)), dev(r(3, 1, 2)), dev(r(2)), st,
                     state_indices=torch.tensor([2, -1, 4], dtype=torch.int32, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == ARG_ERROR
    assert bool((out[1:] == 9.0).all()) and torch.equal(st[[0, 1, 3]], before[[0, 1, 3]]) and not torch.equal(st[2], before[2])


@pytest.mark.parametrize("lengths,tail,dim,dtype,bias,state,silu", CONV_CASES)
@pytest.mark.parametrize("first", [0, 2])
def test_short_conv_bwd(lengths, tail, dim, dtype, bias, state, silu, first):
    offs, T, x, w, b, st, r = conv_inputs(lengths, tail, dim, dtype, bias, state, seed=dim, first=first)
    dout = dev(r(T, dim), dtype)
    dlast = dev(r(len(lengths), dim, 3)) if state else None
    dx, dw, db, ds = gdn.gdn_short_conv_bwd(dout, x, w, b, cu_seqlens=cu(offs), conv_state=st, dconv_state_out=dlast, silu=silu)
    X, W, Bb, S, DO, DL = (wide(t) for t in (x, w, b, st, dout, dlast))
    _, c, _ = _layer.conv(X, W, Bb, offs, S, silu)
    mag = lambda t: None if t is None else t.abs()  # noqa: E731
    cmag, _, _ = _layer.conv(X.abs(), W.abs(), mag(Bb), offs, mag(S), False)
    inside = torch.zeros(T, 1, dtype=F64)
    inside[offs[0]:offs[-1]] = 1
    ref = _layer.conv_bwd(DO * inside * (_layer.silu_slope(c) if silu else 1.0), X, W, offs, S, DL)
    # the slope of the SiLU is at most 1.1 and changes by at most half of c's error
    terms = _layer.conv_bwd(DO.abs() * inside * (1.1 + cmag), X.abs(), W.abs(), offs, mag(S), mag(DL))
    check("dx", dx, ref[0], terms[0])                 # rows outside the sequences are zeros
    check("dweight", dw, ref[1], terms[1])
    if bias:
        check("dbias", db, ref[2], terms[2])
    else:
        assert db is None
    if state:
        check("dstate", ds, ref[3], terms[3])
    given = torch.full_like(dx, 3.0)
    gdn.gdn_short_conv_bwd(dout, x, w, b, cu_seqlens=cu(offs), conv_state=st, dconv_state_out=dlast, silu=silu, dx=given)
    assert torch.equal(given[offs[0]:offs[-1]], dx[offs[0]:offs[-1]])
    assert bool((given[:offs[0]] == 3.0).all()) and bool((given[offs[-1]:] == 3.0).all())


def test_short_conv_pieces_have_the_whole_sequences_gradients():
    """A sequence cut in two: the later part's dconv_state is the earlier part's dconv_state_out."""
    _, T, x, w, b, st, r = conv_inputs([50], 0, 64, F32, True, True, seed=8)
    dout = dev(r(50, 64))
    dx, dw, db, ds = gdn.gdn_short_conv_bwd(dout, x, w, b, conv_state=st)
    _, mid = gdn.gdn_short_conv_fwd(x[:48], w, b, conv_state=st)
    dx2, dw2, db2, dmid = gdn.gdn_short_conv_bwd(dout[48:], x[48:], w, b, conv_state=mid)
    dx1, dw1, db1, ds1 = gdn.gdn_short_conv_bwd(dout[:48], x[:48], w, b, conv_state=st, dconv_state_out=dmid)
    assert torch.allclose(torch.cat([dx1, dx2]), dx, rtol=1e-6, atol=1e-6) and torch.allclose(ds1, ds, rtol=1e-6, atol=1e-6)
    assert torch.allclose(dw1 + dw2, dw, rtol=1e-5, atol=1e-5) and torch.allclose(db1 + db2, db, rtol=1e-5, atol=1e-5)


# ---- selective scan ------------------------------------------------------------------------------

SCAN_CASES = [  # lengths, tokens behind, H, G, P, N, dtype, carried, dt_bias and D
    ([1], 0, 1, 1, 64, 64, F32, True, True), ([63], 0, 2, 1, 64, 128, BF, False, True), ([64], 0, 3, 3, 128, 64, F32, True, False),
    ([65, 0, 1], 5, 4, 2, 128, 128, BF, True, True), ([130, 64, 3], 0, 6, 2, 64, 128, F32, True, True),
    ([200, 129, 1, 0, 0, 77], 70, 4, 1, 64, 64, BF, True, False), ([300], 0, 5, 1, 128, 128, F32, False, True),
    ([2] * 40, 1, 2, 2, 64, 64, BF, True, True), ([257, 127], 0, 10, 2, 64, 128, BF, True, True),
]


def scan_inputs(lengths, tail, H, G, P, N, dtype, carried, extra, seed, first=0, a_scale=1.0, a_shift=-2.0):
    r = draw(seed)
    offs = offsets(lengths, first)
    T, n = offs[-1] + tail, len(lengths)
    mixed = dev(r(T, H * P + 2 * G * N), dtype)
    x, B, C = mixed.split([H * P, G * N, G * N], -1)
    s = dict(x=x.unflatten(-1, (H, P)), B=B.unflatten(-1, (G, N)), C=C.unflatten(-1, (G, N)),
             a=dev(r(T, H) * a_scale + a_shift), A_log=dev(r(H)), dt_bias=dev(r(H)) if extra else None,
             D=dev(r(H)) if extra else None)
    return offs, T, s, dev(r(n, H, P, N)) if carried else None, r


def scan_reference(s, offs, S0):
    w = {k: wide(t) for k, t in s.items()}
    S = wide(S0)
    _, dt, alpha = _layer.gates(w["a"], w["A_log"], w["dt_bias"])
    ref = _layer.ssm(w["x"], w["B"], w["C"], dt, alpha, w["D"], offs, S)
    mag = lambda t: None if t is None else t.abs()  # noqa: E731
    terms = _layer.ssm(w["x"].abs(), w["B"].abs(), w["C"].abs(), dt, alpha, mag(w["D"]), offs, mag(S))
    return ref, terms


@pytest.mark.parametrize("lengths,tail,H,G,P,N,dtype,carried,extra", SCAN_CASES)
def test_scan(lengths, tail, H, G, P, N, dtype, carried, extra):
    offs, T, s, S0, _ = scan_inputs(lengths, tail, H, G, P, N, dtype, carried, extra, seed=H + sum(lengths))
    out = torch.full((T, H, P), 7.0, dtype=dtype, device="cuda")
    got, last = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=S0, out=out)
    (ref, ref_last), (terms, terms_last) = scan_reference(s, offs, S0)
    n = offs[-1]
    check("out", got[:n], ref[:n], terms[:n])
    check("state", last, ref_last, terms_last)
    assert bool((got[n:] == 7.0).all())
    again, last2 = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=S0, out=out.clone())
    assert torch.equal(again, got) and torch.equal(last2, last)


SEGMENT_CASES = [  # long sequences of few heads, which are walked along in segments
    ([1700], 0, 1, 1, 64, 64, BF, True, True), ([0, 5200, 1], 9, 2, 2, 64, 64, BF, True, False),
    ([1600], 0, 2, 1, 128, 128, BF, True, True), ([2048], 0, 3, 3, 64, 128, BF, False, True),
    ([900], 0, 2, 1, 64, 128, F32, True, True), ([0, 2500, 1], 9, 2, 2, 64, 64, F32, True, False), ([1024], 0, 1, 1, 128, 128, F32, False, True),
]


@pytest.mark.parametrize("first", [0, 77])
@pytest.mark.parametrize("lengths,tail,H,G,P,N,dtype,carried,extra", SEGMENT_CASES)
def test_scan_in_segments(lengths, tail, H, G, P, N, dtype, carried, extra, first):
    offs, T, s, S0, r = scan_inputs(lengths, tail, H, G, P, N, dtype, carried, extra, seed=H + sum(lengths), first=first)
    assert dtype == F32 or gdn.lib().gdn_ssm_chunk_fwd_workspace_size(len(lengths), T, H, G, P, N, 1) > 0
    out = torch.full((T, H, P), 7.0, dtype=dtype, device="cuda")
    got, last = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=S0, out=out)
    (ref, ref_last), (terms, terms_last) = scan_reference(s, offs, S0)
    check("out", got[first:offs[-1]], ref[first:offs[-1]], terms[first:offs[-1]])
    check("state", last, ref_last, terms_last)
    assert bool((got[:first] == 7.0).all()) and bool((got[offs[-1]:] == 7.0).all())
    if carried:  # the final states in the initial ones' place
        keep = S0.clone()
        again, same = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=keep, final_state=keep, out=out.clone())
        assert torch.equal(again, got) and torch.equal(keep, last) and same is keep
    dout = dev(r(T, H, P), dtype)
    dlast = dev(r(len(lengths), H, P, N)) if carried else None
    args = dict(cu_seqlens=cu(offs), initial_state=S0)
    grads = gdn.gdn_ssm_chunk_bwd(dout, **s, **args, dfinal_state=dlast)
    check_grads(grads, dout, s, offs, S0, dlast, dtype)
    if carried:
        keep = dlast.clone()
        for a, b in zip(grads, gdn.gdn_ssm_chunk_bwd(dout, **s, **args, dfinal_state=keep, dinitial_state=keep)):
            assert a is None or torch.equal(a, b)
    # a workspace of just the size, of NaN, with a guard behind it
    L, sizes = gdn.lib(), (len(lengths), T, H, G, P, N, int(dtype == BF))
    for need, call in ((L.gdn_ssm_chunk_fwd_workspace_size(*sizes), lambda ws: gdn.gdn_ssm_chunk_fwd(**s, **args, workspace=ws)),
                       (L.gdn_ssm_chunk_bwd_workspace_size(*sizes),
                        lambda ws: gdn.gdn_ssm_chunk_bwd(dout, **s, **args, dfinal_state=dlast, workspace=ws))):
        ws = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")
        results = call(ws[:need])
        assert bool((ws[need:] == 255).all())
        for a, b in zip(results, (got, last) if len(results) == 2 else grads):
            rows = slice(first, offs[-1]) if a is not None and a.shape[0] == T else slice(None)
            assert a is None or torch.equal(a[rows], b[rows])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale,shift,a_log", [(30.0, 0.0, 0.0), (1.0, 60.0, 3.0), (1.0, -40.0, 0.0), (1.0, 0.0, -20.0)])
def test_scan_in_segments_with_extreme_steps_and_decays(dtype, scale, shift, a_log):
    offs, T, s, S0, r = scan_inputs([1600], 0, 1, 1, 64, 64, dtype, True, True, seed=58, a_scale=scale, a_shift=shift)
    s["A_log"] = torch.full_like(s["A_log"], a_log)
    got, last = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=S0)
    (ref, ref_last), (terms, terms_last) = scan_reference(s, offs, S0)
    check("out", got, ref, terms)
    check("state", last, ref_last, terms_last)
    dout = dev(r(*s["x"].shape), dtype)
    check_grads(gdn.gdn_ssm_chunk_bwd(dout, **s, cu_seqlens=cu(offs), initial_state=S0), dout, s, offs, S0, None, dtype)


def test_scan_in_segments_of_packed_prompts_that_differ():
    """More blocks than SMs, and one sequence that outlasts the others."""
    lengths, H, P, N = [1, 37, 513, 2901, 0, 1333, 700], 24, 64, 64
    assert gdn.lib().gdn_ssm_chunk_fwd_workspace_size(len(lengths), sum(lengths), H, 1, P, N, 1) > 0
    offs, T, s, S0, _ = scan_inputs(lengths, 0, H, 1, P, N, BF, True, True, seed=57)
    got, last = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=S0)
    (ref, ref_last), (terms, terms_last) = scan_reference(s, offs, S0)
    check("out", got, ref, terms)
    check("state", last, ref_last, terms_last)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_scan_of_many_sequences_without_offsets_and_states_in_place(dtype):
    offs, T, s, S0, _ = scan_inputs([70] * 5, 0, 2, 1, 64, 64, dtype, True, True, seed=9)
    ref, last = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=S0)
    keep = S0.clone()
    out, same = gdn.gdn_ssm_chunk_fwd(**s, num_seqs=5, initial_state=keep, final_state=keep)
    assert torch.equal(out, ref) and torch.equal(keep, last) and same is keep
    out, none = gdn.gdn_ssm_chunk_fwd(**s, num_seqs=5, initial_state=S0, output_final_state=False)
    assert none is None and torch.equal(out, ref)
    empty = {k: (v[:0] if k in ("x", "B", "C", "a") else v) for k, v in s.items()}
    out, last = gdn.gdn_ssm_chunk_fwd(**empty, num_seqs=5, initial_state=S0)
    assert out.shape[0] == 0 and torch.equal(last, S0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scale,shift,a_log", [(30.0, 0.0, 0.0), (1.0, 60.0, 3.0), (1.0, -40.0, 0.0), (1.0, 0.0, -20.0)])
def test_scan_with_extreme_steps_and_decays(dtype, scale, shift, a_log):
    """Steps near zero and of tens, decays to zero and of one."""
    offs, T, s, S0, r = scan_inputs([150, 3], 0, 2, 1, 64, 64, dtype, True, True, seed=11, a_scale=scale, a_shift=shift)
    s["A_log"] = torch.full_like(s["A_log"], a_log)
    got, last = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=S0)
    (ref, ref_last), (terms, terms_last) = scan_reference(s, offs, S0)
    check("out", got, ref, terms)
    check("state", last, ref_last, terms_last)
    dout = dev(r(*s["x"].shape), dtype)
    grads = gdn.gdn_ssm_chunk_bwd(dout, **s, cu_seqlens=cu(offs), initial_state=S0)
    check_grads(grads, dout, s, offs, S0, None, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_scan_keeps_sequences_apart(dtype):
    """NaN and infinities in one sequence, and in rows of no sequence, reach no other sequence."""
    offs, T, s, S0, r = scan_inputs([70, 30, 65], 40, 2, 1, 64, 64, dtype, True, True, seed=13, first=3)
    dout = dev(r(*s["x"].shape), dtype)
    args = dict(cu_seqlens=cu(offs), initial_state=S0)
    out, last = gdn.gdn_ssm_chunk_fwd(**s, **args, out=torch.zeros_like(dout))
    grads = gdn.gdn_ssm_chunk_bwd(dout, **s, **args)
    bad = {k: (v.clone() if k in ("x", "B", "C", "a") else v) for k, v in s.items()}
    bad_out = dout.clone()
    for t in (bad["x"], bad["B"], bad["C"], bad["a"], bad_out):
        t[:3] = float("nan")
        t[offs[-1]:] = float("inf")
        t[73 + 4] = float("nan")                      # in the second sequence
    out2, last2 = gdn.gdn_ssm_chunk_fwd(**bad, **args, out=torch.zeros_like(dout))
    grads2 = gdn.gdn_ssm_chunk_bwd(bad_out, **bad, **args)
    for a, b in [(out, out2), *zip(grads[:4], grads2[:4])]:
        assert torch.equal(a[3:73], b[3:73]) and torch.equal(a[103:168], b[103:168])
        assert bool(torch.isnan(b[73 + 4]).any())
    for a, b in ((last, last2), (grads[7], grads2[7])):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    # the convolution and its gradient too
    dim = 64
    w, st = dev(r(dim, 4)), dev(r(3, dim, 3))
    x, xb = s["x"].flatten(1)[:, :dim], bad["x"].flatten(1)[:, :dim]
    g, gb = dout.flatten(1)[:, :dim].contiguous(), bad_out.flatten(1)[:, :dim].contiguous()
    a, b = (gdn.gdn_short_conv_fwd(v, w, cu_seqlens=cu(offs), conv_state=st)[0] for v in (x, xb))
    assert torch.equal(a[3:73], b[3:73]) and torch.equal(a[103:168], b[103:168])
    a, b = (gdn.gdn_short_conv_bwd(u, v, w, cu_seqlens=cu(offs), conv_state=st)[0] for u, v in ((g, x), (gb, xb)))
    assert torch.equal(a[3:73], b[3:73]) and torch.equal(a[103:], b[103:])


@pytest.mark.parametrize("offs", [[0, 40, 30, 64], [-1, 30, 50, 64], [0, 30, 50, 65], [5, 4, 3, 2]])
def test_malformed_offsets_write_nothing(offs):
    _, T, s, S0, r = scan_inputs([64], 0, 2, 1, 64, 64, F32, False, True, seed=14)
    S0 = dev(r(3, 2, 64, 64))
    bad = torch.tensor(offs, dtype=torch.int32, device="cuda")
    full = lambda *sh: torch.full(sh, 5.0, device="cuda")  # noqa: E731
    outs = dict(out=full(64, 2, 64), final_state=full(3, 2, 64, 64))
    gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=bad, initial_state=S0, **outs)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == CU_ERROR
    grads = dict(dx=full(64, 2, 64), dB=full(64, 1, 64), dC=full(64, 1, 64), da=full(64, 2), dinitial_state=full(3, 2, 64, 64))
    gdn.gdn_ssm_chunk_bwd(full(64, 2, 64), **s, cu_seqlens=bad, initial_state=S0, **grads)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == CU_ERROR
    x, w = dev(r(64, 64)), dev(r(64, 4))
    conv = dict(out=full(64, 64), conv_state_out=full(3, 64, 3))
    gdn.gdn_short_conv_fwd(x, w, cu_seqlens=bad, **conv)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == CU_ERROR
    cgrads = dict(dx=full(64, 64), dconv_state=full(3, 64, 3))
    gdn.gdn_short_conv_bwd(x, x, w, cu_seqlens=bad, **cgrads)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == CU_ERROR
    for name, t in {**outs, **grads, **conv, **cgrads}.items():
        assert bool((t == 5.0).all()), name


GRADS = ("dx", "dB", "dC", "da", "dA_log", "ddt_bias", "dD", "dinitial_state")


def check_grads(grads, dout, s, offs, S0, dlast, dtype):
    w = {k: wide(t) for k, t in s.items()}
    ref, terms = _layer.scan_grads(wide(dout), w["x"], w["B"], w["C"], w["a"], w["A_log"], w["dt_bias"], w["D"], offs, wide(S0),
                                   wide(dlast))
    for name, got in zip(GRADS, grads):
        if got is not None:
            check(name, got, ref[name], terms[name])


@pytest.mark.parametrize("first", [0, 3])
@pytest.mark.parametrize("lengths,tail,H,G,P,N,dtype,carried,extra", SCAN_CASES)
def test_scan_bwd(lengths, tail, H, G, P, N, dtype, carried, extra, first):
    offs, T, s, S0, r = scan_inputs(lengths, tail, H, G, P, N, dtype, carried, extra, seed=H + sum(lengths), first=first)
    dout = dev(r(T, H, P), dtype)
    dlast = dev(r(len(lengths), H, P, N)) if carried else None
    args = dict(cu_seqlens=cu(offs), initial_state=S0, dfinal_state=dlast)
    grads = gdn.gdn_ssm_chunk_bwd(dout, **s, **args)
    assert (grads[7] is not None) == carried and (grads[6] is not None) == extra
    check_grads(grads, dout, s, offs, S0, dlast, dtype)   # zeros outside the sequences
    given = {k: torch.full_like(g, 3.0) for k, g in zip(GRADS[:4], grads)}
    more = gdn.gdn_ssm_chunk_bwd(dout, **s, **args, **given)
    for k, a, b in zip(GRADS, grads, more):
        if k in given:
            assert torch.equal(a[offs[0]:offs[-1]], b[offs[0]:offs[-1]])
            assert bool((b[:offs[0]] == 3.0).all()) and bool((b[offs[-1]:] == 3.0).all())
        elif a is not None:
            assert torch.equal(a, b), k


def test_scan_bwd_in_pieces_and_in_place_state():
    """A sequence cut where the forward handed out a state has the whole sequence's gradients."""
    _, T, s, S0, r = scan_inputs([150], 0, 2, 1, 64, 128, F32, True, True, seed=21)
    dout, dlast = dev(r(150, 2, 64)), dev(r(1, 2, 64, 128))
    whole = gdn.gdn_ssm_chunk_bwd(dout, **s, initial_state=S0, dfinal_state=dlast)
    part = lambda lo, hi: {k: (v[lo:hi] if k in ("x", "B", "C", "a") else v) for k, v in s.items()}  # noqa: E731
    _, mid = gdn.gdn_ssm_chunk_fwd(**part(0, 97), initial_state=S0)
    carry = dlast.clone()
    late = gdn.gdn_ssm_chunk_bwd(dout[97:].clone(), **part(97, 150), initial_state=mid, dfinal_state=carry, dinitial_state=carry)
    assert late[7] is carry
    early = gdn.gdn_ssm_chunk_bwd(dout[:97], **part(0, 97), initial_state=S0, dfinal_state=carry)
    for i, name in enumerate(GRADS):
        got = torch.cat([early[i], late[i]]) if i < 4 else (early[i] if i == 7 else early[i] + late[i])
        off = (got - whole[i]).norm() / whole[i].norm()
        assert off <= 1e-5, (name, off)                # two orders of the additions


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("P,N,H,G,dtype", [(64, 64, 4, 2, F32), (64, 128, 6, 1, BF), (128, 128, 2, 1, F32), (128, 64, 3, 3, BF)])
def test_step_continues_a_prompt(T, P, N, H, G, dtype):
    n, L = 4, 70
    offs, _, s, S0, _ = scan_inputs([L] * n, 0, H, G, P, N, dtype, True, True, seed=T + P + N)
    (ref, ref_last), (terms, terms_last) = scan_reference(s, offs, S0)
    part = lambda t, lo, hi: t.unflatten(0, (n, L))[:, lo:hi]  # noqa: E731
    first = {k: (part(v, 0, L - T).flatten(0, 1) if k in ("x", "B", "C", "a") else v) for k, v in s.items()}
    _, mid = gdn.gdn_ssm_chunk_fwd(**first, num_seqs=n, initial_state=S0)
    pool, idx = torch.full((7, H, P, N), 2.0, device="cuda"), [6, 0, 3, 2]
    pool[idx] = mid
    tok = [torch.cat([part(s[k], L - T, L).flatten(2) for k in ("x", "B", "C")], -1)]   # [n, T, mixed]: rows with a stride
    x, B, C = tok[0].split([H * P, G * N, G * N], -1)
    out = gdn.gdn_ssm_step(x.unflatten(-1, (H, P)), B.unflatten(-1, (G, N)), C.unflatten(-1, (G, N)),
                           part(s["a"], L - T, L).contiguous(), s["A_log"], pool, dt_bias=s["dt_bias"], D=s["D"],
                           state_indices=torch.tensor(idx, dtype=torch.int32, device="cuda"))
    rows = lambda t: t.unflatten(0, (n, L))[:, L - T:]  # noqa: E731
    check("out", out, rows(ref), rows(terms))
    check("state", pool[idx], ref_last, terms_last)
    assert bool((pool[[1, 4, 5]] == 2.0).all())


# ---- norm and rotation -------------------------------------------------------------------------------

QK_CASES = [  # T, H, H_k, d, rot, l2, interleaved, weights, dtype
    (1, 1, 1, 64, 64, False, False, True, F32), (5, 3, 1, 128, 64, False, True, True, BF), (33, 2, 2, 96, 24, True, False, False, F32),
    (257, 4, 0, 64, 16, False, False, True, BF), (70, 1, 5, 256, 256, True, True, True, BF), (9, 2, 1, 8, 4, False, False, True, F32),
    (40, 3, 3, 128, 0, False, False, True, F32), (1030, 5, 2, 40, 20, False, False, True, BF), (64, 8, 8, 128, 128, True, False, False, BF),
]


def qk_inputs(T, H, H_k, d, rot, weights, dtype, seed):
    r = draw(seed)
    mixed = dev(r(T, H + H_k + 1, d), dtype)
    q, k = mixed[:, :H], mixed[:, H:H + H_k] if H_k else None
    ang = r(300, max(rot // 2, 1))[:, :rot // 2] * 10
    table = dev(torch.cat([ang.cos(), ang.sin()], -1)) if rot else None
    gen = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, 300, (T,), generator=gen, dtype=torch.int32).cuda() if rot else None
    w = [dev(1 + r(d, scale=0.1)) if weights else None for _ in range(2)]
    return q, k, table, pos, w, r


def angles(table, pos, rot, T):
    if not rot:
        return torch.zeros(T, 0, dtype=F64), torch.zeros(T, 0, dtype=F64)
    rows = wide(table)[pos.cpu().long()]
    return rows[:, :rot // 2], rows[:, rot // 2:]


@pytest.mark.parametrize("T,H,H_k,d,rot,l2,interleaved,weights,dtype", QK_CASES)
def test_qk_norm_rope(T, H, H_k, d, rot, l2, interleaved, weights, dtype):
    q, k, table, pos, w, r = qk_inputs(T, H, H_k, d, rot, weights, dtype, seed=T)
    kw = dict(positions=pos, q_weight=w[0], k_weight=w[1] if H_k else None, norm=gdn.GDN_NORM_L2 if l2 else gdn.GDN_NORM_RMS,
              eps=1e-5, interleaved=interleaved)
    qo, ko = gdn.gdn_qk_norm_rope(q, k, table, **kw)
    cos, sin = angles(table, pos, rot, T)
    for x, wt, got in ((q, w[0], qo), (k, w[1], ko)):
        if x is None:
            assert got is None
            continue
        ref, terms = _layer.qk(wide(x), wide(wt), cos, sin, l2, 1e-5, interleaved)
        check("rotated", got, ref, terms)
    dq_out, dk_out = dev(r(T, H, d), dtype), dev(r(T, H_k, d), dtype) if H_k else None
    grads = gdn.gdn_qk_norm_rope_bwd(dq_out, dk_out, q, k, table, **kw)
    for x, wt, do, dx, dw in ((q, w[0], dq_out, grads[0], grads[2]), (k, w[1], dk_out, grads[1], grads[3])):
        if x is None:
            assert dx is None and dw is None
            continue
        ref = _layer.qk_bwd(wide(do), wide(x), wide(wt), cos, sin, l2, 1e-5, interleaved)
        check("dx", dx, ref[0], ref[2])
        if wt is not None:
            check("dw", dw, ref[1], ref[3])
        else:
            assert dw is None
    # in place, on the slices they came from
    keep = (q.clone(), None if k is None else k.clone())
    a, b = gdn.gdn_qk_norm_rope(q, k, table, **kw, q_out=q, k_out=k)
    assert a is q and torch.equal(q, qo) and (k is None or torch.equal(k, ko))
    again = gdn.gdn_qk_norm_rope_bwd(dq_out, dk_out, *keep, table, **kw, dq=dq_out, dk=dk_out)
    for u, v in zip(again, grads):
        assert (u is None) == (v is None) and (u is None or torch.equal(u, v))


def test_rotation_without_positions_and_with_some_outside_the_table():
    q, k, table, pos, w, r = qk_inputs(50, 2, 1, 64, 32, True, F32, seed=2)
    rows = torch.arange(50, dtype=torch.int32, device="cuda")
    a, b = gdn.gdn_qk_norm_rope(q, k, table, q_weight=w[0], k_weight=w[1])
    c, d = gdn.gdn_qk_norm_rope(q, k, table, positions=rows, q_weight=w[0], k_weight=w[1])
    assert torch.equal(a, c) and torch.equal(b, d)
    rows[7], rows[20] = 300, -1
    qo, ko = torch.full_like(a, 4.0), torch.full_like(b, 4.0)
    gdn.gdn_qk_norm_rope(q, k, table, positions=rows, q_weight=w[0], k_weight=w[1], q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == ARG_ERROR
    good = [t for t in range(50) if t not in (7, 20)]
    assert torch.equal(qo[good], a[good]) and torch.equal(ko[good], b[good])
    assert bool((qo[[7, 20]] == 4.0).all()) and bool((ko[[7, 20]] == 4.0).all())
    do, dk = dev(r(50, 2, 64)), dev(r(50, 1, 64))
    ref = gdn.gdn_qk_norm_rope_bwd(do[good], dk[good], q[good], k[good], table, positions=rows[good], q_weight=w[0], k_weight=w[1])
    got = gdn.gdn_qk_norm_rope_bwd(do, dk, q, k, table, positions=rows, q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    assert gdn.gdn_get_device_error() == ARG_ERROR
    assert torch.equal(got[0][good], ref[0]) and torch.allclose(got[2], ref[2], rtol=1e-5, atol=1e-5)


def test_l2_norm_is_the_delta_rules_own():
    """gdn_chunk_fwd on q and k normalised here equals its own normalisation (a rotation by zero changes nothing)."""
    r = draw(31)
    q, k, v = (dev(r(130, 2, 64)) for _ in range(3))
    g, beta = -dev(r(130, 2)).abs() * 0.1, dev(r(130, 2)).sigmoid()
    ref, S = gdn.gdn_chunk_fwd(q, k, v, g, beta)
    qn, kn = gdn.gdn_qk_norm_rope(q, k, None, norm=gdn.GDN_NORM_L2, eps=1e-6)
    out, S2 = gdn.gdn_chunk_fwd(qn, kn, v, g, beta, use_qk_l2norm=False)
    assert (out - ref).norm() <= 1e-5 * ref.norm() and (S2 - S).norm() <= 1e-5 * S.norm()


# ---- workspaces, guards, streams, graphs ---------------------------------------------------------------

def all_calls(dtype, seed=41, lengths=(70, 1, 0, 64, 30)):
    """Every call once, on given outputs: name -> (function of a dict of outputs, outputs)."""
    H, G, P, N, dim, d = 4, 2, 64, 128, 512, 64
    offs, T, s, S0, r = scan_inputs(list(lengths), 6, H, G, P, N, dtype, True, True, seed=seed, first=2)
    n, c = len(lengths), cu(offs)
    w, b, st = dev(r(dim, 4)), dev(r(dim)), dev(r(n, dim, 3))
    x = s["x"].flatten(1)[:, :256]
    xc = torch.cat([x, x], 1)
    dout, dlast, dst = dev(r(T, H, P), dtype), dev(r(n, H, P, N)), dev(r(n, dim, 3))
    dconv = dev(r(T, dim), dtype)
    pool, cpool = dev(r(9, H, P, N)), dev(r(9, dim, 3))
    idx = torch.tensor([8, 0, 4], dtype=torch.int32, device="cuda")
    step = {k: s[k][:6].unflatten(0, (3, 2)) for k in ("x", "B", "C", "a")}
    q, k, table, pos, qw, _ = qk_inputs(T, 3, 2, d, 32, True, dtype, seed)
    do, dk = dev(r(T, 3, d), dtype), dev(r(T, 2, d), dtype)

    def e(*shape, dt=F32):
        return torch.zeros(*shape, dtype=dt, device="cuda")

    return {
        "conv_fwd": (lambda o: gdn.gdn_short_conv_fwd(xc, w, b, cu_seqlens=c, conv_state=st, **o),
                     dict(out=e(T, dim, dt=dtype), conv_state_out=e(n, dim, 3))),
        "conv_step": (lambda o: (o["conv_state"].copy_(cpool), gdn.gdn_short_conv_step(
            xc[:6].unflatten(0, (3, 2)), w, o["conv_state"], b, state_indices=idx, out=o["out"])),
                      dict(out=e(3, 2, dim, dt=dtype), conv_state=e(9, dim, 3))),
        "conv_bwd": (lambda o: gdn.gdn_short_conv_bwd(dconv, xc, w, b, cu_seqlens=c, conv_state=st, dconv_state_out=dst, **o),
                     dict(dx=e(T, dim, dt=dtype), dweight=e(dim, 4), dbias=e(dim), dconv_state=e(n, dim, 3))),
        "ssm_fwd": (lambda o: gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=c, initial_state=S0, **o),
                    dict(out=e(T, H, P, dt=dtype), final_state=e(n, H, P, N))),
        "ssm_step": (lambda o: (o["state"].copy_(pool), gdn.gdn_ssm_step(
            *(step[k] for k in ("x", "B", "C", "a")), s["A_log"], o["state"], dt_bias=s["dt_bias"], D=s["D"],
            state_indices=idx, out=o["out"])), dict(out=e(3, 2, H, P, dt=dtype), state=e(9, H, P, N))),
        "ssm_bwd": (lambda o: gdn.gdn_ssm_chunk_bwd(dout, **s, cu_seqlens=c, initial_state=S0, dfinal_state=dlast, **o),
                    dict(dx=e(T, H, P, dt=dtype), dB=e(T, G, N, dt=dtype), dC=e(T, G, N, dt=dtype), da=e(T, H), dA_log=e(H),
                         ddt_bias=e(H), dD=e(H), dinitial_state=e(n, H, P, N))),
        "qk_fwd": (lambda o: gdn.gdn_qk_norm_rope(q, k, table, positions=pos, q_weight=qw[0], k_weight=qw[1], **o),
                   dict(q_out=e(T, 3, d, dt=dtype), k_out=e(T, 2, d, dt=dtype))),
        "qk_bwd": (lambda o: gdn.gdn_qk_norm_rope_bwd(do, dk, q, k, table, positions=pos, q_weight=qw[0], k_weight=qw[1], **o),
                   dict(dq=e(T, 3, d, dt=dtype), dk=e(T, 2, d, dt=dtype), dq_weight=e(d), dk_weight=e(d))),
    }


NAMES = ("conv_fwd", "conv_step", "conv_bwd", "ssm_fwd", "ssm_step", "ssm_bwd", "qk_fwd", "qk_bwd")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("name", NAMES)
def test_writes_stay_inside_the_outputs(name, dtype):
    call, outs = all_calls(dtype)[name]
    call(outs)
    ref = {k: v.clone() for k, v in outs.items()}
    guarded = {}
    for k, v in outs.items():
        buf = torch.full((v.numel() + 128,), 3.5, dtype=v.dtype, device="cuda")
        guarded[k] = (buf, buf[64:64 + v.numel()].view(v.shape))
        guarded[k][1].zero_()
    call({k: v for k, (_, v) in guarded.items()})
    for k, (buf, view) in guarded.items():
        assert torch.equal(view, ref[k]), k
        assert bool((buf[:64] == 3.5).all()) and bool((buf[-64:] == 3.5).all()), k


@pytest.mark.parametrize("name,size", [("conv_bwd", "gdn_short_conv_bwd_workspace_size"), ("ssm_fwd", "gdn_ssm_chunk_fwd_workspace_size"),
                                       ("ssm_bwd", "gdn_ssm_chunk_bwd_workspace_size"), ("qk_bwd", "gdn_qk_norm_rope_bwd_workspace_size")])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_workspaces_hold_nothing_that_is_read_before_it_is_written(name, size, dtype):
    call, outs = all_calls(dtype)[name]
    call(outs)
    ref = {k: v.clone() for k, v in outs.items()}
    L = gdn.lib()
    T, dt = 2 + 165 + 6, int(dtype == BF)
    need = {"conv_bwd": (5, T, 512), "ssm_fwd": (5, T, 4, 2, 64, 128, dt), "ssm_bwd": (5, T, 4, 2, 64, 128, dt),
            "qk_bwd": (T, 3, 2, 64)}[name]
    bytes_ = getattr(L, size)(*need)
    buf = torch.full((bytes_ + 512,), 255, dtype=torch.uint8, device="cuda")   # NaN in every type
    start = (-buf.data_ptr()) % 256
    ws = buf[start:start + bytes_]
    call({**{k: v.zero_() for k, v in outs.items()}, "workspace": ws})
    for k, v in outs.items():
        assert torch.equal(v, ref[k]), k
    assert bool((buf[:start] == 255).all()) and bool((buf[start + bytes_:] == 255).all())
    if bytes_:
        with pytest.raises(gdn.GdnError):
            call({**outs, "workspace": ws[:bytes_ - 256] if bytes_ > 256 else ws[:0]})


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name):
    call, outs = all_calls(BF)[name]
    call(outs)
    ref = {k: v.clone() for k, v in outs.items()}
    for v in outs.values():
        v.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs)
    torch.cuda.current_stream().wait_stream(side)
    for k, v in outs.items():
        assert torch.equal(v, ref[k]), k


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    """A captured call, replayed twice, beside eager calls of other sizes: the same bits."""
    call, outs = all_calls(BF)[name]
    call(outs)
    ref = {k: v.clone() for k, v in outs.items()}
    other, other_outs = all_calls(BF, seed=7, lengths=(200, 33))[name]
    other(other_outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs)
    for _ in range(2):
        for v in outs.values():
            v.zero_()
        graph.replay()
        other(other_outs)
        torch.cuda.synchronize()
        for k, v in outs.items():
            assert torch.equal(v, ref[k]), k


def test_a_given_stream_is_used():
    _, _, s, S0, _ = scan_inputs([100], 0, 2, 1, 64, 64, BF, True, True, seed=3)
    ref, last = gdn.gdn_ssm_chunk_fwd(**s, initial_state=S0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, last2 = gdn.gdn_ssm_chunk_fwd(**s, initial_state=S0, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(last, last2)


def test_more_sequences_than_a_block_has_threads():
    lengths = [(i * 7) % 5 for i in range(700)]
    offs, T, s, S0, r = scan_inputs(lengths, 2, 1, 1, 64, 64, F32, False, True, seed=17)
    S0 = dev(r(700, 1, 64, 64))
    got, last = gdn.gdn_ssm_chunk_fwd(**s, cu_seqlens=cu(offs), initial_state=S0)
    (ref, ref_last), (terms, terms_last) = scan_reference(s, offs, S0)
    check("out", got[:offs[-1]], ref[:offs[-1]], terms[:offs[-1]])
    check("state", last, ref_last, terms_last)
    w, st = dev(r(64, 4)), dev(r(700, 64, 3))
    x = s["x"][:, 0]
    out, h = gdn.gdn_short_conv_fwd(x, w, cu_seqlens=cu(offs), conv_state=st)
    ref, _, ref_h = _layer.conv(wide(x), wide(w), None, offs, wide(st))
    terms = _layer.conv(wide(x).abs(), wide(w).abs(), None, offs, wide(st).abs(), False)[0]
    check("conv", out[:offs[-1]], ref[:offs[-1]], 2 * terms[:offs[-1]])
    assert torch.equal(h.cpu().to(F64), ref_h)


# ---- a layer ---------------------------------------------------------------------------------------

def test_a_layer_of_prompts_tokens_and_gradients():
    """Convolution, norm and rotation of C and B, scan, gated norm: a prompt in one piece equals the same prompt cut into
    a prefill and single tokens, and its gradients equal differences of the 64-bit layer."""
    H, G, P, N, T, n = 4, 1, 64, 64, 90, 2
    r = draw(51)
    dim = H * P + 2 * G * N
    mixed, z = dev(r(n * T, dim)), dev(r(n * T, H, P))
    w, b, A_log, bias, D = dev(r(dim, 4, scale=0.5)), dev(r(dim, scale=0.1)), dev(r(H, scale=0.3)), dev(r(H) - 2), dev(r(H))
    a, cw, bw = dev(r(n * T, H)), dev(1 + 0.1 * r(N)), dev(1 + 0.1 * r(N))
    ang = torch.arange(T, dtype=F64)[:, None] * 10000.0 ** (-torch.arange(0, N, 2, dtype=F64) / N)
    table = dev(torch.cat([ang.cos(), ang.sin()], -1).float())
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(n)

    def parts(c):
        x, B, C = c.split([H * P, G * N, G * N], -1)
        return x.unflatten(-1, (H, P)), B.unflatten(-1, (G, N)), C.unflatten(-1, (G, N))

    def forward(mixed, a, z, pos, conv_state, state):
        c, conv_state = gdn.gdn_short_conv_fwd(mixed, w, b, num_seqs=n, conv_state=conv_state)
        x, B, C = parts(c)
        C, B = gdn.gdn_qk_norm_rope(C, B, table, positions=pos, q_weight=cw, k_weight=bw)
        y, state = gdn.gdn_ssm_chunk_fwd(x, B, C, a, A_log, dt_bias=bias, D=D, num_seqs=n, initial_state=state)
        return gdn.gdn_gate_rmsnorm_silu(y, z), conv_state, state, (c, x, B, C, y)

    out, conv_state, state, (c, x, B, C, y) = forward(mixed, a, z, pos, None, None)
    cut = T - 3
    head = lambda t: t.unflatten(0, (n, T))[:, :cut].flatten(0, 1).contiguous()  # noqa: E731
    o1, cs, S, _ = forward(head(mixed), head(a), head(z), head(pos), None, None)
    outs = [o1.unflatten(0, (n, cut))]
    for t in range(cut, T):
        at = lambda v: v.unflatten(0, (n, T))[:, t].contiguous()  # noqa: E731
        ct = gdn.gdn_short_conv_step(at(mixed), w, cs, b)
        xt, Bt, Ct = parts(ct)
        Ct, Bt = gdn.gdn_qk_norm_rope(Ct, Bt, table, positions=at(pos), q_weight=cw, k_weight=bw)
        yt = gdn.gdn_ssm_step(xt, Bt, Ct, at(a), A_log, S, dt_bias=bias, D=D)
        outs.append(gdn.gdn_gate_rmsnorm_silu(yt, at(z))[:, None])
    whole = out.unflatten(0, (n, T))
    pieces = torch.cat(outs, 1)
    assert (pieces - whole).norm() <= 1e-5 * whole.norm()     # fp32 throughout, other orders of the sums
    assert torch.equal(cs, conv_state) and (S - state).norm() <= 1e-5 * state.norm()

    dout = dev(r(n * T, H, P))
    dy, dz, _ = gdn.gdn_gate_rmsnorm_silu_bwd(dout, y, z)
    dx, dB, dC, da, dA_log, dbias, dD, _ = gdn.gdn_ssm_chunk_bwd(dy, x, B, C, a, A_log, dt_bias=bias, D=D, num_seqs=n)
    _, B0, C0 = parts(c)
    dC, dB, dcw, dbw = gdn.gdn_qk_norm_rope_bwd(dC, dB, C0, B0, table, positions=pos, q_weight=cw, k_weight=bw)
    dc = torch.cat([dx.flatten(1), dB.flatten(1), dC.flatten(1)], 1)
    dmixed, dw, db, _ = gdn.gdn_short_conv_bwd(dc, mixed, w, b, num_seqs=n)

    offs, tab = [0, T, 2 * T], wide(table)[pos.cpu().long()]
    cos, sin = tab[:, :N // 2], tab[:, N // 2:]

    def layer64(mixed, w, b, a, A_log, bias, D, cw, bw, z):
        c = _layer.conv(mixed, w, b, offs, None)[0]
        x, B, C = parts(c)
        C = _layer.qk(C, cw, cos, sin, False, 1e-6, False)[0]
        B = _layer.qk(B, bw, cos, sin, False, 1e-6, False)[0]
        _, dt, alpha = _layer.gates(a, A_log, bias)
        y = _layer.ssm(x, B, C, dt, alpha, D, offs, None)[0]
        return (y * _layer.norm_factor(y, False, 1e-6) * _layer.silu(z) * wide(dout)).sum()

    args = [wide(t) for t in (mixed, w, b, a, A_log, bias, D, cw, bw, z)]
    grads = [wide(t) for t in (dmixed, dw, db, da, dA_log, dbias, dD, dcw, dbw, dz)]
    gen = torch.Generator().manual_seed(6)
    for i, g in enumerate(grads):
        u = torch.randn(args[i].shape, generator=gen, dtype=F64)
        ends = [layer64(*args[:i], args[i] + s * 1e-6 * u, *args[i + 1:]) for s in (1, -1)]
        num = (ends[0] - ends[1]) / 2e-6
        assert abs(num - (g * u).sum()) <= 1e-4 * (g * u).norm(), i
