"""The training operators on the GPU, against fp64 forms on the same inputs (tests/_train.py)."""
import ctypes

import pytest
import torch

import gated_deltanet_recurrence_gb300 as gdn
from tests import _train
from tests._train import decay_grads, delta_grads, delta_inputs, norm_grads, rel_l2, tol_of

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state")


def dev(x):
    return x.cuda() if isinstance(x, torch.Tensor) else x


def chunk_bwd(inp, **kw):
    cu = torch.tensor(inp["cu"], dtype=torch.int32, device="cuda")
    args = [dev(inp[x]) for x in ("q", "k", "v", "g", "beta", "dout")]
    got = gdn.gdn_chunk_bwd(*args, cu_seqlens=cu, initial_state=dev(inp["initial_state"]),
                            dfinal_state=dev(inp["dfinal_state"]), **kw)
    assert gdn.gdn_get_device_error() == 0
    return dict(zip(NAMES, got))


def check_chunk(inp, got, use_l2=True, scale=None):
    ref = delta_grads(inp, use_l2=use_l2, scale=scale)
    lo, hi = inp["cu"][0], inp["cu"][-1]
    for name in NAMES:
        if got[name] is None:
            continue
        x, r = got[name], ref[name]
        if name != "dinitial_state":
            x, r = x[lo:hi], r[lo:hi]
        assert rel_l2(x, r) <= tol_of(x), (name, rel_l2(x, r))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,H,Hk,carried", [
    ([1], 1, 1, False),
    ([1, 2, 0, 3], 2, 2, True),
    ([63, 64, 65], 2, 1, True),
    ([200], 3, 3, False),
    ([130, 0, 257, 5], 4, 2, True),
    ([321], 6, 2, False),
])
def test_chunk_bwd(lengths, H, Hk, carried, d, dtype):
    inp = delta_inputs(lengths, H, Hk, d, dtype, seed=sum(lengths) + d, carried=carried)
    check_chunk(inp, chunk_bwd(inp))


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F32)])
@pytest.mark.parametrize("a_mean", [-4.0, 3.0])
def test_chunk_bwd_slow_and_fast_decay(d, dtype, a_mean):
    inp = delta_inputs([300, 77], 2, 2, d, dtype, seed=7, a_mean=a_mean)
    check_chunk(inp, chunk_bwd(inp))


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F32)])
def test_chunk_bwd_without_normalisation(d, dtype):
    inp = delta_inputs([150, 20], 2, 1, d, dtype, seed=9)
    for x in ("q", "k"):
        inp[x] = (inp[x].float() * d ** -0.5).to(dtype)
    check_chunk(inp, chunk_bwd(inp, use_qk_l2norm=False, scale=0.7), use_l2=False, scale=0.7)


def _exponents(pattern, lengths):
    """Powers of two of a batch's tokens, spread over 2^30 in every chunk of 64."""
    gen = torch.Generator().manual_seed(len(pattern))
    out = []
    for n in lengths:
        t = torch.arange(n) % 64
        out.append({"first": torch.where(t == 0, 30, 0), "falling": 15 - t // 2, "rising": t // 2 - 15,
                    "mixed": torch.randint(-15, 16, (n,), generator=gen)}[pattern])
    return torch.cat(out).double()


def check_tokens(inp, got, **kw):
    """Each token's and head's gradients by themselves: off by their own rounding and at most ten standard
    deviations of what the roundings of their terms leave.  (Against the gradient itself no such bound holds, in
    fp32 neither: with a_mean = 1 and "mixed" below, token 147 of head 0 has dR = 0.0012 from terms of 0.12,
    0.054, 0.041, 0.024, ..., and half a step of 22 bits of the first alone is 0.12 * 2^-23 / 0.0012 = 1.2e-5.)"""
    ref, size = delta_grads(inp, **kw), _train.delta_errors(inp, device="cuda", **kw)
    lo, hi = inp["cu"][0], inp["cu"][-1]
    for name, sigma in size.items():
        x, r = (y.detach().cpu().double()[lo:hi] for y in (got[name], ref[name]))
        assert torch.isfinite(x).all(), name
        half = 2.0 ** -8 if got[name].dtype == BF16 else 2.0 ** -24
        off, most = (x - r).abs(), r.abs() * half
        if x.dim() == 3:
            off, most = off.norm(dim=-1), most.norm(dim=-1)
        most = most + 10 * sigma[lo:hi]
        assert (off <= most).all(), (name, float((off / most).max()), int((off / most).argmax()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("a_mean", [-4.0, 1.0])
@pytest.mark.parametrize("pattern", ["first", "falling", "rising", "mixed"])
def test_chunk_bwd_tokens_whose_gradients_are_far_apart(d, dtype, a_mean, pattern):
    """The output's gradient 2^30 apart between tokens of a chunk: a token's results keep their accuracy beside
    the others' (those behind a token with a large one depend on the small ones alone)."""
    lengths = [64, 100]
    inp = delta_inputs(lengths, 4, 2, d, dtype, seed=61, a_mean=a_mean, carried=False)
    e = _exponents(pattern, lengths)
    inp["dout"] = (inp["dout"].double() * 2.0 ** e[:, None, None]).to(dtype)
    check_tokens(inp, chunk_bwd(inp))


@pytest.mark.parametrize("d,dtype", [(64, F32), (64, BF16), (128, F32), (128, BF16)])
@pytest.mark.parametrize("a_mean", [-4.0, 1.0])
@pytest.mark.parametrize("pattern", ["first", "falling", "mixed"])
def test_chunk_bwd_queries_and_keys_far_apart_without_normalisation(d, dtype, a_mean, pattern):
    """Rows of q and of k 2^30 apart where no norm takes their sizes off: small ones keep their accuracy."""
    lengths = [64, 100]
    inp = delta_inputs(lengths, 4, 2, d, dtype, seed=65, a_mean=a_mean)
    e = _exponents(pattern, lengths)
    for x, most in (("q", 0.0), ("k", float(e.max()))):  # keys of length one at most
        inp[x] = (inp[x].double() * d ** -0.5 * 2.0 ** (e - most)[:, None, None]).to(dtype)
    check_tokens(inp, chunk_bwd(inp, use_qk_l2norm=False, scale=0.5), use_l2=False, scale=0.5)


@pytest.mark.parametrize("d,dtype", [(64, F32), (64, BF16), (128, F32), (128, BF16)])
@pytest.mark.parametrize("a_mean", [-4.0, 1.0])
@pytest.mark.parametrize("pattern", ["rising", "mixed"])
def test_chunk_bwd_tokens_whose_values_are_far_apart(d, dtype, a_mean, pattern):
    """v 2^30 apart: a token's results depend on its own and earlier tokens' v and keep their accuracy beside
    later ones."""
    lengths = [64, 100]
    inp = delta_inputs(lengths, 4, 2, d, dtype, seed=63, a_mean=a_mean)
    e = _exponents(pattern, lengths)
    inp["v"] = (inp["v"].double() * 2.0 ** e[:, None, None]).to(dtype)
    inp["initial_state"] *= 2.0 ** -15
    check_tokens(inp, chunk_bwd(inp))


def test_chunk_bwd_first_token_has_no_decay_gradient():
    inp = delta_inputs([1, 1], 2, 2, 128, BF16, seed=3, carried=False)
    assert torch.count_nonzero(chunk_bwd(inp)["dg"]) == 0


@pytest.mark.parametrize("Hk", [1, 3])
def test_chunk_bwd_leaves_rows_outside_the_sequences(Hk):
    inp = delta_inputs([70, 0, 9], 3, Hk, 64, BF16, seed=5, lead=4, behind=6)
    T = inp["q"].shape[0]
    outs = {x: torch.full_like(dev(inp[x[1:]]), 3.5) for x in ("dq", "dk", "dv", "dg", "dbeta")}
    got = chunk_bwd(inp, **outs)
    check_chunk(inp, got)
    for x in outs:
        assert (got[x][:4] == 3.5).all() and (got[x][T - 6:] == 3.5).all(), x


@pytest.mark.parametrize("dtype,d,Hk", [(BF16, 64, 1), (F32, 128, 3)])
def test_chunk_bwd_allocated_rows_outside_the_sequences_are_zero(dtype, d, Hk):
    """Tokens of no sequence (a padded batch) have zero gradients in what the binding allocates, also where the
    memory held something else before, and on another stream; given outputs keep their rows."""
    inp = delta_inputs([70, 0, 9], 3, Hk, d, dtype, seed=5, lead=4, behind=60)
    T = inp["q"].shape[0]
    shapes = [tuple(inp[x].shape) for x in ("q", "k", "v", "g", "beta")]
    for stream in (None, torch.cuda.Stream()):
        with torch.cuda.stream(stream):  # None: as it is
            before = [torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in zip(shapes, (dtype,) * 3 + (F32,) * 2)]
            torch.cuda.synchronize()
            del before
        dv = torch.full(shapes[2], 3.5, dtype=dtype, device="cuda")
        torch.cuda.synchronize()
        got = chunk_bwd(inp, stream=stream, dv=dv)
        torch.cuda.synchronize()
        check_chunk(inp, got)
        for x in ("dq", "dk", "dg", "dbeta"):
            assert (got[x][:4] == 0).all() and (got[x][T - 60:] == 0).all(), x
        assert (dv[:4] == 3.5).all() and (dv[T - 60:] == 3.5).all()


def test_chunk_bwd_without_any_token_in_a_sequence():
    inp = delta_inputs([0, 0], 2, 1, 64, F32, seed=5, lead=3, behind=2)
    del inp["cu"][:]
    inp["cu"] += [3, 3, 3]
    nan = [torch.full((5, 2, 64), float("nan"), device="cuda") for _ in range(8)]
    del nan
    got = chunk_bwd(inp)
    assert all(torch.count_nonzero(got[x]) == 0 for x in NAMES[:5])
    assert torch.equal(got["dinitial_state"].cpu(), inp["dfinal_state"])


def test_chunk_bwd_fp32_dout_of_bf16_inputs_and_equal_lengths():
    inp = delta_inputs([96, 96], 2, 2, 128, BF16, seed=6)
    inp["dout"] = torch.randn(192, 2, 128, generator=torch.Generator().manual_seed(1))
    args = [dev(inp[x]) for x in ("q", "k", "v", "g", "beta", "dout")]
    got = gdn.gdn_chunk_bwd(*args, num_seqs=2, initial_state=dev(inp["initial_state"]),
                            dfinal_state=dev(inp["dfinal_state"]))
    check_chunk(inp, dict(zip(NAMES, got)))


@pytest.mark.parametrize("num,length,H,Hk,d,dtype", [
    (7, 100, 15, 5, 64, BF16), (3, 129, 14, 2, 128, BF16), (5, 64, 11, 11, 64, F32), (9, 1, 7, 1, 128, F32), (2, 700, 13, 1, 128, BF16)])
def test_chunk_bwd_equal_lengths_of_odd_counts(num, length, H, Hk, d, dtype):
    """Blocks find their head, group and sequence by division: counts that are no powers of two, and more
    blocks than fit the device at once."""
    inp = delta_inputs([length] * num, H, Hk, d, dtype, seed=num + H)
    args = [dev(inp[x]) for x in ("q", "k", "v", "g", "beta", "dout")]
    got = gdn.gdn_chunk_bwd(*args, num_seqs=num, initial_state=dev(inp["initial_state"]),
                            dfinal_state=dev(inp["dfinal_state"]))
    assert gdn.gdn_get_device_error() == 0
    check_chunk(inp, dict(zip(NAMES, got)))
    packed = chunk_bwd(inp)
    for x, y in zip(NAMES, got):
        assert torch.equal(packed[x], y), x


@pytest.mark.parametrize("lengths,H,Hk,d,dtype", [([2300], 1, 1, 128, BF16), ([1500, 40], 2, 1, 64, F32),
                                                  ([1300], 1, 1, 128, F32)])
def test_chunk_bwd_long_chains(lengths, H, Hk, d, dtype):
    """Tens of chunks in a row: the scan's warps run far ahead of one another, and every chunk's states, U and E
    still come from that chunk.  The same call gives the same bits."""
    inp = delta_inputs(lengths, H, Hk, d, dtype, seed=sum(lengths), a_mean=-4.0)
    got = chunk_bwd(inp)
    check_chunk(inp, got)
    for _ in range(20):
        again = chunk_bwd(inp)
        assert all(torch.equal(got[x], again[x]) for x in NAMES)


def test_chunk_bwd_is_reproducible_and_aliases_the_state_gradient():
    inp = delta_inputs([200, 33], 4, 2, 128, BF16, seed=8)
    one, two = chunk_bwd(inp), None
    dS = dev(inp["dfinal_state"]).clone()
    cu = torch.tensor(inp["cu"], dtype=torch.int32, device="cuda")
    args = [dev(inp[x]) for x in ("q", "k", "v", "g", "beta", "dout")]
    two = dict(zip(NAMES, gdn.gdn_chunk_bwd(*args, cu_seqlens=cu, initial_state=dev(inp["initial_state"]),
                                            dfinal_state=dS, dinitial_state=dS)))
    for x in NAMES:
        assert torch.equal(one[x], two[x]), x


def test_chunk_bwd_malformed_cu_seqlens_writes_nothing():
    inp = delta_inputs([64, 64], 2, 1, 64, F32, seed=4)
    outs = {x: torch.full_like(dev(inp[x[1:]]), 3.5) for x in ("dq", "dk", "dv", "dg", "dbeta")}
    outs["dinitial_state"] = torch.full_like(dev(inp["initial_state"]), 3.5)
    args = [dev(inp[x]) for x in ("q", "k", "v", "g", "beta", "dout")]
    for cu in ([0, 100, 64], [0, 64, 129], [-1, 64, 128]):
        gdn.gdn_chunk_bwd(*args, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                          initial_state=dev(inp["initial_state"]), dfinal_state=dev(inp["dfinal_state"]), **outs)
        assert gdn.gdn_get_device_error() == -3
        assert gdn.gdn_get_device_error() == 0
        assert all((x == 3.5).all() for x in outs.values())


def test_chunk_bwd_empty_batch_passes_the_state_gradient_through():
    inp = delta_inputs([0, 0], 2, 2, 64, F32, seed=2)
    got = chunk_bwd(inp)
    assert torch.equal(got["dinitial_state"].cpu(), inp["dfinal_state"])
    assert got["dq"].numel() == 0


@pytest.mark.parametrize("reset", [-float("inf"), -3e38, -200.0])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, F32)])
def test_chunk_bwd_decay_to_zero(d, dtype, reset):
    """Tokens that forget everything (documents packed into one sequence): nothing passes them, and the
    tokens behind them keep their own decays."""
    inp = delta_inputs([180], 2, 2, d, dtype, seed=17)
    for t in (0, 30, 31, 64, 130):
        inp["g"][t] = reset
    got = chunk_bwd(inp)
    check_chunk(inp, got)
    assert torch.count_nonzero(got["dinitial_state"]) == 0
    assert torch.count_nonzero(got["dg"][[0, 30, 31, 64, 130]]) == 0


def test_chunk_bwd_many_sequences():
    """More sequences than a block looks over by itself."""
    gen = torch.Generator().manual_seed(2)
    lengths = torch.randint(0, 3, (1500,), generator=gen).tolist()
    lengths[700] = 130
    inp = delta_inputs(lengths, 2, 1, 64, F32, seed=3)
    check_chunk(inp, chunk_bwd(inp))
    inp["cu"][900] += 5
    inp["cu"][901] = inp["cu"][900] - 1
    outs = {x: torch.full_like(dev(inp[x[1:]]), 3.5) for x in ("dq", "dk", "dv", "dg", "dbeta")}
    args = [dev(inp[x]) for x in ("q", "k", "v", "g", "beta", "dout")]
    gdn.gdn_chunk_bwd(*args, cu_seqlens=torch.tensor(inp["cu"], dtype=torch.int32, device="cuda"), **outs)
    assert gdn.gdn_get_device_error() == -3
    assert all((x == 3.5).all() for x in outs.values())


def test_chunk_bwd_degenerate_values():
    """Zero queries and keys, no update (beta = 0), full overwrite without decay."""
    for mode in ("zero", "beta0", "full"):
        inp = delta_inputs([100, 30], 2, 2, 128, BF16, seed=21)
        if mode == "zero":
            inp["q"][::5] = 0
            inp["k"][::7] = 0
            inp["dout"][::3] = 0
        elif mode == "beta0":
            inp["beta"].zero_()
        else:
            inp["beta"].fill_(1.0)
            inp["g"].zero_()
        check_chunk(inp, chunk_bwd(inp))


@pytest.mark.parametrize("big,small", [(2.0 ** 60, 2.0 ** -70), (2.0 ** -50, 2.0 ** 40)])
def test_chunk_bwd_scales_with_its_inputs(big, small):
    """Values (and the output's gradient) far from one: v and the states times a power of two, dout and
    dfinal_state times another, scale every output by exact powers of two."""
    inp = delta_inputs([150, 7], 2, 1, 128, BF16, seed=23)
    one = chunk_bwd(inp)
    far = dict(inp, v=inp["v"] * big, initial_state=inp["initial_state"] * big, dout=inp["dout"] * small,
               dfinal_state=inp["dfinal_state"] * small)
    got = chunk_bwd(far)
    for name, f in (("dq", big * small), ("dk", big * small), ("dg", big * small), ("dbeta", big * small),
                    ("dv", small), ("dinitial_state", small)):
        assert torch.equal(got[name], one[name] * f), name


def _streams_and_graph(call):
    """The call's result eagerly, on a side stream beside another call, and from a replayed graph."""
    eager = [x for x in call() if x is not None]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = call(stream=side)
    b = call()
    c = call(stream=side.cuda_stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = call()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for other in (a, b, c, g):
        for x, y in zip(eager, [x for x in other if x is not None]):
            assert torch.equal(x, y)


def test_calls_on_streams_and_in_graphs():
    inp = delta_inputs([200, 0, 70, 33], 4, 2, 128, BF16, seed=41)
    cu = torch.tensor(inp["cu"], dtype=torch.int32, device="cuda")
    args = [dev(inp[x]) for x in ("q", "k", "v", "g", "beta", "dout")]
    S0, dS = dev(inp["initial_state"]), dev(inp["dfinal_state"])
    _streams_and_graph(lambda **kw: gdn.gdn_chunk_bwd(*args, cu_seqlens=cu, initial_state=S0, dfinal_state=dS, **kw))
    x = _norm_inputs(300, 4, 64, BF16, seed=2)
    y, z, w, b, do = (dev(x[k]) for k in ("y", "z", "w", "b", "dout"))
    _streams_and_graph(lambda **kw: gdn.gdn_gate_groupnorm_silu_bwd(do, y, z, w, b, **kw))
    _streams_and_graph(lambda **kw: gdn.gdn_gate_rmsnorm_silu_bwd(do, y, z, w[0].contiguous(), **kw))
    _streams_and_graph(lambda **kw: (gdn.gdn_gate_groupnorm_silu(y, z, w, b, **kw),))
    a = torch.randn(777, 8, device="cuda")
    _streams_and_graph(lambda **kw: gdn.gdn_decay_from_logits_bwd(a, a[0].contiguous(), a[1].contiguous(), a, a, a, **kw))


# ---- norms -----------------------------------------------------------------------------------------

def _norm_inputs(rows, groups, size, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(y=(rn(rows, groups, size) * 0.7 + 0.3).to(dtype), z=rn(rows, groups, size) * 2,
                w=1 + 0.2 * rn(groups, size), b=0.3 * rn(groups, size), dout=rn(rows, groups, size).to(dtype))


@pytest.mark.parametrize("rows,heads,d,dtype,weight", [
    (1, 1, 32, F32, True), (3, 2, 64, BF16, False), (5, 3, 96, BF16, True), (1000, 16, 128, BF16, True),
    (2500, 1, 1024, F32, True), (7, 5, 128, F32, False), (301, 4, 512, BF16, True)])
def test_rmsnorm_bwd(rows, heads, d, dtype, weight):
    x = _norm_inputs(rows, heads, d, dtype, seed=rows + d)
    w = x["w"][0] if weight else None
    got = gdn.gdn_gate_rmsnorm_silu_bwd(dev(x["dout"]), dev(x["y"]), dev(x["z"]), dev(w))
    ref = norm_grads(x["dout"], x["y"], x["z"], w, None, 1e-6, True)
    for g, r, name in zip(got, ref, ("dy", "dz", "dw")):
        assert (g is None) == (r is None)
        if g is not None:
            assert rel_l2(g, r) <= tol_of(g), (name, rel_l2(g, r))


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("rows,groups,size,dtype", [
    (1, 1, 2, F32), (2, 3, 5, BF16), (4, 16, 64, F32), (1000, 16, 128, BF16), (333, 12, 80, F32),
    (65, 7, 41, BF16), (50, 2, 1023, F32), (19, 4, 1024, BF16), (3, 700, 4, F32), (9, 1500, 3, BF16)])
def test_groupnorm(rows, groups, size, dtype, affine, gated):
    x = _norm_inputs(rows, groups, size, dtype, seed=rows + size)
    z = x["z"] if gated else None
    w, b = (x["w"], x["b"]) if affine else (None, None)
    out = gdn.gdn_gate_groupnorm_silu(dev(x["y"]), dev(z), dev(w), dev(b))
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    ref = _train.norm_forward(*(f64(t) for t in (x["y"], z, w, b)), 1e-6, False)
    assert rel_l2(out, ref) <= tol_of(out), rel_l2(out, ref)
    got = gdn.gdn_gate_groupnorm_silu_bwd(dev(x["dout"]), dev(x["y"]), dev(z), dev(w), dev(b))
    for g, r, name in zip(got, norm_grads(x["dout"], x["y"], z, w, b, 1e-6, False), ("dy", "dz", "dw", "db")):
        assert (g is None) == (r is None), name
        if g is not None and not (size == 2 and name == "dy"):   # n = +-1 there: dy is what eps leaves
            assert rel_l2(g, r) <= tol_of(g), (name, rel_l2(g, r))


def test_groupnorm_of_constant_and_single_channel_groups():
    y = torch.full((6, 3, 40), 1.75)
    w, b = torch.randn(3, 40), torch.randn(3, 40)
    out = gdn.gdn_gate_groupnorm_silu(dev(y), None, dev(w), dev(b))
    assert rel_l2(out, (b * torch.sigmoid(b)).expand_as(y)) <= 2e-6   # n is 0 exactly
    one = gdn.gdn_gate_groupnorm_silu(dev(torch.randn(4, 9, 1)), None, None, dev(torch.ones(9, 1)))
    assert rel_l2(one, torch.full((4, 9, 1), 1.0) * torch.sigmoid(torch.tensor(1.0))) <= 2e-6


def test_norm_bwd_in_place_and_mixed_types():
    x = _norm_inputs(77, 4, 64, BF16, seed=1)
    y, z, dout = dev(x["y"]), dev(x["z"]), dev(x["dout"].float())
    ref = gdn.gdn_gate_rmsnorm_silu_bwd(dout, y, z)
    rr = norm_grads(x["dout"], x["y"], x["z"], None, None, 1e-6, True)
    assert rel_l2(ref[0], rr[0]) <= tol_of(ref[0]) and rel_l2(ref[1], rr[1]) <= tol_of(ref[1])
    y2, z2 = y.clone(), z.clone()
    gdn.gdn_gate_rmsnorm_silu_bwd(dout, y2, z2, dy=y2, dz=z2)
    assert torch.equal(y2, ref[0]) and torch.equal(z2, ref[1])
    w, b = dev(x["w"]), dev(x["b"])
    ref = gdn.gdn_gate_groupnorm_silu(y, z, w, b)
    y2 = y.clone()
    gdn.gdn_gate_groupnorm_silu(y2, z, w, b, out=y2)
    assert torch.equal(y2, ref)


def _off(x, ref, most):
    """The largest error of an element beside what it may be, `most` times its value."""
    ref = ref.double()
    return float(((x.detach().cpu().double() - ref).abs() / (ref.abs() * most)).max())


def test_small_gates_keep_their_relative_accuracy():
    """Gates far from zero: silu(z) and its slope are tiny on the negative side and each element is right by
    itself.  Per element: the exponential (2 + 1.16 |z|) 2^-23, 1 + e 2^-24, the division 2^-22, the norm's rsqrt
    and sum of squares 2^-22 each, and eight products and sums 2^-24 each."""
    x = _norm_inputs(64, 2, 128, F32, seed=15)
    gen = torch.Generator().manual_seed(16)
    z = (2 + 78 * torch.rand(64, 2, 128, generator=gen)) * torch.where(torch.rand(64, 2, 128, generator=gen) < 0.8, -1, 1)
    tol = 3 * 2.0 ** -22 + 9 * 2.0 ** -24 + (2 + 1.16 * z.double().abs()) * 2.0 ** -23
    y = torch.rand(64, 2, 128, generator=gen) + 0.5
    _, dz, _ = gdn.gdn_gate_rmsnorm_silu_bwd(dev(x["dout"]), dev(y), dev(z))
    assert _off(dz, norm_grads(x["dout"], y, z, None, None, 1e-6, True)[1], tol) <= 1
    one = torch.full((64, 2, 1), 1.0)  # a group of one channel: n = 0, m = bias
    out = gdn.gdn_gate_groupnorm_silu(dev(one), dev(z[..., :1].contiguous()), None, dev(torch.ones(2, 1)))
    assert _off(out, z[..., :1].double() * torch.sigmoid(z[..., :1].double()), tol[..., :1]) <= 1
    a, b, dg = (t.contiguous() for t in (z[:, 0], z[:, 1], x["dout"][:, 0]))
    A_log = torch.rand(128, generator=gen)
    got = gdn.gdn_decay_from_logits_bwd(dev(a), dev(A_log), None, dev(b), dev(dg), dev(dg))
    assert _off(got[0], decay_grads(a, A_log, None, b, dg, dg)[0], tol[:, 0]) <= 1
    bb = b.double()  # sigma(b) sigma(-b): 1 - sigma(80) is zero in 64 bits
    assert _off(got[3], dg.double() * torch.sigmoid(bb) * torch.sigmoid(-bb), tol[:, 1]) <= 1
    for v in (float("inf"), 1000.0):  # what the formulas give at the ends
        ends = torch.tensor([[v, -v]], device="cuda")
        da, _, _, db = gdn.gdn_decay_from_logits_bwd(ends, torch.zeros(2, device="cuda"), None, ends, *[torch.ones(1, 2, device="cuda")] * 2)
        assert da.tolist() == [[-1.0, 0.0]] and db.tolist() == [[0.0, 0.0]]
        out = gdn.gdn_gate_groupnorm_silu(dev(one[:1]), ends[..., None], None, dev(torch.ones(2, 1)))
        assert out[0, 0, 0] == v and (out[0, 1, 0].isnan() if v == float("inf") else out[0, 1, 0] == 0)


def test_norm_bwd_of_no_rows_gives_zero_sums():
    y = torch.empty(0, 3, 32, device="cuda")
    _, _, dw, db = gdn.gdn_gate_groupnorm_silu_bwd(y, y, y, torch.ones(3, 32, device="cuda"),
                                                   torch.ones(3, 32, device="cuda"))
    assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_norm_bwd_zero_eps():
    """Rows past the end take part in no sum even where eps = 0 makes an empty row's factor infinite."""
    x = _norm_inputs(3, 2, 64, F32, seed=12)
    got = gdn.gdn_gate_groupnorm_silu_bwd(dev(x["dout"]), dev(x["y"]), dev(x["z"]), dev(x["w"]), dev(x["b"]), eps=0.0)
    for g, r in zip(got, norm_grads(x["dout"], x["y"], x["z"], x["w"], x["b"], 0.0, False)):
        assert rel_l2(g, r) <= tol_of(g)


# ---- gate preparation --------------------------------------------------------------------------------

@pytest.mark.parametrize("T,H", [(1, 1), (7, 3), (513, 6), (4096, 32), (1000, 33), (20, 300), (3, 2052)])
@pytest.mark.parametrize("full", [True, False])
def test_decay_bwd(T, H, full):
    gen = torch.Generator().manual_seed(T + H)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    a, A_log, dg = rn(T, H) * 8, torch.rand(H, generator=gen) * 2, rn(T, H)
    dt, b, dbeta = (rn(H), rn(T, H) * 3, rn(T, H)) if full else (None, None, None)
    got = gdn.gdn_decay_from_logits_bwd(dev(a), dev(A_log), dev(dt), dev(b), dev(dg), dev(dbeta))
    for g, r, name in zip(got, decay_grads(a, A_log, dt, b, dg, dbeta), ("da", "dA_log", "ddt_bias", "db")):
        assert (g is None) == (r is None), name
        if g is not None:
            assert rel_l2(g, r) <= tol_of(g), (name, rel_l2(g, r))


def test_decay_bwd_of_no_tokens_gives_zero_sums():
    a = torch.empty(0, 5, device="cuda")
    _, dA, ddt, _ = gdn.gdn_decay_from_logits_bwd(a, torch.ones(5, device="cuda"), torch.ones(5, device="cuda"), a, a, a)
    assert torch.count_nonzero(dA) == 0 and torch.count_nonzero(ddt) == 0


def test_decay_bwd_in_place():
    a, dg, b, dbeta = (torch.randn(100, 7, device="cuda") for _ in range(4))
    A = torch.rand(7, device="cuda")
    ref = gdn.gdn_decay_from_logits_bwd(a, A, None, b, dg, dbeta)
    a2, b2 = a.clone(), b.clone()
    got = gdn.gdn_decay_from_logits_bwd(a2, A, None, b2, dg, dbeta, da=a2, db=b2)
    for x, y in zip(ref, got):
        assert (x is None and y is None) or torch.equal(x, y)


# ---- guard bands -----------------------------------------------------------------------------------------

GUARD = 64


def _guarded(shape, dtype):
    """A tensor of `shape` between two bands of GUARD sentinel elements; returns (tensor, whole buffer)."""
    n = 1
    for x in shape:
        n *= x
    buf = torch.full((GUARD + n + GUARD,), 7.0 if dtype != torch.uint8 else 7, dtype=dtype, device="cuda")
    return buf[GUARD:GUARD + n].view(shape), buf


def _intact(bufs):
    torch.cuda.synchronize()
    return all(bool((b[:GUARD] == 7).all()) and bool((b[-GUARD:] == 7).all()) for b in bufs)


def _workspace(need):
    """`need` bytes, 256-byte aligned, between two bands."""
    buf = torch.full((256 + need + GUARD,), 7, dtype=torch.uint8, device="cuda")
    return buf[256:256 + need], buf[256 - GUARD:]


@pytest.mark.parametrize("d,dtype,Hk", [(128, BF16, 2), (128, F32, 1), (64, BF16, 1), (64, F32, 2)])
def test_chunk_bwd_stays_inside_its_outputs(d, dtype, Hk):
    inp = delta_inputs([1, 0, 130, 64, 63], 2, Hk, d, dtype, seed=50)
    bufs, outs = [], {}
    for x in ("dq", "dk", "dv", "dg", "dbeta"):
        outs[x], b = _guarded(tuple(inp[x[1:]].shape), inp[x[1:]].dtype)
        bufs.append(b)
    outs["dinitial_state"], b = _guarded(tuple(inp["initial_state"].shape), F32)
    bufs.append(b)
    T = inp["q"].shape[0]
    ws, b = _workspace(gdn.lib().gdn_chunk_bwd_workspace_size(5, T, 2, Hk, d, d))
    bufs.append(b)
    check_chunk(inp, chunk_bwd(inp, workspace=ws, **outs))
    assert _intact(bufs)


@pytest.mark.parametrize("rows,groups,size,dtype", [(7, 3, 41, BF16), (1, 2, 64, F32), (300, 5, 128, BF16), (3, 400, 8, F32)])
def test_norms_and_gates_stay_inside_their_outputs(rows, groups, size, dtype):
    x = _norm_inputs(rows, groups, size, dtype, seed=4)
    y, z, w, b, do = (dev(x[k]) for k in ("y", "z", "w", "b", "dout"))
    shapes = dict(dy=(y.shape, dtype), dz=(y.shape, F32), dweight=(w.shape, F32), dbias=(w.shape, F32))
    outs = {k: _guarded(tuple(s), t) for k, (s, t) in shapes.items()}
    ws, band = _workspace(gdn.lib().gdn_gate_bwd_workspace_size(rows, groups, size))
    gdn.gdn_gate_groupnorm_silu_bwd(do, y, z, w, b, workspace=ws, **{k: v[0] for k, v in outs.items()})
    out, out_buf = _guarded(tuple(y.shape), dtype)
    gdn.gdn_gate_groupnorm_silu(y, z, w, b, out=out)
    H = groups * size
    a = torch.randn(rows, H, device="cuda")
    dec = [_guarded((rows, H), F32), _guarded((H,), F32), _guarded((H,), F32), _guarded((rows, H), F32)]
    ws2, band2 = _workspace(gdn.lib().gdn_decay_bwd_workspace_size(rows, H))
    gdn.gdn_decay_from_logits_bwd(a, a[0].contiguous(), a[0].contiguous(), a, a, a, *[t for t, _ in dec], workspace=ws2)
    assert _intact([v[1] for v in outs.values()] + [band, out_buf, band2] + [v for _, v in dec])


# ---- together ------------------------------------------------------------------------------------------

def test_training_step_together():
    """Forward and backward of a whole layer core from its logits, as a training step runs it, against
    fp64 autograd through the same chain."""
    lengths, H, Hk, d, dtype = [150, 41], 4, 2, 128, BF16
    inp = delta_inputs(lengths, H, Hk, d, dtype, seed=31, carried=False)
    gen = torch.Generator().manual_seed(32)
    T = sum(lengths)
    a, b, z = (torch.randn(T, *s, generator=gen) for s in ((H,), (H,), (H, d)))
    A_log, dt, w = torch.rand(H, generator=gen), torch.randn(H, generator=gen) * 0.3, 1 + 0.1 * torch.randn(d, generator=gen)
    do = torch.randn(T, H, d, generator=gen)
    cu = torch.tensor(inp["cu"], dtype=torch.int32, device="cuda")
    q, k, v, A, B, Z, AL, DT, Wt, DO = (dev(x) for x in (inp["q"], inp["k"], inp["v"], a, b, z, A_log, dt, w, do))
    g, beta = gdn.gdn_decay_from_logits(A, AL, DT, B)
    y, _ = gdn.gdn_chunk_fwd(q, k, v, g, beta, cu_seqlens=cu, out_dtype=F32)
    dy, dz, dw = gdn.gdn_gate_rmsnorm_silu_bwd(DO, y, Z, Wt)
    dq, dk, dv, dg, dbeta, _ = gdn.gdn_chunk_bwd(q, k, v, g, beta, dy, cu_seqlens=cu)
    da, dAL, ddt, db = gdn.gdn_decay_from_logits_bwd(A, AL, DT, B, dg, dbeta)
    assert gdn.gdn_get_device_error() == 0
    names = ("q", "k", "v", "a", "b", "z", "A_log", "dt", "w")
    leaves = [x.double().clone().requires_grad_() for x in (inp["q"], inp["k"], inp["v"], a, b, z, A_log, dt, w)]
    lq, lk, lv, la, lb, lz, lA, ldt, lw = leaves
    yy, _ = _train.delta_forward(lq, lk, lv, -lA.exp() * torch.nn.functional.softplus(la + ldt), torch.sigmoid(lb),
                                 inp["cu"], torch.zeros(2, H, d, d, dtype=torch.float64), d ** -0.5, True)
    out = _train.norm_forward(yy, lz, lw, None, 1e-6, True)
    ref = torch.autograd.grad(out, leaves, do.double())
    # y comes from the bf16 tensor-core forward, which is within 1e-2 of the exact one; the norm and its
    # gradient pass that on with a factor of about two
    for name, x, r in zip(names, (dq, dk, dv, da, db, dz, dAL, ddt, dw), ref):
        assert rel_l2(x, r) <= 2e-2 + tol_of(x), (name, rel_l2(x, r))


# ---- sums over rows: one cluster, or a grid and a second kernel -----------------------------------------

@pytest.mark.parametrize("rows,groups,size", [
    (2, 1, 64), (33, 1, 64), (256, 1, 64), (257, 1, 64), (512, 1, 64), (513, 1, 64), (100, 3, 40), (32, 1, 1024), (33, 1, 1024),
    (20, 6, 680), (20, 7, 680), (1, 9, 1)])
@pytest.mark.parametrize("which", ["both", "weight", "bias"])
def test_sums_over_rows_on_either_side_of_a_cluster(rows, groups, size, which):
    x = _norm_inputs(rows, groups, size, F32, seed=rows)
    w = x["w"] if which != "bias" else None
    b = x["b"] if which != "weight" else None
    args = [dev(t) for t in (x["dout"], x["y"], x["z"], w, b)]
    got = gdn.gdn_gate_groupnorm_silu_bwd(*args)
    for g, r, name in zip(got, norm_grads(x["dout"], x["y"], x["z"], w, b, 1e-6, False), ("dy", "dz", "dw", "db")):
        assert (g is None) == (r is None), name
        if g is not None and not (size == 1 and name == "dy"):   # n = 0 there: dy is a rounding
            assert rel_l2(g, r) <= tol_of(g), (name, rel_l2(g, r))
    again = gdn.gdn_gate_groupnorm_silu_bwd(*args)
    assert all(a is None and g is None or torch.equal(a, g) for a, g in zip(again, got))


@pytest.mark.parametrize("T,H", [(2, 1), (255, 5), (256, 7), (1170, 7), (1171, 7), (8191, 1), (8193, 1), (31, 1024), (33, 1024),
                                 (20, 255), (1, 257)])
@pytest.mark.parametrize("which", ["both", "A_log", "dt_bias"])
def test_decay_sums_on_either_side_of_a_cluster(T, H, which):
    gen = torch.Generator().manual_seed(T + H)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    a, A_log, dt, b, dg, dbeta = rn(T, H), torch.rand(H, generator=gen), rn(H), rn(T, H), rn(T, H), rn(T, H)
    outs = [torch.full((T, H), 5.0, device="cuda"), *(torch.full((H,), 5.0, device="cuda") for _ in range(2)),
            torch.full((T, H), 5.0, device="cuda")]
    ws = torch.empty(gdn.lib().gdn_decay_bwd_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    ins = [dev(t) for t in (a, A_log, dt, b, dg, dbeta)]
    given = [t.data_ptr() for t in ins + outs]
    if which != "both":
        given[8 if which == "A_log" else 7] = None
    rc = gdn.lib().gdn_decay_from_logits_bwd(*given, T, H, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    for i, (g, r) in enumerate(zip(outs, decay_grads(a, A_log, dt, b, dg, dbeta))):
        if given[6 + i] is None:
            assert bool((g == 5).all())
        else:
            assert rel_l2(g, r) <= tol_of(g), (i, rel_l2(g, r))


@pytest.mark.parametrize("which", ["decay", "norm", "chunk"])
def test_a_launch_that_fails_leaves_no_error_to_the_next_call(which):
    """A launch into a stream whose capture has been broken off fails on the host; the call says so, and the next
    call on another stream is not told of it."""
    rt = next(r for r in (_cudart(n) for n in ("libcudart.so.13", "libcudart.so")) if r is not None)
    L, s = gdn.lib(), torch.cuda.Stream()
    x = torch.randn(40, 2, 64, device="cuda")
    c, st = torch.ones(2, 64, device="cuda"), torch.zeros(1, 2, 64, 64, device="cuda")
    outs, sums, ws = [torch.empty_like(x) for _ in range(6)], torch.empty(4, 128, device="cuda"), torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(ctypes.c_void_p(s.cuda_stream), 2) == 0
    assert rt.cudaStreamSynchronize(ctypes.c_void_p(s.cuda_stream)) != 0  # not allowed: the capture is broken off
    if which == "decay":
        rc = L.gdn_decay_from_logits_bwd(p(x), p(c), None, None, p(x), None, p(outs[0]), p(sums), None, None, 40, 128,
                                         p(ws), ws.numel(), s.cuda_stream)
    elif which == "norm":
        rc = L.gdn_gate_groupnorm_silu_bwd(p(x), 0, p(x), 0, None, p(c), None, 1e-6, p(outs[0]), None, p(sums), None, 40, 2,
                                           64, p(ws), ws.numel(), s.cuda_stream)
    else:
        rc = L.gdn_chunk_bwd(p(x), p(x), p(x), p(x), p(x), None, 1, 40, 2, 2, 64, 64, 0, 0, 0.0, 1, None, p(x), 0, None,
                             *(p(t) for t in outs[:5]), None, p(ws), ws.numel(), s.cuda_stream)
    graph = ctypes.c_void_p()
    assert rt.cudaStreamEndCapture(ctypes.c_void_p(s.cuda_stream), ctypes.byref(graph)) != 0
    rt.cudaGetLastError()
    assert rc == -5
    assert torch.isfinite(gdn.gdn_gate_groupnorm_silu(x)).all()


def _cudart(name):
    try:
        return ctypes.CDLL(name)
    except OSError:
        return None


def test_small_calls_on_two_streams_at_once():
    """Clusters of two calls in flight together keep their sums apart."""
    xs = [_norm_inputs(60, 2, 64, F32, seed=s) for s in (1, 2)]
    args = [[dev(x[k]) for k in ("dout", "y", "z", "w", "b")] for x in xs]
    want = [gdn.gdn_gate_groupnorm_silu_bwd(*a) for a in args]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(50):
        for i in (0, 1):
            got[i].append(gdn.gdn_gate_groupnorm_silu_bwd(*args[i], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in (0, 1) for g in got[i] for a, b in zip(g, want[i]))
