"""The gated delta rule on the GPU against the float64 oracle: the prompt scan and the
decode step, over types, head layouts, odd sizes, strides, resets, exact decays, streams
and graphs; and a run of prompt, decode and norm as a layer uses them.

Outputs use scale 1 and unit q and k unless said otherwise, so that they and the states
are of order one; the tolerance is the framework's, max |d| / (1 + |ref|) <= 1e-4 for
float32 tensors and 1e-2 for bfloat16 ones.  A float32 output's error: every token adds
less than 40 roundings of 2^-24 to a state that the delta rule does not amplify (beta in
[0, 1], unit keys: the state maps are contractions), 300 tokens of memory at most, so
below 300 * 40 * 6e-8 = 7e-4 if all had one sign and 1e-5 as they fall.  A bfloat16
output's: half a step of the output, 2^-8 |ref|, and up to three operands rounded to
bfloat16 whose errors (2^-8 of each term at most) add up over 128 signed terms."""
import math

import pytest
import torch

from gpu_util import TOL, assert_close
from selective_state_space_18_b200 import ssscan
from selective_state_space_18_b200.inputs import make_delta_inputs

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def _cuda_dict(inp):
    return {k: (None if v is None else v.cuda()) for k, v in inp.items()}


def _scan(inp, **kw):
    out = ssscan.ss_delta_scan(**_cuda_dict(inp), **kw)
    torch.cuda.synchronize()
    assert ssscan.ss_debug_status() == "SS_OK"
    return out["outputs"].cpu(), out["final_state"].cpu()


def _check(orc, inp, what="", scale=1.0, qk_l2norm=True, grow=1.0, **kw):
    y, fs = _scan(inp, scale=scale, qk_l2norm=qk_l2norm, **kw)
    ref = orc.delta_scan(**inp, scale=scale, qk_l2norm=qk_l2norm)
    assert y.dtype == inp["q"].dtype and fs.dtype == F32
    assert_close(y, ref["outputs"], grow * TOL[y.dtype], f"{what} outputs")
    assert_close(fs, ref["final_state"], grow * TOL[F32], f"{what} final_state")
    return y, fs


SHAPES = [  # batch, seq, heads_k, heads_v, dk, dv
    (1, 1, 1, 1, 128, 128), (2, 5, 1, 2, 128, 64), (1, 63, 2, 2, 128, 128), (1, 64, 2, 4, 128, 128),
    (2, 65, 1, 1, 128, 128), (1, 129, 2, 2, 64, 64), (2, 200, 2, 6, 96, 80), (1, 300, 1, 4, 128, 200),
    (1, 150, 1, 1, 8, 8), (1, 90, 1, 2, 40, 24), (3, 130, 2, 2, 128, 256), (1, 77, 1, 1, 33, 17), (1, 70, 1, 2, 200, 40),
    (1, 1, 1, 1, 1, 1), (1, 40, 1, 1, 256, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(orc, shape, dtype):
    seed = 3000 + sum(shape) + len(dtype)
    _check(orc, make_delta_inputs(*shape, dtype, seed=seed, h0=True), str(shape))
    _check(orc, make_delta_inputs(*shape, dtype, seed=seed + 1, reset_mean_doc=20), f"{shape} resets")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_ragged(orc, dtype):
    _check(orc, make_delta_inputs(1, 2051, 1, 2, 128, 128, dtype, seed=3100, h0=True), "long")


@pytest.mark.parametrize("shape", [(1, 6000, 1, 1, 128, 128), (1, 3024, 2, 4, 64, 256), (2, 2400, 1, 3, 40, 24),
                                   (1, 2305, 4, 32, 128, 128), (3, 2331, 4, 12, 96, 64)])
@pytest.mark.parametrize("resets", [0, 150])
def test_segments(orc, shape, resets):
    """Few heads and a long prompt: the sequence is cut and walked in two passes.  With
    decays near one the segments' entering states matter over the whole sequence."""
    inp = make_delta_inputs(*shape, "bf16", seed=3170 + sum(shape), h0=True, reset_mean_doc=resets or None)
    _check(orc, inp, f"{shape}")
    inp["g"] = inp["g"] * 1e-3
    _check(orc, inp, f"{shape}, slow decay")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("workspace", [True, False])
def test_without_norm_or_gates(orc, dtype, workspace):
    """No norm, no g, no beta: keys scaled to below unit length by hand."""
    inp = make_delta_inputs(2, 140, 1, 2, 128, 128, dtype, seed=3110, h0=True)
    inp["q"], inp["k"] = (inp["q"] * 0.125).to(inp["q"].dtype), (inp["k"] * 0.0625).to(inp["k"].dtype)
    inp["g"] = inp["beta"] = None
    _check(orc, inp, "plain delta rule", qk_l2norm=False, workspace=workspace)
    _check(orc, inp, "default scale", qk_l2norm=False, scale=None, workspace=workspace)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pattern", ["minus_inf", "strong", "zero", "growing", "reset_all", "reset_edges", "beta_edges"])
def test_exact_gates(orc, dtype, pattern):
    inp = make_delta_inputs(2, 200, 1, 2, 128, 64, dtype, seed=3120, h0=True)
    g, beta = inp["g"].clone(), inp["beta"].clone()
    if pattern == "minus_inf":
        g[:, ::64] = -float("inf")      # on chunk starts
        g[1, 63] = g[1, 70] = g[1, 71] = -float("inf")
    elif pattern == "strong":
        g = g * 1000                    # decays that underflow, and sums that pass 1e3
        g[:, 100:110] = -0.001
    elif pattern == "zero":
        g[:] = 0.0
    elif pattern == "growing":
        g[:, 50:60] = 0.3               # e^3 over ten tokens
    elif pattern == "reset_all":
        inp["reset"] = torch.ones(2, 200, dtype=torch.bool)
    elif pattern == "reset_edges":
        inp["reset"] = torch.zeros(2, 200, dtype=torch.uint8)
        inp["reset"][0, 0] = inp["reset"][0, 64] = inp["reset"][0, 127] = inp["reset"][1, 199] = 7
    else:
        beta[:, ::3] = 0.0
        beta[:, 1::3] = 1.0
        beta[0, 2::3] = 1.9             # beyond 1: the write overshoots
    inp["g"], inp["beta"] = g, beta
    if inp["reset"] is not None:        # the oracle keeps the type, the binding takes both
        inp["reset"] = inp["reset"].to(torch.uint8)
    # growing: ten decays of e^0.3 make the state, and with it every term of an output and
    # its rounding, up to e^3 times what the tolerance is meant for: 128 terms q_i H_ij of
    # |q| = 1 and columns of length 0.3 sqrt(128) e^3 = 68, each rounded by up to 2^-8, may
    # differ by 0.27 in all, whatever their sum is
    _check(orc, inp, pattern, grow=math.exp(3.0) if pattern == "growing" else 1.0)


def test_reset_forgets_what_came_before():
    """Outputs from a reset on do not depend on earlier tokens or on h0, bit for bit, and
    equal the later document run alone where it starts a chunk."""
    inp = make_delta_inputs(1, 256, 1, 2, 128, 128, "bf16", seed=3130, h0=True)
    inp["reset"] = torch.zeros(1, 256, dtype=torch.bool)
    inp["reset"][0, 128] = True
    y, fs = _scan(inp, qk_l2norm=True)
    other = dict(inp, h0=inp["h0"] * 3, v=inp["v"].clone(), k=inp["k"].clone())
    other["v"][:, :128] *= -2
    other["k"][:, :100] *= 0.5
    y2, fs2 = _scan(other, qk_l2norm=True)
    assert torch.equal(y[:, 128:], y2[:, 128:]) and torch.equal(fs, fs2)
    alone = {k: (None if v is None else v[:, 128:]) for k, v in inp.items() if k not in ("h0", "reset")}
    y3, fs3 = _scan(alone, qk_l2norm=True)
    assert torch.equal(y[:, 128:], y3) and torch.equal(fs, fs3)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta", "h0"])
@pytest.mark.parametrize("seq,heads_v,dtype,workspace", [(250, 2, "bf16", True), (250, 150, "bf16", True), (2400, 2, "bf16", True),
                                                         (250, 2, "f32", True), (250, 2, "bf16", False)])
def test_values_that_are_not_finite_stay_where_they_belong(orc, seq, heads_v, dtype, workspace, where, value):
    """An infinity or NaN in one token reaches neither earlier tokens nor those behind a
    reset, wherever in a chunk both lie; one in h0 nothing behind the first reset.  In every
    form: one walk, many, segments, token by token."""
    if where == "g" and value == math.inf:
        pytest.skip("log decays lie below infinity")
    for at, cut in ((200, 201), (191, 192), (100, 180), (0, 70), (seq - 1, None)):
        clean = make_delta_inputs(1, seq, 1, heads_v, 64, 136, dtype, seed=3125, h0=True)
        clean["reset"] = torch.zeros(1, seq, dtype=torch.uint8)
        if cut is not None:
            clean["reset"][0, cut] = 1
        inp = {k: v.clone() for k, v in clean.items()}
        if where == "h0":
            inp["h0"][0, heads_v - 1] = value
        else:
            inp[where][0, at, -1] = value
        y, fs = _scan(inp, scale=1.0, qk_l2norm=True, workspace=workspace)
        ref = orc.delta_scan(**clean, scale=1.0, qk_l2norm=True)
        before = at if where != "h0" else 0
        assert_close(y[:, :before], ref["outputs"][:, :before], TOL[y.dtype], f"before {at}")
        if cut is not None:
            assert_close(y[:, cut:], ref["outputs"][:, cut:], TOL[y.dtype], f"from the reset at {cut}")
            assert_close(fs, ref["final_state"], TOL[F32], "final state")
        elif where in "kv":
            assert not torch.isfinite(y[:, at:]).all() or not torch.isfinite(fs).all()
        if where in ("v", "h0", "g", "beta") and heads_v > 1:   # the other heads know nothing of it
            assert_close(y[:, :, 0], ref["outputs"][:, :, 0], TOL[y.dtype], "another head")


@pytest.mark.parametrize("dtype,workspace", [("bf16", True), ("bf16", False), ("f32", True)])
@pytest.mark.parametrize("at", [0, 1, 2, 3, 62, 63, 64])
def test_growth_of_an_empty_state(orc, dtype, workspace, at):
    """Decays of e^80 twice over, whose product float32 does not hold, on a state that is
    still empty: nothing has grown."""
    inp = make_delta_inputs(1, 100, 1, 2, 64, 32, dtype, seed=3127)
    inp["g"], inp["beta"] = inp["g"].clone(), inp["beta"].clone()
    inp["g"][:, at:at + 2] = 80.0
    inp["beta"][:, :at + 1] = 0.0
    _check(orc, inp, f"growth at {at}", workspace=workspace)


@pytest.mark.parametrize("seq", [1, 2, 3, 4, 5, 31, 32, 33, 36, 37])
@pytest.mark.parametrize("dv", [4, 30, 600])
@pytest.mark.parametrize("dk", [16, 72])
def test_token_form_steps_and_tiles(orc, seq, dv, dk):
    """Prompts that end inside steps of four tokens and tiles of 32, resets on every place
    of a step, in narrow and in wide blocks of columns."""
    inp = make_delta_inputs(2, seq, 1, 1, dk, dv, "f32", seed=3128, h0=True)
    _check(orc, inp, "no resets")
    for place in range(min(seq, 4)):
        reset = torch.zeros(2, seq, dtype=torch.uint8)
        reset[0, place::8] = 1
        reset[1, place::5] = 1
        _check(orc, dict(inp, reset=reset), f"resets from {place}")


@pytest.mark.parametrize("seq", [250, 2400])
def test_chaining_in_place_after_a_nan(orc, seq):
    """The final state may take h0's place in columns that are walked token by token too."""
    clean = make_delta_inputs(1, seq, 1, 2, 128, 128, "bf16", seed=3126, h0=True)
    clean["reset"] = torch.zeros(1, seq, dtype=torch.uint8)
    clean["reset"][0, 30] = 1
    ref = orc.delta_scan(**clean, scale=1.0, qk_l2norm=True)
    inp = _cuda_dict(clean)
    inp["v"][0, 20, 1, 5] = math.nan
    inp["h0"][0, 0] = math.nan
    out = ssscan.ss_delta_scan(**inp, scale=1.0, qk_l2norm=True, final_state=inp["h0"])
    assert ssscan.ss_debug_status() == "SS_OK"
    assert_close(out["outputs"].cpu()[:, 30:], ref["outputs"][:, 30:], TOL[BF16], "outputs")
    assert_close(out["outputs"].cpu()[:, :20, 1], ref["outputs"][:, :20, 1], TOL[BF16], "outputs before")
    assert_close(inp["h0"].cpu(), ref["final_state"], TOL[F32], "final state in h0's place")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_one_projection(orc, dtype):
    """q, k and v as views of one buffer, read in place, equal the packed copies; rows
    that no vector load divides too; the buffer is left as it was."""
    for hk, hv, dk, dv, pad in ((2, 4, 128, 128, 0), (1, 2, 64, 32, 8), (1, 3, 40, 20, 3)):
        inp = make_delta_inputs(2, 100, hk, hv, dk, dv, dtype, seed=3140 + pad)
        parts = [inp[n].flatten(-2) for n in ("q", "k", "v")]
        buf = torch.cat(parts + [torch.full((2, 100, pad), float("nan"), dtype=parts[0].dtype)], -1).cuda()
        keep = buf.clone()
        at = [0, hk * dk, 2 * hk * dk, 2 * hk * dk + hv * dv]
        views = [buf[..., at[i]:at[i + 1]].unflatten(-1, s) for i, s in enumerate(((hk, dk), (hk, dk), (hv, dv)))]
        out = ssscan.ss_delta_scan(*views, inp["g"].cuda(), inp["beta"].cuda(), qk_l2norm=True)
        y, fs = _scan(inp, qk_l2norm=True)
        assert_close(out["outputs"].cpu(), y.double().numpy(), TOL[y.dtype], "views")
        assert_close(out["final_state"].cpu(), fs.double().numpy(), TOL[F32], "views, state")
        assert torch.equal(buf.view(torch.uint8), keep.view(torch.uint8))


def test_chaining_in_place(orc):
    inp = make_delta_inputs(2, 333, 1, 2, 128, 128, "bf16", seed=3150, h0=True)
    ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
    d = _cuda_dict(inp)
    state, ys = d["h0"].clone(), []
    for a, b in ((0, 100), (100, 101), (101, 333)):
        part = {n: d[n][:, a:b] for n in ("q", "k", "v", "g", "beta")}
        out = ssscan.ss_delta_scan(**part, h0=state, final_state=state, scale=1.0, qk_l2norm=True)
        ys.append(out["outputs"])
        assert out["final_state"] is state
    assert_close(torch.cat(ys, 1).cpu(), ref["outputs"], TOL[BF16], "outputs")
    assert_close(state.cpu(), ref["final_state"], TOL[F32], "state")


def test_chaining_in_place_over_segments(orc):
    """The final state in h0's place while the sequence is walked in segments (the first
    segment's second walk reads h0 after the last one may have written it)."""
    inp = make_delta_inputs(1, 3000, 1, 4, 128, 128, "bf16", seed=3155, h0=True)
    inp["g"] = inp["g"] * 1e-2
    ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
    d = _cuda_dict(inp)
    apart = ssscan.ss_delta_scan(**d, scale=1.0, qk_l2norm=True)
    for _ in range(3):
        state = d["h0"].clone()
        out = ssscan.ss_delta_scan(**dict(d, h0=state), final_state=state, scale=1.0, qk_l2norm=True)
        assert torch.equal(out["outputs"], apart["outputs"]) and torch.equal(state, apart["final_state"])
    assert_close(out["outputs"].cpu(), ref["outputs"], TOL[BF16], "outputs")
    assert_close(state.cpu(), ref["final_state"], TOL[F32], "state")


def test_supplied_buffers_and_no_final_state():
    inp = _cuda_dict(make_delta_inputs(1, 130, 1, 1, 128, 128, "bf16", seed=3160))
    ref = ssscan.ss_delta_scan(**inp)
    need = ssscan.ss_delta_workspace_bytes(1, 130, 1, 1, 128, 128)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")  # contents mean nothing
    y = torch.empty_like(ref["outputs"])
    out = ssscan.ss_delta_scan(**inp, outputs=y, return_final_state=False, workspace=ws)
    assert out["outputs"] is y and out["final_state"] is None
    assert torch.equal(y, ref["outputs"])
    assert bool((ws[need:] == 0xff).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 128, 128), (3, 2, 4, 128, 64), (5, 1, 3, 96, 80), (2, 1, 1, 33, 17),
                                   (2, 1, 2, 200, 40), (1, 1, 1, 1, 1), (130, 1, 1, 64, 128), (2, 2, 2, 256, 36)])
def test_decode(orc, shape, dtype):
    bt, hk, hv, dk, dv = shape
    inp = make_delta_inputs(bt, 1, hk, hv, dk, dv, dtype, seed=3200 + sum(shape), h0=True)
    ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
    d = _cuda_dict(inp)
    guard = torch.full((bt * hv * dk * dv + 8,), 7.0, device="cuda")  # 4-byte aligned only
    for state in (d["h0"].clone(), guard[1:1 + bt * hv * dk * dv].view(bt, hv, dk, dv).copy_(d["h0"])):
        y = ssscan.ss_delta_update(state, *(d[n][:, 0] for n in ("q", "k", "v", "g", "beta")), scale=1.0,
                                   qk_l2norm=True)
        assert_close(y.cpu(), ref["outputs"][:, 0], TOL[y.dtype], "y")
        # one step of float32: 20 roundings of 2^-24 on values of order one
        assert_close(state.cpu(), ref["final_state"], 1e-5, "state")
    assert float(guard[0]) == 7.0 and bool((guard[-7:] == 7.0).all())


def test_decode_gates(orc):
    """No gates, no norm; a decay of zero discards a state that holds infinities."""
    inp = make_delta_inputs(4, 1, 1, 2, 64, 64, "f32", seed=3250, h0=True)
    inp["k"] = inp["k"] * 0.1
    d = _cuda_dict(inp)
    state = d["h0"].clone()
    y = ssscan.ss_delta_update(state, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0])
    ref = orc.delta_scan(inp["q"], inp["k"], inp["v"], h0=inp["h0"])
    assert_close(y.cpu(), ref["outputs"][:, 0], 1e-5, "y")
    assert_close(state.cpu(), ref["final_state"], 1e-5, "state")
    state[0] = float("inf")
    state[1] = float("nan")
    g = torch.full((4, 2), -float("inf"), device="cuda")
    y = ssscan.ss_delta_update(state, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], g)
    ref = orc.delta_scan(inp["q"], inp["k"], inp["v"])
    assert_close(y.cpu(), ref["outputs"][:, 0], 1e-5, "y after the cut")
    assert_close(state.cpu(), ref["final_state"], 1e-5, "state after the cut")


def test_decode_large_batch_and_views(orc):
    inp = make_delta_inputs(67, 1, 2, 4, 128, 128, "bf16", seed=3260, h0=True)
    d = _cuda_dict(inp)
    buf = torch.cat([d[n][:, 0].flatten(-2) for n in ("q", "k", "v")], -1)
    q, k, v = buf[:, :256].unflatten(-1, (2, 128)), buf[:, 256:512].unflatten(-1, (2, 128)), \
        buf[:, 512:].unflatten(-1, (4, 128))
    state = d["h0"].clone()
    y = ssscan.ss_delta_update(state, q, k, v, d["g"][:, 0], d["beta"][:, 0], scale=1.0, qk_l2norm=True)
    ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
    assert_close(y.cpu(), ref["outputs"][:, 0], TOL[BF16], "y")
    assert_close(state.cpu(), ref["final_state"], 1e-5, "state")


def test_other_stream_and_graph():
    """A side stream (with a copied view and a workspace of its own) and a captured graph
    replayed on new inputs give what plain calls give."""
    a = _cuda_dict(make_delta_inputs(2, 150, 1, 2, 128, 128, "bf16", seed=3300, h0=True))
    b = _cuda_dict(make_delta_inputs(2, 150, 1, 2, 128, 128, "bf16", seed=3301, h0=True))
    ref = [ssscan.ss_delta_scan(**x, qk_l2norm=True) for x in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    strided = dict(a, q=a["q"].transpose(1, 2).contiguous().transpose(1, 2))
    outs = [ssscan.ss_delta_scan(**x, qk_l2norm=True, stream=side) for x in (strided, b)]
    torch.cuda.current_stream().wait_stream(side)
    for o, r in zip(outs, ref):
        assert torch.equal(o["outputs"], r["outputs"]) and torch.equal(o["final_state"], r["final_state"])
    static = {k: (None if v is None else v.clone()) for k, v in a.items()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = ssscan.ss_delta_scan(**static, qk_l2norm=True)
        y = ssscan.ss_delta_update(out["final_state"], *(static[n][:, 0] for n in ("q", "k", "v", "g", "beta")))
        n = ssscan.ss_group_norm(y, 1, gate=y, center=False)
    for x, r in ((b, ref[1]), (a, ref[0])):
        for name, t in x.items():
            if t is not None:
                static[name].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["outputs"], r["outputs"])
        fs = r["final_state"].clone()
        y2 = ssscan.ss_delta_update(fs, *(x[m][:, 0] for m in ("q", "k", "v", "g", "beta")))
        assert torch.equal(out["final_state"], fs) and torch.equal(y, y2)
        assert torch.equal(n, ssscan.ss_group_norm(y2, 1, gate=y2, center=False))
    with pytest.raises(ValueError):
        ssscan.ss_delta_scan(a["q"], a["k"], a["v"][:, :10])
    with pytest.raises(TypeError):
        ssscan.ss_delta_scan(a["q"], a["k"].float(), a["v"])
    with pytest.raises(ssscan.SSError):
        ssscan.ss_delta_scan(a["q"].repeat(1, 1, 1, 3), a["k"].repeat(1, 1, 1, 3), a["v"])


def test_same_call_twice_is_bit_identical():
    inp = _cuda_dict(make_delta_inputs(3, 517, 2, 4, 128, 128, "bf16", seed=3310, h0=True, reset_mean_doc=100))
    a, b = (ssscan.ss_delta_scan(**inp, qk_l2norm=True) for _ in range(2))
    assert torch.equal(a["outputs"], b["outputs"]) and torch.equal(a["final_state"], b["final_state"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_prompt_decode_norm(orc, dtype):
    """Prompt, then decode steps from its state, each followed by the gated norm: the
    whole sequence through the oracle."""
    L, n = 130, 6
    inp = make_delta_inputs(2, L + n, 2, 4, 128, 128, dtype, seed=3400, h0=False)
    gen = torch.Generator().manual_seed(3401)
    z = torch.randn(2, L + n, 512, generator=gen).to(inp["q"].dtype)
    w = 1 + 0.1 * torch.randn(128, generator=gen)
    d = _cuda_dict(inp)
    names = ("q", "k", "v", "g", "beta")
    out = ssscan.ss_delta_scan(*(d[m][:, :L] for m in names), qk_l2norm=True, scale=1.0)
    state, ys = out["final_state"], [out["outputs"]]
    for t in range(L, L + n):
        ys.append(ssscan.ss_delta_update(state, *(d[m][:, t] for m in names), qk_l2norm=True, scale=1.0)[:, None])
    y = torch.cat(ys, 1).flatten(-2)
    o = ssscan.ss_group_norm(y, 4, w.cuda(), gate=z.cuda(), center=False, eps=1e-6)
    ref = orc.delta_scan(**{m: inp[m] for m in names}, qk_l2norm=True, scale=1.0)
    assert_close(y.cpu(), ref["outputs"].reshape(2, L + n, 512), TOL[y.dtype], "outputs")
    assert_close(state.cpu(), ref["final_state"], TOL[F32], "state")
    assert_close(o.cpu(), orc.group_norm(y.cpu(), 4, w, gate=z, center=False, eps=1e-6), TOL[o.dtype], "norm")


@pytest.mark.parametrize("shape", [(2, 300, 1, 2, 128, 128), (1, 2400, 1, 2, 128, 128)])
def test_timed_out_waits_report_and_recover(shape):
    """Failure detection without a GPU fault: with an arrival of the first chunk withheld
    and the wait limit cut to 2 ms, the walk's waits give up, the status word reports
    SS_ERR_TIMEOUT, and the next call gives the normal answer."""
    d = _cuda_dict(make_delta_inputs(*shape, "bf16", seed=3500, h0=True))
    ref = ssscan.ss_delta_scan(**d, qk_l2norm=True)
    assert ssscan.ss_debug_status() == "SS_OK"
    ssscan.ss_debug_set_wait_limit(2000)
    ssscan.ss_debug_set_gated_path(3)
    try:
        ssscan.ss_delta_scan(**d, qk_l2norm=True)
        torch.cuda.synchronize()
        assert ssscan.ss_debug_status() == "SS_ERR_TIMEOUT"
    finally:
        ssscan.ss_debug_set_gated_path(0)
        ssscan.ss_debug_set_wait_limit(0)
    out = ssscan.ss_delta_scan(**d, qk_l2norm=True)
    torch.cuda.synchronize()
    assert ssscan.ss_debug_status() == "SS_OK"
    assert torch.equal(out["outputs"], ref["outputs"]) and torch.equal(out["final_state"], ref["final_state"])
