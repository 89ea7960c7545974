"""The gated delta rule and the group norm on unusual values: states near the ends of
float32's range, infinities and NaN where they belong, exact factors; and the parts of the
chunked form that results alone do not show."""
import math

import pytest
import torch

from gpu_util import TOL, assert_close
from selective_state_space_18_b200 import ssscan
from selective_state_space_18_b200.inputs import make_delta_inputs

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# one walk an SM, two walks an SM, segments, token by token
FORMS = [(250, 2, "bf16", True), (250, 150, "bf16", True), (2400, 2, "bf16", True), (250, 2, "f32", True),
         (250, 2, "bf16", False)]


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


@pytest.mark.parametrize("seq,heads_v,dtype,workspace", FORMS)
@pytest.mark.parametrize("power", [-60, 70, 90, 115])
def test_large_and_small_writes(orc, seq, heads_v, dtype, workspace, power):
    """The rule is linear in v and h0, so a power of two on both is one on the outputs and the
    state, and the tolerances are those without it.  The decays reach 2^-50 within a chunk of
    64 tokens and no further: factors of the order of their inverse stay in use."""
    inp = make_delta_inputs(1, seq, 1, heads_v, 64, 136, dtype, seed=3600, h0=True)
    inp["g"] = torch.full_like(inp["g"], -0.55)
    ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
    inp["v"], inp["h0"] = inp["v"] * 2.0 ** power, inp["h0"] * 2.0 ** power
    y, fs = _scan(inp, scale=1.0, qk_l2norm=True, workspace=workspace)
    assert_close(y.double() * 2.0 ** -power, ref["outputs"], TOL[y.dtype], "outputs")
    assert_close(fs.double() * 2.0 ** -power, ref["final_state"], TOL[F32], "final state")


@pytest.mark.parametrize("dk", [16, 24, 64, 72, 96, 112, 128])
def test_maps_of_segments_that_forget_are_zero(dk):
    """36 chunks of one head are three segments.  With a decay of e^-1 a token the middle one's
    map from state to state is exactly 0 after two chunks, whatever the key size: the last word
    of the workspace says so, and the walk for the map ends there."""
    inp = _cuda_dict(make_delta_inputs(1, 36 * 64, 1, 1, dk, 64, "bf16", seed=3610, h0=True))
    need = ssscan.ss_delta_workspace_bytes(1, 36 * 64, 1, 1, dk, 64)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    flag = ws[need - 4:need].view(torch.int32)
    for g, zero in ((-1.0, 1), (-1e-3, 0)):
        inp["g"] = torch.full_like(inp["g"], g)
        ssscan.ss_delta_scan(**inp, qk_l2norm=True, workspace=ws)
        assert flag.item() == zero, g
    assert bool((ws[need:] == 0xff).all())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta", "h0"])
@pytest.mark.parametrize("seq,heads_v,dtype,workspace", FORMS)
def test_values_that_are_not_finite_arrive(orc, seq, heads_v, dtype, workspace, where, value):
    """From the token of an infinity or NaN to the next reset, outputs (and the final state
    where no reset comes) are finite exactly where the definition's are; in other value columns
    of the head that holds it in v or h0 they are what they are without it."""
    if where == "g" and not math.isnan(value):
        pytest.skip("log decays lie below infinity, and minus infinity is a decay of 0")
    for at, cut, h0 in ((200, 201, True), (100, 180, True), (0, 70, True), (0, 70, False), (seq - 1, None, True)):
        if where == "h0" and not h0:
            continue
        clean = make_delta_inputs(1, seq, 1, heads_v, 64, 136, dtype, seed=3620, h0=h0)
        clean["reset"] = torch.zeros(1, seq, dtype=torch.uint8)
        if cut is not None:
            clean["reset"][0, cut] = 1
        inp = {k: (None if v is None else v.clone()) for k, v in clean.items()}
        if where == "h0":
            inp["h0"][0, -1, 5, -1] = value
        else:
            inp[where][0, at].view(-1)[-1] = value
        y, fs = _scan(inp, scale=1.0, qk_l2norm=True, workspace=workspace)
        ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
        first = 0 if where == "h0" else at
        finite = torch.from_numpy(ref["outputs"][:, first:cut]).isfinite()
        assert torch.equal(y[:, first:cut].isfinite(), finite), f"outputs from {first} to {cut}"
        assert not finite.all()
        if cut is None:
            assert torch.equal(fs.isfinite(), torch.from_numpy(ref["final_state"]).isfinite()), "final state"
        if where in ("v", "h0"):
            ref = orc.delta_scan(**clean, scale=1.0, qk_l2norm=True)
            assert_close(y[..., :-1], ref["outputs"][..., :-1], TOL[y.dtype], "other columns")
            assert_close(fs[..., :-1], ref["final_state"][..., :-1], TOL[F32], "other columns, final state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta", "h0"])
def test_values_that_are_not_finite_in_a_decode_step(orc, dtype, where, value):
    """The same of one step: in the head that holds it, and in v or h0 in its column alone."""
    if where == "g" and value == math.inf:
        pytest.skip("log decays lie below infinity")
    inp = make_delta_inputs(3, 1, 1, 2, 64, 72, dtype, seed=3630, h0=True)
    clean = {k: (None if v is None else v.clone()) for k, v in inp.items()}
    inp[where][1].view(-1)[-1] = value
    d = _cuda_dict(inp)
    y = ssscan.ss_delta_update(d["h0"], *(d[n][:, 0] for n in ("q", "k", "v", "g", "beta")), scale=1.0, qk_l2norm=True)
    ref, well = (orc.delta_scan(**x, scale=1.0, qk_l2norm=True) for x in (inp, clean))
    for out, name in ((y.cpu(), "outputs"), (d["h0"].cpu(), "final_state")):
        r = torch.from_numpy(ref[name]).view(out.shape)
        w = torch.from_numpy(well[name]).view(out.shape)
        assert torch.equal(out.isfinite(), r.isfinite()), name
        f = r.isfinite()
        assert_close(out[f], w[f].numpy(), TOL[out.dtype], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [8, 24, 33, 640, 2900])
def test_norm_keeps_a_nan_in_its_group(dtype, size):
    """Groups side by side in a warp, in a warp each and in a CTA each: the others of a row
    and the other rows give the same bits with a NaN beside them as without."""
    t = BF16 if dtype == "bf16" else F32
    x = torch.randn(9, 5 * size, generator=torch.Generator().manual_seed(3640)).to(t).cuda()
    ref = ssscan.ss_group_norm(x, 5, activation="silu").view(9, 5, size)
    bad = x.clone()
    bad[4, 2 * size + 3] = math.nan
    y = ssscan.ss_group_norm(bad, 5, activation="silu").view(9, 5, size)
    assert bool(y[4, 2].isnan().all())
    y[4, 2] = ref[4, 2]
    assert torch.equal(y, ref)


@pytest.mark.parametrize("decay", ["constant", "random", "growing", "strong"])
def test_factors_of_a_chunk(decay):
    """The decays from a chunk's start to its tokens (c and s in the workspace block, for unit
    scale and no norm), from them to its end (w), and over it, against 64 bits.  Two
    exponentials with a relative error of up to 2^-22 each, their product (2^-24), and up to
    eight roundings of a sum below one half (2^-26 each, times ln 2): 6.2e-7 in all."""
    inp = make_delta_inputs(1, 64, 1, 1, 128, 128, "bf16", seed=3650)
    u = torch.rand(inp["g"].shape, generator=torch.Generator().manual_seed(3651))
    inp["g"] = {"constant": torch.full_like(u, -0.63), "random": -0.9 * u, "growing": 0.3 + 0.3 * u,
                "strong": -3.0 * u}[decay]
    need = ssscan.ss_delta_workspace_bytes(1, 64, 1, 1, 128, 128)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    ssscan.ss_delta_scan(**_cuda_dict(dict(inp, h0=torch.zeros(1, 1, 128, 128))), scale=1.0, workspace=ws)
    c, w, s, e = ws[2 * 6144:2 * 6144 + 4 * 256].view(F32).double().cpu().view(4, 64)
    if e[1]:    # strong decays: w and s are kept as factors of powers of two, whose exponents' bits follow
        power = torch.exp2(ws[2 * 6144 + 3 * 256 + 16:][:128].double().cpu().view(2, 64) - 127)
        w, s = w * power[0], s * power[1]
    G = inp["g"].double().view(-1).cumsum(0)
    for got, log, what in ((c, G, "c"), (s, G, "s"), (w, G[-1] - G, "w"), (e[:1], G[-1:], "E_63")):
        rel = ((got - log.exp()) / log.exp()).abs()[log > -86.0]   # (below: under float32's normal range)
        assert float(rel.max() if rel.numel() else 0.0) <= 6.2e-7, what


@pytest.mark.parametrize("shape", [(1, 500, 1, 2, 128, 128), (2, 700, 1, 2, 64, 64), (1, 300, 2, 160, 96, 64),
                                   (1, 3000, 1, 2, 128, 136), (1, 2500, 2, 4, 96, 128)])
@pytest.mark.parametrize("slow", [False, True])
def test_error_of_the_chunked_form_in_norm(orc, shape, slow):
    """Rounding a value to bfloat16 costs 1.66e-3 of the norm (half a step, uniform over the
    mantissa); keeping the remainder in bfloat16 too leaves the square of it, 2.8e-6.  The
    state: five such splits on the way of a chunk (H, R, T, w o U and the product of two
    remainders that is left out), 6.2e-6 as they fall, tripled for the chunks that a state
    remembers.  The outputs: the rounding of their own, 1.66e-3; 1.8e-3 for what a sample of a few
    thousand may differ from it.  A lost remainder would cost either 1e-3 more."""
    inp = make_delta_inputs(*shape, "bf16", seed=3660 + sum(shape), h0=True)
    if slow:
        inp["g"] = inp["g"] * 1e-2
    y, fs = _scan(inp, scale=1.0, qk_l2norm=True)
    ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
    for got, want, tol, what in ((y, ref["outputs"], 1.8e-3, "outputs"), (fs, ref["final_state"], 1.9e-5, "state")):
        want = torch.from_numpy(want)
        err = float((got.double() - want).norm() / want.norm())
        assert err <= tol, f"{what}: {err:.2e}"


@pytest.mark.parametrize("seq,heads_v,dtype,workspace", FORMS)
def test_largest_growth(orc, seq, heads_v, dtype, workspace):
    """A decay of e^88.5, close to the largest that float32 holds, on a state that is still
    empty, and one of e^40 on a state of 1e-20."""
    inp = make_delta_inputs(1, seq, 1, heads_v, 64, 32, dtype, seed=3670)
    inp["g"], inp["beta"] = inp["g"].clone(), inp["beta"].clone()
    inp["g"][:, 10] = inp["g"][:, 75] = 88.5
    inp["beta"][:, :76] = 0.0
    _check_forms(orc, inp, workspace, 1.0)
    inp = make_delta_inputs(1, seq, 1, heads_v, 64, 32, dtype, seed=3671, h0=True)
    inp["g"], inp["h0"] = inp["g"].clone(), inp["h0"] * 1e-20
    inp["g"][:, :20] = -0.01
    inp["g"][:, 20] = 40.0
    inp["beta"] = torch.cat((torch.zeros_like(inp["beta"][:, :21]), inp["beta"][:, 21:]), 1)
    _check_forms(orc, inp, workspace, 1.0)


def _check_forms(orc, inp, workspace, scale):
    y, fs = _scan(inp, scale=scale, qk_l2norm=True, workspace=workspace)
    ref = orc.delta_scan(**inp, scale=scale, qk_l2norm=True)
    assert_close(y, ref["outputs"], TOL[y.dtype], "outputs")
    assert_close(fs, ref["final_state"], TOL[F32], "final state")


@pytest.mark.parametrize("heads_v,seq", [(2, 500), (150, 200), (2, 2400)])
@pytest.mark.parametrize("decay", ["none", "slow", "strong", "resets"])
@pytest.mark.parametrize("spread", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("same", [True, False])
def test_keys_that_resemble_each_other(orc, heads_v, seq, decay, spread, same):
    """Keys around one direction (spread: their own part to the common one), read with
    themselves or with other queries: every write replaces most of the one before, and the
    terms of an output add up to a multiple of it.  The tolerances are the framework's, and in
    norm that of any other outputs (see above)."""
    inp = make_delta_inputs(1, seq, 1, heads_v, 128, 64, "bf16", seed=3680, h0=True)
    gen = torch.Generator().manual_seed(3681)
    k = torch.randn(1, 1, 1, 128, generator=gen) + spread * torch.randn(1, seq, 1, 128, generator=gen)
    inp["k"] = k.to(BF16)
    inp["q"] = inp["k"] if same else torch.randn(1, seq, 1, 128, generator=gen).to(BF16)
    inp["v"] = torch.randn(1, seq, heads_v, 64, generator=gen).to(BF16)
    inp["g"] = torch.full_like(inp["g"], {"none": 0.0, "slow": -0.03, "strong": -1.0, "resets": -0.03}[decay])
    inp["beta"] = 0.5 + 0.5 * torch.rand(inp["beta"].shape, generator=gen)
    inp["beta"][..., 0] = 1.0
    if decay == "resets":
        inp["reset"] = torch.rand(1, seq, generator=gen) < 0.02
    y, fs = _scan(inp, scale=1.0, qk_l2norm=True)
    ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
    assert_close(y, ref["outputs"], TOL[BF16], "outputs")
    want = torch.from_numpy(ref["outputs"])
    assert float((y.double() - want).norm() / want.norm()) <= 1.8e-3
    assert_close(fs, ref["final_state"], TOL[F32], "final state")


@pytest.mark.parametrize("shape", [(1, 300, 1, 200, 128, 128), (3, 2400, 1, 60, 64, 64)])
@pytest.mark.parametrize("resets", [None, 40])
def test_timed_out_waits_with_two_walks_an_sm(shape, resets):
    """An arrival of every walk's first chunk withheld, under a limit of 2 ms: the waits give
    up, the status says so, and the next call gives the normal answer."""
    d = _cuda_dict(make_delta_inputs(*shape, "bf16", seed=3690, h0=True, reset_mean_doc=resets))
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
