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
