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
