"""The gated delta rule and the group norm on tensors of more than 2^31 elements, where 32-bit
index arithmetic would wrap: sampled heads, states and rows against the float64 oracle."""
import pytest
import torch

from gpu_util import TOL, assert_close
from selective_state_space_18_b200 import ssscan

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    free, _ = torch.cuda.mem_get_info()
    if free < 40 * 2**30:
        pytest.skip("needs 40 GB of free device memory")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("workspace", [True, False])
def test_scan(orc, workspace):
    """8 x 16400 tokens x 128 heads of 32 x 128: 2.15e9 values and outputs, and 5.1 GB of
    workspace blocks for the chunked form."""
    b, L, hv, dk, dv = 8, 16400, 128, 32, 128
    assert b * L * hv * dv > 2**31
    gen = _gen(3800)
    q, k = (torch.randn(b, L, 2, dk, generator=gen, device="cuda").to(BF16) for _ in range(2))
    v = torch.randn(b, L, hv, dv, generator=gen, device="cuda", dtype=BF16)
    g = -0.2 * torch.rand(b, L, hv, generator=gen, device="cuda")
    beta = torch.rand(b, L, hv, generator=gen, device="cuda")
    out = ssscan.ss_delta_scan(q, k, v, g, beta, scale=1.0, qk_l2norm=True, workspace=workspace)
    assert ssscan.ss_debug_status() == "SS_OK"
    for i, h in ((0, 0), (4, 1), (7, 63), (7, 127)):
        at = slice(h // 64, h // 64 + 1)
        ref = orc.delta_scan(q[i:i + 1, :, at].cpu(), k[i:i + 1, :, at].cpu(), v[i:i + 1, :, h:h + 1].cpu(),
                             g[i:i + 1, :, h:h + 1].cpu(), beta[i:i + 1, :, h:h + 1].cpu(), scale=1.0, qk_l2norm=True)
        assert_close(out["outputs"][i:i + 1, :, h:h + 1].cpu(), ref["outputs"], TOL[BF16], f"outputs {i} {h}")
        assert_close(out["final_state"][i:i + 1, h:h + 1].cpu(), ref["final_state"], TOL[F32], f"state {i} {h}")


@pytest.mark.parametrize("dk,dv", [(128, 128), (127, 130)])
def test_update(orc, dk, dv):
    """4100 x 32 states: 2.15e9 elements, as vectors and as single elements."""
    b, hv = 4100, 32
    assert b * hv * dk * dv > 2**31
    gen = _gen(3810)
    state = torch.randn(b, hv, dk, dv, generator=gen, device="cuda")
    q, k = (torch.randn(b, 16, dk, generator=gen, device="cuda").to(BF16) for _ in range(2))
    v = torch.randn(b, hv, dv, generator=gen, device="cuda").to(BF16)
    g, beta = -torch.rand(b, hv, generator=gen, device="cuda"), torch.rand(b, hv, generator=gen, device="cuda")
    rows = [0, 2047, 2048, 4099]
    before = state[rows].cpu()
    y = ssscan.ss_delta_update(state, q, k, v, g, beta, scale=1.0, qk_l2norm=True)
    ref = orc.delta_scan(*(t[rows][:, None].cpu() for t in (q, k, v, g, beta)), h0=before, scale=1.0, qk_l2norm=True)
    assert_close(y[rows].cpu(), ref["outputs"][:, 0], TOL[BF16], "y")
    assert_close(state[rows].cpu(), ref["final_state"], 1e-5, "state")


@pytest.mark.parametrize("rows,groups,size", [(524416, 32, 128), (5175000, 5, 83)])
def test_norm(orc, rows, groups, size):
    assert rows * groups * size > 2**31
    gen = _gen(3820)
    ch = groups * size
    x = torch.randn(rows, ch, generator=gen, device="cuda", dtype=BF16)
    w = torch.rand(size, generator=gen, device="cuda")
    y = ssscan.ss_group_norm(x, groups, w, center=False, activation="silu")
    at = [0, 1, rows // 2 - 1, rows // 2, rows - 2, rows - 1]
    ref = orc.group_norm(x[at].cpu(), groups, w.cpu(), center=False, activation="silu")
    assert_close(y[at].cpu(), ref, 2.0 ** -8 + 2e-5, "rows")
