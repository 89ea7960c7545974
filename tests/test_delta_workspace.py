"""The workspace of the gated delta rule's prompt scan: its size against the layout that the
kernels use, its refusals (on the host, before any CUDA call, with fake addresses that no
accepted call is made with), and on the GPU that nothing is written behind it."""
import pytest
import torch

from gpu_util import TOL, assert_close
from selective_state_space_18_b200 import build as ssbuild
from selective_state_space_18_b200 import ssscan
from selective_state_space_18_b200.inputs import make_delta_inputs

BLOCK = 4 * 6144 + 4 * 256  # T and P in two parts each, and four arrays of 64 floats, per chunk and head
P = [0x7f0000000000 + i * 0x100000000 for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    ssbuild.build()
    return ssscan.load_library()


def _two_pass(heads, segments, dk, dv):
    """N of all segments but the last, M of those between the first and the last, a copy of h0,
    and a flag for each M, beside the blocks."""
    return heads * 4 * (dk * ((segments - 1) * dv + (segments - 2) * dk) + dk * dv + segments - 2)


@pytest.mark.parametrize("batch,seq,hk,hv,dk,dv,segments", [
    (2, 130, 2, 4, 128, 64, 1), (8, 2048, 16, 32, 128, 128, 1), (1, 17, 1, 1, 16, 8, 1), (1, 35 * 64, 1, 1, 64, 64, 1),
    (1, 36 * 64, 1, 1, 64, 64, 3), (1, 16384, 16, 32, 128, 128, 6), (1, 16384, 1, 1, 128, 128, 21),
    (1, 16384, 1, 8, 128, 256, 12), (3, 6000, 4, 12, 96, 64, 5)])
def test_sizes(lib, batch, seq, hk, hv, dk, dv, segments):
    heads, chunks = batch * hv, (seq + 63) // 64
    need = heads * chunks * BLOCK + (_two_pass(heads, segments, dk, dv) if segments > 1 else 0)
    assert lib.ss_delta_workspace_bytes(batch, seq, hk, hv, dk, dv, 1) == need
    assert ssscan.ss_delta_workspace_bytes(batch, seq, hk, hv, dk, dv) == need


def test_no_workspace_where_the_token_form_runs(lib):
    for seq, dk, dv, dtype in ((16, 128, 128, 1), (2048, 128, 128, 0), (2048, 100, 128, 1), (2048, 128, 100, 1),
                               (2048, 136, 128, 1), (2048, 8, 128, 1)):
        assert lib.ss_delta_workspace_bytes(1, seq, 2, 4, dk, dv, dtype) == 0


@pytest.mark.parametrize("seq", [256, 4096])
def test_refusals(lib, seq):
    need = lib.ss_delta_workspace_bytes(2, seq, 2, 4, 128, 128, 1)
    assert need > 0

    def call(ws, nbytes):
        return lib.ss_delta_scan(2, seq, 2, 4, 128, 128, 1, P[0], 256, P[1], 256, P[2], 512, P[3], P[4], None, P[7], 1.0,
                                 0, P[5], P[6], ws, nbytes, None)

    assert call(P[8], need - 1) == 9 and call(P[8], 0) == 9
    assert call(P[8] + 8, need) == 4
    for i in (0, 1, 2, 3, 4, 5, 6, 7):                # inputs, outputs, both states
        assert call(P[i], need) == 8, i
        assert call(P[i] - need + 16, need) == 8, i


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 2305, 1, 2, 128, 128), (1, 3000, 2, 4, 72, 200), (2, 300, 2, 4, 128, 128)])
def test_nothing_is_written_behind_it(orc, shape):
    """A workspace of exactly the size, filled with NaN before and followed by guard bytes; the
    final state takes h0's place, so that the copy of h0 is used as well."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    inp = make_delta_inputs(*shape, "bf16", seed=3700, h0=True)
    inp["g"] = inp["g"] * 1e-2
    ref = orc.delta_scan(**inp, scale=1.0, qk_l2norm=True)
    d = {k: (None if v is None else v.cuda()) for k, v in inp.items()}
    need = ssscan.ss_delta_workspace_bytes(*shape)
    buf = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device="cuda")
    out = ssscan.ss_delta_scan(**d, scale=1.0, qk_l2norm=True, final_state=d["h0"], workspace=buf[:need])
    assert ssscan.ss_debug_status() == "SS_OK"
    assert bool((buf[need:] == 0xff).all())
    assert_close(out["outputs"].cpu(), ref["outputs"], TOL[torch.bfloat16], "outputs")
    assert_close(d["h0"].cpu(), ref["final_state"], TOL[torch.float32], "final state")
