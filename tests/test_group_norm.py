"""ss_group_norm on the GPU against the float64 oracle: every form, group sizes from one
element to the largest (each team of lanes), unaligned rows and strided views.

Tolerance: float32 sums of at most 16384 terms in trees of 32 lanes (under 100 roundings
in a row, 6e-6 of the sum at most), SiLU through a 2-ulp exponential and division: 2e-5
(1 + |ref|).  bfloat16: half a step, 2^-8 |ref|, on top."""
import pytest
import torch

from gpu_util import assert_close
from selective_state_space_18_b200 import ssscan

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOLS = {torch.bfloat16: 2.0 ** -8 + 2e-5, torch.float32: 2e-5}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def _inputs(rows, ch, n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, ch, generator=g) + 0.3).to(DT[dtype])
    z = torch.randn(rows, ch, generator=g).to(DT[dtype])
    return x, z, 1 + 0.2 * torch.randn(n, generator=g), 0.2 * torch.randn(n, generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", [dict(), dict(center=False), dict(activation="silu"), dict(gate=True),
                                  dict(gate=True, gate_first=True), dict(gate=True, activation="silu", center=False),
                                  dict(bare=True), dict(shared=True, gate=True), dict(bias=False, eps=0.0)])
@pytest.mark.parametrize("size", [128, 24, 7])
def test_forms(orc, dtype, form, size):
    form = dict(form)
    groups, rows = 5, 37
    shared, bare, bias = form.pop("shared", False), form.pop("bare", False), form.pop("bias", True)
    x, z, w, b = _inputs(rows, groups * size, size if shared else groups * size, dtype, 4000 + size)
    w, b = (None, None) if bare else (w, b if bias else None)
    if form.pop("gate", False):
        form["gate"] = z
    ref = orc.group_norm(x, groups, w, b, **form)
    if "gate" in form:
        form["gate"] = z.cuda()
    y = ssscan.ss_group_norm(x.cuda(), groups, None if w is None else w.cuda(), None if b is None else b.cuda(), **form)
    assert y.dtype == x.dtype and y.shape == x.shape
    assert_close(y.cpu(), ref, TOLS[x.dtype], f"{form.keys()}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1, 2, 8, 31, 64, 100, 257, 512, 640, 1000, 1024, 1025, 2048, 2056, 4097, 5120, 8192,
                                  16383, 16384])
def test_sizes(orc, dtype, size):
    """One element up to the largest group; a group of one is its bias when centred."""
    for rows, groups in ((3, 2), (1, 1)):
        x, z, w, b = _inputs(rows, groups * size, groups * size, dtype, 4100 + size)
        y = ssscan.ss_group_norm(x.cuda(), groups, w.cuda(), b.cuda(), gate=z.cuda(), eps=1e-3)
        assert_close(y.cpu(), orc.group_norm(x, groups, w, b, gate=z, eps=1e-3), TOLS[x.dtype], f"{rows} {groups}")
    if size > 1:
        y = ssscan.ss_group_norm(x.cuda(), 1, center=False, eps=1e-3)
        assert_close(y.cpu(), orc.group_norm(x, 1, center=False, eps=1e-3), TOLS[x.dtype], "no mean")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_and_odd_addresses(orc, dtype):
    """Column slices (a row stride of their own), a transposed view (copied), an address
    that no vector load takes; nothing beside the output is written."""
    x, z, w, b = _inputs(21, 3 * 64, 64, dtype, 4200)
    wide = torch.randn(21, 400).to(x.dtype)
    wide[:, 100:292] = x
    ref = orc.group_norm(x, 3, w, b, gate=z)
    dw, db, dz = w.cuda(), b.cuda(), z.cuda()
    cases = [wide.cuda()[:, 100:292], x.t().contiguous().cuda().t(), x.cuda()]
    odd = torch.empty(21 * 192 + 1, dtype=x.dtype, device="cuda")
    cases.append(odd[1:].view(21, 192).copy_(x.cuda()))
    for c in cases:
        assert_close(ssscan.ss_group_norm(c, 3, dw, db, gate=dz).cpu(), ref, TOLS[x.dtype], "view")
    buf = torch.full((21 * 192 + 32,), 9.0, dtype=x.dtype, device="cuda")
    y = buf[16:-16].view(21, 192)
    assert ssscan.ss_group_norm(cases[0], 3, dw, db, gate=dz, y=y) is y
    assert_close(y.cpu(), ref, TOLS[x.dtype], "supplied output")
    assert bool((buf[:16] == 9).all()) and bool((buf[-16:] == 9).all())
    h = x.view(3, 7, 192)
    assert_close(ssscan.ss_group_norm(h.cuda(), 3, dw, db, gate=dz.view(3, 7, 192)).cpu(),
                 ref.reshape(3, 7, 192), TOLS[x.dtype], "three dimensions")


def test_extremes(orc):
    """Equal values (no variance), values near the largest bfloat16's square root, gates
    far out on both sides, and a row of NaN that stays in its row."""
    x = torch.full((4, 256), 3.0)
    x[1] = 1e18
    x[1, ::2] = -1e18
    x[2] = torch.linspace(-1e-3, 1e-3, 256)
    x[3] = float("nan")
    z = torch.full((4, 256), 200.0)
    z[:, ::2] = -200.0
    y = ssscan.ss_group_norm(x.cuda(), 2, gate=z.cuda(), eps=1e-6).cpu()
    ref = orc.group_norm(x[:3], 2, gate=z[:3], eps=1e-6)
    assert_close(y[:3], ref, 2e-5, "extremes")
    assert bool(torch.isnan(y[3]).all())


def test_many_rows_and_stream(orc):
    """More groups than teams in one wave, on a side stream; sampled rows."""
    x, z, w, b = _inputs(20011, 256, 256, "bf16", 4300)
    side = torch.cuda.Stream()
    dx, dw, db = x.cuda(), w.cuda(), b.cuda()
    side.wait_stream(torch.cuda.current_stream())
    y = ssscan.ss_group_norm(dx, 8, dw, db, activation="silu", stream=side)
    side.synchronize()
    rows = [0, 1, 9999, 20009, 20010]
    assert_close(y[rows].cpu(), orc.group_norm(x[rows], 8, w, b, activation="silu"), TOLS[x.dtype], "rows")


def test_refusals():
    x = torch.randn(4, 64, device="cuda")
    for kw in (dict(groups=3), dict(groups=0), dict(groups=2, weight=torch.ones(16, device="cuda")),
               dict(groups=2, weight=torch.ones(64, device="cuda"), bias=torch.ones(32, device="cuda")),
               dict(groups=2, gate=torch.ones(4, 32, device="cuda")), dict(groups=2, activation="gelu")):
        with pytest.raises(ValueError):
            ssscan.ss_group_norm(x, **kw)
    with pytest.raises(ssscan.SSError):
        ssscan.ss_group_norm(torch.randn(1, 20000, device="cuda"), 1)
    with pytest.raises(ssscan.SSError):
        ssscan.ss_group_norm(x, 2, eps=-1.0)
    with pytest.raises(ssscan.SSError):
        ssscan.ss_group_norm(x, 2, y=x)
