"""The gated delta rule's and the group norm's refusals, on the host before any CUDA call.
Pointers are fake addresses that no accepted call is made with."""
import ctypes

import pytest
import torch

from selective_state_space_18_b200 import build as ssbuild
from selective_state_space_18_b200 import ssscan


@pytest.fixture(scope="module")
def lib():
    ssbuild.build()
    return ssscan.load_library()


P = [0x7f0000000000 + i * 0x100000000 for i in range(12)]
BIG = 1 << 40


def _scan(lib, **kw):
    a = dict(batch=2, seq=32, hk=2, hv=4, dk=64, dv=32, dtype=1, q=P[0], qs=128, k=P[1], ks=128, v=P[2], vs=128,
             g=P[3], beta=P[4], reset=None, h0=None, scale=1.0, flags=0, y=P[5], fs=P[6], ws=None, wsb=0)
    a.update(kw)
    return lib.ss_delta_scan(*(a[n] for n in ("batch", "seq", "hk", "hv", "dk", "dv", "dtype", "q", "qs", "k", "ks",
                                              "v", "vs", "g", "beta", "reset", "h0", "scale", "flags", "y", "fs", "ws",
                                              "wsb")), None)


def _update(lib, **kw):
    a = dict(batch=2, hk=2, hv=4, dk=64, dv=32, dtype=1, state=P[6], q=P[0], qs=128, k=P[1], ks=128, v=P[2], vs=128,
             g=P[3], beta=P[4], scale=1.0, flags=0, y=P[5])
    a.update(kw)
    return lib.ss_delta_update(*(a[n] for n in ("batch", "hk", "hv", "dk", "dv", "dtype", "state", "q", "qs", "k",
                                                "ks", "v", "vs", "g", "beta", "scale", "flags", "y")), None)


def _norm(lib, **kw):
    a = dict(rows=4, groups=2, size=64, dtype=1, x=P[0], xs=128, gate=P[1], zs=128, w=P[2], b=P[3], eps=1e-5, flags=0,
             y=P[4])
    a.update(kw)
    return lib.ss_group_norm(*(a[n] for n in ("rows", "groups", "size", "dtype", "x", "xs", "gate", "zs", "w", "b",
                                              "eps", "flags", "y")), None)


@pytest.mark.parametrize("call,names", [(_scan, "q k v y"), (_update, "state q k v y"), (_norm, "x y")])
def test_null_pointers(lib, call, names):
    for n in names.split():
        assert call(lib, **{n: None}) == 1, n


@pytest.mark.parametrize("call,names", [(_scan, "batch seq hk hv dk dv"), (_update, "batch hk hv dk dv"),
                                        (_norm, "rows groups size")])
def test_sizes(lib, call, names):
    for n in names.split():
        for value in (0, -1):
            assert call(lib, **{n: value}) == 2, n


@pytest.mark.parametrize("call", [_scan, _update])
def test_delta_shapes(lib, call):
    assert call(lib, hv=3) == 2                       # not a multiple of the key heads
    assert call(lib, qs=127) == 2 and call(lib, ks=0) == 2 and call(lib, vs=-128) == 2  # rows overlap
    assert call(lib, batch=BIG << 10) == 2 and call(lib, qs=BIG << 19) == 2
    assert call(lib, dk=257, qs=1024, ks=1024) == 5
    assert call(lib, dtype=2) == 3
    assert call(lib, flags=1) == 5 and call(lib, flags=8) == 5


@pytest.mark.parametrize("call", [_scan, _update])
def test_delta_alignment_and_overlap(lib, call):
    for n, off in (("q", 1), ("k", 1), ("v", 1), ("y", 1), ("g", 2), ("beta", 2)):
        base = {"q": P[0], "k": P[1], "v": P[2], "y": P[5], "g": P[3], "beta": P[4]}[n]
        assert call(lib, **{n: base + off}) == 4, n
    for n in ("q", "k", "v", "g", "beta"):
        base = {"q": P[0], "k": P[1], "v": P[2], "g": P[3], "beta": P[4]}[n]
        assert call(lib, y=base + 16) == 8, n
    assert call(lib, y=P[6]) == 8                     # the state


def test_scan_buffers(lib):
    assert _scan(lib, h0=P[7] + 2) == 4 and _scan(lib, fs=P[6] + 2) == 4
    assert _scan(lib, h0=P[6] + 4) == 8               # overlaps the final state without being it
    assert _scan(lib, reset=P[5]) == 8
    assert _scan(lib, fs=P[0]) == 8
    big = dict(seq=4096, dk=128, dv=128, qs=256, ks=256, vs=512)
    need = lib.ss_delta_workspace_bytes(2, 4096, 2, 4, 128, 128, 1)
    assert need >= 0
    if need:
        assert _scan(lib, ws=P[8], wsb=need - 1, **big) == 9
        assert _scan(lib, ws=P[8] + 8, wsb=need, **big) == 4
        assert _scan(lib, ws=P[5], wsb=need, **big) == 8
        assert _scan(lib, ws=P[0] - need + 16, wsb=need, **big) == 8
    for bad in ((0, 1, 1, 1, 8, 8, 1), (1, 1, 2, 3, 8, 8, 1), (1, 1, 1, 1, 300, 8, 1), (BIG, BIG, 1, 1, 8, 8, 1),
                (1, 1, 1, 1, 8, 8, 9)):
        assert lib.ss_delta_workspace_bytes(*bad) == 0


def test_norm_refusals(lib):
    assert _norm(lib, dtype=5) == 3
    assert _norm(lib, size=16385, xs=1 << 20, zs=1 << 20) == 5
    assert _norm(lib, flags=16) == 5
    assert _norm(lib, eps=-1.0) == 5 and _norm(lib, eps=float("nan")) == 5
    assert _norm(lib, xs=127) == 2 and _norm(lib, zs=127) == 2
    assert _norm(lib, rows=BIG, xs=BIG) == 2
    assert _norm(lib, x=P[0] + 1) == 4 and _norm(lib, gate=P[1] + 1) == 4 and _norm(lib, w=P[2] + 1) == 4
    assert _norm(lib, y=P[0] + 2) == 8 and _norm(lib, y=P[1]) == 8 and _norm(lib, y=P[2] + 4) == 8


def test_binding_refuses():
    q, v = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 4, 8)
    with pytest.raises(ValueError):
        ssscan.ss_delta_scan(q, q, v)
    with pytest.raises(ValueError):
        ssscan.ss_delta_update(torch.zeros(1, 4, 8, 8), q[:, 0], q[:, 0], v[:, 0])
    with pytest.raises(ValueError):
        ssscan.ss_group_norm(torch.zeros(4, 8), 2)


def test_row_views_are_recognised():
    """Slices of one projection are read in place; other views are copied."""
    qkv = torch.arange(2 * 3 * 40.0).view(2, 3, 40)
    k = qkv[..., 8:24].unflatten(-1, (2, 8))
    t, step = ssscan._rows_of(k, "k", -1, torch.float32, (2, 3, 2, 8))
    assert step == 40 and t.data_ptr() == k.data_ptr()
    assert ssscan._rows_of(k[:, :1], "k", -1, torch.float32, (2, 1, 2, 8))[1] == 120
    assert ssscan._rows_of(k[1:, :1], "k", -1, torch.float32, (1, 1, 2, 8))[1] == 16
    for bad in (k[:, ::2], k.transpose(0, 1), k[..., ::2], k[:, :, ::2], k[:1].expand(2, -1, -1, -1)):
        t, step = ssscan._rows_of(bad, "k", -1, torch.float32, bad.shape)
        assert torch.equal(t, bad)
        rows = t.as_strided((bad.shape[0] * bad.shape[1], bad.shape[2] * bad.shape[3]), (step, 1), t.storage_offset())
        assert torch.equal(rows, bad.reshape(rows.shape))
