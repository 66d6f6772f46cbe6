"""Host-only checks of the served forms' and the norm's C ABI (no GPU needed): bad arguments are
refused before anything is launched, and the workspace queries follow the plan."""
import ctypes

import pytest
import torch

import mamba_ssd_scan_03_b200 as ssd
from mamba_ssd_scan_03_b200 import build as ssd_build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load()


def test_status_string_of_a_bad_index(lib):
    assert lib.ssd_status_string(6).decode().startswith(ssd.STATUS[6])


def _conv(lib, **kw):
    a = dict(u=None, us=64, w=None, bias=None, cu=None, state=None, slots=None, resume=None,
             out=None, os=64, ntok=10, nseq=2, nslots=0, cdim=64, K=4, io=1, stream=None)
    a.update(kw)
    return lib.ssd_conv_silu_varlen(*a.values())


@pytest.mark.parametrize("bad", [
    dict(ntok=-1), dict(nseq=-1), dict(cdim=0), dict(K=0), dict(K=9), dict(io=2), dict(us=63),
    dict(os=63), dict(nslots=-1), dict(slots=256), dict(resume=256),
    dict(state=256, K=1, nslots=2),       # a history of no rows
    dict(state=256, nslots=1),            # fewer slots than sequences, no slots given
    dict(state=256, nslots=1 << 32),
    dict(),                               # NULL pointers
])
def test_conv_varlen_refuses(lib, bad):
    assert _conv(lib, **bad) == INVALID


def test_conv_with_nothing_to_do(lib):
    assert _conv(lib, nseq=0) == 0


def _conv_step(lib, **kw):
    a = dict(state=256, u=None, us=64, w=None, bias=None, slots=None, out=None, os=64, batch=2,
             nslots=2, cdim=64, K=4, io=1, stream=None)
    a.update(kw)
    return lib.ssd_conv_silu_step(*a.values())


@pytest.mark.parametrize("bad", [dict(state=None), dict(batch=-1), dict(K=1), dict(K=9),
                                 dict(nslots=1), dict(us=1), dict(io=-1), dict()])
def test_conv_step_refuses(lib, bad):
    assert _conv_step(lib, **bad) == INVALID


def _args(**kw):
    a = ssd.SelectiveArgs()
    base = dict(x_stride=64, dt_stride=64, b_stride=16, c_stride=16, z_stride=64, y_stride=64,
                nslots=0, dim=64, dstate=16, ngroups=1, io=1, dt_dtype=0, y_dtype=0, softplus=1)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


BAD_ARGS = [dict(dim=0), dict(dstate=0), dict(ngroups=0), dict(ngroups=3), dict(io=5),
            dict(io=0, dt_dtype=1), dict(io=0, y_dtype=1), dict(dt_dtype=4), dict(x_stride=63),
            dict(dt_stride=0), dict(y_stride=-64), dict(b_stride=15), dict(c_stride=15),
            dict(z=256, z_stride=63), dict(nslots=-1), dict(slots=256),
            dict(state=256, nslots=1), dict()]


@pytest.mark.parametrize("bad", BAD_ARGS)
def test_selective_varlen_refuses(lib, bad):
    a = _args(**bad)
    assert lib.ssd_selective_scan_varlen(ctypes.byref(a), 256, None, 10, 2, 0, None, 0,
                                         None) == INVALID


def test_selective_varlen_refuses_its_own(lib):
    call = lib.ssd_selective_scan_varlen
    a = ctypes.byref(_args())
    assert call(None, 256, None, 10, 2, 0, None, 0, None) == INVALID
    assert call(a, None, None, 10, 2, 0, None, 0, None) == INVALID       # no bounds
    assert call(a, 256, None, -1, 2, 0, None, 0, None) == INVALID
    assert call(a, 256, None, 10, -1, 0, None, 0, None) == INVALID
    assert call(a, 256, None, 10, 2, -1, None, 0, None) == INVALID
    assert call(a, 256, 256, 10, 2, 0, None, 0, None) == INVALID         # resume without state
    # a plan in chunks needs its workspace, aligned and large enough
    need = lib.ssd_selective_varlen_workspace_size(4096, 1, 64, 16, 1, 0)
    assert need > 0 and need % 256 == 0
    assert call(a, 256, None, 4096, 1, 0, None, 0, None) == WORKSPACE
    assert call(a, 256, None, 4096, 1, 0, 256, need - 1, None) == WORKSPACE
    assert call(a, 256, None, 4096, 1, 0, 300, need, None) == WORKSPACE


def test_selective_varlen_workspace(lib):
    size = lib.ssd_selective_varlen_workspace_size
    assert size(4096, 64, 5120, 16, 1, 0) == 0        # enough sequences and channels
    assert size(50, 1, 64, 16, 1, 0) == 0             # too short to cut
    for bad in ((-1, 1, 64, 16, 1, 0), (10, 0, 64, 16, 1, 0), (10, 1, 64, 129, 1, 0),
                (10, 1, 64, 16, 3, 0), (10, 1, 64, 16, 1, -1)):
        assert size(*bad) == 0


@pytest.mark.parametrize("bad", BAD_ARGS + [dict(state=256, nslots=2, dstate=0)])
def test_selective_step_refuses(lib, bad):
    a = _args(**bad)
    assert lib.ssd_selective_step(ctypes.byref(a), 2, None) == INVALID


def _norm(lib, **kw):
    a = dict(y=None, ys=64, w=None, b=None, z=None, zs=0, out=None, os=64, rows=3, cdim=64,
             groups=2, eps=1e-5, center=0, first=1, yd=0, zd=0, od=0, stream=None)
    a.update(kw)
    return lib.ssd_group_norm_gate(*a.values())


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(cdim=0), dict(groups=0), dict(groups=5), dict(eps=-1e-9),
    dict(eps=float("nan")), dict(ys=63), dict(os=1), dict(z=256, zs=63), dict(z=256, zs=64, zd=2),
    dict(yd=-1), dict(od=2), dict()])
def test_norm_refuses(lib, bad):
    assert _norm(lib, **bad) == INVALID


def test_norm_of_no_rows(lib):
    assert _norm(lib, rows=0) == 0


def _norm_bwd(lib, **kw):
    a = dict(dout=None, ds=64, y=None, ys=64, w=None, b=None, z=None, zs=0, dy=None, dz=None,
             dw=None, db=None, rows=3, cdim=64, groups=2, eps=1e-5, center=0, first=1, dd=0, yd=0,
             zd=0, ws=256, bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.ssd_group_norm_gate_bwd(*a.values())


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(groups=7), dict(eps=-1.0), dict(ds=63), dict(ys=63), dict(dd=3),
    dict(b=256), dict(db=256), dict(z=256, zs=64), dict(dz=256), dict()])
def test_norm_bwd_refuses(lib, bad):
    assert _norm_bwd(lib, **bad) == INVALID


def test_norm_bwd_workspace(lib):
    size = lib.ssd_group_norm_gate_bwd_workspace_size
    need = size(3, 64, 2)
    assert need > 0 and need % 256 == 0
    assert size(0, 64, 2) == 0 and size(3, 64, 5) == 0
    assert _norm_bwd(lib, ws=None) == WORKSPACE
    assert _norm_bwd(lib, bytes=need - 1) == WORKSPACE
    assert _norm_bwd(lib, ws=264) == WORKSPACE


def test_binding_refuses_on_the_host(lib):
    x, w = torch.zeros(4, 8), torch.zeros(8, 4)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ssd.conv_silu_varlen(x, w, cu)
    with pytest.raises(ValueError):
        ssd.conv_silu_step(torch.zeros(4, 3, 8), x, w)
    with pytest.raises(ValueError):
        ssd.selective_scan_varlen(x, x, torch.zeros(8, 16), torch.zeros(4, 1, 16),
                                  torch.zeros(4, 1, 16), cu)
    with pytest.raises(ValueError):
        ssd.selective_step(torch.zeros(4, 8, 16), x, x, torch.zeros(8, 16),
                           torch.zeros(4, 1, 16), torch.zeros(4, 1, 16))
    with pytest.raises(ValueError):
        ssd.group_norm_gate(x, torch.zeros(8))
    with pytest.raises(ValueError):
        ssd.group_norm_gate_bwd(x, x, torch.zeros(8))
    with pytest.raises(TypeError):
        ssd.group_norm_gate([1.0], torch.zeros(8))
