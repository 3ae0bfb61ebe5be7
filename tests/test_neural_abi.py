"""The neural decoder's entry points refuse bad arguments on the host, before anything reaches the GPU
(these calls never touch a device), and their workspace queries follow the sizes."""
import ctypes
import os

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 3
P = 1 << 20  # a 256-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def gs():
    from differentiable_raster_amd import gsmi
    if not os.path.exists(gsmi.LIB_PATH):
        from differentiable_raster_amd import build
        build.build()
    gsmi.load()
    return gsmi


def lin(gs, rows=10, n_in=16, out=24, type=1, y_type=1, grad_type=1, act=0, cm=0, ld_x=0, ld_w=0, ld_y=0, ld_r=0):
    return gs.gs_linear_desc(rows, n_in, out, type, y_type, grad_type, act, cm, ld_x, ld_w, ld_y, ld_r)


def norm(gs, rows=10, width=16, type=1, eps=1e-6, ld_x=0, ld_r=0, ld_s=0, ld_y=0):
    return gs.gs_norm_desc(rows, width, type, eps, ld_x, ld_r, ld_s, ld_y)


def linear(gs, d, x=P, sx=None, w=P, sw=None, b=None, r=None, y=P, ws=P, n=1 << 30):
    return gs.load().gs_linear(ctypes.byref(d), x, sx, w, sw, b, r, y, ws, n, None)


def linear_bwd(gs, d, x=P, w=P, b=None, dy=P, dx=P, dw=P, db=None, ws=P, n=1 << 30, name="gs_linear_bwd"):
    return getattr(gs.load(), name)(ctypes.byref(d), x, w, b, dy, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("field", [dict(rows=-1), dict(n_in=0), dict(out=0), dict(n_in=1 << 21), dict(type=0), dict(type=9),
                                   dict(y_type=3), dict(act=4), dict(act=-1), dict(cm=2), dict(ld_x=15), dict(ld_w=8),
                                   dict(ld_y=23), dict(ld_r=23), dict(ld_x=1 << 21), dict(cm=1, ld_y=9)])
def test_linear_refuses_descriptors(gs, field):
    d = lin(gs, **field)
    assert linear(gs, d) == INVALID
    assert gs.load().gs_last_error()
    assert gs.gs_linear_workspace_size(d) == 0
    if "ld_r" in field:
        return  # the backward's ld_r is dx's stride (in = 16): see test_backward_refuses_arguments
    assert linear_bwd(gs, d) == INVALID
    assert gs.gs_linear_bwd_workspace_size(d) == 0


def test_linear_refuses_arguments(gs):
    d = lin(gs)
    assert gs.load().gs_linear(None, P, None, P, None, None, None, P, None, 0, None) == INVALID
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(x=P + 2), dict(w=P + 8), dict(y=P + 1), dict(b=P + 2),
                dict(r=P + 1), dict(sx=P), dict(sw=P), dict(sx=P, sw=P)):
        assert linear(gs, d, **bad) == INVALID, bad
    eight = lin(gs, type=3)
    for bad in (dict(), dict(sx=P), dict(sw=P)):
        assert linear(gs, eight, **bad) == INVALID, bad
    # 100 rows of 17 values need an operand copy: a workspace, large and aligned enough
    odd = lin(gs, rows=100, n_in=17)
    need = gs.gs_linear_workspace_size(odd)
    assert need >= 124 * 24 * 2
    for bad in (dict(ws=None), dict(n=need - 1), dict(ws=P + 128)):
        assert linear(gs, odd, **bad) == INVALID, bad
    assert linear(gs, lin(gs, rows=0), x=None, y=None) == OK


def test_backward_refuses_arguments(gs):
    assert linear_bwd(gs, lin(gs, type=3)) == UNSUPPORTED
    assert linear_bwd(gs, lin(gs, grad_type=2)) == INVALID
    assert linear_bwd(gs, lin(gs, ld_r=15)) == INVALID
    d = lin(gs)
    for bad in (dict(x=None), dict(w=None), dict(dy=None), dict(x=P + 2), dict(w=P + 4), dict(dy=P + 8), dict(dx=P + 1),
                dict(dw=P + 1), dict(db=P + 2), dict(ws=None), dict(n=0), dict(ws=P + 16)):
        for name in ("gs_linear_bwd", "gs_gated_bwd"):
            assert linear_bwd(gs, d, name=name, **bad) == INVALID, (name, bad)


def test_gated_refuses_arguments(gs):
    call = lambda d, **k: gs.load().gs_gated(ctypes.byref(d), k.get("x", P), None, P, None, None, k.get("h", P), P, 1 << 30, None)  # noqa: E731
    assert call(lin(gs, cm=1)) == INVALID
    assert call(lin(gs), x=None) == INVALID
    assert call(lin(gs), h=P + 1) == INVALID
    assert call(lin(gs, out=1 << 20, n_in=512)) == UNSUPPORTED
    assert call(lin(gs, rows=0)) == OK


def test_norm_refuses_arguments(gs):
    lib = gs.load()

    def fwd(d, x=P, r=None, w=None, s=P, y=P, q=None, qs=None):
        return lib.gs_rmsnorm(ctypes.byref(d), x, r, w, s, y, q, qs, None)

    for bad in (dict(rows=-1), dict(width=0), dict(width=32769), dict(type=3), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(ld_x=15), dict(ld_r=3), dict(ld_s=-4), dict(ld_y=8)):
        d = norm(gs, **bad)
        assert fwd(d) == INVALID, bad
        assert lib.gs_quantize_rows(ctypes.byref(d), P, P, P, None) == INVALID, bad
        assert lib.gs_rmsnorm_bwd(ctypes.byref(d), P, None, P, None, P, P, P, 1 << 30, None) == INVALID, bad
        assert gs.gs_rmsnorm_bwd_workspace_size(d) == 0
    d = norm(gs)
    for bad in (dict(x=None), dict(s=None, y=None), dict(q=P), dict(qs=P), dict(x=P + 1), dict(r=P + 1), dict(w=P + 2), dict(y=P + 1)):
        assert fwd(d, **bad) == INVALID, bad
    assert fwd(norm(gs, rows=0), x=None, s=None, y=None) == OK
    assert lib.gs_quantize_rows(ctypes.byref(d), P, None, P, None) == INVALID
    for bad in ((None, P, P, P), (P, None, P, P), (P, P, None, P), (P, P, P, None)):
        s, dy, dx, ws = bad
        assert lib.gs_rmsnorm_bwd(ctypes.byref(d), s, None, dy, None, dx, P, ws, 1 << 30, None) == INVALID, bad


def test_workspace_queries(gs):
    assert gs.gs_linear_workspace_size(lin(gs, rows=1000, n_in=64, out=64)) == 0  # nothing to copy or join
    assert gs.gs_linear_workspace_size(lin(gs, rows=1000, n_in=63, out=64)) > 1000 * 64 * 2
    assert gs.gs_gated_bwd_workspace_size(lin(gs, rows=1000, n_in=64, out=128)) >= 1000 * 256 * 2
    assert gs.gs_rmsnorm_bwd_workspace_size(norm(gs, rows=1000, width=64)) > 0


def test_python_plans_refuse_tensors(gs):
    torch = pytest.importorskip("torch")
    from differentiable_raster_amd import neural
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="expected torch.bfloat16"):
        neural._rows(torch.zeros(4, 8), "x", 4, 8, bf)
    with pytest.raises(ValueError, match=r"\[4, 9\]"):
        neural._rows(torch.zeros(4, 8, dtype=bf), "x", 4, 9, bf)
    with pytest.raises(ValueError, match="device tensor"):
        neural._rows(torch.zeros(4, 8, dtype=bf), "x", 4, 8, bf)
    with pytest.raises(ValueError, match="float32"):
        neural._vector(torch.zeros(4, dtype=bf), "bias", 4)
    with pytest.raises(ValueError, match=r"\[5\]"):
        neural._vector(torch.zeros(4), "bias", 5)
    with pytest.raises(KeyError):
        neural.ACTS["tanh"]
