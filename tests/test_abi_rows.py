"""Host-side checks of the norm, the routing and the combination of rows: bad
arguments are refused with a status and a message before any GPU call, empty
work is fine without one, and the workspace queries agree with the calls.  No
kernel runs."""
import ctypes
import os

import pytest

FAKE = 0x100000  # never dereferenced: every call below fails validation first
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    import sparse_ternary_bit_amd as stq
    if not os.path.exists(stq.lib_path()):
        from sparse_ternary_bit_amd import build
        build.build(verbose=False)
    return stq.lib()


def _refused(L, name, args, kw, status):
    a = dict(args)
    a.update(kw)
    assert getattr(L, name)(*a.values(), None) == status
    assert L.stq_last_error().decode().startswith(name)


def _done(L, name, args, kw):
    a = dict(args)
    a.update(kw)
    assert getattr(L, name)(*a.values(), None) == 0


NORM = dict(x=FAKE, xd=BF16, xs=100, r=FAKE, rd=F32, rs=100, h=FAKE + 4096, hs=100, w=FAKE, eps=1e-6, n=4, d=100, rstd=FAKE, q=FAKE,
            qs=112, sc=FAKE, y=FAKE, ys=100)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), 1), (dict(d=0), 2), (dict(d=(1 << 26) + 1), 2), (dict(n=(1 << 22) + 1), 2), (dict(xd=2), 1), (dict(rd=5), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(q=None), 1), (dict(sc=None), 1), (dict(x=None), 1), (dict(w=None), 1),
    (dict(h=None), 1), (dict(qs=96), 2), (dict(qs=120), 3), (dict(q=FAKE + 8), 3), (dict(w=FAKE + 2), 3), (dict(rstd=FAKE + 1), 3),
    (dict(sc=FAKE + 2), 3), (dict(xs=99), 2), (dict(rs=99), 2), (dict(hs=99), 2), (dict(ys=99), 2), (dict(xs=1 << 62), 2),
    (dict(x=FAKE + 1), 3), (dict(r=FAKE + 2), 3), (dict(h=FAKE + 2), 3), (dict(y=FAKE + 1), 3), (dict(h=FAKE, hs=104), 1),
    (dict(h=FAKE, r=FAKE + 8192), 1), (dict(h=FAKE, r=FAKE + 8192, xd=F32, xs=104), 1),
])
def test_norm_refusals(L, kw, status):
    _refused(L, "stq_rmsnorm_rows", NORM, kw, status)


def test_norm_nothing_to_do(L):
    _done(L, "stq_rmsnorm_rows", NORM, dict(n=0, x=None, r=None, h=None, w=None, q=None, sc=None, y=None, rstd=None))


NORM_BWD = dict(h=FAKE, hd=BF16, hs=100, w=FAKE, rstd=FAKE, dy=FAKE, yd=F32, ys=100, dh=FAKE, dhs=100, dx=FAKE + 4096, dxs=100,
                dw=FAKE, n=4, d=100, ws=FAKE, wsb=1 << 40)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), 1), (dict(d=0), 2), (dict(hd=3), 1), (dict(yd=3), 1), (dict(h=None), 1), (dict(w=None), 1), (dict(rstd=None), 1),
    (dict(dy=None), 1), (dict(w=FAKE + 2), 3), (dict(dw=FAKE + 2), 3), (dict(hs=99), 2), (dict(ys=99), 2), (dict(dhs=99), 2),
    (dict(dxs=99), 2), (dict(dh=FAKE + 1), 3), (dict(dx=FAKE + 1), 3), (dict(dy=FAKE + 2), 3), (dict(wsb=-1), 1),
    (dict(dx=FAKE + 64, dh=FAKE + 64, dxs=104), 1), (dict(dx=FAKE), 1), (dict(dx=FAKE, dh=None, hd=F32, dxs=104), 1),
])
def test_norm_backward_refusals(L, kw, status):
    _refused(L, "stq_rmsnorm_rows_backward", NORM_BWD, kw, status)


def test_norm_backward_workspace(L):
    need = ctypes.c_int64()
    query = L.stq_rmsnorm_rows_backward_workspace
    assert query(300, 100, 1, 256, ctypes.byref(need)) == 0 and need.value == 300 * 100 * 4
    assert query(5000, 7168, 1, 256, ctypes.byref(need)) == 0 and need.value == 512 * 7168 * 4
    for args in [(4, 100, 0), (0, 100, 1), (256, 100, 1), (300, 100, 0)]:
        assert query(*args, 256, ctypes.byref(need)) == 0 and need.value == 0
    assert query(4, 0, 1, 256, ctypes.byref(need)) == 2
    assert query(4, 100, 1, -1, ctypes.byref(need)) == 1
    assert query(4, 100, 1, 256, None) == 1
    none = dict(h=None, w=None, rstd=None, dy=None, dh=None, ws=None, wsb=0)
    _done(L, "stq_rmsnorm_rows_backward", NORM_BWD, dict(none, dx=None, dw=None))
    _done(L, "stq_rmsnorm_rows_backward", NORM_BWD, dict(none, n=0, dw=None))


ROUTE = dict(x=FAKE, xd=F32, xs=64, n=100, e=64, k=4, renorm=1, pe=FAKE, pw=FAKE, counts=FAKE, off=FAKE, row=FAKE, tok=FAKE, rw=FAKE,
             bal=FAKE, ws=FAKE, wsb=1 << 40)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), 1), (dict(e=0), 2), (dict(e=1025, xs=1025), 2), (dict(k=0), 2), (dict(k=33), 2), (dict(k=5, e=4), 2),
    (dict(n=(1 << 22) + 1), 2), (dict(xd=2), 1), (dict(x=None), 1), (dict(pe=None), 1), (dict(pw=None), 1), (dict(counts=None), 1),
    (dict(off=None), 1), (dict(row=None), 1), (dict(tok=None), 1), (dict(rw=None), 1), (dict(bal=None), 1), (dict(xs=63), 2),
    (dict(xs=1 << 62), 2), (dict(x=FAKE + 2), 3), (dict(xd=BF16, x=FAKE + 1), 3), (dict(pe=FAKE + 1), 3), (dict(bal=FAKE + 2), 3),
    (dict(ws=None), 1), (dict(wsb=8), 1), (dict(wsb=-1), 1), (dict(ws=FAKE + 16), 3),
])
def test_route_refusals(L, kw, status):
    _refused(L, "stq_route_tokens", ROUTE, kw, status)


def test_route_workspace(L):
    need = ctypes.c_int64()
    query = L.stq_route_tokens_workspace
    for n in (0, 1, 64):
        assert query(n, 256, 8, ctypes.byref(need)) == 0 and need.value == 0
    assert query(65, 256, 8, ctypes.byref(need)) == 0 and need.value == 2 * 2 * 256 * 4 + 256 * 4
    assert query(65, 0, 8, ctypes.byref(need)) == 2
    assert query(65, 256, 40, ctypes.byref(need)) == 2
    assert query(-1, 256, 8, ctypes.byref(need)) == 1
    assert query(65, 256, 8, None) == 1


ROUTE_BWD = dict(x=FAKE, xd=F32, xs=64, n=100, e=64, k=4, renorm=1, pe=FAKE, counts=FAKE, gw=FAKE, row=FAKE, gb=FAKE, d=FAKE + 65536, ds=64)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), 1), (dict(e=0), 2), (dict(k=33), 2), (dict(xd=2), 1), (dict(x=None), 1), (dict(d=None), 1), (dict(pe=None), 1),
    (dict(counts=None), 1), (dict(xs=63), 2), (dict(ds=63), 2), (dict(d=FAKE, ds=65), 1), (dict(d=FAKE + 2), 3), (dict(gw=FAKE + 2), 3),
    (dict(gb=FAKE + 1), 3), (dict(row=FAKE + 3), 3),
])
def test_route_backward_refusals(L, kw, status):
    _refused(L, "stq_route_tokens_backward", ROUTE_BWD, kw, status)


COMBINE = dict(z=FAKE, zd=F32, zs=100, rows=80, row=FAKE, w=FAKE, n=10, k=8, d=100, y=FAKE, yd=BF16, ys=100)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 2), (dict(d=0), 2), (dict(k=0), 2), (dict(k=33), 2), (dict(zd=2), 1),
    (dict(yd=2), 1), (dict(z=None), 1), (dict(row=None), 1), (dict(y=None), 1), (dict(zs=99), 2), (dict(ys=99), 2), (dict(zs=1 << 60), 2),
    (dict(z=FAKE + 2), 3), (dict(y=FAKE + 1), 3), (dict(row=FAKE + 1), 3), (dict(w=FAKE + 2), 3),
    (dict(n=1 << 22, d=7168, zs=7168, ys=7168), 2),
])
def test_combine_refusals(L, kw, status):
    _refused(L, "stq_combine_rows", COMBINE, kw, status)


COMBINE_BWD = dict(dy=FAKE, yd=F32, ys=100, z=FAKE, zd=F32, zs=100, rows=80, row=FAKE, w=FAKE, n=10, k=8, d=100, dz=FAKE, dzd=BF16,
                   dzs=100, dw=FAKE)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), 1), (dict(k=0), 2), (dict(yd=2), 1), (dict(zd=2), 1), (dict(dzd=2), 1), (dict(dy=None), 1), (dict(row=None), 1),
    (dict(z=None), 1), (dict(ys=99), 2), (dict(zs=99), 2), (dict(dzs=99), 2), (dict(dw=FAKE + 2), 3), (dict(dz=FAKE + 1), 3),
])
def test_combine_backward_refusals(L, kw, status):
    _refused(L, "stq_combine_rows_backward", COMBINE_BWD, kw, status)


def test_combine_nothing_to_do(L):
    _done(L, "stq_combine_rows", COMBINE, dict(n=0, z=None, row=None, y=None))
    _done(L, "stq_combine_rows_backward", COMBINE_BWD, dict(n=0, z=None, row=None, dy=None))
    _done(L, "stq_combine_rows_backward", COMBINE_BWD, dict(dz=None, dw=None, dy=None, row=None, z=None))


HEAD = dict(x=FAKE, xd=BF16, xs=104, sx=None, w=FAKE, ws=104, sw=None, n=10, v=1000, k=100, t=FAKE, loss=FAKE, lse=FAKE, wsp=FAKE,
            wsb=1 << 40)


@pytest.mark.parametrize("kw, status", [
    (dict(xd=F32), 1), (dict(xd=7), 1), (dict(n=-1), 1), (dict(k=0), 2), (dict(k=131072, xs=131072, ws=131072), 2), (dict(v=0), 2),
    (dict(v=(1 << 26) + 1), 2), (dict(n=(1 << 20) + 1), 2), (dict(n=1 << 20, v=1 << 19), 2), (dict(xs=96), 2), (dict(ws=96), 2),
    (dict(xs=108), 3), (dict(ws=108), 3), (dict(xs=1 << 22 | 8), 2), (dict(ws=1 << 62), 2), (dict(x=None), 1), (dict(w=None), 1),
    (dict(t=None), 1), (dict(loss=None), 1), (dict(lse=None), 1), (dict(x=FAKE + 8), 3), (dict(w=FAKE + 8), 3), (dict(t=FAKE + 2), 3),
    (dict(loss=FAKE + 1), 3), (dict(lse=FAKE + 2), 3), (dict(wsp=None), 1), (dict(wsb=8), 1), (dict(wsb=-1), 1), (dict(wsp=FAKE + 64), 3),
    (dict(xd=2, xs=112, ws=112), 1), (dict(xd=2, xs=112, ws=112, sx=FAKE), 1), (dict(xd=2, xs=112, ws=112, sx=FAKE, sw=FAKE + 2), 3),
])
def test_head_refusals(L, kw, status):
    _refused(L, "stq_head_cross_entropy", HEAD, kw, status)


def test_head_nothing_to_do(L):
    _done(L, "stq_head_cross_entropy", HEAD, dict(n=0, x=None, w=None, t=None, loss=None, lse=None, wsp=None, wsb=0))


HEAD_BWD = dict(x=FAKE, xd=BF16, xs=104, sx=None, w=FAKE, ws=104, sw=None, n=10, v=1000, k=100, t=FAKE, lse=FAKE, g=FAKE, dx=FAKE,
                dxs=100, dw=FAKE, dws=100, wsp=FAKE, wsb=1 << 40)


@pytest.mark.parametrize("kw, status", [
    (dict(xd=F32), 1), (dict(n=-1), 1), (dict(k=0), 2), (dict(v=0), 2), (dict(xs=96), 2), (dict(ws=108), 3), (dict(x=None), 1),
    (dict(w=None), 1), (dict(t=None), 1), (dict(lse=None), 1), (dict(g=None), 1), (dict(lse=FAKE + 2), 3), (dict(g=FAKE + 1), 3),
    (dict(dxs=99), 2), (dict(dws=99), 2), (dict(dx=FAKE + 1), 3), (dict(dw=FAKE + 1), 3), (dict(wsp=None), 1), (dict(wsb=64), 1),
    (dict(wsb=-1), 1), (dict(xd=2, xs=112, ws=112, sx=FAKE, sw=FAKE), 1), (dict(dws=1 << 61), 2),
])
def test_head_backward_refusals(L, kw, status):
    _refused(L, "stq_head_cross_entropy_backward", HEAD_BWD, kw, status)


def test_head_workspaces(L):
    need = ctypes.c_int64()
    fwd, bwd = L.stq_head_cross_entropy_workspace, L.stq_head_cross_entropy_backward_workspace
    # (maximum, sum) of every row for each 16 words, or for two wavefronts a tile of 64, and the rows' target logits
    assert fwd(BF16, 10, 1000, 100, 256, ctypes.byref(need)) == 0 and need.value == 5120 + 256 and 63 * 10 * 8 <= 5120
    assert fwd(BF16, 20, 1000, 100, 256, ctypes.byref(need)) == 0 and need.value == 2 * 16 * 20 * 8 + 256
    assert fwd(BF16, 0, 1000, 100, 256, ctypes.byref(need)) == 0 and need.value == 0
    assert fwd(F32, 10, 1000, 100, 256, ctypes.byref(need)) == 1
    assert fwd(BF16, 10, 1000, 100, -1, ctypes.byref(need)) == 1
    assert fwd(BF16, 10, 1000, 100, 256, None) == 1
    for dx, dw in [(0, 0), (1, 0), (0, 1), (1, 1)]:
        assert bwd(BF16, 10, 1000, 100, dx, dw, 256, ctypes.byref(need)) == 0 and (need.value > 0) == bool(dx or dw)
    assert bwd(2, 10, 1000, 100, 1, 1, 256, ctypes.byref(need)) == 1
    assert bwd(BF16, 10, 0, 100, 1, 1, 256, ctypes.byref(need)) == 2
    # a piece's gradients and weights stay within a few hundred MB whatever the vocabulary
    assert bwd(BF16, 4096, 1 << 20, 7168, 1, 1, 256, ctypes.byref(need)) == 0 and need.value < 1 << 30
    _done(L, "stq_head_cross_entropy_backward", HEAD_BWD, dict(dx=None, dw=None, lse=None, g=None, wsp=None, wsb=0))
    _done(L, "stq_head_cross_entropy_backward", HEAD_BWD, dict(n=0, dw=None, x=None, w=None, t=None, lse=None, g=None, wsp=None, wsb=0))


def test_norm_gradient_in_the_place_of_h(L):
    # with few rows the workgroups of dweight read h beside those that write dx
    far = dict(dy=FAKE + 4096, dh=None, yd=BF16)
    _refused(L, "stq_rmsnorm_rows_backward", NORM_BWD, dict(far, dx=FAKE), 1)
    _refused(L, "stq_rmsnorm_rows_backward", NORM_BWD, dict(far, dx=FAKE, dw=None), 1)


def test_head_gradients_in_an_operands_place(L):
    far = dict(x=FAKE, w=FAKE + 65536, dx=FAKE + 131072, dw=FAKE + 262144)
    for kw in [dict(dx=FAKE), dict(dx=FAKE + 65536), dict(dw=FAKE, dws=104), dict(dw=FAKE + 65536, dws=104), dict(dw=FAKE + 131072)]:
        _refused(L, "stq_head_cross_entropy_backward", HEAD_BWD, dict(far, **kw), 1)


def test_combine_gradient_in_an_operands_place(L):
    far = dict(dy=FAKE + 4096, z=FAKE + 8192, zd=BF16)
    _refused(L, "stq_combine_rows_backward", COMBINE_BWD, dict(far, dz=FAKE + 4096), 1)
    _refused(L, "stq_combine_rows_backward", COMBINE_BWD, dict(far, dz=FAKE + 8192, zd=F32), 1)
    _refused(L, "stq_combine_rows_backward", COMBINE_BWD, dict(far, dz=FAKE + 8192, dzs=104), 1)
