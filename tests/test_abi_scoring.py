"""Host-side checks of the gated feed-forward, the 8-bit product and the token scoring:
bad arguments are refused with a status and a message before any GPU call,
empty work is fine without one, and the workspace queries agree with the
calls.  No kernel runs."""
import ctypes
import os

import pytest

FAKE = 0x100000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    import sparse_ternary_bit_amd as stq
    if not os.path.exists(stq.lib_path()):
        from sparse_ternary_bit_amd import build
        build.build(verbose=False)
    return stq.lib()


def _err(L):
    return L.stq_last_error().decode()


def _quant(L, **kw):
    a = dict(x=FAKE, xd=1, xs=100, n=4, k=100, q=FAKE, qs=112, sc=FAKE)
    a.update(kw)
    return L.stq_q8_quantize_rows(a["x"], a["xd"], a["xs"], a["n"], a["k"], a["q"], a["qs"], a["sc"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(n=-1), 1), (dict(k=0), 2), (dict(k=-3), 2), (dict(xd=2), 1), (dict(xs=99), 2), (dict(qs=96), 2),
    (dict(qs=120), 3), (dict(q=FAKE + 8), 3), (dict(x=FAKE + 1), 3), (dict(xd=0, x=FAKE + 2), 3),
    (dict(sc=FAKE + 2), 3), (dict(x=None), 1), (dict(q=None), 1), (dict(sc=None), 1), (dict(n=(1 << 22) + 1), 2),
    (dict(xs=1 << 62), 2), (dict(k=1 << 31, xs=1 << 31, qs=1 << 31), 2),
])
def test_quantize_refusals(L, kw, status):
    assert _quant(L, **kw) == status
    assert _err(L).startswith("stq_q8_quantize_rows")


def test_quantize_nothing_to_do(L):
    assert _quant(L, n=0, x=None, q=None, sc=None) == 0


def _mm(L, **kw):
    a = dict(a=FAKE, lda=112, as_=FAKE, w=FAKE, ldw=112, ws=FAKE, m=128, n=64, k=100, y=FAKE, yd=1, ldy=64)
    a.update(kw)
    return L.stq_q8_matmul(a["a"], a["lda"], a["as_"], a["w"], a["ldw"], a["ws"], a["m"], a["n"], a["k"], a["y"],
                           a["yd"], a["ldy"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(m=-1), 1), (dict(n=-1), 1), (dict(k=0), 2), (dict(k=131072, lda=131072, ldw=131072), 2), (dict(yd=3), 1),
    (dict(lda=96), 2), (dict(ldw=96), 2), (dict(lda=120), 3), (dict(ldw=120), 3), (dict(lda=(1 << 23) + 16), 2),
    (dict(ldw=(1 << 23) + 16), 2), (dict(ldy=63), 2), (dict(a=None), 1), (dict(as_=None), 1), (dict(w=None), 1),
    (dict(ws=None), 1), (dict(y=None), 1), (dict(a=FAKE + 8), 3), (dict(w=FAKE + 8), 3), (dict(as_=FAKE + 2), 3),
    (dict(ws=FAKE + 2), 3), (dict(y=FAKE + 1), 3), (dict(yd=0, y=FAKE + 2), 3), (dict(m=(1 << 22) + 1), 2),
    (dict(n=(1 << 26) + 1, ldy=1 << 27), 2), (dict(m=1 << 20, n=1 << 20, ldy=1 << 20), 2), (dict(ldy=1 << 62), 2),
])
def test_matmul_refusals(L, kw, status):
    assert _mm(L, **kw) == status
    assert _err(L).startswith("stq_q8_matmul")


def test_matmul_nothing_to_do(L):
    none = dict(a=None, as_=None, w=None, ws=None, y=None)
    assert _mm(L, m=0, **none) == 0
    assert _mm(L, n=0, **none) == 0


def _lp(L, **kw):
    a = dict(x=FAKE, xd=1, xs=1000, n=4, v=1000, t=FAKE, lp=FAKE, lse=FAKE, ent=FAKE, top=5, ids=FAKE, tlp=FAKE,
             ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.stq_token_logprobs(a["x"], a["xd"], a["xs"], a["n"], a["v"], a["t"], a["lp"], a["lse"], a["ent"],
                                a["top"], a["ids"], a["tlp"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(xd=7), 1), (dict(n=-1), 1), (dict(v=0), 2), (dict(v=(1 << 30) + 1, xs=1 << 31), 2), (dict(n=(1 << 22) + 1), 2),
    (dict(top=-1), 1), (dict(top=33), 2), (dict(v=4, top=5), 2), (dict(xs=999), 2), (dict(wsb=-1), 1),
    (dict(x=None), 1), (dict(t=None), 1), (dict(lp=None), 1), (dict(ids=None), 1), (dict(tlp=None), 1),
    (dict(xs=1 << 62), 2), (dict(x=FAKE + 1), 3), (dict(xd=0, x=FAKE + 2), 3), (dict(t=FAKE + 2), 3),
    (dict(lp=FAKE + 2), 3), (dict(lse=FAKE + 2), 3), (dict(ent=FAKE + 2), 3), (dict(ids=FAKE + 2), 3),
    (dict(tlp=FAKE + 2), 3),
])
def test_logprobs_refusals(L, kw, status):
    assert _lp(L, **kw) == status
    assert _err(L).startswith("stq_token_logprobs")


def test_logprobs_nothing_to_do(L):
    assert _lp(L, n=0, x=None, t=None, lp=None, lse=None, ent=None, ids=None, tlp=None, ws=None, wsb=0) == 0


def test_logprobs_workspace_query_and_refusal(L):
    wb = ctypes.c_int64(-7)
    f = L.stq_token_logprobs_workspace
    assert f(1, 0, 1000, 5, 256, ctypes.byref(wb)) == 0 and wb.value == 0
    assert f(1, 4096, 131072, 5, 256, ctypes.byref(wb)) == 0 and wb.value == 0      # enough rows to fill the chip
    assert f(0, 1, 131072, 20, 256, ctypes.byref(wb)) == 0 and wb.value > 0          # one row is split
    assert f(5, 1, 1000, 5, 256, ctypes.byref(wb)) == 1
    assert f(1, 1, 1000, 33, 256, ctypes.byref(wb)) == 2
    assert f(1, 1, 1000, 5, -2, ctypes.byref(wb)) == 1
    assert f(1, 1, 1000, 5, 256, None) == 1
    assert f(0, 1, 131072, 20, 0, ctypes.byref(wb)) == 0
    need = wb.value
    big = dict(xd=0, n=1, v=131072, xs=131072, top=20)
    assert _lp(L, ws=None, wsb=0, **big) == 1 and "workspace" in _err(L)
    assert _lp(L, ws=FAKE, wsb=need - 1, **big) == 1
    assert _lp(L, ws=FAKE + 16, wsb=need, **big) == 3


def _bw(L, **kw):
    a = dict(x=FAKE, xd=1, xs=1000, n=4, v=1000, t=FAKE, lse=FAKE, ent=FAKE, g=FAKE, ge=FAKE, d=2 * FAKE, ds=1000)
    a.update(kw)
    return L.stq_token_logprobs_backward(a["x"], a["xd"], a["xs"], a["n"], a["v"], a["t"], a["lse"], a["ent"],
                                         a["g"], a["ge"], a["d"], a["ds"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(xd=7), 1), (dict(n=-1), 1), (dict(v=0), 2), (dict(n=(1 << 22) + 1), 2), (dict(xs=999), 2), (dict(ds=999), 2),
    (dict(x=None), 1), (dict(t=None), 1), (dict(lse=None), 1), (dict(d=None), 1), (dict(ent=None), 1),
    (dict(d=FAKE, ds=1008), 1), (dict(x=FAKE + 1), 3), (dict(d=2 * FAKE + 1), 3), (dict(t=FAKE + 2), 3),
    (dict(lse=FAKE + 2), 3), (dict(ent=FAKE + 2), 3), (dict(g=FAKE + 2), 3), (dict(ge=FAKE + 2), 3),
    (dict(ds=1 << 62), 2), (dict(n=1 << 22, v=1 << 20, xs=1 << 20, ds=1 << 20), 2),
])
def test_logprobs_backward_refusals(L, kw, status):
    assert _bw(L, **kw) == status
    assert _err(L).startswith("stq_token_logprobs_backward")


def test_logprobs_backward_nothing_to_do(L):
    assert _bw(L, n=0, x=None, t=None, lse=None, ent=None, g=None, ge=None, d=None) == 0


ROWB = 4096 // 256 * 42      # packed bytes of a row of 4096
STRIDE = 2 * 512 * ROWB


def _fw(L, **kw):
    a = dict(w=FAKE, st=STRIDE, ne=4, d=4096, f=512, x=FAKE, off=FAKE, m=10, h=FAKE, gu=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.stq_grouped_swiglu(a["w"], a["st"], a["ne"], a["d"], a["f"], a["x"], a["off"], a["m"], a["h"], a["gu"],
                                a["ws"], a["wsb"], None)


SHAPE_REFUSALS = [(dict(ne=0), 1), (dict(m=-1), 1), (dict(d=100), 2), (dict(f=128), 2), (dict(f=0), 2),
                  (dict(ne=65536), 2), (dict(m=(1 << 23) + 1), 2), (dict(d=1 << 23), 2), (dict(f=1 << 22), 2),
                  (dict(d=1 << 17, f=1 << 17, st=1 << 60), 2), (dict(st=STRIDE - 16), 2), (dict(off=None), 1),
                  (dict(st=STRIDE + 8), 3), (dict(w=FAKE + 8), 3), (dict(off=FAKE + 2), 3), (dict(w=None), 1)]


@pytest.mark.parametrize("kw, status", SHAPE_REFUSALS + [
    (dict(x=None), 1), (dict(h=None), 1), (dict(x=FAKE + 8), 3), (dict(h=FAKE + 8), 3), (dict(gu=FAKE + 8), 3),
    (dict(wsb=-1), 1)])
def test_swiglu_refusals(L, kw, status):
    assert _fw(L, **kw) == status
    assert _err(L).startswith("stq_grouped_swiglu")


def _bwd(L, **kw):
    a = dict(w=FAKE, st=STRIDE, ne=4, d=4096, f=512, x=FAKE, off=FAKE, m=10, gu=FAKE, dh=FAKE, dx=FAKE, dw=FAKE,
             ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.stq_grouped_swiglu_backward(a["w"], a["st"], a["ne"], a["d"], a["f"], a["x"], a["off"], a["m"], a["gu"],
                                         a["dh"], a["dx"], a["dw"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw, status", SHAPE_REFUSALS + [
    (dict(gu=None), 1), (dict(dh=None), 1), (dict(x=None), 1), (dict(gu=FAKE + 8), 3), (dict(dh=FAKE + 8), 3),
    (dict(x=FAKE + 8), 3), (dict(dx=FAKE + 4), 3), (dict(dw=FAKE + 8), 3), (dict(wsb=-1), 1),
    (dict(ne=60000, d=1 << 16, f=1 << 14, st=1 << 40), 2)])
def test_swiglu_backward_refusals(L, kw, status):
    assert _bwd(L, **kw) == status
    assert _err(L).startswith("stq_grouped_swiglu_backward")


def test_swiglu_workspace(L, monkeypatch):
    monkeypatch.delenv("STQ_GEMV_PLAN", raising=False)
    wb = ctypes.c_int64(-7)
    f = L.stq_grouped_swiglu_workspace
    assert f(256, 7168, 2048, 16384, 256, ctypes.byref(wb)) == 0 and wb.value == 0    # the matrix-core kernel
    assert f(4, 4096, 512, 0, 256, ctypes.byref(wb)) == 0 and wb.value == 0
    assert f(4, 4096, 500, 10, 256, ctypes.byref(wb)) == 2
    assert f(4, 4096, 512, -1, 256, ctypes.byref(wb)) == 1
    assert f(4, 4096, 512, 10, -1, ctypes.byref(wb)) == 1
    assert f(4, 4096, 512, 10, 256, None) == 1
    # few rows: the rows' experts, their fp32 pre-activations, and the GEMV's split outputs
    assert f(4, 4096, 512, 10, 256, ctypes.byref(wb)) == 0
    sp, mp, scratch = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
    assert L.stq_gemv_plan(4, 1024, 4096, 10, 256, ctypes.byref(sp), ctypes.byref(mp), ctypes.byref(scratch)) == 0
    assert wb.value == (scratch.value + 255) // 256 * 256 + 256 + 10 * 1024 * 4
    assert f(4, 4096, 512, 10, 0, ctypes.byref(wb)) == 0
    need = wb.value
    assert _fw(L, ws=None, wsb=0) == 1 and "workspace" in _err(L)
    assert _fw(L, wsb=need - 1) == 1
    assert _fw(L, ws=FAKE + 16, wsb=need) == 3


def test_swiglu_nothing_to_do(L):
    assert _fw(L, m=0, w=None, x=None, h=None, gu=None, ws=None, wsb=0) == 0
    assert _bwd(L, dx=None, dw=None, w=None, x=None, gu=None, dh=None, ws=None, wsb=0) == 0
    assert _bwd(L, m=0, dw=None, w=None, x=None, gu=None, dh=None, ws=None, wsb=0) == 0


def test_swiglu_backward_workspace(L):
    wb = ctypes.c_int64(-7)
    f = L.stq_grouped_swiglu_backward_workspace
    z = 10 * 1024 * 2
    assert f(4, 4096, 512, 10, 1, 0, ctypes.byref(wb)) == 0 and wb.value == z + 256
    assert f(4, 4096, 512, 10, 0, 1, ctypes.byref(wb)) == 0 and wb.value == z
    assert f(4, 4096, 512, 10, 1, 1, ctypes.byref(wb)) == 0 and wb.value == 2 * z + 256
    need = wb.value
    assert f(4, 4096, 512, 0, 1, 1, ctypes.byref(wb)) == 0 and wb.value == 0
    assert f(4, 4096, 500, 10, 1, 1, ctypes.byref(wb)) == 2
    assert f(4, 4096, 512, -1, 1, 1, ctypes.byref(wb)) == 1
    assert f(4, 4096, 512, 10, 1, 1, None) == 1
    assert _bwd(L, ws=None, wsb=0) == 1 and "workspace" in _err(L)
    assert _bwd(L, wsb=need - 1) == 1 and str(need) in _err(L)
    assert _bwd(L, ws=FAKE + 16, wsb=need) == 3


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    import sparse_ternary_bit_amd as stq
    x = torch.zeros(2, 32)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        stq.q8_quantize_rows(x)
    with pytest.raises(ValueError, match="GPU"):
        stq.token_logprobs(x, i)
    with pytest.raises(ValueError, match="GPU"):
        stq.token_logprobs_backward(x, i, x[:, 0], None, x[:, 0])
    q = torch.zeros(2, 32, dtype=torch.int8)
    with pytest.raises(ValueError, match="GPU"):
        stq.q8_matmul(q, x[:, 0], q, x[:, 0])


def test_logprobs_backward_takes_what_a_gpu_can_hold(L):
    """The joint limit on rows and vocabulary lies above any GPU's memory; calls below it get as far as
    the alignment check."""
    odd = dict(t=FAKE + 2)
    for n, v, xd in ((1 << 20, 131072, 1), (1 << 22, 32768, 1), (1 << 22, 40000, 1), (1 << 21, 50021, 0), (4, 1 << 30, 1)):
        assert _bw(L, n=n, v=v, xs=v + 8, ds=v + 8, xd=xd, **odd) == 3, (n, v)
        assert _bw(L, n=n, v=v, xs=v + 1, ds=v + 1, xd=xd, **odd) == 3, (n, v)   # rows that start inside 16 bytes
    assert _bw(L, n=1 << 22, v=65536, xs=65536, ds=65536, **odd) == 2             # 550 GB
    assert "too many rows" in _err(L)


def _units(ne, m):
    e = min(ne, m)
    return e + (m - e) // 32 + 8


@pytest.mark.parametrize("ne, d, f", [(256, 4096, 16384), (1, 256, 65536), (65535, 256, 1024), (65535, 512, 32768)])
def test_swiglu_limits_are_the_documented_ones(L, ne, d, f):
    """The largest row count below the joint limit is taken as far as the alignment checks, the next
    is not."""
    stride = 2 * f * (d // 256) * 42
    ok = [m for m in (1 << i for i in range(24)) if _units(ne, m) * (f // 128) <= 1 << 23]
    assert _fw(L, ne=ne, d=d, f=f, st=stride, m=ok[-1], x=FAKE + 2) == 3
    lo, hi = ok[-1], 1 << 23
    if _units(ne, hi) * (f // 128) <= 1 << 23:
        assert _fw(L, ne=ne, d=d, f=f, st=stride, m=hi + 1, x=FAKE + 2) == 2
        return
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if _units(ne, mid) * (f // 128) <= 1 << 23 else (lo, mid)
    assert _fw(L, ne=ne, d=d, f=f, st=stride, m=lo, x=FAKE + 2) == 3
    assert _fw(L, ne=ne, d=d, f=f, st=stride, m=hi, x=FAKE + 2) == 2
    assert "too many rows" in _err(L)


@pytest.mark.parametrize("ne, d, f", [(256, 65536, 256), (1, 1 << 17, 256), (65535, 8192, 256)])
def test_swiglu_backward_limits_are_the_documented_ones(L, ne, d, f):
    stride = 2 * f * (d // 256) * 42
    lo, hi = 1, 1 << 23
    assert _units(ne, lo) * (d // 256) <= 1 << 23 < _units(ne, hi) * (d // 256)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if _units(ne, mid) * (d // 256) <= 1 << 23 else (lo, mid)
    args = dict(ne=ne, d=d, f=f, st=stride, dh=FAKE + 2)
    assert _bwd(L, m=lo, dw=None, **args) == 3
    assert _bwd(L, m=hi, dw=None, **args) == 2
    ne = (1 << 23) // ((f // 64) * (d // 128))                 # dw's experts
    args["ne"] = ne
    assert _bwd(L, m=10, dx=None, **args) == 3
    args["ne"] = ne + 1
    assert _bwd(L, m=10, dx=None, **args) == 2
    assert "weight gradients" in _err(L)


def _cases(test):
    return next(m for m in test.pytestmark if m.name == "parametrize").args[1]


def test_swiglu_tests_reach_every_form():
    """The form follows from estimates in the library: the GPU tests written for one of them still take it
    on the 256 compute units of an MI355X."""
    import sparse_ternary_bit_amd as stq
    import test_gpu_swiglu as T

    def fwd(counts, d, f, tail=0):
        return stq.grouped_swiglu_plan(len(counts), d, f, sum(counts) + tail, 256)

    def bwd(counts, d, f, tail=0):
        return stq.grouped_swiglu_backward_plan(len(counts), d, f, sum(counts) + tail, 256)
    assert {fwd(*c) for c in _cases(T.test_forward)} == {32}
    assert {bwd(*c) for c in _cases(T.test_backward)} == {32, 96}
    assert {fwd(*c) for c in _cases(T.test_few_rows_through_the_gemv)} == {0}
    assert [fwd(*c[:3], 5) for c in _cases(T.test_long_passes)] == [80] + 5 * [160]
    assert {fwd(*c[:3], 2) for c in _cases(T.test_passes_of_80)} == {80}
    assert fwd([160] * 130, 768, 1024) == 160                                 # blocks of no scale
    assert [bwd(*c[:3]) for c in _cases(T.test_long_passes_of_the_gradients)] == 5 * [96]
    far = {bwd(c[1], 512, 256) for m in T.test_gradient_of_x_beside_rows_of_a_large_scale.pytestmark
           if m.name == "parametrize" and m.args[0].startswith("at") for c in m.args[1]}
    assert far == {32, 96}


def test_swiglu_plan_refusals(L):
    rows = ctypes.c_int32(-7)
    for f in (L.stq_grouped_swiglu_plan, L.stq_grouped_swiglu_backward_plan):
        assert f(4, 4096, 512, 0, 256, ctypes.byref(rows)) == 0 and rows.value == 0
        assert f(256, 7168, 2048, 16384, 0, ctypes.byref(rows)) == 0 and rows.value > 32
        assert f(4, 4096, 500, 10, 256, ctypes.byref(rows)) == 2
        assert f(0, 4096, 512, 10, 256, ctypes.byref(rows)) == 1
        assert f(4, 4096, 512, -1, 256, ctypes.byref(rows)) == 1
        assert f(4, 4096, 512, 10, -1, ctypes.byref(rows)) == 1
        assert f(4, 4096, 512, 10, 256, None) == 1
        assert "_plan" in _err(L)
    # the form that needs a workspace is the one that reports no passes
    wb = ctypes.c_int64()
    for m in (1, 10, 300, 2000, 20000):
        assert L.stq_grouped_swiglu_plan(256, 7168, 2048, m, 256, ctypes.byref(rows)) == 0
        assert L.stq_grouped_swiglu_workspace(256, 7168, 2048, m, 256, ctypes.byref(wb)) == 0
        assert (wb.value > 0) == (rows.value == 0)
