"""Norm rows and their gradients against 64-bit arithmetic.

h, q and step have one right value each (one rounding apiece) and are compared
bit for bit, the integers through test_gpu_q8's exact quotients.  Tolerances (u
= 2^-24): a row's sum of squares meets at most J = 8 ceil(d / 512) + 20
additions, all of positive terms, so rstd errs by u ((J + 3) / 2 + 3) relative
(halved by the root; the division, eps, root and reciprocal add theirs) and y
and scale by 2 u more.  In the gradient g w and h rstd round once each, the
dot product meets J + 4 roundings of its terms' magnitudes, and
    |dx error| <= rstd (10 u (|g w| + |u m|) + |u| dm) + 2 u |dh| + half a step,
dm = (J + 6) u sum|g w u| / d.  dweight adds at most K = ceil(n / 512) + 56
terms in a row (256 compute units or more: 512 parts, added 16 a thread and
then 32)."""
import numpy as np
import pytest
import torch

import test_gpu_q8 as TQ

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6


@pytest.fixture(scope="module")
def stq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_ternary_bit_amd as m
    return m


def _rand(shape, seed, std=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std


def _inputs(n, d, xt, rt, seed):
    x = _rand((n, d), seed).to(xt)
    r = None if rt is None else _rand((n, d), seed + 1, 3.0).to(rt)
    return x, r, 1.0 + _rand((d,), seed + 2, 0.2)


def _j(d):
    return 8 * -(-d // 512) + 20


def _check(got, x, r, w, eps=EPS):
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    n, d = x.shape
    assert torch.equal(got.h.cpu().view(torch.uint8), h.view(torch.uint8)) if r is not None else got.h.dtype == x.dtype
    f = h.double()
    rstd = 1.0 / torch.sqrt(f.square().mean(1) + eps)
    rel = U * ((_j(d) + 3) / 2 + 3)
    assert bool(((got.rstd.cpu().double() - rstd).abs() <= rel * rstd).all())
    v = h.float() * w
    if got.q is not None:
        want_q, step = TQ._quant_ref(v)
        assert np.array_equal(got.q.cpu().numpy(), want_q)
        scale = torch.from_numpy(step).double() * rstd
        assert bool(((got.scale.cpu().double() - scale).abs() <= (rel + 2 * U) * scale + 2.0 ** -149).all())
        if d % 16:
            pad = got.q.as_strided((n, (d + 15) // 16 * 16), (got.q.stride(0), 1))[:, d:]
            assert not pad.any()
    if got.y is not None:
        y = f * w.double() * rstd[:, None]
        assert bool(((got.y.cpu().double() - y).abs() <= (rel + 2 * U + B * (1 + rel + 2 * U)) * y.abs() + 2.0 ** -126).all())


SHAPES = [(1, 1), (1, 64), (3, 7), (5, 511), (2, 512), (4, 513), (1, 2048), (3, 2049), (1, 7168), (17, 4099), (2, 8192),
          (3, 8200), (1, 20001), (600, 4104), (515, 2056)]


@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rt", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, d", SHAPES)
def test_forward(stq, n, d, xt, rt):
    x, r, w = _inputs(n, d, xt, rt, n + d)
    got = stq.rmsnorm_rows(x.cuda(), w.cuda(), EPS, residual=None if r is None else r.cuda(), need_q=True, need_y=True)
    _check(got, x, r, w)


# many rows of more than a thread's held columns
@pytest.mark.parametrize("rt", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, d", [(520, 8203), (513, 16385)])
def test_forward_of_many_wide_rows(stq, n, d, rt):
    x, r, w = _inputs(n, d, torch.bfloat16, rt, n + d)
    _check(stq.rmsnorm_rows(x.cuda(), w.cuda(), EPS, residual=None if r is None else r.cuda(), need_y=True), x, r, w)


# the row's last columns are read whole, over those that a neighbour writes
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, d", [(5, 9), (9, 87), (600, 87), (3, 515), (7, 4099), (600, 4099), (4, 9001), (530, 9001)])
def test_in_place_of_ragged_rows(stq, n, d, t):
    x, r, w = _inputs(n, d, t, t, n + d)
    xc, rc, wc = x.cuda(), r.cuda(), w.cuda()
    want = stq.rmsnorm_rows(xc, wc, EPS, rc, need_y=True)
    for over_x in (False, True):
        a, b = xc.clone(), rc.clone()
        got = stq.rmsnorm_rows(a, wc, EPS, b, need_y=True, h=a if over_x else b)
        assert got.h.data_ptr() == (a if over_x else b).data_ptr() and all(torch.equal(g, e) for g, e in zip(got, want))
    dy, dh = _rand((n, d), 1).to(t).cuda(), _rand((n, d), 2).to(t).cuda()
    dx, dw = stq.rmsnorm_rows_backward(want.h, wc, want.rstd, dy, dh=dh)
    for name in ("dy", "dh"):
        g = dict(dy=dy.clone(), dh=dh.clone())
        dx2, dw2 = stq.rmsnorm_rows_backward(want.h, wc, want.rstd, g["dy"], dh=g["dh"], dx=g[name])
        assert dx2.data_ptr() == g[name].data_ptr() and torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_forward_single_outputs_and_given_ones(stq):
    x, r, w = _inputs(33, 1000, torch.bfloat16, torch.float32, 5)
    xc, rc, wc = x.cuda(), r.cuda(), w.cuda()
    both = stq.rmsnorm_rows(xc, wc, EPS, rc, need_y=True)
    only_q = stq.rmsnorm_rows(xc, wc, EPS, rc)
    only_y = stq.rmsnorm_rows(xc, wc, EPS, rc, need_q=False, need_y=True)
    assert only_q.y is None and only_y.q is None and only_y.scale is None
    assert torch.equal(only_q.q, both.q) and torch.equal(only_q.scale, both.scale) and torch.equal(only_y.y, both.y)
    # wide strides, an offset, and memory around the rows that must stay
    q = torch.full((33, 1040), 77, dtype=torch.int8, device="cuda")
    y = torch.full((33, 1003), 7.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.full((33, 1005), 7.0, device="cuda")
    wide[:, 2:1002] = rc
    got = stq.rmsnorm_rows(xc, wc, EPS, wide[:, 2:1002], need_y=True, h=wide[:, 2:1002], q=q[:, :1000], y=y[:, :1000])
    assert got.h.data_ptr() == wide.data_ptr() + 8
    assert torch.equal(wide[:, 2:1002], both.h) and torch.equal(q[:, :1000], both.q) and torch.equal(y[:, :1000], both.y)
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 1002:] == 7).all()) and bool((y[:, 1000:] == 7).all())
    assert bool((q[:, 1008:] == 77).all()) and not q[:, 1000:1008].any()


def test_forward_in_x_place(stq):
    x, r, w = _inputs(9, 9000, torch.float32, torch.float32, 6)
    xc = x.cuda()
    got = stq.rmsnorm_rows(xc, w.cuda(), EPS, r.cuda(), h=xc, need_y=True)
    assert got.h.data_ptr() == xc.data_ptr()
    _check(got, x, r, w)


@pytest.mark.parametrize("d", [100, 700, 4000, 9000])
def test_rows_that_are_empty_or_not_finite(stq, d):
    n = 8
    x, _, w = _inputs(n, d, torch.float32, None, d)
    x[1] = 0.0
    x[2, d // 2] = float("nan")
    x[3, d - 1] = float("inf")
    x[4, 0] = -float("inf")
    x[5] = 1e-38
    x[6] *= 1e-30                       # the sum of squares leaves fp32's range downwards: eps is what is left
    got = stq.rmsnorm_rows(x.cuda(), w.cuda(), EPS, need_y=True)
    rows = [0, 1, 5, 6, 7]
    _check(stq.Norm(got.h[rows], got.rstd[rows], got.q[rows].contiguous() if d % 16 == 0 else None,
                    got.scale[rows], got.y[rows]), x[rows], None, w)
    assert np.array_equal(got.q.cpu().numpy()[rows], TQ._quant_ref((x * w)[rows])[0])
    assert not got.q[1].any() and got.scale[1].item() == 0.0 and not got.y[1].any()
    for i in (2, 3, 4):
        assert np.isnan(got.scale[i].item()) and not got.q[i].any()
    assert np.isnan(got.rstd[2].item()) and got.rstd[3].item() == 0.0 and got.rstd[4].item() == 0.0


@pytest.mark.parametrize("n, d", [(3, 100), (3, 700), (2, 4000), (2, 9000), (600, 2500)])
def test_rows_of_zeros_without_eps(stq, n, d):
    x, _, w = _inputs(n, d, torch.float32, None, d)
    x[1] = 0.0
    got = stq.rmsnorm_rows(x.cuda(), w.cuda(), 0.0)
    assert got.scale[1].item() == 0.0 and not got.q[1].any() and np.isinf(got.rstd[1].item())
    rest = [i for i in range(n) if i != 1]
    assert bool(torch.isfinite(got.scale[rest]).all()) and bool((got.scale[rest] > 0).all())


def test_halves_go_to_even(stq):
    # weight 1 and max 127: the quotients are the values themselves
    row = torch.tensor([127.0] + [i + 0.5 for i in range(-126, 126)] + [0.25, -0.75, 63.0])
    got = stq.rmsnorm_rows(row[None].cuda(), torch.ones(len(row)).cuda(), EPS)
    assert np.array_equal(got.q.cpu().numpy(), TQ._quant_ref(row[None])[0])


def test_no_rows(stq):
    w = torch.ones(64, device="cuda")
    got = stq.rmsnorm_rows(torch.empty(0, 64, device="cuda"), w, need_y=True)
    assert got.q.shape == (0, 64) and got.y.shape == (0, 64) and got.rstd.shape == (0,)
    e = torch.empty(0, 64, device="cuda")
    dw = torch.full((64,), 3.0, device="cuda")
    dx, dw = stq.rmsnorm_rows_backward(e, w, torch.empty(0, device="cuda"), e, dweight=dw)
    assert dx.shape == (0, 64) and not dw.any()


def _bwd_inputs(n, d, ht, yt, joined, seed):
    h = _rand((n, d), seed, 2.0).to(ht)
    w = 1.0 + _rand((d,), seed + 1, 0.2)
    dy = _rand((n, d), seed + 2).to(yt)
    dh = _rand((n, d), seed + 3).to(ht) if joined else None
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    return h, w, rstd, dy, dh


def _bwd_ref(h, w, rstd, dy, dh):
    n, d = h.shape
    u, gw = h.double() * rstd.double()[:, None], dy.double() * w.double()
    dot = gw * u
    m = dot.mean(1, keepdim=True)
    dx = rstd.double()[:, None] * (gw - u * m)
    dm = (_j(d) + 6) * U * dot.abs().mean(1, keepdim=True)
    tol = rstd.double()[:, None] * (10 * U * (gw.abs() + (u * m).abs()) + u.abs() * dm)
    if dh is not None:
        dx, tol = dx + dh.double(), tol + 2 * U * dh.double().abs()
    half = B if h.dtype == torch.bfloat16 else U
    tol = tol * (1 + half) + half * dx.abs()
    terms = dy.double() * u
    k = -(-n // 512) + 56
    return dx, tol, terms.sum(0), (k + 3) * U * terms.abs().sum(0)


def _bwd_check(got, args):
    dx, tol, dw, tol_w = _bwd_ref(*args)
    if got[0] is not None:
        assert bool(((got[0].cpu().double() - dx).abs() <= tol + 2.0 ** -126).all())
    if got[1] is not None:
        assert bool(((got[1].cpu().double() - dw).abs() <= tol_w + 2.0 ** -126).all())


@pytest.mark.parametrize("ht", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("yt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, d", SHAPES + [(1030, 300), (2000, 2000), (256, 700), (257, 700), (270, 8200), (260, 9001)])
def test_backward(stq, n, d, ht, yt):
    for joined in (False, True):
        args = _bwd_inputs(n, d, ht, yt, joined, n + 3 * d)
        h, w, rstd, dy, dh = (None if t is None else t.cuda() for t in args)
        _bwd_check(stq.rmsnorm_rows_backward(h, w, rstd, dy, dh), args)


@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("d", [200, 4096, 9001])
def test_backward_one_output_and_in_place(stq, n, d):
    args = _bwd_inputs(n, d, torch.float32, torch.float32, True, d)
    h, w, rstd, dy, dh = (t.cuda() for t in args)
    both = stq.rmsnorm_rows_backward(h, w, rstd, dy, dh)
    dx, none = stq.rmsnorm_rows_backward(h, w, rstd, dy, dh, need_dweight=False)
    assert none is None and torch.equal(dx, both[0])
    none, dw = stq.rmsnorm_rows_backward(h, w, rstd, dy, dh, need_dx=False)
    assert none is None and torch.equal(dw, both[1])
    at_dh, dw = stq.rmsnorm_rows_backward(h, w, rstd, dy, dh, dx=dh)
    assert at_dh.data_ptr() == dh.data_ptr() and torch.equal(dh, both[0]) and torch.equal(dw, both[1])
    dh = args[4].cuda()
    at_dy, dw = stq.rmsnorm_rows_backward(h, w, rstd, dy, dh, dx=dy)
    assert torch.equal(dy, both[0]) and torch.equal(dw, both[1])


@pytest.mark.parametrize("d", list(range(8, 26)) + list(range(1200, 1208)))
def test_every_end_of_a_row(stq, d):
    for xt, rt in ((torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        x, r, w = _inputs(6, d, xt, rt, d)
        _check(stq.rmsnorm_rows(x.cuda(), w.cuda(), EPS, r.cuda(), need_y=True), x, r, w)
        for n in (6, 270):
            args = _bwd_inputs(n, d, xt, rt, True, d)
            _bwd_check(stq.rmsnorm_rows_backward(*(t.cuda() for t in args)), args)


def test_gradient_against_differences(stq):
    # the loss is a fixed weighting c of y; central differences of the 64-bit norm, whose error is of the
    # order of step^2 and far below the bound
    n, d, step = 3, 70, 1e-5
    h, w, rstd, c, _ = _bwd_inputs(n, d, torch.float32, torch.float32, False, 2)
    exact = torch.rsqrt(h.double().square().mean(1) + EPS)

    def loss(hh, ww):
        return (c.double() * hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + EPS) * ww).sum().item()
    dx, dw = (t.cpu().double() for t in stq.rmsnorm_rows_backward(h.cuda(), w.cuda(), exact.float().cuda(), c.cuda()))
    for i, j in [(0, 0), (1, 33), (2, 69)]:
        e = torch.zeros(n, d, dtype=torch.float64)
        e[i, j] = step
        diff = (loss(h.double() + e, w.double()) - loss(h.double() - e, w.double())) / (2 * step)
        assert abs(diff - dx[i, j].item()) < 1e-4
        e = torch.zeros(d, dtype=torch.float64)
        e[j] = step
        diff = (loss(h.double(), w.double() + e) - loss(h.double(), w.double() - e)) / (2 * step)
        assert abs(diff - dw[j].item()) < 1e-4


def test_under_a_graph_with_work_between(stq):
    n, d = 700, 4096
    x, r, w = (t.cuda() for t in _inputs(n, d, torch.bfloat16, torch.bfloat16, 1))
    dy = _rand((n, d), 9).cuda()
    out = stq.rmsnorm_rows(x, w, EPS, r, need_y=True)
    ws = torch.empty(stq.rmsnorm_rows_backward_workspace(n, d), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")

    def call():
        stq.rmsnorm_rows(x, w, EPS, r, True, True, out.h, out.rstd, out.q, out.scale, out.y)
        stq.rmsnorm_rows_backward(out.h, w, out.rstd, dy, out.h, dx=dx, dweight=dw, workspace=ws)
    call()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(_rand((n, d), 50 + i))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, dx, dw)]
        want = stq.rmsnorm_rows(x, w, EPS, r, need_y=True)
        want = [*want, *stq.rmsnorm_rows_backward(want.h, w, want.rstd, dy, want.h)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i


def test_on_another_stream(stq):
    x, r, w = _inputs(64, 2048, torch.bfloat16, torch.float32, 3)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = stq.rmsnorm_rows(x.cuda(), w.cuda(), EPS, r.cuda(), need_y=True)
    s.synchronize()
    _check(got, x, r, w)


def test_binding_refusals(stq):
    x, w = torch.zeros(2, 32, device="cuda"), torch.ones(32, device="cuda")
    with pytest.raises(ValueError, match="weight must hold 32"):
        stq.rmsnorm_rows(x, w[:31])
    with pytest.raises(ValueError, match="weight must be"):
        stq.rmsnorm_rows(x, w.bfloat16())
    with pytest.raises(ValueError, match="x must be"):
        stq.rmsnorm_rows(x.half(), w)
    with pytest.raises(ValueError, match="contiguous rows"):
        stq.rmsnorm_rows(x.t().contiguous().t(), w)
    with pytest.raises(ValueError, match="residual must be"):
        stq.rmsnorm_rows(x, w, residual=x[:1])
    with pytest.raises(ValueError, match="without a residual"):
        stq.rmsnorm_rows(x, w, h=x)
    with pytest.raises(ValueError, match="need_q"):
        stq.rmsnorm_rows(x, w, need_q=False, scale=w)
    with pytest.raises(ValueError, match="need_y"):
        stq.rmsnorm_rows(x, w, y=x.bfloat16())
    with pytest.raises(stq.StqError, match="eps"):
        stq.rmsnorm_rows(x, w, eps=-1.0)
    with pytest.raises(ValueError, match="one GPU"):
        stq.rmsnorm_rows(x, w.cpu())
    r = torch.ones(2, device="cuda")
    with pytest.raises(ValueError, match="dy must be"):
        stq.rmsnorm_rows_backward(x, w, r, x[:1])
    with pytest.raises(ValueError, match="dh must be"):
        stq.rmsnorm_rows_backward(x, w, r, x, dh=x.bfloat16())
    with pytest.raises(ValueError, match="need_dx"):
        stq.rmsnorm_rows_backward(x, w, r, x, need_dx=False, dx=x)
    with pytest.raises(stq.StqError, match="workspace"):
        many = x.repeat(150, 1)
        stq.rmsnorm_rows_backward(many, w, r.repeat(150), many, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
