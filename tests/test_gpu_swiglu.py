"""The gated feed-forward over packed experts and its gradients against
64-bit arithmetic on the decoded weights.

Tolerances (u = 2^-24; bf16 half step b = 2^-8, fp16 f = 2^-11).  A sum of k
exact products on the matrix cores goes through k / 32 accumulations of 32
products each: its error is at most 2 u (k / 32 + 40) times the sum of the
products' magnitudes (40 covers the 32 products inside one and the block
scale).  exp, the reciprocal and the products of silu err by at most
e = u (2 |g| + 10) relative.  So
    h        1.1 dg (|u| + du) + |silu(g)| du + e |h| + b |h|     (silu' < 1.1)
    gate_up  dz + b |z|
    dz       |dh u| e s (1 + 2 |g|) and |dh g s| e for the two halves, then
             its roundings: for dx two to fp16, dz itself and its product with
             the block scale d / D, 2 f |dz| |w|; dz is scaled so that the row's
             largest is at least 2^14, where a subnormal step errs by 2^-25,
             2^-39 of it, and once more for the product, 2^-39 max |dz| times
             D, a power of two at most twice the largest |d| of the column block
             (or 2^-15); for dw one to bf16, b |dz|
    dx, dw   the sums of those against the other factor's magnitudes, the
             accumulation, and b of the result."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
B = 2.0 ** -8
QK, BLOCK = 256, 42


@pytest.fixture(scope="module")
def stq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_ternary_bit_amd as m
    return m


class Case:
    """Random packed experts (any code bits are valid) with block scales in +-[0.01, 0.03], some of
    them 0, subnormal or large, and rows grouped by expert."""

    def __init__(self, stq, counts, d, f, seed=0, tail=0, slack=0, odd_scales=False, x_std=1.0):
        g = torch.Generator().manual_seed(seed)
        self.stq, self.E, self.d, self.f = stq, len(counts), d, f
        nbytes = 2 * f * (d // QK) * BLOCK
        self.stride = nbytes + slack
        t = torch.randint(0, 256, (self.E, self.stride), dtype=torch.uint8, generator=g)
        sc = 0.01 + 0.02 * torch.rand((self.E, nbytes // BLOCK), generator=g)
        if odd_scales:
            sc[:, ::7] = 0.0
            sc[:, 3::11] = 3e-6
            sc[:, 5::13] *= -40.0
        blocks = t[:, :nbytes].reshape(self.E, -1, BLOCK)
        blocks[:, :, :2] = sc.half().view(torch.uint8).view(self.E, -1, 2)
        t[:, :nbytes] = blocks.reshape(self.E, nbytes)
        self.table = t.view(-1).cuda()
        self.bounds = [0] + list(np.cumsum(counts))
        self.m = self.bounds[-1] + tail                       # `tail` rows behind the last expert
        self.offsets = torch.tensor(self.bounds, dtype=torch.int32, device="cuda")
        self.x = (torch.randn((self.m, d), generator=g) * x_std).bfloat16().cuda()
        self.gu = (torch.randn((self.m, 2 * f), generator=g) * 1.5).bfloat16().cuda()
        self.dh = (torch.randn((self.m, f), generator=g) * 1e-3).bfloat16().cuda()

    def args(self):
        return self.table, self.stride, self.E, self.d, self.f, self.x, self.offsets

    def weights(self, e):
        q = self.table[e * self.stride:(e + 1) * self.stride]
        return self.stq.dequantize_rows(q, 2 * self.f, self.d).double()   # bit-exact by its own tests

    def forward(self, **kw):
        return self.stq.grouped_swiglu(*self.args(), **kw)

    def check_forward(self, h, gu=None):
        f = self.f
        for e, (lo, hi) in enumerate(zip(self.bounds, self.bounds[1:])):
            if lo == hi:
                continue
            w, x = self.weights(e), self.x[lo:hi].double()
            z, A = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
            dz = 2 * U * (self.d / 32 + 40) * A
            g, u, dg, du = z[:, :f], z[:, f:], dz[:, :f], dz[:, f:]
            silu = g * torch.sigmoid(g)
            ref = silu * u
            tol = (1.1 * dg * (u.abs() + du) + silu.abs() * du + U * (2 * g.abs() + 10) * ref.abs()) * (1 + B) + B * ref.abs()
            err = (h[lo:hi].double() - ref).abs()
            assert bool((err <= tol + 1e-30).all()), (e, (err - tol).max().item())
            if gu is not None:
                err = (gu[lo:hi].double() - z).abs()
                assert bool((err <= dz * (1 + B) + B * z.abs() + 1e-30).all()), e

    def dz_ref(self):
        g, u, dh = self.gu[:, :self.f].double(), self.gu[:, self.f:].double(), self.dh.double()
        s = torch.sigmoid(g)
        dz = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1)
        e = U * (2 * g.abs() + 10)
        return dz, torch.cat([(dh * u).abs() * e * s * (1 + 2 * g.abs()), (dh * g * s).abs() * e], 1)

    def backward(self, **kw):
        return self.stq.grouped_swiglu_backward(*self.args(), self.gu, self.dh, **kw)

    def dx_tol(self, dz, err, w):
        F = 2.0 ** -11
        top = 2.0 ** -39 * dz.abs().amax(1, keepdim=True)
        t = (err + F * dz.abs() + top) * (1 + F) + F * dz.abs()
        D = 2 * w.abs().amax(0).view(-1, QK).amax(1).clamp(min=2.0 ** -16).repeat_interleave(QK)   # per column
        return (t + 2 * U * (2 * self.f / 32 + 40) * dz.abs()) @ w.abs() + top * 2 * self.f * D

    def check_backward(self, dx, dw):
        dz, err = self.dz_ref()
        for e, (lo, hi) in enumerate(zip(self.bounds, self.bounds[1:])):
            z, ez = dz[lo:hi], err[lo:hi]
            if dx is not None and hi > lo:
                w = self.weights(e)
                ref = z @ w
                tol = self.dx_tol(z, ez, w) * (1 + B) + B * ref.abs() + 1e-30
                d = (dx[lo:hi].double() - ref).abs()
                assert bool((d <= tol).all()), (e, (d - tol).max().item())
            if dw is not None:
                x = self.x[lo:hi].double()
                zt = z.t().contiguous()
                ref = zt @ x
                t = ez + B * z.abs() * (1 + B) + 2 * U * ((hi - lo) / 32 + 40) * z.abs()
                tol = (t.t().contiguous() @ x.abs()) * (1 + B) + B * ref.abs() + 1e-30
                d = (dw[e].double() - ref).abs()
                assert bool((d <= tol).all()), (e, (d - tol).max().item())


CASES = [([1], 256, 256), ([16], 512, 256), ([17, 0, 3], 256, 512), ([0, 64, 0, 33, 0, 0, 1, 15, 16], 512, 256),
         ([80, 81, 79, 5], 768, 256), ([128, 129, 127], 256, 768), ([300], 1024, 512), ([97, 111, 255, 256, 257], 256, 256),
         ([2] * 19, 512, 512)]


@pytest.mark.parametrize("counts, d, f", CASES)
def test_forward(stq, counts, d, f):
    c = Case(stq, counts, d, f, seed=len(counts) + d)
    gu = torch.empty((c.m, 2 * f), dtype=torch.bfloat16, device="cuda")
    h = c.forward(gate_up=gu)
    c.check_forward(h, gu)
    assert torch.equal(h, c.forward())


@pytest.mark.parametrize("counts, d, f", CASES)
def test_backward(stq, counts, d, f):
    c = Case(stq, counts, d, f, seed=len(counts) + d + 1)
    dx, dw = c.backward()
    c.check_backward(dx, dw)
    only_x, none = c.backward(need_dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = c.backward(need_dx=False)
    assert none is None and torch.equal(only_w, dw)


def test_odd_block_scales_and_expert_stride(stq):
    c = Case(stq, [20, 0, 50], 512, 256, seed=3, slack=4096, odd_scales=True)
    c.check_forward(c.forward())
    c.check_backward(*c.backward())


@pytest.mark.parametrize("counts, d, f, tail", [([1], 7168, 2048, 0), ([0, 3, 0, 17, 1, 0], 7168, 512, 5),
                                                 ([1, 1, 0, 2] * 10, 7168, 1024, 1), ([40], 7168, 1024, 0), ([1, 0, 5], 7168, 256, 3)])
def test_few_rows_through_the_gemv(stq, counts, d, f, tail):
    c = Case(stq, counts, d, f, seed=d + f, tail=tail)
    need = stq.grouped_swiglu_workspace(c.E, d, f, c.m)
    assert need > 0                                        # the GEMV's form
    h = torch.full((c.m, f), 3.0, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((c.m, 2 * f), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    c.forward(out=h, gate_up=gu, workspace=ws)
    c.check_forward(h, gu)
    used = c.bounds[-1]
    assert bool((h[used:] == 3.0).all()) and bool((gu[used:] == 3.0).all())
    assert torch.equal(c.forward()[:used], h[:used])
    c.x[0, 1] = float("nan")                               # stays in its row
    assert torch.equal(c.forward()[1:used], h[1:used])
    for bad in ([c.m + 7] * (c.E + 1), [-3] * (c.E + 1), list(range(c.E + 1))[::-1]):
        c.offsets.copy_(torch.tensor(bad, dtype=torch.int32))
        guard = torch.full((c.m + 8, f), 3.0, dtype=torch.bfloat16, device="cuda")
        c.forward(out=guard[:c.m])
        torch.cuda.synchronize()
        assert bool((guard[c.m:] == 3.0).all())


def test_few_rows_under_graph(stq):
    c = Case(stq, [1, 0, 2, 1], 7168, 512, seed=15)
    h = torch.empty((c.m, c.f), dtype=torch.bfloat16, device="cuda")
    need = stq.grouped_swiglu_workspace(c.E, c.d, c.f, c.m)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    c.forward(out=h, workspace=ws)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            c.forward(out=h, workspace=ws)
    torch.cuda.synchronize()
    for r in range(4):
        c.x.copy_(torch.randn(c.x.shape, generator=torch.Generator().manual_seed(r)).bfloat16())
        c.offsets.copy_(torch.tensor([[0, 1, 1, 3, 4], [0, 4, 4, 4, 4], [0, 0, 0, 0, 4], [0, 1, 2, 3, 4]][r], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = h.clone()
        assert torch.equal(got, c.forward()), r


def test_full_width_expert(stq):
    c = Case(stq, [0, 70, 131], 7168, 2048, seed=4)
    c.check_forward(c.forward())
    c.check_backward(*c.backward())


def test_rows_behind_the_last_expert_stay_as_they_were(stq):
    c = Case(stq, [5, 0, 40], 256, 256, seed=5, tail=23)
    h = torch.full((c.m, c.f), 3.0, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((c.m, 2 * c.f), 3.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((c.m, c.d), 3.0, dtype=torch.bfloat16, device="cuda")
    c.forward(out=h, gate_up=gu)
    _, dw = c.backward(dx=dx)
    for t in (h, gu, dx):
        assert bool((t[45:] == 3.0).all())
    c.check_forward(h, gu)
    c.check_backward(dx, dw)


def test_rows_of_uneven_experts_beyond_one_pass(stq):
    # hundreds of experts, most without rows, one with many passes: the passes are found on the device
    counts = [0] * 600
    counts[3], counts[255], counts[256], counts[599] = 500, 1, 81, 160
    c = Case(stq, counts, 256, 256, seed=14)
    c.check_forward(c.forward())
    dx, _ = c.backward(need_dw=False)
    c.check_backward(dx, None)


def test_nothing_routed(stq):
    c = Case(stq, [0, 0, 0], 256, 256)
    assert c.forward().shape == (0, 256)
    dx, dw = c.backward()
    assert dx.shape == (0, 256) and not dw.any()
    c = Case(stq, [0, 0], 256, 256, tail=7)
    h = torch.full((7, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    assert bool((c.forward(out=h) == 3.0).all())
    assert not c.backward(need_dx=False)[1].any()


@pytest.mark.parametrize("offsets", [[-5, 10, 20], [0, 90, 20], [0, 10, 500], [7, 3, 1]])
def test_offsets_outside_the_contract_stay_in_bounds(stq, offsets):
    c = Case(stq, [30, 20], 256, 256, seed=6)
    c.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
    guard = torch.full((c.m + 64, c.f), 3.0, dtype=torch.bfloat16, device="cuda")
    gx = torch.full((c.m + 64, c.d), 3.0, dtype=torch.bfloat16, device="cuda")
    c.forward(out=guard[:c.m])
    c.backward(dx=gx[:c.m])
    torch.cuda.synchronize()
    assert bool((guard[c.m:] == 3.0).all()) and bool((gx[c.m:] == 3.0).all())


def test_not_finite_rows_do_not_spread(stq):
    c = Case(stq, [40, 30], 512, 256, seed=7)
    clean = c.forward(), c.backward()
    c.x[11, 5] = float("nan")
    c.x[50, 7] = float("inf")
    c.dh[3, 9] = float("nan")
    c.dh[20, 100] = float("inf")
    c.dh[45] = 3e38                                        # overflows the row's fp32 products
    c.gu[45] = 4.0
    h, (dx, dw) = c.forward(), c.backward()
    rows = torch.arange(70, device="cuda")
    keep = (rows != 11) & (rows != 50)
    assert torch.equal(h[keep], clean[0][keep]) and torch.isnan(h[11].float()).all()
    keep = (rows != 3) & (rows != 20) & (rows != 45)
    assert torch.equal(dx[keep], clean[1][0][keep])
    assert not torch.isfinite(dx[3].float()).any() and not torch.isfinite(dx[20].float()).any()
    assert torch.isnan(dw[0].float()).any()


@pytest.mark.parametrize("std", [1e-30, 1e-12, 1e12])
def test_gradient_scale_does_not_matter(stq, std):
    # the fp16 form of dz is scaled row by row: tiny and huge gradients keep their digits
    c = Case(stq, [33, 20], 256, 256, seed=8)
    c.dh = (c.dh.float() * (std / 1e-3)).bfloat16()
    c.dh[4] = 0.0
    c.dh[5, 1:] = (c.dh[5, 1:].float() * 1e-6).bfloat16()   # one large entry beside small ones
    dx, dw = c.backward()
    c.check_backward(dx, dw)
    assert bool((dx[4] == 0).all())


def test_large_pre_activations(stq):
    c = Case(stq, [40], 256, 256, seed=9, x_std=30.0)
    c.gu = (c.gu.float() * 40).bfloat16()                  # silu saturated either way
    c.check_forward(c.forward())
    c.check_backward(*c.backward())


def test_gradients_against_differences(stq):
    """Central differences of the fp64 objective sum(dh h(z)) along random directions of x and of the
    weights; h's third derivative is below 2 in every |u| <= 8, so a step t leaves at most
    t^2 sum |dh| |dz/dt|^2 (|dz/dt| + 3) of it."""
    c = Case(stq, [9], 256, 256, seed=10)
    w = c.weights(0)
    x = c.x.double()
    z = x @ w.t().contiguous()
    c.gu = z.bfloat16()
    z0 = c.gu.double()                                     # the point the saved values name
    f = c.f
    dx, dw = c.backward()
    dz, err = c.dz_ref()

    def objective(z):
        g, u = z[:, :f], z[:, f:]
        return (c.dh.double() * g * torch.sigmoid(g) * u).sum()
    gen = torch.Generator().manual_seed(1)
    t = 1e-4
    for _ in range(4):
        v = torch.randn(x.shape, generator=gen).double().cuda()
        dzt = v @ w.t().contiguous()
        diff = (objective(z0 + t * dzt) - objective(z0 - t * dzt)) / (2 * t)
        third = t * t * (c.dh.double().abs().sum() * (dzt.abs().max() ** 2) * (dzt.abs().max() + 3) * 8)
        tol = (v.abs() * (c.dx_tol(dz, err, w) * (1 + B) + B * (dz @ w).abs())).sum() + third
        assert abs((dx.double() * v).sum() - diff) <= tol
        V = torch.randn(w.shape, generator=gen).double().cuda()
        dzt = x @ V.t().contiguous()
        t2 = 1e-5
        diff = (objective(z0 + t2 * dzt) - objective(z0 - t2 * dzt)) / (2 * t2)
        third = t2 * t2 * (c.dh.double().abs().sum() * (dzt.abs().max() ** 2) * (dzt.abs().max() + 3) * 8)
        lo = (err + 2 * B * dz.abs()).t().contiguous() @ x.abs()
        tol = (V.abs() * (lo + B * (dz.t().contiguous() @ x).abs())).sum() + third
        assert abs((dw[0].double() * V).sum() - diff) <= tol


def test_calls_repeat_bit_for_bit_whatever_the_workspace_held(stq):
    c = Case(stq, [70, 3, 150], 512, 512, seed=11)
    a = c.backward()
    need = stq.grouped_swiglu_backward_workspace(c.E, c.d, c.f, c.m)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    b = c.backward(workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(c.forward(), c.forward())


def test_step_under_graph_beside_another(stq):
    """Forward and backward of two sets of experts, each captured with a workspace of its own, replayed
    with new inputs and eager calls in between."""
    cases = [Case(stq, [30, 0, 90], 512, 256, seed=12), Case(stq, [140, 7], 256, 512, seed=13)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for c in cases:
        h = torch.empty((c.m, c.f), dtype=torch.bfloat16, device="cuda")
        dx = torch.empty((c.m, c.d), dtype=torch.bfloat16, device="cuda")
        dw = torch.empty((c.E, 2 * c.f, c.d), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(stq.grouped_swiglu_backward_workspace(c.E, c.d, c.f, c.m), dtype=torch.uint8, device="cuda")

        def call(c=c, h=h, dx=dx, dw=dw, ws=ws):
            c.forward(out=h, gate_up=c.gu)
            c.backward(dx=dx, dw=dw, workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                call()
        torch.cuda.synchronize()
        graphs.append(g)
        outs.append((h, dx, dw, ws))
    for r in range(4):
        for i, c in enumerate(cases):
            gen = torch.Generator().manual_seed(100 * r + i)
            c.x.copy_(torch.randn(c.x.shape, generator=gen).bfloat16())
            c.dh.copy_((torch.randn(c.dh.shape, generator=gen) * 0.1).bfloat16())
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for c, (h, dx, dw, _) in zip(cases, outs):
            got = h.clone(), dx.clone(), dw.clone()
            want = (c.forward(), *c.backward())
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), r


def test_binding_refusals(stq):
    c = Case(stq, [4, 4], 256, 256)
    with pytest.raises(ValueError, match="x_sorted must be"):
        stq.grouped_swiglu(c.table, c.stride, c.E, c.d, c.f, c.x[:, :128], c.offsets)
    with pytest.raises(ValueError, match="offsets must hold"):
        stq.grouped_swiglu(c.table, c.stride, c.E, c.d, c.f, c.x, c.offsets[:2])
    with pytest.raises(ValueError, match="w_gate_up holds"):
        stq.grouped_swiglu(c.table[:-1], c.stride, c.E, c.d, c.f, c.x, c.offsets)
    with pytest.raises(ValueError, match="gate_up must be"):
        stq.grouped_swiglu(*c.args(), gate_up=c.gu[:, :c.f].contiguous())
    with pytest.raises(stq.StqError, match="expert stride"):
        stq.grouped_swiglu(c.table, 16, c.E, c.d, c.f, c.x, c.offsets)
    with pytest.raises(ValueError, match="dh must be"):
        stq.grouped_swiglu_backward(*c.args(), c.gu, c.dh.float())
    with pytest.raises(ValueError, match="dw is given"):
        c.backward(need_dw=False, dw=torch.empty(2, 512, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(stq.StqError, match="workspace"):
        c.backward(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


LOADS = [1, 0, 16, 17, 33, 48, 49, 64, 65, 79, 80, 81, 95, 96, 97, 113, 127, 128, 129, 145, 159, 160, 161, 319, 320, 321, 333, 480]


@pytest.mark.parametrize("counts, d, f, odd", [([50, 300, 0, 200, 81, 112, 449, 1400], 2048, 1024, False),
                                               (LOADS * 5 + [3000], 256, 1024, False), (LOADS * 5, 768, 1024, True),
                                               ([20000, 1, 12345], 512, 256, True), (LOADS * 4 + [400] * 10, 1280, 2048, False),
                                               (LOADS * 19, 256, 256, True)])
def test_long_passes(stq, counts, d, f, odd):
    """Enough rows for passes of 80 and of 160, of every number of token tiles.

    Their sums change units between two blocks: a quotient and a product, so two roundings more every
    eight accumulations.  An accumulation rounds its result once and has 2 u above: u k / 32 of the
    bound is for these u k / 128."""
    c = Case(stq, counts, d, f, seed=len(counts), tail=5, odd_scales=odd, slack=256)
    h = torch.full((c.m, f), 3.0, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((c.m, 2 * f), 3.0, dtype=torch.bfloat16, device="cuda")
    c.forward(out=h, gate_up=gu)
    c.check_forward(h, gu)
    used = c.bounds[-1]
    assert bool((h[used:] == 3.0).all()) and bool((gu[used:] == 3.0).all())
    assert torch.equal(c.forward()[:used], h[:used])
    c.x[0, 1] = float("nan")                               # stays in its row
    assert torch.equal(c.forward()[1:used], h[1:used])
    for bad in ([c.m + 7] * (c.E + 1), [-3] * (c.E + 1), list(range(c.E + 1))[::-1]):
        c.offsets.copy_(torch.tensor(bad, dtype=torch.int32))
        guard = torch.full((c.m + 8, f), 3.0, dtype=torch.bfloat16, device="cuda")
        c.forward(out=guard[:c.m])
        torch.cuda.synchronize()
        assert bool((guard[c.m:] == 3.0).all())


def test_long_passes_with_blocks_of_no_scale(stq):
    """Rows whose blocks are all 0, whose first or last is, and an infinite or NaN scale, which stay in their columns."""
    counts, d, f = [160] * 130, 768, 1024
    c = Case(stq, counts, d, f, seed=7)
    blocks = c.table.view(c.E, -1)[:, :2 * f * (d // QK) * BLOCK].view(c.E, 2 * f // 64, d // QK, 64, BLOCK)
    zero = torch.tensor([0, 0], dtype=torch.uint8, device="cuda")
    blocks[:, 1, :, 5, :2] = zero                          # row 69
    blocks[:, 2, 0, 6, :2] = zero                          # row 134's first block
    blocks[:, 3, 2, 7, :2] = zero                          # row 199's last
    blocks[:, 4, 1, 8, :2] = torch.tensor([0, 128], dtype=torch.uint8, device="cuda")  # row 264: -0
    gu = torch.empty((c.m, 2 * f), dtype=torch.bfloat16, device="cuda")
    h = c.forward(gate_up=gu)
    c.check_forward(h, gu)
    assert bool((gu[:, 69] == 0).all()) and bool((h[:, 69] == 0).all())
    for at, bits in ((5, [0, 0x7C]), (6, [0, 0x7E])):      # rows 325 and 390
        blocks[0, at, 1, at, :2] = torch.tensor(bits, dtype=torch.uint8, device="cuda")
    bad = c.forward()
    keep = torch.ones(f, dtype=torch.bool, device="cuda")
    keep[[325, 390]] = False
    assert torch.equal(bad[:, keep], h[:, keep]) and torch.equal(bad[160:], h[160:])
    assert not bool(torch.isfinite(bad[:160, 390]).any())


@pytest.mark.parametrize("counts, d, f, odd", [(LOADS * 4 + [1500], 2048, 256, False), (LOADS * 5, 1280, 512, True),
                                               ([96] * 40 + [95, 97, 81, 1, 0, 66, 50], 3584, 256, False),
                                               ([9000, 1, 7000], 1024, 256, True), (LOADS * 12, 512, 256, True)])
def test_long_passes_of_the_gradients(stq, counts, d, f, odd):
    """Enough rows for passes of 96 in the gradient of x, of every number of token tiles."""
    c = Case(stq, counts, d, f, seed=len(counts) + 2, odd_scales=odd, slack=512)
    dx, dw = c.backward()
    c.check_backward(dx, dw)
    only_x, _ = c.backward(need_dw=False)
    assert torch.equal(only_x, dx)


def test_long_passes_under_graph_with_other_loads(stq):
    """One capture serves any spread of the same number of rows over the experts."""
    E, d, f, rows = 40, 1024, 512, 9000
    c = Case(stq, [rows // E] * E, d, f, seed=21)
    h = torch.empty((c.m, f), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((c.m, 2 * f), dtype=torch.bfloat16, device="cuda")
    dx = torch.empty((c.m, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(stq.grouped_swiglu_backward_workspace(E, d, f, c.m, True, False), dtype=torch.uint8, device="cuda")
    need = stq.grouped_swiglu_workspace(E, d, f, c.m)
    assert need == 0                                       # the matrix cores' form

    def call():
        c.forward(out=h, gate_up=gu)
        c.stq.grouped_swiglu_backward(*c.args(), gu, c.dh, need_dw=False, dx=dx, workspace=ws)
    call()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.synchronize()
    rng = np.random.default_rng(3)
    for loads in (rng.multinomial(rows, np.ones(E) / E), rng.multinomial(rows, 1 / np.arange(1, E + 1) / (1 / np.arange(1, E + 1)).sum()),
                  np.eye(E, dtype=int)[7] * rows, np.minimum(np.arange(E), 1) * (rows // (E - 1))):
        c.bounds = [0] + np.cumsum(loads).tolist()
        c.offsets.copy_(torch.tensor(c.bounds, dtype=torch.int32))
        c.x.copy_(torch.randn(c.x.shape, generator=torch.Generator().manual_seed(int(loads[1]))).bfloat16())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        used = c.bounds[-1]
        got = h[:used].clone(), gu[:used].clone(), dx[:used].clone()
        gu2 = torch.empty_like(gu)
        eager = c.forward(gate_up=gu2)
        dx2, _ = c.stq.grouped_swiglu_backward(*c.args(), gu2, c.dh, need_dw=False)
        assert all(torch.equal(a, b[:used]) for a, b in zip(got, (eager, gu2, dx2)))
        c.check_forward(eager, gu2)


def test_gradient_of_x_eight_bytes_into_a_buffer(stq):
    """dx needs 8-byte alignment only, and nothing beside it is written."""
    c = Case(stq, [70, 0, 33, 5], 512, 256, seed=31)
    want, _ = c.backward(need_dw=False)
    buf = torch.full((c.m * c.d + 8,), 3.0, dtype=torch.bfloat16, device="cuda")
    dx = buf[4:4 + c.m * c.d].view(c.m, c.d)
    c.backward(need_dw=False, dx=dx)
    assert torch.equal(dx, want)
    assert bool((buf[:4] == 3.0).all()) and bool((buf[4 + c.m * c.d:] == 3.0).all())


@pytest.mark.parametrize("at, counts", [(0, [40, 0, 70, 100]), (1, [1, 16, 33]), (255, LOADS * 12), (511, [40, 0, 70, 100])])
@pytest.mark.parametrize("steps, large", [(848, 17.0), (1000, 30.0), (26.5 * 2 ** 15, 3.0e4), (10.5 * 2 ** 15, 3.0e4),
                                          (33000, 6.0e4), (40000, 6.0e4)])
def test_gradient_of_x_beside_rows_of_a_large_scale(stq, steps, large, at, counts):
    """Rows of W whose scales are small, `steps` of fp16's subnormal ones, beside rows with a large one
    through which no gradient flows (dh is 0 there): what the small ones carry keeps its digits, however
    far below the largest they lie, wherever that one stands.

    Weights and dz are positive, so nothing cancels: an element errs by fp16's f for dz and once more for
    its product with the scale, the accumulation (module docstring) and its own rounding, relative to
    itself.  dz's lie within a factor of 6.2 of each other (dg up to 1.1 * 2e-3 * 2, du from 0.73e-3), so
    scaled they are above 2^14 / 6.2 and their products with 2^-25 (33000 steps beside a D of 2^16) above
    2^-13.7: normal fp16 numbers."""
    d, f = 512, 256
    c = Case(stq, counts, d, f, seed=int(steps) + at)
    blocks = c.table.view(c.E, 2 * f // 64, d // QK, 64, BLOCK)
    blocks[..., 2:34] &= 0x88                              # sign bits 0: three +d and a zero a group
    scale = torch.full((2 * f,), steps * 2.0 ** -24)
    scale[[at, at ^ f]] = large                            # a gate row and the up row of the same column
    scale = scale.half().view(torch.uint8).view(1, 2 * f // 64, 1, 64, 2).cuda()
    blocks[..., :2] = scale
    g = torch.Generator().manual_seed(at)
    c.gu = (1.0 + torch.rand(c.gu.shape, generator=g)).bfloat16().cuda()
    c.dh = (1e-3 * (1.0 + torch.rand(c.dh.shape, generator=g))).bfloat16().cuda()
    c.dh[:, at % f] = 0.0
    dx, _ = c.backward(need_dw=False)
    F = 2.0 ** -11
    dz, err = c.dz_ref()
    assert bool((dz >= 0).all())
    for e, (lo, hi) in enumerate(zip(c.bounds, c.bounds[1:])):
        if lo == hi:
            continue
        w = c.weights(e)
        assert bool((w >= 0).all()) and w[at].max() == torch.tensor(large).half().item()
        ref = dz[lo:hi] @ w
        tol = ((err[lo:hi] @ w) * (1 + F) + (2 * F + F * F + 2 * U * (2 * f / 32 + 40)) * ref) * (1 + B) + B * ref
        bad = ((dx[lo:hi].double() - ref).abs() - tol).amax()
        assert bad <= 0, (e, (dx[lo:hi].double() / ref - 1).abs().max().item())


def test_gradients_without_the_operand_of_the_other(stq):
    """dx reads no x and dw no weights: the one not wanted needs none."""
    c = Case(stq, [40, 0, 33], 512, 256, seed=41, tail=3)
    dx, dw = c.backward()
    dims = c.E, c.d, c.f
    only_x, none = stq.grouped_swiglu_backward(c.table, c.stride, *dims, None, c.offsets, c.gu, c.dh, need_dw=False)
    assert none is None and torch.equal(only_x[:73], dx[:73])
    none, only_w = stq.grouped_swiglu_backward(None, 0, *dims, c.x, c.offsets, c.gu, c.dh, need_dx=False)
    assert none is None and torch.equal(only_w, dw)
    with pytest.raises(ValueError, match="dx needs w_gate_up"):
        stq.grouped_swiglu_backward(None, 0, *dims, c.x, c.offsets, c.gu, c.dh)
    with pytest.raises(ValueError, match="dw needs x_sorted"):
        stq.grouped_swiglu_backward(c.table, c.stride, *dims, None, c.offsets, c.gu, c.dh)
    with pytest.raises(ValueError, match="x_sorted must be"):
        stq.grouped_swiglu_backward(c.table, c.stride, *dims, c.x[:-1], c.offsets, c.gu, c.dh)
    with pytest.raises(ValueError, match="gate_up must be"):
        stq.grouped_swiglu_backward(c.table, c.stride, *dims, c.x, c.offsets, c.gu[0], c.dh)


@pytest.mark.parametrize("counts, d, f, odd", [(LOADS, 512, 512, False), (LOADS * 2, 768, 256, True), (LOADS * 3, 1280, 256, False)])
def test_passes_of_80(stq, counts, d, f, odd):
    """Every number of token tiles that passes of 80 have, cut from loads of up to 480 rows (tolerances as in
    test_long_passes)."""
    c = Case(stq, counts, d, f, seed=len(counts) + 9, tail=2, odd_scales=odd, slack=256)
    assert stq.grouped_swiglu_plan(c.E, d, f, c.m) == 80
    gu = torch.full((c.m, 2 * f), 3.0, dtype=torch.bfloat16, device="cuda")
    h = c.forward(out=torch.full((c.m, f), 3.0, dtype=torch.bfloat16, device="cuda"), gate_up=gu)
    c.check_forward(h, gu)
    assert bool((h[-2:] == 3.0).all()) and bool((gu[-2:] == 3.0).all())
