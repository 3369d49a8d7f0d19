"""Routing, its gradient, and the combination of expert rows against 64-bit
arithmetic.

Experts, counts, offsets and rows are compared exactly.  Tolerances (u =
2^-24): a term exp(l - m) errs by u (3 |l - m| + 4) relative (difference,
product and constant of the exponent, one step of exp2); a sum of E of them by
u (3 T + J + 4) with T = sum p |l - m| and J = E / 16 + 10 additions at most, so
p and w by R = u (3 |l - m| + 3 T + J + 16).  The balance adds p over a chunk's
passes, lanes, wavefronts and the chunks (24 + n / 4096 additions of positive
terms), then E / 64 + 12 more with the counts.  In the gradient every factor
errs by R, every dot product by its terms' magnitudes times 2 R + J u, and the
output by its type's half step.  What is below 2^-126 may be flushed."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -126
INF = float("inf")


@pytest.fixture(scope="module")
def stq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_ternary_bit_amd as m
    return m


def _logits(n, e, dtype, seed, pads=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, e), generator=g) + torch.randn((e,), generator=g)
    if pads:
        x[torch.randperm(n, generator=g)[:pads]] = -INF
    return x.to(dtype)


def _ref(x, k, renorm):
    """On the host, in 64 bits, for rows of numbers and -inf."""
    l = x.double()
    n, e = l.shape
    live = ~torch.isneginf(l).all(1)
    order = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :k]
    m = torch.where(live, l.amax(1), 0.0)[:, None]
    ex = torch.exp(l - m)
    s = torch.where(live[:, None], ex.sum(1, keepdim=True), 1.0)
    p = ex / s
    w = ex.gather(1, order)
    w = w / torch.where(live[:, None], w.sum(1, keepdim=True), 1.0) if renorm else p.gather(1, order)
    gap = torch.where(torch.isneginf(l), 0.0, (l - m).abs())
    T = (p * gap).sum(1, keepdim=True)
    R = U * (3 * gap + 3 * T + e / 16 + 10 + 16)
    expert = torch.where(live[:, None], order, -1)
    flat = torch.where(expert.reshape(-1) < 0, e, expert.reshape(-1))
    by = torch.sort(flat, stable=True)[1]
    counts = torch.bincount(flat, minlength=e + 1)[:e]
    total = int(counts.sum())
    row = torch.full((n * k,), -1)
    row[by[:total]] = torch.arange(total)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    token = torch.where(torch.arange(n * k) < total, by // k, 0)
    w = torch.where(live[:, None], w, 0.0)
    balance = (e * (counts.double() / max(total, 1)) * (p.sum(0) / max(int(live.sum()), 1))).sum()
    return dict(l=l, live=live, order=order, p=p, w=w, R=R, expert=expert, counts=counts, offsets=offsets, row=row, token=token,
                by=by, total=total, balance=balance, m=m, gap=gap)


def _check(got, x, k, renorm):
    r = _ref(x, k, renorm)
    n, e = x.shape
    got = type(got)(*(t.cpu() for t in got))
    assert torch.equal(got.pair_expert.long().view(n, k), r["expert"])
    assert torch.equal(got.counts.long(), r["counts"]) and torch.equal(got.offsets.long(), r["offsets"])
    assert torch.equal(got.pair_row.long(), r["row"]) and torch.equal(got.row_token.long(), r["token"])
    tol = 2 * r["R"].gather(1, r["order"]) * r["w"] + TINY
    assert bool(((got.pair_weight.double().view(n, k) - r["w"]).abs() <= tol).all())
    want = torch.zeros(n * k)
    want[:r["total"]] = got.pair_weight[r["by"][:r["total"]]]
    assert torch.equal(got.row_weight, want)
    worst = r["R"].max().item() + U * (24 + n / 4096 + e / 64 + 12)
    assert abs(got.balance.double().item() - r["balance"].item()) <= worst * r["balance"].item() + TINY
    return r


CASES = [(1, 256, 8), (1, 1, 1), (2, 3, 3), (5, 17, 4), (64, 256, 8), (65, 256, 8), (63, 64, 1), (200, 60, 6), (129, 130, 32),
         (1000, 512, 8), (70, 1000, 31), (66, 1024, 32), (40, 1024, 2), (4097, 128, 2), (300, 33, 17), (33, 100, 16)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("n, e, k", CASES)
def test_routing(stq, n, e, k, renorm, dtype):
    x = _logits(n, e, dtype, n + e + k)
    _check(stq.route_tokens(x.cuda(), k, renorm), x, k, renorm)


def test_probabilities_far_below_the_largest(stq):
    # Two experts x = 0 and -i / 8, whose difference is exact: exp errs by 3 u (2 u the instruction, u its last step),
    # the sum by as much and u more, its reciprocal and the product by u each: 9 u at any distance.  In the gradient at
    # the lower expert, p (1 - p) with g = 1 there alone, the second factor adds at most 9 u p / (1 - p) + 2 u and the
    # last product u.
    low = torch.arange(1, 680) / 8.0
    x = torch.stack([torch.zeros_like(low), -low], 1)
    p = 1.0 / (1.0 + torch.exp(low.double()))
    r = stq.route_tokens(x.cuda(), 2, False)
    got = r.pair_weight.cpu().double().view(-1, 2)
    assert bool(((got[:, 1] - p).abs() <= 9 * U * p).all()) and bool(((got[:, 0] - (1 - p)).abs() <= 9 * U * (1 - p)).all())
    g = torch.tensor([0.0, 1.0]).repeat(len(low))
    d = stq.route_tokens_backward(x.cuda(), r.pair_expert, None, 2, False, grad_weight=g.cuda()).cpu().double()
    want = p * (1 - p)
    assert bool(((d[:, 1] - want).abs() <= U * (12 + 9 * p / (1 - p)) * want).all())


# more chunks than the prefix sums take at once
@pytest.mark.parametrize("n, e, k, pads", [(16450, 20, 2, 300), (33000, 70, 3, 0), (49153, 5, 1, 7)])
def test_routing_of_long_prompts(stq, n, e, k, pads):
    x = _logits(n, e, torch.float32, n, pads)
    _check(stq.route_tokens(x.cuda(), k), x, k, True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, e, k, pads", [(1, 16, 2, 1), (50, 64, 4, 20), (500, 256, 8, 77), (130, 40, 3, 130), (64, 512, 8, 64)])
def test_padding(stq, n, e, k, pads, dtype):
    x = _logits(n, e, dtype, 3, pads)
    _check(stq.route_tokens(x.cuda(), k), x, k, True)


@pytest.mark.parametrize("n", [6, 300])
def test_ties_go_to_the_lowest_expert(stq, n):
    g = torch.Generator().manual_seed(n)
    for e, k in [(256, 8), (40, 32), (1000, 20)]:
        x = torch.randint(-2, 3, (n, e), generator=g).float()
        x[:, 3] = -0.0
        _check(stq.route_tokens(x.cuda(), k), x, k, True)
        _check(stq.route_tokens(x.bfloat16().cuda(), k), x.bfloat16(), k, True)
        same = torch.zeros(n, e)
        same[:, ::2] = -0.0
        _check(stq.route_tokens(same.cuda(), k, False), same, k, False)


@pytest.mark.parametrize("n", [5, 200])
def test_logits_that_differ_in_their_last_bits(stq, n):
    # equal in the 22 bits of a key, different in 32, in orders that the index alone would get wrong
    g = torch.Generator().manual_seed(n)
    base = torch.full((n, 256), 1.0)
    steps = torch.stack([torch.randperm(256, generator=g) for _ in range(n)])
    x = (base.view(torch.int32) + steps.int()).view(torch.float32)
    _check(stq.route_tokens(x.cuda(), 8), x, 8, True)
    neg = -x
    _check(stq.route_tokens(neg.cuda(), 8), neg, 8, True)
    mixed = _logits(n, 256, torch.float32, 1)
    mixed[::2, :40] = 5.0 + steps[::2, :40] * 2.0 ** -21
    _check(stq.route_tokens(mixed.cuda(), 8), mixed, 8, True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_experts(stq, dtype):
    x = _logits(150, 96, dtype, 4)
    x[:, 10:] = -INF                      # fewer left than are chosen: the lowest masked ones follow, with weight 0
    x[7, 1:] = -INF
    x[9, 2] = torch.finfo(dtype).min
    x[11] = torch.finfo(dtype).min        # masked by the type's lowest value throughout: all alike
    _check(stq.route_tokens(x.cuda(), 12), x, 12, True)
    _check(stq.route_tokens(x.cuda(), 12, False), x, 12, False)
    big = x * 1e30 if dtype == torch.float32 else x
    _check(stq.route_tokens(big.cuda(), 5), big, 5, True)


@pytest.mark.parametrize("n", [20, 200])
def test_tokens_without_a_distribution(stq, n):
    x = _logits(n, 64, torch.float32, 8)
    x[3, 5] = float("nan")
    x[17, 63] = INF
    clean = x.clone()
    clean[[3, 17]] = -INF
    r = _ref(clean, 4, True)
    got = stq.route_tokens(x.cuda(), 4)
    assert torch.equal(got.pair_expert.cpu().long().view(n, 4), r["expert"])
    assert torch.equal(got.offsets.cpu().long(), r["offsets"]) and torch.equal(got.pair_row.cpu().long(), r["row"])
    w = got.pair_weight.cpu().view(n, 4)
    assert bool(torch.isnan(w[[3, 17]]).all()) and bool(torch.isfinite(w[[0, 1, 2, 4, 5, 19]]).all())
    assert torch.isnan(got.balance).item() and bool(torch.isfinite(got.row_weight).all())
    d = stq.route_tokens_backward(x.cuda(), got.pair_expert, got.counts, 4, grad_weight=torch.ones(4 * n, device="cuda"))
    assert bool(torch.isnan(d[[3, 17]]).all()) and bool(torch.isfinite(d[[0, 1, 2, 4, 5, 19]]).all())


@pytest.mark.parametrize("n", [0, 3, 100])
def test_no_tokens_and_given_outputs(stq, n):
    x = _logits(n, 40, torch.float32, 2)
    wide = torch.zeros(max(n, 1), 43, device="cuda")[:n]
    wide[:, 1:41] = x.cuda()
    first = stq.route_tokens(x.cuda(), 3)
    out = stq.Routing(*(torch.full_like(t, 5) for t in first))
    got = stq.route_tokens(wide[:, 1:41], 3, out=out)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(got, first))
    if n == 0:
        assert not got.counts.any() and not got.offsets.any() and got.balance.item() == 0.0
    d = stq.route_tokens_backward(wide[:, 1:41], got.pair_expert, got.counts, 3, grad_balance=torch.ones(1, device="cuda"))
    assert d.shape == (n, 40)


def _bwd_ref(x, k, renorm, r, g, gb):
    n, e = x.shape
    p, R, live = r["p"], r["R"], r["live"][:, None]
    order = r["order"]
    if r["total"]:
        c = gb * e * (r["counts"].double() / r["total"]) / (r["total"] / k)
    else:
        c = torch.zeros(e, dtype=torch.float64)
    d = p * (c - (p * c).sum(1, keepdim=True))
    S = (p * c.abs()).sum(1, keepdim=True)
    Rm = R.amax(1, keepdim=True)
    tol = p * (4 * R * (c.abs() + S) + 4 * Rm * S)
    if renorm:
        w = torch.where(live, r["w"], 0.0)
        S = (w * g.abs()).sum(1, keepdim=True)
        dc = w * (g - (w * g).sum(1, keepdim=True))
        tc = w * (8 * Rm * (g.abs() + 2 * S))
        d = d.scatter_add(1, order, dc)
        tol = tol.scatter_add(1, order, tc)
    else:
        full = torch.zeros_like(p).scatter_add(1, order, g)
        S2 = (p * full.abs()).sum(1, keepdim=True)
        d = d + p * (full - (p * full).sum(1, keepdim=True))
        tol = tol + p * (4 * R * (full.abs() + S2) + 4 * Rm * (S2 + full.abs()))
    d, tol = torch.where(live, d, 0.0), torch.where(live, tol, 0.0)
    half = B if x.dtype == torch.bfloat16 else U
    return d, tol * (1 + half) + (half + 2 * U) * d.abs() + TINY


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("n, e, k, pads", [(1, 256, 8, 0), (1, 1, 1, 0), (37, 17, 4, 5), (100, 256, 8, 9), (66, 1024, 32, 3),
                                           (300, 60, 6, 0), (65, 512, 20, 65), (1000, 128, 2, 50)])
def test_gradient(stq, n, e, k, pads, renorm, dtype):
    x = _logits(n, e, dtype, n + e, pads)
    r = _ref(x, k, renorm)
    got = stq.route_tokens(x.cuda(), k, renorm)
    gen = torch.Generator().manual_seed(1)
    g, gb = torch.randn(n * k, generator=gen), 0.7
    b = torch.full((1,), gb, device="cuda")
    gb = float(b.item())
    want, tol = _bwd_ref(x, k, renorm, r, g.double().view(n, k), gb)
    d = stq.route_tokens_backward(x.cuda(), got.pair_expert, got.counts, k, renorm, grad_weight=g.cuda(), grad_balance=b)
    assert bool(((d.cpu().double() - want).abs() <= tol).all())
    # the same gradient in the order of the sorted rows, pads' shares anywhere
    rows = torch.full((n * k,), 9.0)
    on = r["row"] >= 0
    rows[r["row"][on]] = g[on]
    in_rows = stq.route_tokens_backward(x.cuda(), got.pair_expert, got.counts, k, renorm, grad_weight=rows.cuda(),
                                        pair_row=got.pair_row, grad_balance=b)
    assert torch.equal(in_rows, d)
    for only in (dict(grad_weight=g.cuda()), dict(grad_balance=b), dict()):
        want, tol = _bwd_ref(x, k, renorm, r, g.double().view(n, k) * ("grad_weight" in only), gb * ("grad_balance" in only))
        d1 = stq.route_tokens_backward(x.cuda(), got.pair_expert, got.counts, k, renorm, **only)
        assert bool(((d1.cpu().double() - want).abs() <= tol).all())
    xc = x.cuda()
    assert torch.equal(stq.route_tokens_backward(xc, got.pair_expert, got.counts, k, renorm, g.cuda(), None, b, out=xc), d)


# wavefronts of four tokens of which the last few are missing, and more tokens than the workgroups of a launch take at once
@pytest.mark.parametrize("n, e, k", [(n, 20, 3) for n in list(range(1, 20)) + [31, 33]] + [(131100, 6, 2), (131083, 5, 1)])
def test_gradient_of_every_number_of_tokens(stq, n, e, k):
    x = _logits(n, e, torch.float32, n, n // 7)
    r = _ref(x, k, True)
    got = stq.route_tokens(x.cuda(), k)
    g = torch.randn(n * k, generator=torch.Generator().manual_seed(n))
    b = torch.full((1,), 0.5, device="cuda")
    want, tol = _bwd_ref(x, k, True, r, g.double().view(n, k), 0.5)
    wide = torch.full((n + 1, e), 7.0, device="cuda")
    d = stq.route_tokens_backward(x.cuda(), got.pair_expert, got.counts, k, grad_weight=g.cuda(), grad_balance=b, out=wide[:n])
    assert bool(((d.cpu().double() - want).abs() <= tol).all()) and bool((wide[n] == 7).all())


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(stq, renorm):
    # differences of the 64-bit weights and balance with the choice and the counts held, the step far from any tie
    n, e, k, step = 6, 12, 3, 1e-6
    x = _logits(n, e, torch.float32, 5)
    got = stq.route_tokens(x.cuda(), k, renorm)
    g = torch.randn(n, k, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    order, counts = got.pair_expert.cpu().long().view(n, k), got.counts.cpu().double()

    def loss(l):
        p = torch.softmax(l, 1)
        w = p.gather(1, order)
        w = w / w.sum(1, keepdim=True) if renorm else w
        return ((g * w).sum() + 2.5 * e * (counts / (n * k) * p.mean(0)).sum()).item()
    d = stq.route_tokens_backward(x.cuda(), got.pair_expert, got.counts, k, renorm, grad_weight=g.float().reshape(-1).cuda(),
                                  grad_balance=torch.full((1,), 2.5, device="cuda")).cpu()
    for i, j in [(0, 0), (3, 7), (5, 11), (2, int(order[2, 0])), (4, int(order[4, 2]))]:
        s = torch.zeros(n, e, dtype=torch.float64)
        s[i, j] = step
        diff = (loss(x.double() + s) - loss(x.double() - s)) / (2 * step)
        assert abs(diff - d[i, j].item()) < 1e-5


# ---- combination --------------------------------------------------------

def _pairs(n, k, extra, dropped, seed):
    """pair_row of n tokens: distinct rows out of n * k + extra, some pairs without one."""
    g = torch.Generator().manual_seed(seed)
    row = torch.randperm(n * k + extra, generator=g)[:n * k].int()
    row[torch.randperm(n * k, generator=g)[:dropped]] = -1
    return row, torch.randn(n * k, generator=g)


def _combine_ref(z, row, w, k, out):
    on = (row >= 0) & (row < len(z))
    terms = torch.zeros(len(row), z.shape[1], dtype=torch.float64)
    terms[on] = z.double()[row[on].long()] * (1.0 if w is None else w.double()[on, None])
    terms = terms.view(-1, k, z.shape[1])
    y = terms.sum(1)
    half = B if out == torch.bfloat16 else U
    return y, (k + 1) * U * terms.abs().sum(1) * (1 + half) + half * y.abs() + TINY


@pytest.mark.parametrize("zt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("yt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, k, d", [(1, 1, 1), (1, 8, 7168), (3, 2, 65), (40, 8, 4099), (7, 9, 512), (5, 32, 520), (300, 3, 264)])
def test_combine(stq, n, k, d, zt, yt):
    row, w = _pairs(n, k, 3, n * k // 5, n + d)
    z = torch.randn((n * k + 3, d), generator=torch.Generator().manual_seed(d)).to(zt)
    unused = torch.ones(len(z), dtype=torch.bool)
    unused[row[row >= 0].long()] = False
    z[unused] = float("nan")                # rows of no pair are not looked at
    for weight in (None, w):
        y = stq.combine_rows(z.cuda(), row.cuda(), k, weight=None if weight is None else weight.cuda(), out_dtype=yt)
        want, tol = _combine_ref(z, row, weight, k, yt)
        assert y.dtype == yt and bool(((y.cpu().double() - want).abs() <= tol).all())
    # rows beyond z count for nothing
    cut = max(1, len(z) // 2)
    y = stq.combine_rows(z[:cut].cuda(), row.cuda(), k, weight=w.cuda(), out_dtype=yt)
    want, tol = _combine_ref(z[:cut], row, w, k, yt)
    assert bool(((y.cpu().double() - want).abs() <= tol).all())


def test_combine_nothing(stq):
    row = torch.full((12,), -1, dtype=torch.int32, device="cuda")
    for rows in (0, 4):
        z = torch.full((rows, 40), float("nan"), device="cuda")
        assert not stq.combine_rows(z, row, 3).any()
        dz, dw = stq.combine_rows_backward(torch.ones(4, 40, device="cuda"), row, 3, z)
        assert not dw.any()
    assert stq.combine_rows(z, row[:0], 3).shape == (0, 40)
    dz, dw = stq.combine_rows_backward(z[:0], row[:0], 3, z, dz=z)
    assert dw.shape == (0,) and bool(torch.isnan(dz).all())


@pytest.mark.parametrize("yt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("zt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, k, d", [(1, 1, 1), (1, 8, 7168), (3, 2, 65), (40, 8, 4099), (7, 9, 512), (5, 32, 520), (300, 3, 264)])
def test_combine_gradients(stq, n, k, d, yt, zt, dt):
    row, w = _pairs(n, k, 3, n * k // 5, n + d)
    g = torch.Generator().manual_seed(d)
    z, dy = torch.randn((n * k + 3, d), generator=g).to(zt), torch.randn((n, d), generator=g).to(yt)
    dz = torch.full((n * k + 3, d), 7.0, dtype=dt, device="cuda")
    got = stq.combine_rows_backward(dy.cuda(), row.cuda(), k, z.cuda(), weight=w.cuda(), dz=dz)
    assert got[0].data_ptr() == dz.data_ptr()
    want = torch.full((n * k + 3, d), 7.0, dtype=torch.float64)
    on = row >= 0
    share = dy.double().repeat_interleave(k, 0)
    want[row[on].long()] = share[on] * w.double()[on, None]
    half = B if dt == torch.bfloat16 else 0.0
    assert bool(((dz.cpu().double() - want).abs() <= (U * (1 + half) + half) * want.abs() + TINY).all())
    terms = torch.zeros(n * k, d, dtype=torch.float64)
    terms[on] = share[on] * z.double()[row[on].long()]
    tol = (8 * -(-d // 512) + 24) * U * terms.abs().sum(1) + TINY
    assert bool(((got[1].cpu().double() - terms.sum(1)).abs() <= tol).all())
    ones, none = stq.combine_rows_backward(dy.cuda(), row.cuda(), k, z.cuda(), need_dweight=False, dz_dtype=dt)
    assert none is None and torch.equal(ones.cpu()[row[on].long()], dy.repeat_interleave(k, 0)[on].to(dt))
    none, dw = stq.combine_rows_backward(dy.cuda(), row.cuda(), k, z.cuda(), weight=w.cuda(), need_dz=False)
    assert none is None and torch.equal(dw, got[1])


@pytest.mark.parametrize("d", list(range(8, 26)) + list(range(1200, 1208)))
def test_combine_every_end_of_a_row(stq, d):
    n, k = 9, 3
    row, w = _pairs(n, k, 2, 4, d)
    on = row >= 0
    for zt, yt in ((torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        g = torch.Generator().manual_seed(d)
        z, dy = torch.randn((n * k + 2, d), generator=g).to(zt), torch.randn((n, d), generator=g).to(yt)
        want, tol = _combine_ref(z, row, w, k, yt)
        assert bool(((stq.combine_rows(z.cuda(), row.cuda(), k, w.cuda(), out_dtype=yt).cpu().double() - want).abs() <= tol).all())
        dz, dw = stq.combine_rows_backward(dy.cuda(), row.cuda(), k, z.cuda(), w.cuda(), dz_dtype=torch.float32)
        share = dy.double().repeat_interleave(k, 0)
        want = share[on] * w.double()[on, None]
        assert bool(((dz.cpu().double()[row[on].long()] - want).abs() <= U * want.abs() + TINY).all())
        terms = torch.zeros(n * k, d, dtype=torch.float64)
        terms[on] = share[on] * z.double()[row[on].long()]
        tol = (8 * -(-d // 512) + 24) * U * terms.abs().sum(1) + TINY
        assert bool(((dw.cpu().double() - terms.sum(1)).abs() <= tol).all())


def test_combine_strides_and_offsets(stq):
    n, k, d = 20, 4, 300
    row, w = (t.cuda() for t in _pairs(n, k, 0, 5, 1))
    g = torch.Generator().manual_seed(3)
    z, dy = torch.randn((n * k, d), generator=g).cuda(), torch.randn((n, d), generator=g).cuda()
    want, (want_dz, want_dw) = stq.combine_rows(z, row, k, w), stq.combine_rows_backward(dy, row, k, z, w, dz=torch.zeros_like(z))
    zw, yw = torch.full((n * k, d + 5), 7.0, device="cuda"), torch.full((n, d + 3), 7.0, device="cuda")
    dyw, dzw = torch.full((n, d + 1), 7.0, device="cuda"), torch.zeros((n * k, d + 2), device="cuda")
    zw[:, 1:d + 1], dyw[:, 1:] = z, dy
    assert torch.equal(stq.combine_rows(zw[:, 1:d + 1], row, k, w, out=yw[:, 2:d + 2]), want)
    assert bool((yw[:, :2] == 7).all()) and bool((yw[:, d + 2:] == 7).all())
    dz, dw = stq.combine_rows_backward(dyw[:, 1:], row, k, zw[:, 1:d + 1], w, dz=dzw[:, 1:d + 1])
    assert torch.equal(dz, want_dz) and torch.equal(dw, want_dw) and not dzw[:, 0].any() and not dzw[:, d + 1].any()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, k, d", [(9, 3, 87), (5, 32, 1203), (40, 8, 4099), (3, 2, 264)])
def test_combine_gradient_in_the_rows_place(stq, n, k, d, dt):
    row, w = (t.cuda() for t in _pairs(n, k, 3, n * k // 5, n + d))
    g = torch.Generator().manual_seed(d)
    z, dy = torch.randn((n * k + 3, d), generator=g).to(dt).cuda(), torch.randn((n, d), generator=g).cuda()
    want, want_dw = stq.combine_rows_backward(dy, row, k, z, w, dz=z.clone())
    got, dw = stq.combine_rows_backward(dy, row, k, z, w, dz=z)
    assert got.data_ptr() == z.data_ptr() and torch.equal(got, want) and torch.equal(dw, want_dw)


def test_rows_past_32_bits(stq):
    # rows of z that start beyond 2^32 bytes and 2^31 elements
    rows, d = 600, 4_000_000
    z = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    z[599] = 3.0
    z[1] = 1.0
    row = torch.tensor([599, 1, 0, 599], dtype=torch.int32, device="cuda")
    y = stq.combine_rows(z, row[:2], 2)
    assert bool((y == 4.0).all())
    dz, dw = stq.combine_rows_backward(torch.ones((1, d), dtype=torch.bfloat16, device="cuda"), row[:2], 2, z, dz=z)
    assert bool((z[599] == 1).all()) and bool((z[1] == 1).all()) and not z[2:599].any()


def test_under_a_graph_with_work_between(stq):
    n, e, k, d = 700, 128, 4, 512
    x = _logits(n, e, torch.float32, 1, 20).cuda()
    z = torch.randn(n * k, d, device="cuda")
    gb = torch.ones(1, device="cuda")
    r = stq.route_tokens(x, k)
    ws = torch.empty(stq.route_tokens_workspace(n, e, k), dtype=torch.uint8, device="cuda")
    y, dz, dw, dl = torch.empty(n, d, device="cuda"), torch.zeros_like(z), torch.empty(n * k, device="cuda"), torch.empty_like(x)

    def call(r, ws, y, dz, dw, dl):
        r = stq.route_tokens(x, k, out=r, workspace=ws)
        y = stq.combine_rows(z, r.pair_row, k, r.pair_weight, out=y)
        dz, dw = stq.combine_rows_backward(y, r.pair_row, k, z, r.pair_weight, dz=dz, dweight=dw)
        dl = stq.route_tokens_backward(x, r.pair_expert, r.counts, k, grad_weight=dw, grad_balance=gb, out=dl)
        return [*r, y, dz, dw, dl]
    call(r, ws, y, dz, dw, dl)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            outs = call(r, ws, y, dz, dw, dl)
    torch.cuda.synchronize()
    for i in range(4):
        x.copy_(_logits(n, e, torch.float32, 30 + i, 10 * i))
        dz.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = call(None, None, None, torch.zeros_like(z), None, None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_binding_refusals(stq):
    x = torch.zeros(4, 16, device="cuda")
    with pytest.raises(stq.StqError, match="top_k"):
        stq.route_tokens(x, 17)
    with pytest.raises(stq.StqError, match="top_k"):
        stq.route_tokens(x, 0)
    with pytest.raises(stq.StqError, match="n_experts"):
        stq.route_tokens(torch.zeros(2, 1025, device="cuda"), 2)
    with pytest.raises(ValueError, match="logits must be"):
        stq.route_tokens(x.double(), 2)
    with pytest.raises(ValueError, match="contiguous rows"):
        stq.route_tokens(x.t(), 2)
    r = stq.route_tokens(x, 2)
    with pytest.raises(ValueError, match="counts must hold"):
        stq.route_tokens(x, 2, out=r._replace(counts=r.counts[:3]))
    with pytest.raises(ValueError, match="must be a Routing"):
        stq.route_tokens(x, 2, out=tuple(r))
    big = torch.zeros(100, 16, device="cuda")
    with pytest.raises(stq.StqError, match="workspace"):
        stq.route_tokens(big, 2, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="pair_expert must hold 8"):
        stq.route_tokens_backward(x, r.pair_expert[:6], r.counts, 2)
    with pytest.raises(ValueError, match="needs counts"):
        stq.route_tokens_backward(x, r.pair_expert, None, 2, grad_balance=r.balance)
    with pytest.raises(ValueError, match="grad_weight must be"):
        stq.route_tokens_backward(x, r.pair_expert, r.counts, 2, grad_weight=r.pair_expert)
    z = torch.zeros(8, 32, device="cuda")
    with pytest.raises(ValueError, match="n_tokens \\* top_k"):
        stq.combine_rows(z, r.pair_row, 3)
    with pytest.raises(ValueError, match="top_k must be positive"):
        stq.combine_rows(z, r.pair_row, 0)
    with pytest.raises(stq.StqError, match="top_k"):
        stq.combine_rows(z, torch.zeros(33, dtype=torch.int32, device="cuda"), 33)
    with pytest.raises(ValueError, match="weight must hold 8"):
        stq.combine_rows(z, r.pair_row, 2, r.pair_weight[:4])
    with pytest.raises(ValueError, match="out must be"):
        stq.combine_rows(z, r.pair_row, 2, out=z)
    with pytest.raises(ValueError, match="dy must be"):
        stq.combine_rows_backward(z, r.pair_row, 2, z)
    with pytest.raises(ValueError, match="dz must be"):
        stq.combine_rows_backward(z[:4], r.pair_row, 2, z, dz=z[:7])
    with pytest.raises(ValueError, match="need_dz"):
        stq.combine_rows_backward(z[:4], r.pair_row, 2, z, need_dz=False, dz=z)
