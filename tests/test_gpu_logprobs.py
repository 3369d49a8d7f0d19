"""Token log probabilities and their gradient against 64-bit arithmetic.

Tolerances (u = 2^-24, half an fp32 step relative).  A term exp(l - m) errs by
at most u (3 |l - m| + 4) relative (difference, product and constant of the
exponent; one step of exp2, with its share of the rescalings' exponents, which
add up to l - m), and on its way into the sum meets at most J additions and
rescalings of 4 u together, J = elements a thread adds + 20 joins (fewer
workgroups' threads a row only shorten it).  With T = sum p |l - m| the sum s
errs by rs = u (3 T + 4 J + 8) relative, log s by rs + 4 u |log s|, and
    logprob, lse: rs + u (4 |log s| + |l_t - m| + |m| + |result|)
    entropy:      rs (1 + 2 T) + u (4 |log s| + 8 T (J + 1) + 2 H).
The gradient's p errs by u (3 |l - lse| + 8) relative, its bracket by
u (4 |g| + 6 |g_H| (|l - lse| + |H|)), the output by its type's half step."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
THREADS = 512


@pytest.fixture(scope="module")
def stq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_ternary_bit_amd as m
    return m


def _logits(n, v, dtype, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, v), generator=g) * std
    x[:, seed % v] += 6.0 * (seed % 3)
    return x.to(dtype)


def _targets(n, v, seed):
    return torch.randint(0, v, (n,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


def _reference(x):
    l = x.double()
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - m)
    s = e.sum(1)
    lp = (l - m) - torch.log(s)[:, None]
    p = e / s[:, None]
    ent = -(p * torch.where(p > 0, lp, 0.0)).sum(1)
    T = (p * torch.where(p > 0, (l - m).abs(), 0.0)).sum(1)
    J = -(-x.shape[1] // THREADS) + 8 + 20
    rs = U * (3 * T + 4 * J + 8)
    return dict(l=l, m=m[:, 0], s=s, lp=lp, p=p, ent=ent, lse=m[:, 0] + torch.log(s), T=T, J=J, rs=rs)


def _check(got, x, targets, top_n):
    logprob, lse, ent, ids, top = (t.cpu() for t in got)
    R = _reference(x)
    n, v = x.shape
    row = torch.arange(n)
    ls = torch.log(R["s"]).abs()

    def ok(value, ref, extra):
        inf = torch.isneginf(ref)
        assert bool((torch.isneginf(value) == inf).all())
        d = (value.double() - ref).abs()
        tol = R["rs"].view(-1, *[1] * (ref.dim() - 1)) + U * (extra + ref.abs())
        assert bool((d <= tol)[~inf].all()), (d - tol)[~inf].max().item()

    t = targets.long()
    ok(logprob, R["lp"][row, t], 4 * ls + (R["l"][row, t] - R["m"]).abs())
    ok(lse, R["lse"], 4 * ls + R["m"].abs())
    tol = R["rs"] * (1 + 2 * R["T"]) + U * (4 * ls + 8 * R["T"] * (R["J"] + 1) + 2 * R["ent"])
    d = (ent.double() - R["ent"]).abs()
    assert bool((d <= tol).all()), (d - tol).max().item()
    if top_n:
        order = torch.sort(R["l"], dim=1, descending=True, stable=True)[1][:, :top_n]
        assert torch.equal(ids.long(), order)
        gap = (R["l"].gather(1, order) - R["m"][:, None]).abs()
        ok(top, R["lp"].gather(1, order), 4 * ls[:, None] + gap)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, v, top_n", [(1, 1, 1), (1, 2, 2), (3, 7, 5), (2, 33, 32), (5, 1000, 0), (4, 4099, 1),
                                         (1, 131072, 20), (2, 50021, 32), (70, 9001, 8), (600, 515, 5), (9, 200003, 5)])
def test_forward(stq, n, v, top_n, dtype):
    x, t = _logits(n, v, dtype, n + v), _targets(n, v, n)
    _check(stq.token_logprobs(x.cuda(), t.cuda(), top_n=top_n), x, t, top_n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 3, 700])
def test_masked_vocabulary_and_masked_targets(stq, n, dtype):
    v = 5003
    x = _logits(n, v, dtype, 1)
    x[:, 3000:] = float("-inf")
    x[:, 7] = float("-inf")
    t = _targets(n, v, 5)
    t[0] = 7                                            # a masked target: log probability -inf
    _check(stq.token_logprobs(x.cuda(), t.cuda(), top_n=6), x, t, 6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [2, 1200])
def test_fewer_unmasked_than_alternatives(stq, n, dtype):
    # masked entries fill the list by lowest id, with log probability -inf
    v = 20000
    x = torch.full((n, v), float("-inf"), dtype=dtype)
    x[:, 11111] = 1.5
    x[:, 40] = 1.5
    x[:, 19999] = -2.0
    t = torch.full((n,), 40, dtype=torch.int32)
    _check(stq.token_logprobs(x.cuda(), t.cuda(), top_n=8), x, t, 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 900])
def test_ties_go_to_the_lowest_id(stq, n, dtype):
    v = 30011
    g = torch.Generator().manual_seed(4)
    x = torch.randint(-3, 4, (n, v), generator=g).to(dtype)      # seven values: thousands of ties
    x[:, 5] = -0.0
    t = _targets(n, v, 6)
    _check(stq.token_logprobs(x.cuda(), t.cuda(), top_n=32), x, t, 32)
    flat = torch.zeros((n, v), dtype=dtype)
    flat[:, ::2] = -0.0                                          # equal to +0
    _check(stq.token_logprobs(flat.cuda(), t.cuda(), top_n=32), flat, t, 32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 640])
def test_largest_logits_of_few_threads(stq, n, dtype):
    # a thread meets chunks 512 apart: put hundreds of the largest values where the same few threads meet
    # them, more than the list of candidates holds
    v = 300000
    per = 16 // x_bytes(dtype)
    x = _logits(n, v, dtype, 3, std=0.5)
    chunk = torch.arange(v) // per
    hot = (chunk % THREADS) < 12
    x[:, hot] += (torch.arange(int(hot.sum())) % 97).to(dtype) + 20
    t = _targets(n, v, 8)
    _check(stq.token_logprobs(x.cuda(), t.cuda(), top_n=9), x, t, 9)


def x_bytes(dtype):
    return 2 if dtype == torch.bfloat16 else 4


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_extreme_values(stq, dtype):
    big = torch.finfo(dtype).max
    v = 2000
    x = _logits(6, v, dtype, 2)
    x[0] = -big                                          # every entry the type's lowest: a uniform row
    x[1, 100:] = -big                                    # masked with the type's lowest
    x[2, 3] = big
    x[3] = 1e30
    x[4, 9] = 1e4                                        # one certain token
    x[5, :] = float("-inf")
    x[5, 77] = -1e30                                     # one token left
    t = torch.tensor([5, 200, 3, 4, 9, 77], dtype=torch.int32)
    got = stq.token_logprobs(x.cuda(), t.cuda(), top_n=4)
    _check(got, x, t, 4)


@pytest.mark.parametrize("n", [8, 700])
def test_rows_without_a_distribution(stq, n):
    v = 3001
    x = _logits(n, v, torch.float32, 2)
    x[1] = float("-inf")
    x[2, 2999] = float("nan")
    x[3, 0] = float("inf")
    x[4] = float("nan")
    t = _targets(n, v, 5)
    t[5], t[6] = -1, v                                   # no such token
    lp, lse, ent, ids, top = (o.cpu() for o in stq.token_logprobs(x.cuda(), t.cuda(), top_n=3))
    for r in (1, 2, 3, 4):
        assert torch.isnan(lp[r]) and torch.isnan(ent[r]) and torch.isnan(top[r]).all() and (ids[r] == -1).all()
    assert torch.isneginf(lse[1]) and torch.isnan(lse[2:5]).all()
    assert torch.isnan(lp[5:7]).all() and torch.isfinite(ent[5:7]).all()
    keep = torch.tensor([0] + list(range(7, n)))
    _check(stq.token_logprobs(x[keep].cuda(), t[keep].cuda(), top_n=3), x[keep], t[keep], 3)
    one = torch.full((1, 131072), float("-inf"), device="cuda")   # an empty row that is split
    out = stq.token_logprobs(one, t[:1].cuda(), top_n=2)
    assert torch.isnan(out[0]).all() and torch.isneginf(out[1]).all() and (out[3] == -1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lead", [0, 1, 3])
def test_strided_rows(stq, dtype, lead):
    n, v = 5, 1537
    big = _logits(n, v + 14, dtype, 9)
    x = big[:, lead:lead + v]
    t = _targets(n, v, 3)
    dev = big.cuda()[:, lead:lead + v]
    _check(stq.token_logprobs(dev, t.cuda(), top_n=7), x, t, 7)
    g = torch.randn(n, generator=torch.Generator().manual_seed(1))
    out = torch.full((n, v + 11), 9.0, dtype=dtype, device="cuda")
    for olead in (0, lead, 2):
        out.fill_(9.0)
        _backward_check(stq, x, dev, t, g, 0.3 * g, out[:, olead:olead + v])
        rest = torch.cat([out[:, :olead], out[:, olead + v:]], 1)
        assert bool((rest == 9.0).all())


def test_top_outputs_are_optional_and_calls_repeat_bit_for_bit(stq):
    x, t = _logits(3, 70001, torch.bfloat16, 4).cuda(), _targets(3, 70001, 4).cuda()
    a = stq.token_logprobs(x, t, top_n=10)
    b = stq.token_logprobs(x, t, top_n=10)
    c = stq.token_logprobs(x, t)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert all(torch.equal(p, q) for p, q in zip(a[:3], c[:3]))
    ws = torch.full((stq.token_logprobs_workspace(stq.X_BF16, 3, 70001, 10),), 255, dtype=torch.uint8, device="cuda")
    d = stq.token_logprobs(x, t, top_n=10, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(a, d))


# -- gradient ---------------------------------------------------------------

def _backward_ref(x, t, lse, ent, g, ge):
    l = x.double()
    lp = l - lse.double()[:, None]
    p = torch.exp(lp)
    lp0 = torch.where(p > 0, lp, 0.0)
    n = x.shape[0]
    valid = (t >= 0) & (t < x.shape[1])
    g = torch.where(valid, g.double(), 0.0)
    d = -p * (g[:, None] + ge.double()[:, None] * (lp0 + ent.double()[:, None]))
    d[torch.arange(n)[valid], t.long()[valid]] += g[valid]
    bracket = 4 * g.abs()[:, None] + 6 * ge.double().abs()[:, None] * (lp0.abs() + ent.double().abs()[:, None])
    tol = p * U * ((3 * lp0.abs() + 8) * bracket + bracket) + 2 * U * (d.abs() + g.abs()[:, None] * (p > 0)) + 2.0 ** -120
    return d, tol


def _backward_check(stq, x, dev, t, g, ge, out=None):
    R = _reference(x)
    lse, ent = R["lse"].float(), R["ent"].float()
    got = stq.token_logprobs_backward(dev, t.cuda(), lse.cuda(), ent.cuda(), g.cuda(), ge.cuda(), out=out)
    d, tol = _backward_ref(x, t, lse, ent, g, ge)
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0
    # below the smallest normal number a bf16 output may hold a subnormal or zero
    err = (got.cpu().double() - d).abs()
    tol = tol * (1 + half) + half * d.abs() + 2.0 ** -126
    assert got.dtype == x.dtype
    assert bool((err <= tol).all()), (err - tol).max().item()
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, v", [(1, 1), (1, 3), (3, 17), (17, 50021), (300, 1030), (2, 131072)])
def test_backward(stq, n, v, dtype):
    x, t = _logits(n, v, dtype, v), _targets(n, v, 2)
    gen = torch.Generator().manual_seed(n)
    _backward_check(stq, x, x.cuda(), t, torch.randn(n, generator=gen), torch.randn(n, generator=gen))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_masks_special_rows_and_missing_gradients(stq, dtype):
    n, v = 6, 2003
    x, t = _logits(n, v, dtype, 5), _targets(n, v, 2)
    x[:, 1500:] = float("-inf")
    t[1], t[2] = -1, v + 5
    t[3] = 1600                                          # masked: keeps its one-hot share
    g, ge = torch.randn(n, generator=torch.Generator().manual_seed(0)), torch.full((n,), 0.5)
    got = _backward_check(stq, x, x.cuda(), t, g, ge)
    assert bool((got[:, 1500:].cpu() == 0).sum() == n * 503 - 1)
    zero = torch.zeros(n)
    R = _reference(x)
    lse, ent = R["lse"].float().cuda(), R["ent"].float().cuda()
    xd, td = x.cuda(), t.cuda()
    a = stq.token_logprobs_backward(xd, td, lse, None, g.cuda())
    b = stq.token_logprobs_backward(xd, td, lse, ent, g.cuda(), zero.cuda())
    assert torch.equal(a, b)
    c = stq.token_logprobs_backward(xd, td, lse, ent, None, ge.cuda())
    d = stq.token_logprobs_backward(xd, td, lse, ent, zero.cuda(), ge.cuda())
    assert torch.equal(c, d)
    # rows without a distribution: masked throughout gives zeros, a NaN gives NaN, neighbours are untouched
    x[4], x[5, 3] = float("-inf"), float("nan")
    out = stq.token_logprobs(x.cuda(), t.clamp(0, v - 1).cuda())
    y = stq.token_logprobs_backward(x.cuda(), td, out[1], out[2], g.cuda(), ge.cuda()).cpu()
    assert bool((y[4] == 0).all()) and bool(torch.isnan(y[5]).all()) and bool(torch.isfinite(y[:4]).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_in_place(stq, dtype):
    x, t = _logits(9, 4001, dtype, 5).cuda(), _targets(9, 4001, 2).cuda()
    _, lse, ent, _, _ = stq.token_logprobs(x, t)
    g = torch.randn(9, generator=torch.Generator().manual_seed(0)).cuda()
    want = stq.token_logprobs_backward(x, t, lse, ent, g, 0.1 * g)
    stq.token_logprobs_backward(x, t, lse, ent, g, 0.1 * g, out=x)
    assert torch.equal(x, want)


def test_backward_against_differences(stq):
    # central differences of the fp64 objective along random directions; a step h leaves h^2 / 6 of the
    # third derivative, which for these sums is below 4 sum |g|
    n, v, h = 4, 61, 1e-4
    gen = torch.Generator().manual_seed(8)
    x, t = _logits(n, v, torch.float32, 3, std=1.0), _targets(n, v, 2)
    g, ge = torch.randn(n, generator=gen), torch.randn(n, generator=gen)
    _, lse, ent, _, _ = stq.token_logprobs(x.cuda(), t.cuda())
    d = stq.token_logprobs_backward(x.cuda(), t.cuda(), lse, ent, g.cuda(), ge.cuda()).cpu().double()

    def objective(z):
        lp = torch.log_softmax(z, 1)
        return (g.double() * lp[torch.arange(n), t.long()]).sum() - (ge.double() * (lp.exp() * lp).sum(1)).sum()
    for _ in range(8):
        u = torch.randn((n, v), generator=gen).double()
        u /= u.norm()
        diff = (objective(x.double() + h * u) - objective(x.double() - h * u)) / (2 * h)
        tol = 4 * (g.abs().sum() + ge.abs().sum()).item() * h * h + 1e-10 + 60 * U * d.abs().sum().item()
        assert abs((d * u).sum().item() - diff.item()) <= tol


@pytest.mark.parametrize("n, v", [(1, 131072), (40, 9001)])
def test_scoring_under_graph(stq, n, v):
    x, t = _logits(n, v, torch.bfloat16, 1).cuda(), _targets(n, v, 1).cuda()
    outs = [o.clone() for o in stq.token_logprobs(x, t, top_n=4)]
    ws = torch.empty(max(1, stq.token_logprobs_workspace(stq.X_BF16, n, v, 4)), dtype=torch.uint8, device="cuda")
    g = torch.ones(n, device="cuda")
    d = torch.empty_like(x)

    def call():
        stq.token_logprobs(x, t, 4, *outs, workspace=ws)
        stq.token_logprobs_backward(x, t, outs[1], outs[2], g, g, out=d)
    call()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for r in range(4):
        x.copy_(_logits(n, v, torch.bfloat16, 10 + r))
        t.copy_(_targets(n, v, 20 + r))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs] + [d.clone()]
        want = list(stq.token_logprobs(x, t, 4))
        want.append(stq.token_logprobs_backward(x, t, want[1], want[2], g, g))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), r


def test_binding_refusals(stq):
    x, t = torch.zeros(2, 10, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="targets must be torch.int32"):
        stq.token_logprobs(x, t.long())
    with pytest.raises(ValueError, match="targets must hold 2"):
        stq.token_logprobs(x, t[:1])
    with pytest.raises(stq.StqError, match="top_n"):
        stq.token_logprobs(x, t, top_n=11)
    with pytest.raises(ValueError, match="contiguous rows"):
        stq.token_logprobs(x.t().contiguous().t(), t)
    with pytest.raises(ValueError, match="logits must be"):
        stq.token_logprobs(x.half(), t)
    with pytest.raises(ValueError, match="top_ids"):
        stq.token_logprobs(x, t, top_n=2, top_ids=torch.zeros(2, 3, dtype=torch.int32, device="cuda"))
    f = torch.zeros(2, device="cuda")
    with pytest.raises(stq.StqError, match="needs entropy"):
        stq.token_logprobs_backward(x, t, f, None, f, f)
    with pytest.raises(ValueError, match="out must be"):
        stq.token_logprobs_backward(x, t, f, f, f, out=x[:1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 3, 1100])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_backward_of_rows_that_end_with_a_workgroups_piece(stq, dtype, n, more):
    """Rows of a whole number of pieces (32 KB, 8 KB where rows are few), one entry less or more, starting on
    16 bytes, inside them all alike, and each elsewhere."""
    size = 2 if dtype == torch.bfloat16 else 4
    v = (32768 if n > 500 else 8192) // size + more
    x, t = _logits(n, v, dtype, 3), _targets(n, v, 2)
    gen = torch.Generator().manual_seed(n)
    g, ge = torch.randn(n, generator=gen), torch.randn(n, generator=gen)
    per = 16 // size
    for lead, row in ((0, -(-v // per) * per), (1, -(-(v + 1) // per) * per), (per - 1, -(-(v + per) // per) * per),
                      (0, (v + per) // per * per + 1)):
        buf = torch.full((n, row), 9.0, dtype=dtype, device="cuda")
        dev = buf[:, lead:lead + v]
        dev.copy_(x)
        out = torch.full((n, row), 9.0, dtype=dtype, device="cuda")
        _backward_check(stq, x, dev, t, g, ge, out[:, lead:lead + v])
        assert bool((torch.cat([out[:, :lead], out[:, lead + v:]], 1) == 9.0).all())
