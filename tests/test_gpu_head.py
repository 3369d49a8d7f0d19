"""The output head's cross entropy and its gradients against 64-bit arithmetic.

Tolerances (u = 2^-24, half an fp32 step relative; b = 2^-8, half a bf16 step).
A bf16 logit is a sum of k exact products, each addition off by at most a step:
dl <= 2 u (k + 2) sum |x w|; an 8-bit one is an exact integer scaled twice, dl
<= 4 u |l|.  A term exp(l - m) errs by u (3 |l - m| + 4) relative beside dl,
its sums meet J = 60 + (tiles of 64) / 16 additions and rescalings of 4 u
together, so with T = sum p |l - m| and D = sum p dl
    lse:  D + u (3 T + 4 J + 8 + 4 |log s| + 2 |m| + 2 |lse|)
    loss: that, dl of the target and u |l_t - m| more.
In the gradient p errs by dl + u (3 |l - lse| + 12) relative, d = g (p - 1) by u
|g| more and by b |d| from its rounding to bf16 (its 8-bit scale adds u); dx
and dw by the magnitudes of those errors times the other operand, 2 u a term
for the sum, and b for their own rounding."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def stq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_ternary_bit_amd as m
    return m


class Case:
    """Operands on the GPU, in rows that start on 16 bytes; what lies between the rows is NaN (or 99)."""

    def __init__(self, n, v, k, i8, seed, ignored=0.2, spread=3.0):
        self.n, self.v, self.k, self.i8 = n, v, k, i8
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
        self.targets = torch.randint(0, v, (n,), device="cuda", generator=g)
        w = randn(v, k) * spread / k ** 0.5
        x = randn(n, k) + (2.0 / spread) * torch.rand((n, 1), device="cuda", generator=g) * k ** 0.5 * torch.nn.functional.normalize(
            w[self.targets], dim=1)
        if ignored:
            self.targets[torch.rand(n, device="cuda", generator=g) < ignored] = -1
        self.targets = self.targets.int()
        self.x_scale = self.w_scale = None
        if i8:
            x, self.x_scale = self._quantize(x)
            w, self.w_scale = self._quantize(w)
        else:
            x, w = x.bfloat16(), w.bfloat16()
        self.x, self.w = self._place(x), self._place(w)
        self.grad = torch.randn(n, device="cuda", generator=g)

    @staticmethod
    def _quantize(t):
        scale = t.abs().amax(1) / 127
        return torch.round(t / scale[:, None]).to(torch.int8), scale

    @staticmethod
    def _place(t):
        unit = 16 // t.element_size()
        wide = torch.full((t.shape[0], (t.shape[1] + unit - 1) // unit * unit), 99 if t.dtype == torch.int8 else float("nan"),
                          dtype=t.dtype, device=t.device)
        wide[:, :t.shape[1]] = t
        return wide[:, :t.shape[1]]

    def args(self):
        return dict(x_scale=self.x_scale, w_scale=self.w_scale)

    def logits(self):
        """(l, its error) in 64 bits."""
        x, w = self.x.double(), self.w.double()
        if self.i8:
            l = (x @ w.t()) * self.x_scale.double()[:, None] * self.w_scale.double()
            return l, 4 * U * l.abs()
        return x @ w.t(), 2 * U * (self.k + 2) * (x.abs() @ w.abs().t())

    def check_forward(self, loss, lse):
        l, dl = self.logits()
        m = l.amax(1)
        p = torch.softmax(l, 1)
        ref = torch.logsumexp(l, 1)
        gap = (l - m[:, None]).abs()
        T, D = (p * gap).sum(1), (p * dl).sum(1)
        J = 60 + self.v / 64 / 16
        tol = D + U * (3 * T + 4 * J + 8 + 4 * (ref - m).abs() + 2 * m.abs() + 2 * ref.abs())
        assert bool(((lse.double() - ref).abs() <= tol).all()), ((lse.double() - ref).abs() / tol).max().item()
        at = self.targets.clamp(min=0).long()[:, None]
        on = self.targets >= 0
        want = torch.where(on, ref - l.gather(1, at)[:, 0], 0.0)
        tol = torch.where(on, tol + dl.gather(1, at)[:, 0] + U * (gap.gather(1, at)[:, 0] + want.abs()), 0.0)
        assert bool(((loss.double() - want).abs() <= tol).all())

    def gradient_ref(self, lse):
        l, dl = self.logits()
        p = torch.exp(l - lse.double()[:, None])
        on = self.targets >= 0
        g = torch.where(on, self.grad.double(), 0.0)[:, None]
        hot = torch.zeros_like(p)
        hot[torch.arange(self.n, device="cuda")[on], self.targets[on].long()] = 1.0
        d = g * (p - hot)
        err = g.abs() * (p * (dl + U * (3 * (l - lse.double()[:, None]).abs() + 12)) + U * hot)
        if self.i8:
            s = self.w_scale.double()
            d, err = d * s, err * s + U * (d * s).abs()
        return d, err * (1 + B) + B * d.abs() + TINY

    def check_backward(self, dx, dw, lse):
        d, err = self.gradient_ref(lse)
        w, x = self.w.double(), torch.where((self.targets >= 0)[:, None], self.x.double(), 0.0)
        if dx is not None:
            ref, tol = d @ w, err @ w.abs() + 2 * U * (self.v + 20) * (d.abs() @ w.abs())
            assert bool(((dx.double() - ref).abs() <= tol * (1 + B) + B * ref.abs() + TINY).all())
        if dw is not None:
            ref = d.t().contiguous() @ x
            tol = err.t().contiguous() @ x.abs() + 2 * U * (self.n + 20) * (d.abs().t().contiguous() @ x.abs())
            assert bool(((dw.double() - ref).abs() <= tol * (1 + B) + B * ref.abs() + TINY).all())


# every tile of either product: 16 channels (up to 16 rows), 64 x 64, 64 x 128 and 64 x 256 (more than 32768 and 65536
# words), 128 x 128, 256 x 256; dx of up to 32 rows and of more (8-bit heads)
SHAPES = [(1, 1, 1), (1, 2, 9), (3, 65, 8), (5, 130, 100), (64, 1000, 64), (65, 257, 130), (37, 16450, 33), (64, 16500, 72),
          (1, 20000, 17), (300, 700, 129), (129, 4099, 200), (700, 9001, 65), (512, 66000, 64), (513, 65537, 40),
          (40, 40000, 24), (50, 70000, 24), (16, 4000, 260), (17, 3000, 96), (128, 3333, 150)]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n, v, k", SHAPES)
def test_forward(stq, n, v, k, i8):
    c = Case(n, v, k, i8, n + v + k)
    c.check_forward(*stq.head_cross_entropy(c.x, c.w, c.targets, **c.args()))


# dW's 256 x 256 tiles; dx's sum shared out or not, in two rounds of tiles or one (all in one piece of the vocabulary)
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n, v, k", SHAPES + [(70, 8192, 2048), (20, 17000, 8000), (900, 17000, 8000),
                                              (1300, 4500, 6501), (4097, 3001, 6999)])
def test_backward(stq, n, v, k, i8):
    c = Case(n, v, k, i8, 2 * n + v + k)
    _, lse = stq.head_cross_entropy(c.x, c.w, c.targets, **c.args())
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dw=not i8, **c.args())
    assert dx.shape == (n, k) and (dw is None if i8 else dw.shape == (v, k))
    c.check_backward(dx, dw, lse)


# Above 2^26 logits the vocabulary is taken in pieces: sums that begin with the pieces before, targets on either side of
# a piece's end, a narrow last piece; dx's sum shared out (short rows) and not (a tile for every compute unit); more rows
# than leave a piece more than its least width.
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n, v, k", [(4100, 40000, 72), (4100, 40003, 4099), (9001, 20011, 40), (263000, 700, 24)])
def test_backward_in_pieces_of_the_vocabulary(stq, n, v, k, i8):
    c = Case(n, v, k, i8, n + v + k)
    width = max(2 ** 26 // n // 256, 1) * 256
    edges = sorted({e for w in (width, width - 256, width - 512) if w > 0 for p in range(w, v, w) for e in (p - 1, p) if e < v} | {0, v - 1})
    for i in range(0, n, 7):
        if i // 7 < 400:
            c.targets[i] = edges[i // 7 % len(edges)]
    kind = stq.X_I8 if i8 else stq.X_BF16
    # (dl of the whole vocabulary alone takes this much, where the outputs' sums are small)
    assert k > 100 or stq.head_cross_entropy_backward_workspace(kind, n, v, k, True, False) < 2 * n * v
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets, **c.args())
    c.check_forward(loss, lse)
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dw=not i8, **c.args())
    c.check_backward(dx, dw, lse)


def test_backward_one_output_and_given_ones(stq):
    c = Case(100, 3000, 203, False, 1)
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    only, none = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dx=False)
    assert none is None and torch.equal(only, dw)
    # any strides and offsets of the outputs, wide rows of the operands
    dxw, dww = torch.full((100, 209), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((3000, 210), 7.0, dtype=torch.bfloat16, device="cuda")
    xw, ww = torch.full((100, 240), float("nan"), dtype=torch.bfloat16, device="cuda"), torch.full((3000, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    xw[:, 8:211], ww[:, 16:219] = c.x, c.w
    loss2, lse2 = torch.empty_like(loss), torch.empty_like(lse)
    stq.head_cross_entropy(xw[:, 8:211], ww[:, 16:219], c.targets, loss=loss2, lse=lse2)
    assert torch.equal(loss2, loss) and torch.equal(lse2, lse)
    stq.head_cross_entropy_backward(xw[:, 8:211], ww[:, 16:219], c.targets, lse, c.grad, dx=dxw[:, 3:206], dw=dww[:, 1:204])
    assert torch.equal(dxw[:, 3:206], dx) and torch.equal(dww[:, 1:204], dw)
    assert bool((dxw[:, :3] == 7).all()) and bool((dxw[:, 206:] == 7).all()) and bool((dww[:, :1] == 7).all()) and bool((dww[:, 204:] == 7).all())


# One word alone has weights: dx is its term d w, which has two roundings, that of d (in fp32: the errors of p and U
# |g|) and its own to bf16.  Every tile of the logits; dx of 8-bit heads by few rows, from parts of the sum, and by the
# tiles themselves.
@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n, v, k", [(1, 40, 24), (12, 500, 72), (20, 1000, 200), (66, 1000, 64), (300, 700, 129), (600, 250, 701),
                                     (513, 9000, 96), (50, 70000, 24)])
def test_the_targets_term_of_the_rows_gradient(stq, n, v, k, i8):
    c = Case(n, v, k, i8, 3 * n, ignored=0.1 if n > 9 else 0.0)
    word = v // 3
    only = c.w[word].clone()
    c.w.zero_()
    c.w[word] = only
    c.targets[c.targets >= 0] = word
    if i8:
        c.w_scale.fill_(c.w_scale[word].item())
    _, lse = stq.head_cross_entropy(c.x, c.w, c.targets, **c.args())
    dx, _ = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dw=False, **c.args())
    d, err = c.gradient_ref(lse)
    d, err = d[:, word:word + 1], (err[:, word:word + 1] - B * d[:, word:word + 1].abs()) / (1 + B)
    w = c.w[word].double()
    ref = d * w
    tol = (err + 2 * U * d.abs()) * w.abs()
    assert bool(((dx.double() - ref).abs() <= tol * (1 + B) + B * ref.abs() + TINY).all())


# Each row of x has two columns of its own, so that dW's row of its target has there one term d x, with two roundings as
# above (and the rest's own, B B |d x|), for up to 32 rows: targets apart, a few that many rows share, one for all, in
# every tile of the logits.
@pytest.mark.parametrize("n, v, words", [(1, 40, 40), (2, 500, 1), (12, 500, 500), (16, 20000, 3), (17, 3000, 3000), (30, 3000, 7), (32, 200, 200),
                                         (31, 40000, 40000), (20, 70000, 1), (9, 33000, 33000)])
def test_the_targets_term_of_the_heads_gradient(stq, n, v, words):
    k = 2 * n + 3
    c = Case(n, v, k, False, n, ignored=0.0)
    own = torch.arange(n, device="cuda") * 2
    keep = torch.zeros(n, k, dtype=torch.bool, device="cuda")
    keep[torch.arange(n, device="cuda"), own] = keep[torch.arange(n, device="cuda"), own + 1] = True
    c.x.copy_(torch.where(keep, c.x * 4, 0))
    c.targets.remainder_(words)
    dead = torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)) < 0.1
    c.targets[dead] = -1
    c.x[dead] = float("nan")
    _, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    _, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dx=False)
    assert bool(torch.isfinite(dw).all())
    r = torch.arange(n, device="cuda")[~dead]
    c.x[dead] = 0
    t = c.targets[r].long()
    d, err = c.gradient_ref(torch.where(dead, 0.0, lse))
    d, err = d[r, t][:, None], ((err[r, t] - B * d[r, t].abs()) / (1 + B))[:, None]
    col = torch.stack([own[r], own[r] + 1], 1)
    x, got = c.x.double()[r[:, None], col], dw.double()[t[:, None], col]
    tol = (err + (2 * U + B * B) * d.abs()) * x.abs()
    assert bool(((got - d * x).abs() <= tol * (1 + B) + B * (d * x).abs() + TINY).all())
    again = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dx=False)[1]
    assert torch.equal(again, dw)


# many rows to a word: sums in the rows' order, targets of every kind beside each other
@pytest.mark.parametrize("n, v, k, words", [(20, 30, 515, 3), (300, 700, 129, 5), (1300, 4000, 701, 40), (2500, 300, 96, 2)])
def test_gradients_of_words_that_rows_share(stq, n, v, k, words):
    c = Case(n, v, k, False, n + k)
    c.targets.copy_(torch.where(c.targets < 0, c.targets, c.targets % words + v - words))
    _, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    c.check_backward(dx, dw, lse)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n, v, k", [(600, 250, 701), (300, 100, 1030), (260, 256, 515)])
def test_rows_of_any_stride_and_offset(stq, n, v, k, i8):
    # one part of the sum: the tiles of 256 x 256 write dx themselves, on odd element boundaries
    c = Case(n, v, k, i8, n + k)
    _, lse = stq.head_cross_entropy(c.x, c.w, c.targets, **c.args())
    wide = torch.full((n, k + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    big = None if i8 else torch.full((v, k + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, dw = wide[:, 3:3 + k], None if i8 else big[:, 1:1 + k]
    stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dw=not i8, dx=dx, dw=dw, **c.args())
    c.check_backward(dx, dw, lse)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 3 + k:] == 7).all())
    if not i8:
        assert bool((big[:, :1] == 7).all()) and bool((big[:, 1 + k:] == 7).all())


def test_rows_left_out_are_not_looked_at(stq):
    c = Case(90, 2000, 96, False, 4, ignored=0.3)
    out = c.targets < 0
    assert bool(out.any()) and not bool(out.all())
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    assert not loss[out].any() and not dx[out].any()
    # padding may hold anything
    c.x[out] = float("nan")
    c.grad[out] = float("inf")
    loss2, lse2 = stq.head_cross_entropy(c.x, c.w, c.targets)
    dx2, dw2 = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse2, c.grad)
    assert torch.equal(loss2, loss) and torch.equal(lse2[~out], lse[~out]) and bool(torch.isnan(lse2[out]).all())
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    c.targets[:] = -100
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    assert not loss.any() and not dx.any() and not dw.any()


def test_targets_past_the_vocabulary(stq):
    c = Case(66, 1000, 64, False, 5, ignored=0.0)
    good = c.targets.clone()
    c.targets[3], c.targets[40] = 1000, 2 ** 31 - 1
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    assert bool(torch.isnan(loss[[3, 40]]).all()) and torch.isnan(loss).sum().item() == 2
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    assert not dx[[3, 40]].any()
    good[[3, 40]] = -1
    want = stq.head_cross_entropy_backward(c.x, c.w, good, lse, c.grad)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


# tiles of 16, 64, 128 and 256; dx joined from parts of the sum, and written by the tiles themselves
@pytest.mark.parametrize("n, v, k", [(12, 500, 72), (66, 1000, 64), (300, 700, 129), (600, 250, 701), (513, 9000, 96)])
def test_rows_without_a_gradient_may_hold_anything(stq, n, v, k):
    c = Case(n, v, k, False, n, ignored=0.1)
    c.targets[[1, 2, 4, 7, 9]] = torch.tensor([v, 2 ** 31 - 1, v + 1, 3, 5], dtype=torch.int32, device="cuda")
    c.x[1, 3], c.x[2, 5], c.x[4] = float("nan"), float("inf"), -float("inf")
    # a row whose logits are all -inf, under a head with one column above zero
    c.w[:, 1] = c.w[:, 1].abs() + 0.125
    c.x[7] = 0
    c.x[7, 1] = -float("inf")
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    assert bool(torch.isneginf(lse[7])) and bool(torch.isnan(loss[[1, 2, 4, 7]]).all())
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    assert not dx[[1, 2, 4, 7]].any() and bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())
    c.targets[[1, 2, 4, 7]] = -1
    c.x[[1, 2, 4, 7]] = 1.0
    want = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    c.check_backward(dx, dw, torch.where(c.targets < 0, 0.0, lse))


@pytest.mark.parametrize("n, v, k", [(12, 500, 72), (66, 1000, 64), (600, 250, 701)])
def test_rows_under_a_head_of_minus_infinity(stq, n, v, k):
    c = Case(n, v, k, False, n, ignored=0.1)
    c.x.abs_()
    c.w[:] = -float("inf")
    _, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    assert bool(torch.isneginf(lse).all())
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("n, v, k", [(12, 500, 72), (66, 1000, 64), (600, 250, 701)])
def test_8_bit_rows_without_a_gradient(stq, n, v, k):
    c = Case(n, v, k, True, n, ignored=0.1)
    c.targets[[1, 2]] = torch.tensor([v, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    c.x_scale[[1, 2]] = torch.tensor([float("nan"), float("inf")], device="cuda")
    _, lse = stq.head_cross_entropy(c.x, c.w, c.targets, **c.args())
    dx, _ = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dw=False, **c.args())
    assert not dx[[1, 2]].any() and bool(torch.isfinite(dx).all())
    c.targets[[1, 2]] = -1
    c.x_scale[[1, 2]] = 1.0
    want = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dw=False, **c.args())
    assert torch.equal(dx, want[0])


@pytest.mark.parametrize("v", [300, 20000])
def test_rows_that_are_not_finite(stq, v):
    c = Case(50, v, 64, False, 6, ignored=0.0)
    c.x[2, 5] = float("nan")
    c.x[7, 1] = float("inf")                      # logits of +inf and -inf
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    bad = torch.zeros(50, dtype=torch.bool, device="cuda")
    bad[[2, 7]] = True
    assert bool(torch.isnan(loss[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    assert bool(torch.isfinite(loss[~bad]).all()) and bool(torch.isfinite(lse[~bad]).all())
    dx, _ = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, need_dw=False)
    assert bool(torch.isnan(dx[bad]).all()) and bool(torch.isfinite(dx[~bad]).all())
    # words that are masked throughout, and a row whose every logit is
    c = Case(50, v, 64, False, 7, ignored=0.0)
    c.x.abs_()
    c.w[v // 2:] = -float("inf")
    c.targets.clamp_(max=v // 2 - 1)
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    half = Case(50, v, 64, False, 7, ignored=0.0)
    half.x, half.w, half.v, half.targets = c.x, c.w[:v // 2], v // 2, c.targets
    half.check_forward(loss, lse)
    c.w[:] = -float("inf")
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    assert bool(torch.isneginf(lse).all()) and bool(torch.isnan(loss).all())


def test_a_target_that_is_almost_sure(stq):
    # p close to 1: the loss is the others' share, and p - 1 keeps its digits
    c = Case(40, 5000, 64, False, 8, ignored=0.0, spread=1.0)
    c.x.copy_((c.w[c.targets.long()].float() * 40).bfloat16())
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    c.check_forward(loss, lse)
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    c.check_backward(dx, dw, lse)


def test_no_rows_and_gradient_of_a_mean(stq):
    c = Case(3, 100, 40, False, 9)
    loss, lse = stq.head_cross_entropy(c.x[:0], c.w, c.targets[:0])
    assert loss.shape == (0,) and lse.shape == (0,)
    dw = torch.full((100, 40), 3.0, dtype=torch.bfloat16, device="cuda")
    dx, dw = stq.head_cross_entropy_backward(c.x[:0], c.w, c.targets[:0], lse, c.grad[:0], dw=dw)
    assert dx.shape == (0, 40) and not dw.any()


def test_gradient_against_differences(stq):
    # central differences of the 64-bit loss; the bound is what the bf16 rounding of dl and dx allows
    c = Case(4, 50, 24, False, 10, ignored=0.0)
    _, lse = stq.head_cross_entropy(c.x, c.w, c.targets)
    dx, dw = stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad)
    x, w, g, t = c.x.double(), c.w.double(), c.grad.double(), c.targets.long()
    lse64 = torch.logsumexp(x @ w.t(), 1)
    assert bool(((lse.double() - lse64).abs() < 1e-5).all())

    def loss(x, w):
        l = x @ w.t()
        return (g * (torch.logsumexp(l, 1) - l.gather(1, t[:, None])[:, 0])).sum().item()
    step = 1e-6
    for i, j in [(0, 0), (1, 13), (3, 23)]:
        e = torch.zeros_like(x)
        e[i, j] = step
        diff = (loss(x + e, w) - loss(x - e, w)) / (2 * step)
        d = g[i].abs() * (torch.softmax(x[i] @ w.t(), 0) @ w[:, j].abs() + w[t[i], j].abs())
        assert abs(diff - dx[i, j].item()) <= 2 * B * (d.item() + abs(diff)) + 1e-6
    for i, j in [(int(t[0]), 3), (7, 11), (49, 0)]:
        e = torch.zeros_like(w)
        e[i, j] = step
        diff = (loss(x, w + e) - loss(x, w - e)) / (2 * step)
        p = torch.softmax(x @ w.t(), 1)[:, i] + (t == i).double()
        d = (g.abs() * p * x[:, j].abs()).sum()
        assert abs(diff - dw[i, j].item()) <= 2 * B * (d.item() + abs(diff)) + 1e-6


@pytest.mark.parametrize("i8", [False, True])
def test_agrees_with_the_logits_kept(stq, i8):
    # the scoring of kept logits gives the same log probabilities
    c = Case(130, 3001, 256, i8, 11, ignored=0.0)
    loss, lse = stq.head_cross_entropy(c.x, c.w, c.targets, **c.args())
    if i8:
        logits = stq.q8_matmul(c.x, c.x_scale, c.w, c.w_scale, out_dtype=torch.float32)
        logprob, lse2, _, _, _ = stq.token_logprobs(logits, c.targets)
        tol = U * (6 * lse.abs() + 600)
        assert bool(((lse - lse2).abs() <= tol).all()) and bool(((loss + logprob).abs() <= tol + U * 8 * loss.abs()).all())
    c.check_forward(loss, lse)


@pytest.mark.parametrize("i8", [False, True])
def test_under_a_graph_with_work_between(stq, i8):
    n, v, k = 200, 17000, 512
    c = Case(n, v, k, i8, 12)
    kind = stq.X_I8 if i8 else stq.X_BF16
    loss, lse = (torch.empty(n, device="cuda") for _ in range(2))
    dx, dw = torch.empty(n, k, dtype=torch.bfloat16, device="cuda"), None if i8 else torch.empty(v, k, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(stq.head_cross_entropy_workspace(kind, n, v, k), dtype=torch.uint8, device="cuda")
    wsb = torch.empty(stq.head_cross_entropy_backward_workspace(kind, n, v, k, True, not i8), dtype=torch.uint8, device="cuda")

    def call():
        stq.head_cross_entropy(c.x, c.w, c.targets, **c.args(), loss=loss, lse=lse, workspace=ws)
        stq.head_cross_entropy_backward(c.x, c.w, c.targets, lse, c.grad, **c.args(), need_dw=not i8, dx=dx, dw=dw, workspace=wsb)
    call()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for i in range(4):
        other = Case(n, v, k, i8, 20 + i)
        for name in ("x", "w", "targets", "grad", "x_scale", "w_scale"):
            if getattr(c, name) is not None:
                getattr(c, name).copy_(getattr(other, name))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (loss, lse, dx, dw) if t is not None]
        want = list(stq.head_cross_entropy(c.x, c.w, c.targets, **c.args()))
        want += [t for t in stq.head_cross_entropy_backward(c.x, c.w, c.targets, want[1], c.grad, **c.args(), need_dw=not i8) if t is not None]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i


def test_on_another_stream_and_twice(stq):
    c = Case(100, 5000, 128, False, 13)
    torch.cuda.synchronize()
    first = stq.head_cross_entropy(c.x, c.w, c.targets)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        second = stq.head_cross_entropy(c.x, c.w, c.targets)
    third = stq.head_cross_entropy(c.x, c.w, c.targets)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, d) for a, b, d in zip(first, second, third))


def test_binding_refusals(stq):
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"), torch.zeros(10, 32, dtype=torch.bfloat16, device="cuda")
    t, f = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="x must be"):
        stq.head_cross_entropy(x.float(), w, t)
    with pytest.raises(ValueError, match="like x"):
        stq.head_cross_entropy(x, w.to(torch.int8), t)
    with pytest.raises(ValueError, match="same length"):
        stq.head_cross_entropy(x, w[:, :16], t)
    with pytest.raises(ValueError, match="targets must be torch.int32"):
        stq.head_cross_entropy(x, w, t.long())
    with pytest.raises(ValueError, match="no scales"):
        stq.head_cross_entropy(x, w, t, x_scale=f)
    with pytest.raises(ValueError, match="need x_scale"):
        stq.head_cross_entropy(x.to(torch.int8), w.to(torch.int8), t)
    with pytest.raises(stq.StqError, match="16-byte"):
        stq.head_cross_entropy(x[:, :30].contiguous(), w[:, :30].contiguous(), t)
    with pytest.raises(ValueError, match="own its bytes"):
        stq.head_cross_entropy(x[:, :30], w.view(-1)[:9 * 32 + 30].clone().as_strided((10, 30), (32, 1)), t)
    with pytest.raises(ValueError, match="contiguous rows"):
        stq.head_cross_entropy(x.t().contiguous().t(), w, t)
    with pytest.raises(stq.StqError, match="workspace"):
        stq.head_cross_entropy(x, w, t, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="need_dw must be False"):
        stq.head_cross_entropy_backward(x.to(torch.int8), w.to(torch.int8), t, f, f, x_scale=f, w_scale=torch.zeros(10, device="cuda"))
    with pytest.raises(ValueError, match="grad_loss must hold"):
        stq.head_cross_entropy_backward(x, w, t, f, f[:3])
    with pytest.raises(ValueError, match="dx must be"):
        stq.head_cross_entropy_backward(x, w, t, f, f, dx=x[:3])
    with pytest.raises(ValueError, match="need_dx"):
        stq.head_cross_entropy_backward(x, w, t, f, f, need_dx=False, dx=x)
