"""8-bit rows and their product against integers and 64-bit arithmetic.

The quantizer's integers and scales are compared exactly.  The product's sum
is exact, its two scalings and the conversion of the sum round to fp32 (three
half steps of 2^-24 relative), and a bf16 output rounds once more (2^-8)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_ternary_bit_amd as m
    return m


def _rand(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * std


def _quant_ref(x):
    """fp64 on the host: exact scale rounding, exact quotients next to halves."""
    x = x.double().numpy()
    amax = np.abs(x).max(1)
    scale = (amax / 127.0).astype(np.float32)
    some = np.isfinite(amax) & (scale > 0)
    q = np.zeros(x.shape, dtype=np.int8)
    q[some] = np.clip(np.rint(x[some] / scale[some, None].astype(np.float64)), -127, 127).astype(np.int8)
    scale[~np.isfinite(amax)] = np.nan
    return q, scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n, k", [(1, 1), (1, 7168), (3, 15), (5, 16), (2, 17), (130, 4099), (64, 256), (1, 20001), (1500, 77), (1030, 9000)])
def test_quantize_is_exact(stq, dtype, n, k):
    x = _rand((n, k), 7 * n + k).to(dtype)
    q, s = stq.q8_quantize_rows(x.cuda())
    want_q, want_s = _quant_ref(x)
    assert tuple(q.shape) == (n, k) and q.stride(0) % 16 == 0
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)
    if k % 16:
        pad = q.as_strided((n, (k + 15) // 16 * 16), (q.stride(0), 1))[:, k:]
        assert not pad.any()


def test_quantize_halves_go_to_even(stq):
    # max 127 makes the scale 1: quotients are the values themselves
    row = torch.tensor([127.0] + [i + 0.5 for i in range(-126, 126)] + [0.25, -0.75, 63.0])
    x = torch.stack([row, row * 2.0 ** -20, row * 3.0])
    q, s = stq.q8_quantize_rows(x.cuda())
    want_q, want_s = _quant_ref(x)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)


def test_quantize_near_halves(stq):
    # values one fp32 step either side of (i + 1/2) * scale
    base = torch.tensor([126.7])
    scale = (base.double() / 127).float()
    half = (torch.arange(-126, 126).double() + 0.5) * scale.double()
    h = half.float()
    x = torch.cat([base, h, torch.nextafter(h, torch.full_like(h, 1e9)), torch.nextafter(h, torch.full_like(h, -1e9))])[None]
    q, s = stq.q8_quantize_rows(x.cuda())
    want_q, want_s = _quant_ref(x)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)


def test_quantize_special_rows(stq):
    x = torch.zeros(8, 33)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3, 32] = float("-inf")
    x[4] = 1e-44                       # the scale underflows or is a subnormal
    x[5] = torch.linspace(-3e-39, 3e-39, 33)
    x[6] = torch.finfo(torch.float32).max
    x[7, 0] = -0.0
    q, s = stq.q8_quantize_rows(x.cuda())
    q, s = q.cpu().numpy(), s.cpu().numpy()
    want_q, want_s = _quant_ref(x)
    assert np.array_equal(s, want_s, equal_nan=True)
    assert np.array_equal(q, want_q)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_strided_rows_and_output(stq, dtype):
    big = _rand((6, 101), 3).to(dtype).cuda()
    x = big[1:5, 3:90]                                   # unaligned rows 101 elements apart
    out = torch.full((4, 160), 77, dtype=torch.int8, device="cuda")
    q, s = stq.q8_quantize_rows(x, out=out[:, :87])
    want_q, want_s = _quant_ref(x.cpu())
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    assert not out[:, 87:96].any() and (out[:, 96:] == 77).all()


def _int8(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def _padded(q, fill=99):
    """The rows on the GPU, with other values behind k."""
    n, k = q.shape
    t = torch.full((n, (k + 15) // 16 * 16), fill, dtype=torch.int8)
    t[:, :k] = q
    return t.cuda()[:, :k]


def _check(y, a, sa, w, sw):
    acc = torch.from_numpy(a.numpy().astype(np.int64) @ w.numpy().astype(np.int64).T) if a.numel() * w.shape[0] < 1 << 24 \
        else (a.cuda().double() @ w.cuda().double().t()).cpu().long()       # below 2^53: exact
    ref = acc.double() * sa.double()[:, None] * sw.double()
    tol = ref.abs() * (3.0 * 2 ** -24 * (1 + 2 ** -20) + (2 ** -8 if y.dtype == torch.bfloat16 else 0))
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (err - tol).max().item()


SHAPES = [(1, 1, 1), (1, 64, 16), (1, 4096, 7168), (2, 100, 130), (7, 333, 1000), (16, 65, 4096), (17, 64, 127),
          (33, 129, 257), (64, 1003, 2049), (65, 128, 128), (100, 77, 15), (128, 256, 512), (129, 513, 333),
          (300, 200, 1111), (512, 640, 4096), (1000, 1000, 100), (257, 300, 20000), (5, 9001, 320), (20, 20011, 500), (50, 17000, 777),
          (1100, 2100, 200), (2100, 4200, 300), (2048, 4096, 1024), (20, 70001, 96), (9, 70001, 130), (64, 131090, 50)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m, n, k", SHAPES)
def test_matmul(stq, m, n, k, out):
    a, w = _int8((m, k), m + n + k), _int8((n, k), m + n + k + 1)
    sa, sw = _rand((m,), 5).abs() + 0.1, _rand((n,), 6)
    y = stq.q8_matmul(_padded(a), sa.cuda(), _padded(w, -77), sw.cuda(), out_dtype=out)
    assert y.dtype == out
    _check(y, a, sa, w, sw)


@pytest.mark.parametrize("m", [1, 8, 40, 64, 200])
def test_matmul_extreme_sums_are_exact(stq, m):
    # every product 2^14, the longest k: sums of 2^31 - 2^14, held exactly
    k, n = 131071, 48
    a = torch.full((m, (k + 15) // 16 * 16), -128, dtype=torch.int8, device="cuda")[:, :k]
    w = torch.full((n, (k + 15) // 16 * 16), -128, dtype=torch.int8, device="cuda")[:, :k]
    one = torch.ones(max(m, n), device="cuda")
    y = stq.q8_matmul(a, one[:m], w, one[:n], out_dtype=torch.float32)
    assert bool((y == float(np.float32(k * 16384))).all())


@pytest.mark.parametrize("m, n, k", [(3, 70, 200), (70, 150, 200), (200, 300, 300)])
def test_matmul_strided_operands_and_output(stq, m, n, k):
    a, w = _int8((m, k), 1), _int8((n, k), 2)
    A = torch.full((m, 512), 55, dtype=torch.int8, device="cuda")
    W = torch.full((n + 4, 384), 44, dtype=torch.int8, device="cuda")
    A[:, :k], W[2:n + 2, :k] = a.cuda(), w.cuda()
    sa, sw = _rand((m,), 5), _rand((n,), 6)
    for dtype, lead in ((torch.bfloat16, 1), (torch.float32, 3), (torch.bfloat16, 0), (torch.float32, 0)):
        out = torch.full((m, n + 9), 7.0, dtype=dtype, device="cuda")
        y = out[:, lead:lead + n]
        stq.q8_matmul(A[:, :k], sa.cuda(), W[2:n + 2, :k], sw.cuda(), out=y)
        _check(y, a, sa, w, sw)
        rest = torch.cat([out[:, :lead], out[:, lead + n:]], 1)
        assert bool((rest == 7.0).all())


@pytest.mark.parametrize("m", [1, 5, 64, 130])
def test_matmul_nan_scale_marks_its_row_only(stq, m):
    x = _rand((m, 300), 9)
    x[m // 2, 17] = float("nan")
    q, s = stq.q8_quantize_rows(x.cuda())
    w = _int8((90, 300), 3)
    y = stq.q8_matmul(q, s, _padded(w), torch.ones(90, device="cuda"), out_dtype=torch.float32)
    bad = torch.isnan(y).all(1).cpu()
    assert bad[m // 2] and int(bad.sum()) == 1 and not torch.isnan(y.cpu()[~bad]).any()


def test_matmul_bits_do_not_depend_on_the_shape_around(stq):
    k = 3000
    a, w = _int8((700, k), 11), _int8((500, k), 12)
    sa, sw = _rand((700,), 5).cuda(), _rand((500,), 6).cuda()
    A, W = _padded(a), _padded(w)
    full = stq.q8_matmul(A, sa, W, sw, out_dtype=torch.float32)
    for m in (1, 9, 33, 64, 128, 300):
        part = stq.q8_matmul(A[:m], sa[:m], W[:77], sw[:77], out_dtype=torch.float32)
        assert torch.equal(part, full[:m, :77]), m


@pytest.mark.parametrize("m", [1, 24, 64, 150])
def test_linear_under_graph_and_on_another_stream(stq, m):
    n, k = 520, 2000
    W, sw = stq.q8_quantize_rows(_rand((n, k), 21).cuda())
    x = _rand((m, k), 22).bfloat16().cuda()
    q, s = stq.q8_quantize_rows(x)
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")

    def call():
        stq.q8_quantize_rows(x, out=q, scale=s)
        stq.q8_matmul(q, s, W, sw, out=y)
    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.synchronize()
    for r in range(4):
        x.copy_(_rand((m, k), 30 + r).bfloat16())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        with torch.cuda.stream(side):
            want = stq.q8_matmul(*stq.q8_quantize_rows(x), W, sw)
        torch.cuda.synchronize()
        assert torch.equal(got, want), r


def test_binding_refusals(stq):
    q = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    s = torch.ones(4, device="cuda")
    with pytest.raises(ValueError, match="same length"):
        stq.q8_matmul(q, s, q[:, :16], s)
    with pytest.raises(ValueError, match="a_scale"):
        stq.q8_matmul(q, s[:3], q, s)
    with pytest.raises(ValueError, match="last row"):
        t = torch.zeros(4 * 32 - 3, dtype=torch.int8, device="cuda").as_strided((4, 29), (32, 1))
        stq.q8_matmul(t, s, t, s)
    with pytest.raises(ValueError, match="contiguous rows"):
        stq.q8_matmul(q.t().contiguous().t(), s, q, s)
    with pytest.raises(stq.StqError, match="16-byte aligned"):
        t = torch.zeros(4, 40, dtype=torch.int8, device="cuda")
        stq.q8_matmul(t[:, 8:40], s, q, s)
    with pytest.raises(stq.StqError, match="row stride"):
        stq.q8_matmul(q[:1].expand(4, 32), s, q, s)
    with pytest.raises(ValueError, match="out_dtype"):
        stq.q8_matmul(q, s, q, s, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="must be torch.float32"):
        stq.q8_quantize_rows(torch.zeros(2, 8, dtype=torch.float16, device="cuda"))


@pytest.mark.parametrize("k", [77, 80, 1])
def test_nothing_to_multiply(stq, k):
    """No tokens or no channels, from the quantizer to the product, whatever k."""
    some, none = _rand((5, k), 41).cuda(), torch.empty((0, k), device="cuda")
    for a, w in ((none, some), (some, none), (none, none)):
        qa, sa = stq.q8_quantize_rows(a)
        qw, sw = stq.q8_quantize_rows(w)
        y = stq.q8_matmul(qa, sa, qw, sw)
        assert y.shape == (a.shape[0], w.shape[0])
        out = torch.empty(y.shape, device="cuda")
        assert stq.q8_matmul(qa, sa, qw, sw, out=out) is out
    q, s = stq.q8_quantize_rows(none, out=torch.empty((0, k), dtype=torch.int8, device="cuda"))
    assert q.shape == (0, k) and s.shape == (0,)


def test_out_of_another_type_than_out_dtype_is_refused(stq):
    q, s = stq.q8_quantize_rows(_rand((3, 32), 51).cuda())
    y = torch.full((3, 3), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="out must be torch.float32"):
        stq.q8_matmul(q, s, q, s, out=y, out_dtype=torch.float32)
    assert bool((y == 7.0).all())
    want = stq.q8_matmul(q, s, q, s)
    assert want.dtype == torch.bfloat16
    assert torch.equal(stq.q8_matmul(q, s, q, s, out=y, out_dtype=torch.bfloat16), want)
    full = torch.empty((3, 3), device="cuda")
    assert torch.equal(stq.q8_matmul(q, s, q, s, out=full).bfloat16(), want)   # out alone says its type
