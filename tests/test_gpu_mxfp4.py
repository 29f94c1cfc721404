"""MXFP4 matrices on the GPU against the 64-bit oracle: codes and scales bit for bit, products within the fp32 bound."""
import numpy as np
import pytest
import torch

from oracle import mxfp4 as oracle

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
SHAPES = [(1, 1), (1, 32), (31, 33), (128, 128), (129, 257), (300, 1000), (64, 4096), (1000, 72), (257, 31), (2, 5000)]


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import split_gemm_gb300
    return split_gemm_gb300


def _values(rows, cols, dtype, seed=0):
    """Normal values over many binades, exact ties, zeros, whole zero blocks, subnormal and huge ones."""
    g = torch.Generator().manual_seed(seed + 7 * rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    pick = torch.randint(0, 12, (rows, cols), generator=g)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.5])[torch.randint(0, 8, (rows, cols), generator=g)]
    x = torch.where(pick == 0, ties, torch.where(pick == 1, torch.zeros(()), x))
    if rows > 8:
        x[1] = 0
        x[2] = 1e-39 * torch.randn(cols, generator=g)
        x[3] = 1e38 * torch.randn(cols, generator=g).clamp(-3, 3)
        x[4] = -0.0
    return x.to(dtype)


def _np(t):
    return t.detach().cpu().double().numpy()


def _check_quantized(q, x):
    rows, cols = x.shape
    codes, scales = oracle.quantize(_np(x))
    assert q.shape == (rows, cols)
    assert np.array_equal(q.scales.cpu().numpy(), oracle.tile_scales(scales))
    got = oracle.unpack(q.data.cpu().numpy())
    fine = (scales != 255).repeat(32, 1)
    assert np.array_equal(got[fine], codes[fine])


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize(sg, rows, cols, dtype):
    x = _values(rows, cols, dtype)
    xd = x.cuda()
    _check_quantized(sg.mxfp4_quantize(xd), x)
    _check_quantized(sg.mxfp4_quantize(xd, transpose=True), x.t())
    q, q_t = sg.mxfp4_quantize_both(xd)
    _check_quantized(q, x)
    _check_quantized(q_t, x.t())
    codes, scales = oracle.quantize(_np(x))
    want = oracle.values(codes, scales, cols)
    for t in (F32, BF16):
        y = sg.mxfp4_dequantize(q, out_dtype=t)
        assert y.dtype == t and np.array_equal(_np(y), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bad_values_mark_their_block(sg, dtype):
    x = _values(40, 100, dtype)
    x[5, 33], x[9, 99], x[20, 0] = float("nan"), float("inf"), -float("inf")
    for q, v in ((sg.mxfp4_quantize(x.cuda()), x), (sg.mxfp4_quantize(x.cuda(), transpose=True), x.t())):
        _check_quantized(q, v)
        codes, scales = oracle.quantize(_np(v))
        assert np.array_equal(_np(sg.mxfp4_dequantize(q)), oracle.values(codes, scales, v.shape[1]), equal_nan=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("step,shift", [(300, 0), (301, 1), (304, 8)])
def test_quantize_strided(sg, dtype, step, shift):
    wide = _values(70, step + 8, dtype)
    x = wide[:, shift:shift + 290]
    xd = wide.cuda()[:, shift:shift + 290]
    q, q_t = sg.mxfp4_quantize_both(xd)
    _check_quantized(q, x)
    _check_quantized(q_t, x.t())


def test_quantize_more_dimensions_and_empty(sg):
    x = _values(2 * 7 * 5, 64, BF16)
    _check_quantized(sg.mxfp4_quantize(x.reshape(2, 7, 5, 64).cuda()), x)
    q = sg.mxfp4_quantize(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and sg.mxfp4_dequantize(q).shape == (0, 64)


def _operand(sg, rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g).float())
    codes, scales = oracle.quantize(_np(x))
    q = sg.Mxfp4(torch.from_numpy(oracle.pack(codes)).cuda(), torch.from_numpy(oracle.tile_scales(scales)).cuda(), rows, cols)
    return q, oracle.values(codes, scales, cols)


def _check_product(y, a, b, bias, relu, dtype):
    want, bound = oracle.matmul(a, b, bias, relu)
    tol = bound + (2.0 ** -8 * (np.abs(want) + bound) if dtype == BF16 else 0.0)
    err = np.abs(_np(y) - want)
    assert y.dtype == dtype and np.all(err <= tol), f"max excess {np.nanmax(err - tol)}"


MNK = [(1, 1, 1), (1, 64, 32), (1, 1000, 4096), (2, 4096, 64), (3, 129, 2000), (5, 300, 16384), (8, 513, 1024), (17, 256, 96),
       (33, 77, 200), (64, 64, 64), (100, 1000, 160), (127, 128, 129), (128, 256, 512), (130, 130, 130), (255, 257, 1000),
       (300, 40, 3000), (777, 1001, 2000), (1024, 256, 5000), (1500, 8, 512), (2049, 640, 256), (512, 2560, 320),
       (2500, 2600, 100), (2304, 1100, 2080), (5000, 1003, 770), (300, 10000, 64), (2561, 2056, 33), (3000, 1284, 1500)]


@pytest.mark.parametrize("m,n,k", MNK)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_matmul(sg, m, n, k, dtype):
    (qa, a), (qb, b) = _operand(sg, m, k, m + k), _operand(sg, n, k, n + 2 * k)
    _check_product(sg.mxfp4_matmul(qa, qb, out_dtype=dtype), a, b, None, False, dtype)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(n))
    y = sg.mxfp4_matmul(qa, qb, bias.cuda(), relu=True, out_dtype=dtype)
    _check_product(y, a, b, _np(bias), True, dtype)
    assert torch.equal(y, sg.mxfp4_matmul(qa, qb, bias.cuda(), relu=True, out_dtype=dtype))


@pytest.mark.parametrize("m,n,k", [(1, 500, 4096), (9, 700, 300), (200, 200, 8192), (300, 520, 1000), (4096, 512, 512)])
def test_matmul_exact(sg, m, n, k):
    """Scales of 1: the sums are whole multiples of a quarter below 2^24 quarters, so every order gives them exactly."""
    g = torch.Generator().manual_seed(k)
    ops = []
    for rows in (m, n):
        codes = torch.randint(0, 16, (rows, 32 * oracle.blocks_of(k)), generator=g, dtype=torch.uint8).numpy()
        codes[:, k:] = 0
        scales = np.full((rows, oracle.blocks_of(k)), 127, dtype=np.uint8)
        ops.append((sg.Mxfp4(torch.from_numpy(oracle.pack(codes)).cuda(), torch.from_numpy(oracle.tile_scales(scales)).cuda(), rows, k),
                    oracle.values(codes, scales, k)))
    assert 36 * k < 2 ** 22
    assert np.array_equal(_np(sg.mxfp4_matmul(ops[0][0], ops[1][0])), ops[0][1] @ ops[1][1].T)


@pytest.mark.parametrize("m,n,k", [(1, 200, 320), (40, 300, 200), (513, 260, 640)])
def test_every_scale_counts(sg, m, n, k):
    """A scale of its own for every block of either operand, powers of two over a range where sums stay exact."""
    rng = np.random.default_rng(k)
    ops = []
    for rows in (m, n):
        nb = oracle.blocks_of(k)
        codes = np.zeros((rows, 32 * nb), dtype=np.uint8)
        at = rng.integers(0, 32, (rows, nb))
        at[:, -1] %= k - 32 * (nb - 1)
        codes[np.arange(rows)[:, None], 32 * np.arange(nb) + (at if rows == n else 0)] = 2  # one element of 1.0 in a block
        if rows == m:
            codes = np.full_like(codes, 2)
            codes[:, k:] = 0
        scales = (127 + rng.integers(-4, 4, (rows, nb))).astype(np.uint8)
        ops.append((sg.Mxfp4(torch.from_numpy(oracle.pack(codes)).cuda(), torch.from_numpy(oracle.tile_scales(scales)).cuda(), rows, k),
                    oracle.values(codes, scales, k)))
    assert np.array_equal(_np(sg.mxfp4_matmul(ops[0][0], ops[1][0])), ops[0][1] @ ops[1][1].T)


@pytest.mark.parametrize("m,n", [(1, 300), (20, 64), (300, 300)])
def test_nan_blocks_reach_their_rows_alone(sg, m, n):
    k = 256
    (qa, a), (qb, b) = _operand(sg, m, k, 1), _operand(sg, n, k, 2)
    x = torch.randn(m, k)
    x[m // 2, 40] = float("nan")
    qa = sg.mxfp4_quantize(x.cuda())
    y = sg.mxfp4_matmul(qa, qb, relu=True)
    assert torch.isnan(y[m // 2]).all() and torch.isfinite(y[torch.arange(m) != m // 2]).all()
    w = torch.randn(n, k)
    w[n - 1, 255] = float("inf")
    y = sg.mxfp4_matmul(_operand(sg, m, k, 1)[0], sg.mxfp4_quantize(w.cuda()))
    assert torch.isnan(y[:, n - 1]).all() and torch.isfinite(y[:, :n - 1]).all()


def test_matmul_empty_and_other_stream(sg):
    (qa, a), (qb, b) = _operand(sg, 200, 512, 3), _operand(sg, 300, 512, 4)
    assert sg.mxfp4_matmul(sg.mxfp4_quantize(torch.empty(0, 512, device="cuda")), qb).shape == (0, 300)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = sg.mxfp4_matmul(qa, qb, stream=s)
    x = torch.randn(100, 512, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    q = sg.mxfp4_quantize(x, stream=s)
    v = sg.mxfp4_dequantize(q, stream=s)
    s.synchronize()
    _check_product(y, a, b, None, False, F32)
    assert torch.equal(v, sg.mxfp4_dequantize(sg.mxfp4_quantize(x)))


def test_matrices_beyond_32_bit_offsets(sg):
    """More than 2^31 elements: the last rows and columns are quantised, and come back, as they do on their own."""
    rows, cols = 1 << 16, (1 << 15) + 128
    x = torch.randn(rows, cols, device="cuda", dtype=BF16)
    q, q_t = sg.mxfp4_quantize_both(x)
    alone, alone_t = sg.mxfp4_quantize(x[-128:]), sg.mxfp4_quantize(x[:, -128:], transpose=True)
    assert torch.equal(q.data.view(-1)[-alone.data.numel():], alone.data.view(-1))
    assert torch.equal(q.scales.view(-1)[-alone.scales.numel():], alone.scales.view(-1))
    assert torch.equal(q_t.data.view(-1)[-alone_t.data.numel():], alone_t.data.view(-1))
    assert torch.equal(q_t.scales.view(-1)[-alone_t.scales.numel():], alone_t.scales.view(-1))
    assert torch.equal(sg.mxfp4_dequantize(q)[-128:], sg.mxfp4_dequantize(alone))


@pytest.mark.parametrize("n", [(1 << 14) + 16, (1 << 14) + 5])
def test_results_beyond_32_bit_offsets(sg, n):
    """More than 2^31 elements of y, stored by boxes and element by element: the last rows come out as they do on their own."""
    m, k = (1 << 17) + 37, 64
    a, b = torch.randn(m, k, device="cuda"), torch.randn(n, k, device="cuda")
    qb = sg.mxfp4_quantize(b)
    y = sg.mxfp4_matmul(sg.mxfp4_quantize(a), qb, out_dtype=BF16)
    assert torch.equal(y[-300:], sg.mxfp4_matmul(sg.mxfp4_quantize(a[-300:]), qb, out_dtype=BF16))


def test_gradients_of_the_product(sg):
    """dx and dw of y = x w^T from the quantised operands are the oracle's products of the oracle's quantisations."""
    m, n, k = 200, 96, 160
    g = torch.Generator().manual_seed(5)
    x, w, dy = torch.randn(m, k, generator=g), torch.randn(n, k, generator=g), torch.randn(m, n, generator=g)
    val = lambda t: oracle.values(*oracle.quantize(_np(t)), t.shape[1])  # noqa: E731
    (qdy, qdy_t), (_, qx_t) = sg.mxfp4_quantize_both(dy.cuda()), sg.mxfp4_quantize_both(x.cuda())
    dx = sg.mxfp4_matmul(qdy, sg.mxfp4_quantize(w.cuda(), transpose=True))
    dw = sg.mxfp4_matmul(qdy_t, qx_t)
    _check_product(dx, val(dy), val(w.t()), None, False, F32)
    _check_product(dw, val(dy.t()), val(x.t()), None, False, F32)
    # and they approximate the gradients of the unrounded product: E2M1 with a block's scale keeps 1 part in 4,
    # so sums of independent errors stay well below half of the gradient's norm
    assert np.linalg.norm(_np(dx) - _np(dy) @ _np(w)) < 0.5 * np.linalg.norm(_np(dy) @ _np(w))


@pytest.mark.parametrize("call,error", [
    (lambda sg, a, b: sg.mxfp4_quantize(torch.zeros(4, 32, device="cuda", dtype=torch.float16)), TypeError),
    (lambda sg, a, b: sg.mxfp4_matmul(a, b._replace(cols=64)), ValueError),
    (lambda sg, a, b: sg.mxfp4_matmul(a, sg.mxfp4_quantize(torch.zeros(4, 64, device="cuda"))), ValueError),
    (lambda sg, a, b: sg.mxfp4_matmul(a, b, torch.zeros(3, device="cuda")), ValueError),
    (lambda sg, a, b: sg.mxfp4_matmul(a, b, torch.zeros(5, device="cuda").double()), TypeError),
    (lambda sg, a, b: sg.mxfp4_matmul(a, b, out_dtype=torch.float16), TypeError),
    (lambda sg, a, b: sg.mxfp4_matmul_into(torch.zeros(4, 4, device="cuda"), a, b), ValueError),
    (lambda sg, a, b: sg.mxfp4_quantize_into(a, torch.zeros(4, 33, device="cuda")), ValueError),
    (lambda sg, a, b: sg.mxfp4_dequantize(a, out_dtype=torch.int8), TypeError),
    (lambda sg, a, b: sg.mxfp4_dequantize(a._replace(scales=a.scales[:256])), ValueError),
    (lambda sg, a, b: sg.mxfp4_dequantize(a._replace(data=a.data.int())), TypeError),
])
def test_refusals(sg, call, error):
    a, b = sg.mxfp4_quantize(torch.zeros(4, 32, device="cuda")), sg.mxfp4_quantize(torch.zeros(5, 32, device="cuda"))
    with pytest.raises(error):
        call(sg, a, b)
