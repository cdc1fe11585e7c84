"""MXFP4 quantizer and linear layer: refusals on the host, codes and scales bit for bit against
the 64-bit definition (mx_reference.py), products within a derived bound of the exact product of
the operands' values."""
import numpy as np
import pytest
import torch

import mx_reference as R
import nvfp4_block_scaled_14_b200 as nv
from gpu_helpers import assert_gemm_close, to_numpy_f64
from nvfp4_block_scaled_14_b200 import _lib as L

FAKE = 0x10000  # never dereferenced: each call below fails its host-side check first


@pytest.fixture(scope="module")
def lib():
    return L.load()


# ---- refusals (no GPU) -----------------------------------------------------------------------


def test_scale_bytes(lib):
    assert lib.nvfp4_mxfp4_scales_bytes(4096, 2048, 0) == 4096 * 64
    assert lib.nvfp4_mxfp4_scales_bytes(4096, 2048, 1) == 4096 * 64
    assert lib.nvfp4_mxfp4_scales_bytes(1, 32, 1) == 512
    assert lib.nvfp4_mxfp4_scales_bytes(129, 160, 1) == 2 * 128 * 8
    assert lib.nvfp4_mxfp4_scales_bytes(-1, 32, 1) == 0


def test_quantize_refusals(lib):
    q = lib.nvfp4_quantize_mxfp4
    rows = [FAKE, FAKE, None]
    none = [None] * 3
    assert q(FAKE, 1, 8, 48, 0, *rows, *none, None) == L.NVFP4_ERR_SHAPE
    assert q(FAKE, 1, -1, 64, 0, *rows, *none, None) == L.NVFP4_ERR_SHAPE
    assert q(FAKE, 1, 8, 1 << 31, 0, *rows, *none, None) == L.NVFP4_ERR_SHAPE
    assert q(FAKE, 2, 8, 64, 0, *rows, *none, None) == L.NVFP4_ERR_INVALID_ARG
    assert q(FAKE, 1, 8, 64, 2, *rows, *none, None) == L.NVFP4_ERR_INVALID_ARG
    assert q(None, 1, 8, 64, 0, *rows, *none, None) == L.NVFP4_ERR_INVALID_ARG
    assert q(FAKE, 1, 8, 64, 0, *none, *none, None) == L.NVFP4_ERR_INVALID_ARG
    assert q(FAKE, 1, 8, 64, 0, FAKE, None, None, *none, None) == L.NVFP4_ERR_INVALID_ARG
    assert q(FAKE, 1, 8, 64, 0, *rows, FAKE, None, None, None) == L.NVFP4_ERR_INVALID_ARG
    assert q(FAKE, 1, 8, 64, 0, *rows, None, FAKE, None, None) == L.NVFP4_ERR_INVALID_ARG
    assert q(FAKE + 8, 1, 8, 64, 0, *rows, *none, None) == L.NVFP4_ERR_ALIGNMENT
    assert q(FAKE, 1, 8, 64, 0, FAKE, FAKE, FAKE + 4, *none, None) == L.NVFP4_ERR_ALIGNMENT
    assert q(FAKE, 1, 8, 64, 0, *none, FAKE, FAKE + 8, None, None) == L.NVFP4_ERR_ALIGNMENT
    assert q(None, 1, 0, 64, 0, *none, *none, None) == L.NVFP4_OK  # empty


def test_dequantize_refusals(lib):
    d = lib.nvfp4_dequantize_mxfp4
    assert d(FAKE, FAKE, 8, 48, 0, FAKE, None) == L.NVFP4_ERR_SHAPE
    assert d(FAKE, FAKE, 8, 64, 5, FAKE, None) == L.NVFP4_ERR_INVALID_ARG
    assert d(FAKE, None, 8, 64, 0, FAKE, None) == L.NVFP4_ERR_INVALID_ARG
    assert d(FAKE, FAKE, 8, 64, 0, FAKE + 8, None) == L.NVFP4_ERR_ALIGNMENT
    assert d(None, None, 0, 64, 0, None, None) == L.NVFP4_OK


def test_linear_refusals(lib):
    li = lib.nvfp4_linear_mxfp4
    ops = [FAKE] * 4
    assert li(*ops, 64, 64, 48, 1, FAKE, None, 0, 0, None) == L.NVFP4_ERR_SHAPE
    assert li(*ops, -1, 64, 64, 1, FAKE, None, 0, 0, None) == L.NVFP4_ERR_SHAPE
    assert li(*ops, 64, 64, 64, 3, FAKE, None, 0, 0, None) == L.NVFP4_ERR_INVALID_ARG
    assert li(*ops, 64, 64, 64, 1, FAKE, None, 0, 2, None) == L.NVFP4_ERR_INVALID_ARG
    assert li(*ops, 64, 64, 64, 1, None, None, 0, 0, None) == L.NVFP4_ERR_INVALID_ARG
    assert li(*ops, 0, 64, 64, 1, None, None, 0, 0, None) == L.NVFP4_OK
    dy = lib.nvfp4_linear_dynamic_mxfp4
    ops = [FAKE, 1, FAKE, FAKE]
    assert dy(FAKE, 4, FAKE, FAKE, 64, 64, 64, 1, FAKE, None, 0, 0, None) == \
        L.NVFP4_ERR_INVALID_ARG
    assert dy(*ops, 64, 64, 33, 1, FAKE, None, 0, 0, None) == L.NVFP4_ERR_SHAPE
    assert dy(*ops, 64, 0, 64, 1, None, None, 0, 0, None) == L.NVFP4_OK


def test_binding_refuses_cpu_tensors_and_bad_arguments():
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        nv.quantize_mxfp4(x)
    q = nv.MXFP4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8),
                       torch.zeros(4, 2, dtype=torch.uint8), 4, 64)
    with pytest.raises(ValueError):
        nv.dequantize_mxfp4(q)
    with pytest.raises(ValueError):
        nv.linear_mxfp4(q, q)
    with pytest.raises(TypeError):
        nv.linear_mxfp4(x, q)
    with pytest.raises(TypeError):
        nv.linear_dynamic_mxfp4(x, q)


def test_reference_against_a_hand_worked_block():
    # m = 7: floor(log2 7) - 2 = 0 (7 saturates to 6); ceil: 7 > 6 so 2^1
    x = np.zeros((1, 32))
    x[0, :8] = [7.0, -5.0, 2.5, 0.25, 0.75, -0.1, 1.25, 3.5]
    p, s = R.quantize(x, "floor")
    assert s[0, 0] == 127
    assert R.values(p, s)[0, :8].tolist() == [6.0, -4.0, 2.0, 0.0, 1.0, -0.0, 1.0, 4.0]
    p, s = R.quantize(x, "ceil")
    assert s[0, 0] == 128
    assert R.values(p, s)[0, :8].tolist() == [8.0, -4.0, 2.0, 0.0, 1.0, -0.0, 1.0, 4.0]


# ---- quantize (GPU) --------------------------------------------------------------------------


@pytest.fixture(scope="module")
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nv.load()


def spread(rows, cols, seed, dtype):
    """Values over many binades, some exact ties, some zeros."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)) * np.exp2(g.integers(-12, 12, (rows, cols // 32)).repeat(32, 1))
    ties = g.random((rows, cols)) < 0.1
    x = np.where(ties, np.exp2(np.floor(np.log2(np.abs(x) + 1e-30))) * 1.25, x)
    x[g.random((rows, cols)) < 0.05] = 0.0
    t = torch.from_numpy(x.astype(np.float32))
    return t.to(dtype).cuda()


def check_side(q, x64, rule):
    p, s = R.quantize(x64, rule)
    assert (q.rows, q.cols) == x64.shape
    got = q.codes.cpu().numpy()
    assert np.array_equal(got, p), np.argwhere(got != p)[:4].tolist()
    if q.scales_lin is not None:
        assert np.array_equal(q.scales_lin.cpu().numpy(), s)
    if q.scales_swz is not None:
        assert np.array_equal(q.scales_swz.cpu().numpy(), R.swizzle(s))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 32), (31, 64), (32, 96), (33, 160), (128, 128),
                                       (129, 288), (300, 1056)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_quantize_both_sides(cuda, rows, cols, dtype, rule):
    x = spread(rows, cols, rows + cols, dtype)
    x64 = x.double().cpu().numpy()
    qr, qc = nv.quantize_mxfp4(x, rule, "both", linear=True)
    check_side(qr, x64, rule)
    check_side(qc, R.transposed(x64), rule)
    check_side(nv.quantize_mxfp4(x, rule, "rows"), x64, rule)
    check_side(nv.quantize_mxfp4(x, rule, "cols", swizzled=False, linear=True),
               R.transposed(x64), rule)


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_extreme_blocks(cuda, dtype, rule):
    tiny = torch.finfo(dtype).smallest_normal
    top = torch.finfo(dtype).max
    x = torch.zeros(9, 64, dtype=dtype)
    x[0, :4] = torch.tensor([top, -top, top / 2, 1.0], dtype=dtype)
    x[1, :4] = torch.tensor([tiny, -tiny / 2, tiny / 4, 0.0], dtype=dtype)
    x[2, 40] = tiny / 64                      # subnormal maximum
    x[3, :] = -0.0
    x[4, 3], x[4, 4] = float("nan"), 5.0
    x[5, 33], x[5, 34] = float("inf"), 1.0    # the first block of the row stays finite
    x[6, 0] = -float("inf")
    x[7, :2] = torch.tensor([6.0, 1.5], dtype=dtype)
    x[8, :3] = torch.tensor([6.03125, 4.0, 2.0 ** -120], dtype=dtype)
    x = x.cuda()
    x64 = x.double().cpu().numpy()
    qr, qc = nv.quantize_mxfp4(x, rule, "both", linear=True)
    check_side(qr, x64, rule)
    check_side(qc, R.transposed(x64), rule)
    assert qr.scales_lin[4, 0] == 255 and qr.scales_lin[5].tolist()[1] == 255
    v = nv.dequantize_mxfp4(qr).cpu().numpy()
    # the value is an fp32 product: the fp32 maximum is just below 4 * 2^126 = 2^128, which its
    # code rounds to under the ceil rule and which overflows fp32
    with np.errstate(over="ignore"):
        ref = R.values(qr.codes.cpu().numpy(), qr.scales_lin.cpu().numpy()).astype(np.float32)
    assert np.array_equal(v, ref, equal_nan=True)


@pytest.mark.gpu
def test_quantize_strided_input_and_empty(cuda):
    x = spread(96, 256, 5, torch.bfloat16)
    check_side(nv.quantize_mxfp4(x[::3, 64:192], linear=True), x[::3, 64:192].double().cpu().numpy(),
               "floor")
    check_side(nv.quantize_mxfp4(x.T, linear=True), x.T.double().cpu().numpy(), "floor")
    e = nv.quantize_mxfp4(x[:0], orient="both")
    assert e[0].codes.shape == (0, 128) and e[1].codes.shape == (256, 0)
    with pytest.raises(ValueError):
        nv.quantize_mxfp4(x[:, :40].contiguous())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(5, 96), (130, 416)])
def test_quantize_writes_nothing_outside_its_arrays(cuda, rows, cols):
    # every output between guard bytes; the C call itself
    x = spread(rows, cols, 9, torch.bfloat16)
    lib, pad = nv.load(), 64
    rp = -(-rows // 32) * 32
    sizes = [rows * cols // 2, lib.nvfp4_mxfp4_scales_bytes(rows, cols, 1), rows * cols // 32,
             cols * rp // 2, lib.nvfp4_mxfp4_scales_bytes(cols, rp, 1), cols * rp // 32]
    bufs = [torch.full((-(-n // 16) * 16 + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
            for n in sizes]
    st = lib.nvfp4_quantize_mxfp4(x.data_ptr(), 1, rows, cols, 0,
                                  *[b.data_ptr() + pad for b in bufs],
                                  torch.cuda.current_stream().cuda_stream or None)
    assert st == 0
    torch.cuda.synchronize()
    for b, n in zip(bufs, sizes):
        assert (b[:pad] == 0xA5).all() and (b[pad + n:] == 0xA5).all()
    p, s = R.quantize(x.double().cpu().numpy())
    assert np.array_equal(bufs[0][pad:pad + sizes[0]].cpu().numpy(), p.reshape(-1))
    assert np.array_equal(bufs[2][pad:pad + sizes[2]].cpu().numpy(), s.reshape(-1))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 160), (257, 1024), (3000, 96)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_dequantize_all_bytes(cuda, rows, cols, out):
    g = torch.Generator().manual_seed(rows)
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g)
    s = torch.randint(0, 256, (rows, cols // 32), dtype=torch.uint8, generator=g)
    q = nv.MXFP4Tensor(codes.cuda(), None, s.cuda(), rows, cols)
    got = nv.dequantize_mxfp4(q, out)
    # exact in fp32 up to overflow (byte 254), and two significant bits fit bf16
    ref = torch.from_numpy(R.values(codes.numpy(), s.numpy())).float().to(out)
    assert torch.equal(got.cpu().nan_to_num(nan=123.0, posinf=9e37, neginf=-9e37),
                       ref.nan_to_num(nan=123.0, posinf=9e37, neginf=-9e37))
    # an output that is aligned to 16 bytes only
    n = 16 // got.element_size()
    off = torch.empty(rows * cols + n, dtype=out, device="cuda")[n:].view(rows, cols)
    assert torch.equal(nv.dequantize_mxfp4(q, out, out=off).view(torch.uint8),
                       got.view(torch.uint8))


# ---- products (GPU) --------------------------------------------------------------------------


def operand(rows, cols, seed, lo=118, hi=134):
    """Random codes with random scales (every block its own), as an MXFP4Tensor on the GPU, and
    its float64 values."""
    g = np.random.default_rng(seed)
    p = g.integers(0, 256, (rows, cols // 2)).astype(np.uint8)
    s = g.integers(lo, hi, (rows, cols // 32)).astype(np.uint8)
    q = nv.MXFP4Tensor(torch.from_numpy(p).cuda(), torch.from_numpy(R.swizzle(s)).cuda(),
                       torch.from_numpy(s).cuda(), rows, cols)
    return q, torch.from_numpy(R.values(p, s)).cuda()


def product_bound(va, vw):
    """|fp32 product - exact| for each element: the K64 MMAs' block sums are exact in fp32 (32
    products of multiples of 1/4 below 36, times powers of two), so the accumulator takes at most
    K/32 additions, each off by at most 2 units in the last place (2^-22 relative) of a running sum
    of size at most S = sum |a w|."""
    return (va.shape[1] / 32) * 2.0 ** -22 * (va.abs() @ vw.abs().T)


def check_product(y, va, vw, what=""):
    ref, tol = (va @ vw.T).cpu().numpy(), product_bound(va, vw).cpu().numpy()
    if y.dtype == torch.float32:
        tol = tol + 2.0 ** -24 * np.abs(ref)
    assert_gemm_close(to_numpy_f64(y) if y.dtype == torch.bfloat16 else
                      y.double().cpu().numpy(), ref, y.dtype == torch.bfloat16, tol, what)


SHAPES = [(1, 8, 32), (1, 4096, 2048), (3, 130, 96), (8, 1000, 4096), (16, 1001, 2080),
          (17, 264, 64), (33, 2048, 1056), (64, 384, 512), (128, 520, 1024), (128, 40000, 256),
          (129, 256, 256), (200, 256, 8192), (257, 1001, 2080), (300, 520, 160),
          (513, 1024, 1376), (1999, 2052, 160), (2100, 1044, 2080), (1290, 2050, 288)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_linear_against_exact_product(cuda, M, N, K, out):
    a, va = operand(M, K, 1)
    w, vw = operand(N, K, 2)
    check_product(nv.linear_mxfp4(a, w, out), va, vw, f"{M}x{N}x{K}")
    if M <= 128:
        check_product(nv.linear_mxfp4(a, w, out, resident_weights=True), va, vw, "resident")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(8, 256, 512), (300, 512, 512)])
def test_linear_wide_scale_range_and_nan_blocks(cuda, M, N, K):
    # scales of both operands over most of E8M0 (sums within fp32), one NaN block
    a, va = operand(M, K, 3, 70, 180)
    w, vw = operand(N, K, 4, 100, 140)
    check_product(nv.linear_mxfp4(a, w, torch.float32), va, vw)
    s = a.scales_lin.cpu().numpy()
    s[2, 1] = 255
    a.scales_swz.copy_(torch.from_numpy(R.swizzle(s)))
    y = nv.linear_mxfp4(a, w, torch.float32)
    assert y[2].isnan().all()
    keep = [i for i in range(M) if i != 2]
    check_product(y[keep], va[keep], vw)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (2, 100, 64), (16, 1001, 2080),
                                   (17, 520, 1024), (150, 256, 384)])
@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16])
def test_linear_dynamic(cuda, M, N, K, x_dtype):
    x = spread(M, K, M + K, x_dtype)
    w, vw = operand(N, K, 6)
    q = nv.quantize_mxfp4(x, linear=True)
    va = torch.from_numpy(R.values(q.codes.cpu().numpy(), q.scales_lin.cpu().numpy())).cuda()
    for out in (torch.float32, torch.bfloat16):
        check_product(nv.linear_dynamic_mxfp4(x, w, out), va, vw)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(100, 96, 160), (500, 256, 384)])
def test_training_products(cuda, M, N, K):
    """y, dx and dw of a layer from one quantize of each tensor along both axes."""
    x, w, dy = (spread(*s, i, torch.bfloat16) for i, s in enumerate([(M, K), (N, K), (M, N)]))
    quant = lambda t: nv.quantize_mxfp4(t, orient="both", linear=True)  # noqa: E731
    val = lambda q: torch.from_numpy(R.values(q.codes.cpu().numpy(),  # noqa: E731
                                              q.scales_lin.cpu().numpy())).cuda()
    (x_, xt), (w_, wt), (d_, dt) = quant(x), quant(w), quant(dy)
    for a, b, out in ((x_, w_, torch.bfloat16), (d_, wt, torch.bfloat16), (dt, xt, torch.float32)):
        check_product(nv.linear_mxfp4(a, b, out), val(a), val(b))
    assert nv.linear_mxfp4(dt, xt).shape == (N, K)


@pytest.mark.gpu
def test_linear_writes_nothing_outside_y(cuda):
    # fp32 and bf16 y between guard bytes, rows and columns that end inside a tile
    M, N, K, pad = 1300, 2060, 96, 256
    a, va = operand(M, K, 7)
    w, vw = operand(N, K, 8)
    for dt, esz in ((torch.float32, 4), (torch.bfloat16, 2)):
        buf = torch.full((M * N * esz + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
        y = buf[pad:-pad].view(dt).view(M, N)
        check_product(nv.linear_mxfp4(a, w, dt, out=y), va, vw)
        torch.cuda.synchronize()
        assert (buf[:pad] == 0xA5).all() and (buf[-pad:] == 0xA5).all()


@pytest.mark.gpu
def test_linear_checks_and_empty(cuda):
    a, _ = operand(4, 64, 1)
    w, _ = operand(8, 96, 1)
    with pytest.raises(ValueError):
        nv.linear_mxfp4(a, w)
    w, _ = operand(8, 64, 1)
    with pytest.raises(ValueError):
        nv.linear_mxfp4(a, w, out=torch.empty(4, 9, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        nv.linear_mxfp4(a, w, torch.float16)
    with pytest.raises(ValueError):  # no operand-layout scales
        nv.linear_mxfp4(nv.MXFP4Tensor(a.codes, None, a.scales_lin, 4, 64), w)
    with pytest.raises(ValueError):  # codes of another size than the tensor says
        nv.linear_mxfp4(nv.MXFP4Tensor(a.codes, a.scales_swz, None, 5, 64), w)
    z = nv.quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    assert nv.linear_mxfp4(z, w).shape == (0, 8)
    k0 = nv.quantize_mxfp4(torch.empty(4, 0, device="cuda"))
    w0 = nv.quantize_mxfp4(torch.empty(8, 0, device="cuda"))
    assert (nv.linear_mxfp4(k0, w0) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 40, 300])
def test_captured_and_replayed_on_new_inputs(cuda, M):
    """quantize -> linear in two graphs over one side stream, replayed at the same time on two
    streams: equal to the eager calls, bit for bit."""
    N, K = 512, 2048
    w = nv.quantize_mxfp4(spread(N, K, 3, torch.bfloat16))
    xs = [spread(M, K, i, torch.bfloat16) for i in range(4)]
    eager = [(nv.linear_mxfp4(nv.quantize_mxfp4(x), w), nv.linear_dynamic_mxfp4(x, w)) for x in xs]
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        inp = torch.empty_like(xs[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = (nv.linear_mxfp4(nv.quantize_mxfp4(inp), w), nv.linear_dynamic_mxfp4(inp, w))
        graphs.append((g, inp, out))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(0, 4, 2):
        torch.cuda.synchronize()
        for s, (g, inp, _), x in zip(streams, graphs, xs[k:]):
            with torch.cuda.stream(s):
                inp.copy_(x)
                g.replay()
        torch.cuda.synchronize()
        for (_, _, out), ref in zip(graphs, eager[k:]):
            assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
