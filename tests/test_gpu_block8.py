"""The FP8 block-128 linear layer against 64-bit references (needs an MI355X).

Quantized values are compared exactly.  A product of K terms is summed in fp32: each of at most K
additions is off by at most one step (2^-23, the matrix cores may truncate) of a partial sum, which the
sum of magnitudes S bounds, so |Y - ref| <= K 2^-23 S, plus half a step of the output type.  A bf16 output
may come from the E4M3 matrix instruction, which drops what lies below 2^-13 of the largest of eight
products: up to seven of them, each below 2^-13 of a part of S, so 2^-10 S more.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def data(r, c, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(r, c, generator=g) * scale
    x[:, torch.randint(0, c, (max(1, c // 64),), generator=g)] *= 37.0
    x[torch.randint(0, r, (max(1, r // 64),), generator=g)] *= 2.0 ** -12
    return x.to(dt)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check_product(Y, a, b, dt, K):
    want, S = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = (K * 2.0 ** -23 + (2.0 ** -10 if dt == torch.bfloat16 else 0)) * S + HALF[dt] * np.abs(want) + 2.0 ** -140
    err = np.abs(f64(Y) - want)
    assert Y.dtype == dt and (err <= tol).all(), float((err / tol).max())


SHAPES = [(1, 1), (1, 129), (7, 128), (128, 128), (130, 777), (300, 64), (257, 513)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("mode", [fp4.FP4_BLOCK_VECTOR, fp4.FP4_BLOCK_SQUARE])
def test_quantize(shape, mode, dt):
    R, C = shape
    x = data(R, C, DT[dt], 3)
    want_r = ref.blocks(f64(x), 128 if mode else 1, 128)
    want_c = ref.blocks(f64(x), 128, 128 if mode else 1)
    both = fp4.block8_quantize(x.to(DEV), mode, rows=True, cols=True)
    for rows, cols in ((True, True), (True, False), (False, True)):
        r, c = fp4.block8_quantize(x.to(DEV), mode, rows=rows, cols=cols)
        if rows:
            assert np.array_equal(f64(fp4.block8_dequantize(r)), want_r)
            assert torch.equal(r.codes, both[0].codes) and int(r.codes[:, C:].sum()) == 0
        if cols:
            assert np.array_equal(f64(fp4.block8_dequantize(c)), want_c.T)
            assert torch.equal(c.codes, both[1].codes) and int(c.codes[:, R:].sum()) == 0
    assert np.array_equal(f64(fp4.block8_dequantize(both[0], torch.bfloat16)), want_r)


def test_quantize_borders():
    """Scale borders, ties, signs of zero, the smallest and largest floats, in one row of blocks."""
    v = torch.zeros(9, 256)
    v[0, 0], v[0, 1:4] = 448.0, torch.tensor([17.0, 19.0, -2.0 ** -10])
    v[1, 0], v[1, 1] = 448.0001, -448.0
    v[2, 0], v[2, 1] = 1e-45, -1e-45
    v[3, 0], v[3, 1] = 3.4e38, 1e38
    v[4, 0], v[4, 1] = 2.0 ** -126, 2.0 ** -119
    v[5, 0] = -0.0
    v[6] = torch.arange(256) * 0.37
    v[7] = torch.exp2(torch.linspace(-40, 40, 256))
    v[8, 130] = 5.0
    r, _ = fp4.block8_quantize(v.to(DEV))
    with np.errstate(over="ignore"):  # 3.4e38 rounds up to 2^128, which fp32 holds as infinity
        want = ref.blocks(f64(v), 1, 128).astype(np.float32)
    got = f64(fp4.block8_dequantize(r))
    assert [i for i in range(9) if not np.array_equal(got[i], want[i])] == []
    assert np.signbit(got[5, 0])


def test_nonfinite_blocks():
    """A block with a NaN or an infinity poisons exactly its own block, and the products that touch it."""
    x = data(70, 300, torch.bfloat16, 5)
    x[3, 140], x[40, 299] = float("nan"), float("-inf")
    w = data(300, 33, torch.bfloat16, 6, 0.05)
    r, c = fp4.block8_quantize(x.to(DEV), rows=True, cols=True)
    for got, want in ((r, ref.blocks(f64(x), 1, 128)), (c, ref.blocks(f64(x), 128, 1).T)):
        assert np.array_equal(f64(fp4.block8_dequantize(got)), want, equal_nan=True)
    wq = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1]
    y = f64(fp4.block8_linear_forward(x.to(DEV), wq))
    bad = np.zeros(70, bool)
    bad[[3, 40]] = True
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()


LINEAR = [(1, 128, 128), (1, 777, 1290), (3, 4096, 40), (16, 130, 17), (17, 512, 129), (33, 640, 256), (48, 1408, 256),
          (64, 2000, 513), (65, 513, 64), (100, 300, 1000), (129, 128, 257), (512, 384, 640), (2100, 256, 2176)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", LINEAR)
def test_linear(shape, dt):
    M, K, N = shape
    x, w = data(M, K, DT[dt], 7), data(K, N, DT[dt], 8, 0.05)
    wq = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1]
    a, b = ref.blocks(f64(x), 1, 128), ref.blocks(f64(w), 128, 128).T
    for out in (torch.bfloat16, torch.float32):
        check_product(fp4.block8_linear_forward(x.to(DEV), wq, out_dtype=out), a, b, out, K)
    wv = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_VECTOR, rows=False, cols=True)[1]  # vector blocks on both sides
    check_product(fp4.block8_linear_forward(x.to(DEV), wv), a, ref.blocks(f64(w), 128, 1).T, DT[dt], K)


def test_linear_extreme_scales():
    """Blocks near both ends of the scale range: exponents add beyond fp32's own range only in the sum."""
    x, w = torch.zeros(20, 256), torch.zeros(256, 40)
    x[:, :128], w[:128] = torch.randn(20, 128) * 1e30, torch.randn(128, 40) * 1e-34
    x[:, 128:], w[128:] = torch.randn(20, 128) * 1e-36, torch.randn(128, 40) * 1e30
    wq = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1]
    a, b = ref.blocks(f64(x), 1, 128), ref.blocks(f64(w), 128, 128).T
    check_product(fp4.block8_linear_forward(x.to(DEV), wq), a, b, torch.float32, 256)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_strided_and_offset_inputs(M, dt):
    """A column range of a wider matrix, from an odd element on; and dy likewise in the backward."""
    K, N = 391, 200
    wide = data(M, K + 26, DT[dt], 9).to(DEV)
    x = wide[:, 13:13 + K]
    w = data(K, N + 3, DT[dt], 10, 0.05).to(DEV)[:, 3:]
    wr, wc = fp4.block8_quantize(w, fp4.FP4_BLOCK_SQUARE, rows=True, cols=True)
    y, xt = fp4.block8_linear_forward(x, wc, for_backward=True)
    y2, xt2 = fp4.block8_linear_forward(x.contiguous(), wc, for_backward=True)
    assert torch.equal(y, y2) and torch.equal(xt.codes, xt2.codes)
    check_product(y, ref.blocks(f64(x), 1, 128), ref.blocks(f64(w), 128, 128).T, DT[dt], K)
    dy = data(M, N + 5, DT[dt], 11, 1e-3).to(DEV)[:, 1:N + 1]
    got, want = fp4.block8_linear_backward(dy, wr, xt), fp4.block8_linear_backward(dy.contiguous(), wr, xt)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


STEP = [(1, 1, 1), (5, 128, 200), (130, 777, 129), (300, 257, 512), (1111, 130, 260)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", STEP)
def test_step(shape, dt):
    M, K, N = shape
    x, w, dy = data(M, K, DT[dt], 12), data(K, N, DT[dt], 13, 0.05), data(M, N, DT[dt], 14, 1e-3)
    wr, wc = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=True, cols=True)
    y, xt = fp4.block8_linear_forward(x.to(DEV), wc, for_backward=True)
    dx, dw = fp4.block8_linear_backward(dy.to(DEV), wr, xt)
    wv = ref.blocks(f64(w), 128, 128)
    check_product(y, ref.blocks(f64(x), 1, 128), wv.T, DT[dt], K)
    check_product(dx, ref.blocks(f64(dy), 1, 128), wv, DT[dt], N)
    check_product(dw, ref.blocks(f64(x), 128, 1).T, ref.blocks(f64(dy), 128, 1).T, DT[dt], M)
    assert torch.equal(fp4.block8_linear_backward(dy.to(DEV), wr, None)[0], dx)
    assert torch.equal(fp4.block8_linear_backward(dy.to(DEV), None, xt)[1], dw)


def test_gradient_against_differences():
    """Where quantization changes nothing (values on the grid), dx and dw are the slopes of sum(y dy):
    differences of the layer's own outputs, exact for a linear function on representable values."""
    g = torch.Generator().manual_seed(1)
    small = lambda *s: torch.randint(-7, 8, s, generator=g).float()  # noqa: E731
    x, w, dy = small(130, 140), small(140, 66), small(130, 66)
    for t in (x, w, dy):
        t[0, 0] = 8.0  # the same scales before and after a step of 1
    run = lambda x, w: fp4.block8_linear_forward(  # noqa: E731
        x.to(DEV), fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1])
    wr, wc = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=True, cols=True)
    y, xt = fp4.block8_linear_forward(x.to(DEV), wc, for_backward=True)
    dx, dw = fp4.block8_linear_backward(dy.to(DEV), wr, xt)
    loss = lambda y: float((y.cpu().double() * dy.double()).sum())  # noqa: E731
    base = loss(y)
    for i, j in ((3, 5), (129, 139), (64, 128)):
        x2 = x.clone()
        x2[i, j] += 1.0
        assert loss(run(x2, w)) - base == float(dx[i, j])
    for i, j in ((3, 5), (139, 65), (128, 1)):
        w2 = w.clone()
        w2[i, j] += 1.0
        assert loss(run(x, w2)) - base == float(dw[i, j])


def test_repeated_and_streamed():
    """The same bits on every run, on another stream, and replayed from a graph."""
    x, w = data(200, 1000, torch.bfloat16, 15).to(DEV), data(1000, 300, torch.bfloat16, 16).to(DEV)
    wq = fp4.block8_quantize(w, fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1]
    for m in (1, 40, 198):
        y = fp4.block8_linear_forward(x[:m], wq)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y2 = fp4.block8_linear_forward(x[:m], wq)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
        g = torch.cuda.CUDAGraph()
        xin = x[:m].clone()
        with torch.cuda.graph(g):
            yg = fp4.block8_linear_forward(xin, wq)
        for k in range(3):
            xin.copy_(x[k:k + m])
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(yg, fp4.block8_linear_forward(x[k:k + m].contiguous(), wq))


def test_refusals():
    x = torch.zeros(4, 256, device=DEV)
    w = fp4.block8_quantize(torch.zeros(256, 8, device=DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1]
    for bad in (x[:, ::2], x.t(), x[:1].expand(4, 256), x[0], x.cpu()):
        with pytest.raises(ValueError):
            fp4.block8_linear_forward(bad, w)
    with pytest.raises(TypeError):
        fp4.block8_linear_forward(x.half(), w)
    with pytest.raises(ValueError):
        fp4.block8_linear_forward(x[:, :255], w)
    with pytest.raises(fp4.Fp4Error):
        fp4.block8_linear_forward(x, w, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert fp4.block8_linear_forward(x[:0], w).shape == (0, 8)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("M", [1, 3, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("K,N", [(1, 1), (130, 17), (777, 48), (2176, 100), (1000, 1290)])
def test_few_rows(M, K, N, dt):
    """A decode batch: few rows, from strided rows at an odd element, with and without the transposed operand."""
    x, w = data(M, K, DT[dt], M + K), data(K, N, DT[dt], N, 0.02)
    wide = torch.zeros(M, K + 3, dtype=DT[dt])
    wide[:, 1:1 + K] = x
    xs = wide.to(DEV)[:, 1:1 + K]
    _, wq = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)
    a, b = ref.blocks(f64(x), 1, 128), ref.blocks(f64(w), 128, 128).T
    for out in (torch.bfloat16, torch.float32):
        y = fp4.block8_linear_forward(xs, wq, out_dtype=out)
        check_product(y, a, b, out, K)
        z, _ = fp4.block8_linear_forward(xs, wq, out_dtype=out, for_backward=True)
        check_product(z, a, b, out, K)
        q = fp4.block8_gemm(fp4.block8_quantize(xs)[0], wq, out)
        assert torch.equal(q, z)


def test_few_rows_nonfinite():
    """A block with a NaN or an infinity makes its row NaN, and no other."""
    for M in (5, 40):
        x, w = data(M, 500, torch.bfloat16, 3), data(500, 40, torch.bfloat16, 4, 0.02)
        x[1, 130], x[3, 499] = float("nan"), float("inf")
        _, wq = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)
        y = f64(fp4.block8_linear_forward(x.to(DEV), wq))
        bad = np.zeros(M, bool)
        bad[[1, 3]] = True
        assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()


@pytest.mark.parametrize("M,N,K", [(4097, 4100, 300), (4200, 4352, 129), (8200, 2100, 640)])
def test_large_tiles(M, N, K):
    """More than one 256 x 256 tile a workgroup: ragged edges, an odd number of blocks, both output types."""
    x, w = data(M, K, torch.bfloat16, 1), data(N, K, torch.bfloat16, 2)
    a, b = fp4.block8_quantize(x.to(DEV))[0], fp4.block8_quantize(w.to(DEV))[0]
    va, vb = ref.blocks(f64(x), 1, 128), ref.blocks(f64(w), 1, 128)
    for out in (torch.bfloat16, torch.float32):
        y = fp4.block8_gemm(a, b, out)
        check_product(y, va, vb, out, K)
        for _ in range(3):
            assert torch.equal(fp4.block8_gemm(a, b, out), y)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("M,K,N", [(1, 7300, 200), (2, 6500, 33), (1, 6150, 40), (16, 9000, 100), (5, 11008, 48), (17, 3300, 130),
                                   (33, 6500, 64), (64, 6500, 17), (48, 4224, 300)])
def test_few_rows_long(M, K, N, dt):
    """More blocks along K than the waves have on their way at once: every wave refills, several times, and ends
    anywhere in its turn."""
    x, w = data(M, K, DT[dt], M + K), data(K, N, DT[dt], N, 0.02)
    _, wq = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)
    a, b = ref.blocks(f64(x), 1, 128), ref.blocks(f64(w), 128, 128).T
    for out in (torch.bfloat16, torch.float32):
        y = fp4.block8_linear_forward(x.to(DEV), wq, out_dtype=out)
        check_product(y, a, b, out, K)
        z, _ = fp4.block8_linear_forward(x.to(DEV), wq, out_dtype=out, for_backward=True)
        check_product(z, a, b, out, K)


@pytest.mark.parametrize("M", [1, 2])
def test_few_rows_wide(M):
    """So many columns that a workgroup has four waves, each with more blocks than it has on their way."""
    K, N = 4000, 16400
    x, w = data(M, K, torch.bfloat16, 21), data(K, N, torch.bfloat16, 22, 0.02)
    _, wq = fp4.block8_quantize(w.to(DEV), fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)
    a = ref.blocks(f64(x), 1, 128)
    for out in (torch.bfloat16, torch.float32):
        y = fp4.block8_linear_forward(x.to(DEV), wq, out_dtype=out)
        for cols in (slice(0, 128), slice(8064, 8192), slice(16384, N)):
            check_product(y[:, cols], a, ref.blocks(f64(w[:, cols]), 128, 128).T, out, K)


def test_dequantize_largest():
    """2^34 elements, the most that an operand may have (16 GiB of codes, 32 of bf16): every value is written."""
    side = 1 << 17
    op = fp4.Block8(side, side, fp4.FP4_BLOCK_SQUARE, DEV)
    op.codes.fill_(0x38)   # 1
    op.scales.fill_(128)   # 2
    op.codes[-1, -3:] = torch.tensor([0x40, 0xB8, 0], dtype=torch.uint8, device=DEV)
    y = fp4.block8_dequantize(op, torch.bfloat16)
    assert y[-1, -4:].tolist() == [2.0, 4.0, -2.0, 0.0]
    y[-1, -3:] = 2.0
    assert all(bool((part == 2).all()) for part in y.split(1 << 13))
    del y, op
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [4, 40, 130])
def test_products_at_the_ends_of_the_range(M):
    """An fp32 output takes the operands as bf16 holds them: values next to the smallest are rounded to its multiples of
    2^-133, and 256 * 2^120 is infinite; 240 * 2^120 is a number.  A bf16 output takes the values themselves."""
    x, w = torch.zeros(M, 128), torch.zeros(128, 70)
    x[0, :3], x[1, 0], x[2, 0], x[3, :2] = torch.tensor([2.0 ** -131, 2.0 ** -135, 5e-39]), 3.2e38, 3.39e38, torch.tensor([1.0, -3.0])
    w[0, 0], w[:3, 1], w[5, 2] = 2.0 ** -100, 2.0 ** 100, 1.0
    xq, wq = fp4.block8_quantize(x.to(DEV))[0], fp4.block8_quantize(w.to(DEV), rows=False, cols=True)[1]
    y, yb = fp4.block8_gemm(xq, wq, torch.float32), fp4.block8_gemm(xq, wq, torch.bfloat16)
    a, b = (f64(fp4.block8_dequantize(t, torch.bfloat16)) for t in (xq, wq))
    with np.errstate(invalid="ignore", over="ignore"):
        want = (a @ b.T).astype(np.float32)
        assert np.isinf(a[2, 0]) and np.isnan(want[2, 2]) and np.isfinite(want[:2]).any()
        got = f64(y)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
        ok = np.isfinite(want)
        assert (np.abs(got[ok] - want[ok]) <= 2.0 ** -20 * np.abs(want[ok])).all()
    av, bv = ref.blocks(f64(x), 1, 128), ref.blocks(f64(w), 128, 1).T
    cols = [0, *range(2, 70)]  # in column 1 the third value and the second leave the type's range
    check_product(yb[:, cols], av, bv[cols], torch.bfloat16, 128)
    check_product(yb[[0, 3], 1:2], av[[0, 3]], bv[1:2], torch.bfloat16, 128)
    assert torch.isinf(yb[1:3, 1]).all()
