"""4-bit operators on the GPU against the float64 oracle: quantisation byte by byte, products and
the gated block over ragged sizes, parts of wider operands, rows and columns that must stay as
they were, streams, and graphs."""
import numpy as np
import pytest
import torch

import tensor_transformer_layer_megatron_b200 as mgt
from oracle import mx4

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def randn(*n, seed=0, scale=1.0, dtype=torch.float32):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(*n, generator=g) * scale).to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def unsigned_zero(packed):
    """Packed codes with -0 as 0 (the sign of a zero is not specified)."""
    lo, hi = packed & 15, packed >> 4
    return np.where(lo == 8, 0, lo) | (np.where(hi == 8, 0, hi) << 4)


def operand(fmt, rows, cols, x=None, f=1.0, fill=0xCB):
    """An operand whose buffers hold a pattern before it is written."""
    q = mgt.Mx4(fmt, rows, cols)
    q.codes.fill_(fill)
    q.scales.fill_(fill)
    if fmt == "nvfp4":
        q.factor.copy_(torch.tensor([0.0, f]))
    if x is not None:
        mgt.mx4_quantize(x, q)
    return q


def check_bytes(q, x, f, fill=0xCB):
    codes, byte, _ = mx4.quantize(x, q.fmt, f)
    packed, tiles = mx4.pack(codes, byte)
    assert np.array_equal(unsigned_zero(q.codes.cpu().numpy()), unsigned_zero(packed))
    got = q.scales.cpu().numpy().astype(np.int16)
    assert np.array_equal(got, np.where(tiles < 0, fill, tiles))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 31, 0), (2, 33, 7), (3, 128, 8), (5, 129, 0),
                                           (64, 256, 0), (65, 300, 4), (130, 515, 1), (257, 1000, 24)])
def test_quantize_both_layouts(fmt, dtype, rows, cols, pad):
    x = randn(rows, cols + pad, seed=rows + cols, scale=3.0, dtype=TYPES[dtype])
    x[:, : cols // 2] *= 2.0 ** -7
    x[rows // 2, :] = 0  # a block of zeros in every row-wise group of that row
    xd = x.cuda()[:, :cols]
    f, fac = 1.0, None
    if fmt == "nvfp4":
        fac = torch.full((2,), -3.0, device="cuda")
        mgt.mx4_tensor_factor(xd, fac)
        amax, f = mx4.tensor_factor(np64(xd))
        assert fac.tolist() == [np.float32(amax), f]
    for t in (False, True):
        q, qt = operand(fmt, rows, cols), operand(fmt, cols, rows)
        if fac is not None:
            q.factor.copy_(fac)
            qt = mgt.Mx4(fmt, cols, rows, codes=qt.codes, scales=qt.scales, factor=q.factor)
        mgt.mx4_quantize(xd, q, qt if t else None)
        check_bytes(q, np64(xd), f)
        if t:
            check_bytes(qt, np64(xd).T, f)
    mgt.mx4_quantize(xd, None, qt)
    check_bytes(qt, np64(xd).T, f)
    for name, dt in TYPES.items():  # and back, exactly, into rows of a wider matrix
        y = torch.full((rows, cols + 3), 7.0, dtype=dt, device="cuda")
        mgt.mx4_dequantize(q, y[:, :cols])
        assert np.array_equal(np64(y[:, :cols]), mx4.values(np64(xd), fmt, f))
        assert (y[:, cols:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_every_tie_and_its_neighbours(fmt):
    """Borders between elements, and the fp32 numbers next to them, for every scale of a block."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    n = mx4.BLOCK[fmt]
    rows = []
    scales = [2.0 ** e for e in (-126, -30, 0, 90)] if fmt == "mxfp4" else \
        [(8 + m) / 8 * 2.0 ** e for m in range(8) for e in (-6, 0, 7)] + [2.0 ** -9, 3 * 2.0 ** -9]
    for s in scales:
        b = (borders * np.float32(s)).astype(np.float32)
        v = np.stack([b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(3e38))]).reshape(-1)
        for lot in (v[:15], v[-15:]):
            r = np.zeros(n, np.float32)
            r[0] = 6 * s if fmt == "nvfp4" else 4 * s  # gives the block the scale s
            r[1:16] = lot if fmt == "nvfp4" else np.minimum(lot, np.float32(7.9 * s))
            rows.append(r * np.where(np.arange(n) % 2, -1, 1).astype(np.float32))
    x = torch.tensor(np.array(rows))
    for y in (x, x.t().contiguous()):
        q, qt = operand(fmt, *y.shape), operand(fmt, y.shape[1], y.shape[0])
        if fmt == "nvfp4":
            qt = mgt.Mx4(fmt, qt.rows, qt.cols, codes=qt.codes, scales=qt.scales, factor=q.factor)
        mgt.mx4_quantize(y.cuda(), q, qt)
        check_bytes(q, np64(y), 1.0)
        check_bytes(qt, np64(y).T, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_non_finite_subnormal_and_huge(fmt, dtype):
    x = randn(40, 200, seed=9, dtype=TYPES[dtype])
    x[0, 5], x[1, 70], x[2, 199], x[39, 0] = float("inf"), float("nan"), -float("inf"), float("nan")
    x[3] *= 2.0 ** -126
    x[4] *= 2.0 ** -133  # subnormal
    x[5] *= 2.0 ** 100
    x[6, :] = torch.finfo(TYPES[dtype]).max
    xd = x.cuda()
    q, qt = operand(fmt, 40, 200), operand(fmt, 200, 40)
    f = 1.0
    if fmt == "nvfp4":
        qt = mgt.Mx4(fmt, 200, 40, codes=qt.codes, scales=qt.scales, factor=q.factor)
        mgt.mx4_tensor_factor(xd, q.factor)
        amax, f = mx4.tensor_factor(np64(xd))
        assert q.factor.tolist() == [amax, f]
    for g in ([f] if fmt == "mxfp4" else [f, 2.0 ** -100]):  # also a factor far too small: saturation
        if fmt == "nvfp4":
            q.factor[1] = g
        mgt.mx4_quantize(xd, q, qt)
        check_bytes(q, np64(xd), g)
        check_bytes(qt, np64(xd).T, g)
        y = torch.empty(40, 200, device="cuda")
        mgt.mx4_dequantize(q, y)
        assert np.array_equal(np64(y), mx4.values(np64(xd), fmt, g).astype(np.float32), equal_nan=True)


def product_bound(a, b, bf16, ref):
    """Per element. Products of two elements and two scales have few bits and are exact; the tensor
    core adds 64 of them to the fp32 accumulator at a time, each time within 4 units in the last
    place of the largest partial sum (alignment of the addends and one rounding; a unit is at most
    2^-23 of it), and the partial sums stay below sum |a b|. The result then meets the factor (two
    fp32 products, 2^-24 each) and the rounding to bf16 (2^-8)."""
    steps = -(-a.shape[1] // 64)
    t = np.abs(a) @ np.abs(b).T * (4 * steps * 2.0 ** -23) + np.abs(ref) * 2.0 ** -23
    return t + (np.abs(ref) * 2.0 ** -8 if bf16 else 0) + 1e-37


SHAPES = [(1, 1, 1), (1, 8, 16), (24, 200, 1500), (49, 384, 700), (144, 260, 512), (200, 128, 900), (2, 130, 33), (1, 4096, 1024), (7, 257, 4096), (16, 128, 128),
          (17, 100, 300), (64, 513, 640), (100, 384, 2000), (128, 128, 256), (129, 129, 144),
          (250, 1000, 777), (300, 520, 4096), (512, 256, 512), (777, 1111, 999), (1500, 640, 384), (300, 257, 256)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, fmt, out):
    x, w = randn(M, K, seed=M + N, scale=2.0), randn(N, K, seed=K, scale=0.05)
    fx, fw = (1.0, 1.0) if fmt == "mxfp4" else (2.0 ** -6, 2.0 ** -11)
    A, B = operand(fmt, M, K, x.cuda(), fx, 0xFF), operand(fmt, N, K, w.cuda(), fw, 0xFF)
    a, b = mx4.values(np64(x), fmt, fx), mx4.values(np64(w), fmt, fw)
    ref = a @ b.T
    for pad in (0, 3, 8, 16 - N % 16):  # the last: aligned rows, whose end may not be
        C = torch.full((M + 1, N + pad), 77.0, dtype=TYPES[out], device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        mgt.gemm_mx4(A, B, C[:M, :N], st)
        assert int(st) == 0
        err = np.abs(np64(C[:M, :N]) - ref)
        bound = product_bound(a, b, out == "bf16", ref)
        assert (err <= bound).all(), (err / bound).max()
        assert (C[M] == 77).all() and (C[:, N:] == 77).all()


def values_of(q):
    y = torch.empty(q.rows, q.cols, device="cuda")
    mgt.mx4_dequantize(q, y)
    return y.double()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(300, 2000, 8100), (700, 1000, 6500), (300, 2700, 11000), (260, 4000, 21000),
                                   (1000, 1999, 24500)])
def test_product_of_long_sums(M, N, K, fmt):
    """Sums split over two to five CTAs, and the same bytes from a second call."""
    x, w = randn(M, K, seed=M).cuda(), randn(N, K, seed=N).cuda()
    fx = 1.0 if fmt == "mxfp4" else 2.0 ** -8
    A, B = operand(fmt, M, K, x, fx), operand(fmt, N, K, w, fx)
    a, b, st = values_of(A), values_of(B), torch.zeros(1, dtype=torch.int32, device="cuda")
    C = torch.full((M + 1, N + 3), 77.0, device="cuda")
    mgt.gemm_mx4(A, B, C[:M, :N], st)
    ref, most = a @ b.T, a.abs() @ b.abs().T  # bound: product_bound's, in fp32
    assert ((C[:M, :N].double() - ref).abs() <= most * (4 * -(-K // 64) * 2.0 ** -23) + ref.abs() * 2.0 ** -23).all()
    assert (C[M] == 77).all() and (C[:, N:] == 77).all() and int(st) == 0
    D = torch.empty(M, N, device="cuda")
    mgt.gemm_mx4(A, B, D, st)
    assert torch.equal(C[:M, :N], D)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_of_every_row_count(fmt):
    """Row counts around every step of the few-row kernel's shapes, with a sum long enough that it
    keeps up to 256 rows, and around its end; against the dequantised operands in float64."""
    K, N = 8500, 300
    f = 2.0 ** -6 if fmt == "nvfp4" else 1.0
    w = operand(fmt, N, K, randn(N, K, seed=1, scale=0.05).cuda(), f)
    x = randn(258, K, seed=2).cuda()
    wv = values_of(w)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    steps = -(-K // 64)
    for M in (1, 15, 16, 17, 31, 33, 48, 49, 64, 65, 79, 81, 95, 97, 111, 112, 127, 128, 129, 143, 145, 176,
              177, 191, 193, 208, 209, 223, 225, 239, 241, 255, 256, 257, 258):
        q = operand(fmt, M, K, x[:M], f, 0xFF)
        C = torch.full((M, N), float("nan"), device="cuda")
        mgt.gemm_mx4(q, w, C, st)
        xv = values_of(q)
        ref = xv @ wv.t()
        bound = xv.abs() @ wv.abs().t() * (4 * steps * 2.0 ** -23) + ref.abs() * 2.0 ** -23
        assert ((C.double() - ref).abs() <= bound).all(), M
    assert int(st) == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_operands_beyond_32_bit_offsets(fmt):
    """70001 x 65500 elements: 4.6e9, 2.3 GB of codes. The last rows' bytes are those of the same rows
    quantised alone, in both layouts, and a product's last rows those of a product of that part."""
    R, C, t = 70001, 65500, 129
    x = torch.randn(R, C, dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    q = operand(fmt, R, C, x)
    r0 = (R - t) // 128 * 128
    part, alone = q.rows_view(r0, R - r0), operand(fmt, R - r0, C, x[r0:].contiguous())
    assert torch.equal(q.codes[r0:], alone.codes)
    a, b = values_of(part), values_of(alone)
    assert torch.equal(a, b) and float(a.abs().max()) > 1
    v = operand(fmt, 33, C, randn(33, C, seed=3).cuda())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for A, B, rows in ((v, q, None), (q, v, slice(r0, None))):
        out = torch.empty(A.rows, B.rows, device="cuda")
        mgt.gemm_mx4(A, B, out, st)
        small = torch.empty((33, R - r0) if A is v else (R - r0, 33), device="cuda")
        mgt.gemm_mx4(v if A is v else part, part if A is v else v, small, st)
        got = out[:, r0:] if A is v else out[rows]
        ref = values_of(v) @ a.t() if A is v else a @ values_of(v).t()
        scale = float(ref.abs().max())
        # 1024 steps of at most 4 units of 2^-23 of the partial sums, which stay below 256 times a
        # result's largest value (sums of 65500 signed products against their magnitudes')
        assert float((got.double() - ref).abs().max()) <= 1024 * 4 * 2.0 ** -23 * 256 * scale
        assert float((small.double() - ref).abs().max()) <= 1024 * 4 * 2.0 ** -23 * 256 * scale
    del q, part
    qt = operand(fmt, C, R)
    mgt.mx4_quantize(x, None, qt)
    last = operand(fmt, 128, R)
    mgt.mx4_quantize(x[:, C // 128 * 128 - 128:C // 128 * 128].contiguous(), None, last)
    c0 = C // 128 * 128 - 128
    assert torch.equal(qt.codes[c0:c0 + 128], last.codes)
    assert torch.equal(values_of(qt.rows_view(c0, 128)), values_of(last))
    assert int(st) == 0


def test_quantize_with_a_factor_that_is_no_power_of_two():
    """A kept scale from elsewhere: x / (f s) is then rounded twice, each by at most 2^-24, so only
    elements within 2^-22 of a border may go to the other side."""
    x, f = randn(64, 512, seed=5).cuda(), float(np.float32(0.0137))
    q = operand("nvfp4", 64, 512, x, f)
    y = values_of(q).cpu().numpy()
    lo, hi = (mx4.quantize(np64(x) * (1 + e), "nvfp4", f) for e in (-2.0 ** -22, 2.0 ** -22))
    sure = (lo[0] == hi[0])[:, :512] & np.repeat(lo[1] == hi[1], 16, 1)[:, :512]
    assert sure.mean() > 0.999
    ref = mx4.values(np64(x), "nvfp4", f)
    assert (np.abs(y - ref)[sure] <= 2.0 ** -22 * np.abs(ref)[sure]).all()


@pytest.mark.parametrize("M", [5, 300])
def test_factors_whose_product_leaves_fp32(M):
    """f_a f_b = 2^-150 is no fp32 number, the results (about 2^-121) are; with f_a f_b = 2^140 a
    sum of zeros stays zero. Of positive sums every partial one is below the result: 32 steps, at
    most 4 units of 2^-23 each; u rounds to bf16."""
    N, K, st = 130, 2048, torch.zeros(1, dtype=torch.int32, device="cuda")
    bar = 32 * 4 * 2.0 ** -23
    for fa, fb in ((2.0 ** -100, 2.0 ** -50), (2.0 ** 70, 2.0 ** 70)):
        x, w = randn(M, K, seed=1).abs() * 512, randn(512, K, seed=2).abs() * 512
        x[M // 2] = 0
        A, W = (operand("nvfp4", t.shape[0], K, (t * f).cuda(), f) for t, f in ((x, fa), (w, fb)))
        C, u = torch.empty(M, N, device="cuda"), torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
        mgt.gemm_mx4(A, W.rows_view(0, N), C, st)
        a = operand("nvfp4", M, N)
        mgt.gemm_mx4_gated(A, W, a, st, u=u)
        gate, up = (values_of(A).double() @ values_of(W.rows_view(r, N)).double().T for r in (0, 256))
        assert (C[M // 2] == 0).all() and (u[M // 2] == 0).all()
        assert (values_of(a)[M // 2] == 0).all()
        if fa > 1:
            rest = torch.arange(M, device="cuda") != M // 2
            assert torch.isinf(C[rest]).all() and torch.isinf(u[rest]).all()
        else:
            assert ((C.double() - gate).abs() <= bar * gate).all()
            both = torch.cat([gate, up], 1)
            assert ((u.double() - both).abs() <= (2.0 ** -8 + 2 * bar) * both).all()
    assert int(st) == 0


def test_dequantised_zeros_of_a_block_beyond_fp32():
    """448 f = 2^133.8 is no fp32 number; 0 * 448 f and 0.5 * 2^-9 f are."""
    q = operand("nvfp4", 3, 64, f=2.0 ** 125, fill=0)
    q.scales.fill_(0x7E)
    for t in TYPES.values():
        y = torch.empty(3, 64, dtype=t, device="cuda")
        mgt.mx4_dequantize(q, y)
        assert (y == 0).all()
    q.codes.fill_(0x11)
    q.scales.fill_(1)
    y = torch.empty(3, 64, device="cuda")
    mgt.mx4_dequantize(q, y)
    assert (y == 2.0 ** 115).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_product_carries_infinities_and_nans(fmt):
    """A block that cannot be scaled makes the sums that it enters NaN, and no others."""
    x, w = randn(40, 300, seed=1), randn(200, 300, seed=2)
    x[3, 7], w[150, 299] = float("inf"), float("nan")
    A, B = operand(fmt, 40, 300, x.cuda()), operand(fmt, 200, 300, w.cuda())
    C = torch.zeros(40, 200, device="cuda")
    mgt.gemm_mx4(A, B, C, torch.zeros(1, dtype=torch.int32, device="cuda"))
    want = np.zeros((40, 200), bool)
    want[3], want[:, 150] = True, True
    assert np.array_equal(np.isnan(np64(C)), want) and np.isfinite(np64(C))[~want].all()


@pytest.mark.parametrize("fmt", FMTS)
def test_parts_of_wider_operands(fmt):
    """A product over columns 128 .. 427 and rows 256 .. of one operand, quantised there in place."""
    q, w = operand(fmt, 400, 640, fill=0xFF), operand(fmt, 500, 300)
    x, y = randn(144, 300, seed=4), randn(500, 300, seed=5)
    part = q.part(256, 144, 128, 300)
    mgt.mx4_quantize(x.cuda(), part)
    mgt.mx4_quantize(y.cuda(), w)
    untouched = q.codes.clone()
    untouched[256:400, 64:64 + 192] = 255
    assert (untouched == 255).all()
    C, st = torch.empty(144, 500, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    mgt.gemm_mx4(part, w, C, st)
    a, b = mx4.values(np64(x), fmt), mx4.values(np64(y), fmt)
    assert (np.abs(np64(C) - a @ b.T) <= product_bound(a, b, False, a @ b.T)).all()
    D = torch.empty(500, 144, device="cuda")
    mgt.gemm_mx4(w, part, D, st)
    assert (np.abs(np64(D) - b @ a.T) <= product_bound(b, a, False, b @ a.T)).all()
    back = torch.empty(144, 300, device="cuda")
    mgt.mx4_dequantize(part, back)
    assert np.array_equal(np64(back), a)


def check_near(q, exact, f, eps, most=0.02):
    """q holds exact (float64), each entry computed within eps of its size (and of its block's) before the
    rounding to 4 bits: where exact (1 - eps) and exact (1 + eps) round alike, q must agree."""
    y = torch.empty(q.rows, q.cols, device="cuda")
    mgt.mx4_dequantize(q, y)
    got = np64(y)
    lo, hi = mx4.values(exact * (1 - eps), q.fmt, f), mx4.values(exact * (1 + eps), q.fmt, f)
    sure = lo == hi
    assert sure.mean() > 1 - most, sure.mean()
    assert np.array_equal(got[sure], lo[sure]), np.abs(got - lo)[sure].max()
    # the others: no further than the scale's rounding (2^-4) and one step (half of the value, or s / 2)
    s = np.abs(exact).max() + 1e-30
    assert (np.abs(got - exact)[~sure] <= 0.6 * np.abs(exact)[~sure] + 0.3 * s).all()


def gated_weights(fmt, F, K, f, seed):
    """Gate and up rows in one operand, rows and scales between them NaN where the format has one."""
    P = (F + 127) // 128 * 128
    w = randn(2 * F, K, seed=seed, scale=0.06)
    q = operand(fmt, 2 * P, K, f=f, fill=0xFF)
    mgt.mx4_quantize(w[:F].cuda(), q.rows_view(0, F))
    mgt.mx4_quantize(w[F:].cuda(), q.rows_view(P, F))
    return q, mx4.values(np64(w[:F]), fmt, f), mx4.values(np64(w[F:]), fmt, f)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,F,K", [(1, 1, 16), (1, 300, 512), (5, 128, 100), (33, 257, 640), (90, 130, 600), (96, 260, 512),
                                   (112, 128, 1024), (128, 64, 256),
                                   (200, 500, 333), (300, 1300, 512), (700, 384, 128)])
def test_gated_product(M, F, K, fmt, act):
    x = randn(M, K, seed=M)
    fx, fw, fa = (1.0,) * 3 if fmt == "mxfp4" else (2.0 ** -8, 2.0 ** -10, 2.0 ** -9)
    X = operand(fmt, M, K, x.cuda(), fx, 0xFF)
    W, wg, wu = gated_weights(fmt, F, K, fw, seed=F)
    a = mx4.values(np64(x), fmt, fx)
    g, u = a @ wg.T, a @ wu.T
    h = mx4.act(g, act)[0] * u
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = []
    for keep in (True, False):
        q = operand(fmt, M, F, f=fa)
        ub = torch.full((M, 2 * F + 5), 3.0, dtype=torch.bfloat16, device="cuda") if keep else None
        mgt.gemm_mx4_gated(X, W, q, st, act=act, u=ub[:, :2 * F] if keep else None)
        assert int(st) == 0
        # columns behind the last are zeros, of scale zero
        P = (F + 127) // 128 * 128
        y = torch.empty(M, P, device="cuda")
        mgt.mx4_dequantize(mgt.Mx4(fmt, M, P, codes=q.codes, scales=q.scales, factor=q.factor), y)
        assert (y[:, F:] == 0).all()
        # gate and up are within the product's bound; act and the product add a few 2^-23, and the
        # activation's slope relative to its value is below 1 + |g|: 64 * 2^-23 covers |g| < 16 and
        # sums that cancel to a quarter of their terms' root mean square
        check_near(q, h, fa, 2.0 ** -15)
        outs.append((q.codes.clone(), q.scales.clone()))
        if keep:
            ref = np.concatenate([g, u], 1)
            bound = product_bound(a, np.concatenate([wg, wu]), True, ref)
            assert (np.abs(np64(ub[:, :2 * F]) - ref) <= bound).all()
            assert (ub[:, 2 * F:] == 3).all()
    assert all(torch.equal(v, w) for v, w in zip(*outs))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,F", [(1, 1), (3, 200), (64, 128), (130, 515), (257, 300)])
def test_gated_backward(M, F, fmt, act):
    da = randn(M, F + 3, seed=M, scale=1e-3, dtype=torch.bfloat16)
    u = randn(M, 2 * F + 1, seed=F, scale=2.0, dtype=torch.bfloat16)
    P = (F + 127) // 128 * 128
    fd, fa = (1.0, 1.0) if fmt == "mxfp4" else (2.0 ** -18, 2.0 ** -8)
    dad, ud = da.cuda()[:, :F], u.cuda()[:, :2 * F]
    dg, dup, a = mx4.gated_bwd(np64(dad), np64(ud[:, :F]), np64(ud[:, F:]), act)
    full = [operand(fmt, M, 2 * P, f=fd), operand(fmt, 2 * P, M, f=fd), operand(fmt, F, M, f=fa)]
    mgt.mx4_gated_bwd(dad, ud, *full, act=act)
    du, dut, at = full
    # two or three fp32 products and an activation within a few units of 2^-23; where act' crosses zero
    # it is the difference of terms of size 1
    eps = 2.0 ** -17
    check_near(du.part(0, M, 0, F), dg, fd, eps)
    check_near(du.part(0, M, P, F), dup, fd, eps)
    check_near(dut.rows_view(0, F), dg.T, fd, eps)
    check_near(dut.rows_view(P, F), dup.T, fd, eps)
    check_near(at, a.T, fa, eps)
    pad = torch.empty(M, 2 * P, device="cuda")
    mgt.mx4_dequantize(du, pad)
    assert (pad[:, F:P] == 0).all() and (pad[:, P + F:] == 0).all()
    for k in range(3):  # one output at a time gives the same bytes
        q = operand(fmt, full[k].rows, full[k].cols, f=(fd, fd, fa)[k])
        mgt.mx4_gated_bwd(dad, ud, *[q if i == k else None for i in range(3)], act=act)
        assert torch.equal(q.codes, full[k].codes) and torch.equal(q.scales, full[k].scales)


def rel(got, ref):
    return float(np.linalg.norm(np64(got) - ref) / np.linalg.norm(ref))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,H,F", [(1, 256, 384), (96, 256, 700), (300, 512, 1000)])
def test_gated_block_forward_and_backward(M, H, F, fmt):
    """A training step through the block, every tensor in 4 bits where a product reads it. bf16
    results are within 2^-9 root mean square of the exact ones (at most 2^-8 each), and the 4-bit
    decisions of `a` and of the gradients that fp32 takes otherwise than float64 (fewer than one in
    10^4, each off by at most half of its value) add less than 2^-8 to that."""
    P = (F + 127) // 128 * 128
    x, dy = randn(M, H, seed=1).bfloat16().cuda(), randn(M, H, seed=2, scale=1e-2).bfloat16().cuda()
    w1, w2 = randn(2 * F, H, seed=3, scale=0.06).cuda(), randn(H, F, seed=4, scale=0.05).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fx, fw, fa, fd = (1.0,) * 4 if fmt == "mxfp4" else (2.0 ** -8, 2.0 ** -11, 2.0 ** -8, 2.0 ** -14)

    def op(r, c, f):
        return operand(fmt, r, c, f=f, fill=0xFF)

    def pair(r, c, f):
        a, b = op(r, c, f), op(c, r, f)
        return a, mgt.Mx4(fmt, c, r, codes=b.codes, scales=b.scales, factor=a.factor)

    xq, xt = pair(M, H, fx)
    mgt.mx4_quantize(x, xq, xt)
    w1q, w1t = op(2 * P, H, fw), op(H, 2 * P, fw)
    for k in (0, 1):
        rows, cols = w1q.rows_view(k * P, F), w1t.part(0, H, k * P, F)
        if fmt == "nvfp4":
            cols.factor = rows.factor
            cols._c.factor = rows._c.factor
        mgt.mx4_quantize(w1[k * F:(k + 1) * F], rows, cols)
    w2q, w2t = pair(H, F, fw)
    mgt.mx4_quantize(w2, w2q, w2t)
    a, u = op(M, F, fa), torch.empty(M, 2 * F, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    mgt.gemm_mx4_gated(xq, w1q, a, st, u=u)
    mgt.gemm_mx4(a, w2q, y, st)
    dyq, dyt = pair(M, H, fd)
    mgt.mx4_quantize(dy, dyq, dyt)
    da = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    mgt.gemm_mx4(dyq, w2t, da, st)
    du, dut, at = op(M, 2 * P, fd), op(2 * P, M, fd), op(F, M, fa)
    mgt.mx4_gated_bwd(da, u, du, dut, at)
    dx = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    dwg, dwu = (torch.empty(F, H, device="cuda") for _ in range(2))
    dw2 = torch.empty(H, F, device="cuda")
    mgt.gemm_mx4(du, w1t, dx, st)
    mgt.gemm_mx4(dut.rows_view(0, F), xt, dwg, st)
    mgt.gemm_mx4(dut.rows_view(P, F), xt, dwu, st)
    mgt.gemm_mx4(dyt, at, dw2, st)
    assert int(st) == 0

    v = lambda t, f: mx4.values(t if isinstance(t, np.ndarray) else np64(t), fmt, f)  # noqa: E731
    xv, wg, wu = v(x, fx), v(w1[:F], fw), v(w1[F:], fw)
    av = v(mx4.act(xv @ wg.T, "silu")[0] * (xv @ wu.T), fa)
    assert rel(y, av @ v(w2, fw).T) < 2.0 ** -8
    ug, uu = np64(u[:, :F]), np64(u[:, F:])  # what the backward reads is what the forward kept
    assert rel(u, np.concatenate([xv @ wg.T, xv @ wu.T], 1)) < 2.0 ** -8
    dav = v(dy, fd) @ v(np64(w2).T, fw).T
    assert rel(da, dav) < 2.0 ** -8
    dg, dup, ar = mx4.gated_bwd(np64(da), ug, uu, "silu")
    xtv = v(np64(x).T, fx)
    ref = v(dg, fd) @ v(np64(w1[:F]).T, fw).T + v(dup, fd) @ v(np64(w1[F:]).T, fw).T
    assert rel(dx, ref) < 2.0 ** -8
    assert rel(dwg, v(dg.T, fd) @ xtv.T) < 2.0 ** -8
    assert rel(dwu, v(dup.T, fd) @ xtv.T) < 2.0 ** -8
    assert rel(dw2, v(np64(dy).T, fd) @ v(ar.T, fa).T) < 2.0 ** -8


@pytest.mark.parametrize("fmt", FMTS)
def test_streams_and_graphs_give_the_same_bytes(fmt):
    """Eager on the current stream, on another one, on two at once, and replayed from a graph over
    new inputs: the same bytes each time."""
    M, F, K = 70, 600, 1024
    x = [randn(M, K, seed=s).bfloat16().cuda() for s in (1, 2)]
    W, _, _ = gated_weights(fmt, F, K, 2.0 ** -10 if fmt == "nvfp4" else 1.0, seed=3)
    w2 = operand(fmt, K, F, randn(K, F, seed=4, scale=0.05).cuda(), 2.0 ** -10)

    class Run:
        def __init__(self):
            self.x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
            self.q, self.a = operand(fmt, M, K), operand(fmt, M, F, f=2.0 ** -8)
            self.y = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
            self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

        def go(self, stream=None):
            if fmt == "nvfp4":
                mgt.mx4_tensor_factor(self.x, self.q.factor, stream)
            mgt.mx4_quantize(self.x, self.q, stream=stream)
            mgt.gemm_mx4_gated(self.q, W, self.a, self.st, stream=stream)
            mgt.gemm_mx4(self.a, w2, self.y, self.st, stream=stream)

    want = []
    for xi in x:
        r = Run()
        r.x.copy_(xi)
        r.go()
        want.append(r.y.clone())
    runs, streams = [Run(), Run()], [torch.cuda.Stream(), torch.cuda.Stream()]
    for r, xi in zip(runs, x):
        r.x.copy_(xi)
    torch.cuda.synchronize()
    for _ in range(8):
        for r, s in zip(runs, streams):
            r.go(s)
    torch.cuda.synchronize()
    assert all(torch.equal(r.y, w) for r, w in zip(runs, want))
    graphs = []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.go()
        graphs.append(g)
    for turn in range(4):
        for k, r in enumerate(runs):
            r.x.copy_(x[(k + turn) % 2])
            r.y.fill_(9)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(r.y, want[(k + turn) % 2]) for k, r in enumerate(runs))
    assert all(int(r.st) == 0 for r in runs)


@pytest.mark.parametrize("M", [1, 40, 600])
@pytest.mark.parametrize("fmt", FMTS)
def test_chains_over_the_same_buffers(fmt, M):
    """Each call rewrites what the one before has read, or reads what it wrote, with nothing between
    them on the stream: the same bytes as with a synchronisation after every call."""
    F, K, st = 700, 1024, torch.zeros(1, dtype=torch.int32, device="cuda")
    W, _, _ = gated_weights(fmt, F, K, 2.0 ** -10 if fmt == "nvfp4" else 1.0, seed=1)
    w2 = operand(fmt, K, F, randn(K, F, seed=2, scale=0.1).cuda(), 2.0 ** -10)
    du_w = operand(fmt, K, 2 * 768, randn(K, 2 * 768, seed=3, scale=0.05).cuda(), 2.0 ** -10)

    def chain(wait):
        x = randn(M, K, seed=4).bfloat16().cuda()
        q, a, u = operand(fmt, M, K), operand(fmt, M, F, f=2.0 ** -8), torch.empty(M, 2 * F, dtype=torch.bfloat16, device="cuda")
        da, du, at = torch.empty(M, F, dtype=torch.bfloat16, device="cuda"), operand(fmt, M, 2 * 768), operand(fmt, F, M)
        qt = mgt.Mx4(fmt, K, M, factor=q.factor)
        for _ in range(6):
            for call in ([lambda: mgt.mx4_tensor_factor(x, q.factor)] if fmt == "nvfp4" else []) + [
                    lambda: mgt.mx4_quantize(x, q, qt),
                    lambda: mgt.gemm_mx4_gated(q, W, a, st, u=u),
                    lambda: mgt.mx4_dequantize(a, da),
                    lambda: mgt.gemm_mx4(a, w2, x, st),
                    lambda: mgt.mx4_gated_bwd(da, u, du, None, at),
                    lambda: mgt.gemm_mx4(du, du_w, x, st),
                    lambda: mgt.mx4_dequantize(q, x)]:
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [t.clone() for t in (x, u, da, q.codes, a.codes, du.codes, at.codes)]

    want = chain(True)
    for _ in range(5):
        assert all(torch.equal(g, w) for g, w in zip(chain(False), want))
    assert int(st) == 0


@pytest.mark.parametrize("rows,cols", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 8), (2, 2 ** 31 - 4), (2 ** 31 - 1, 1)])
def test_factor_of_the_longest_rows_and_columns(rows, cols):
    """Sizes at the end of int32, whose groups of eight columns end behind it; the largest element is
    the last one, then the first."""
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(2, device="cuda")
    for at, v in ((-1, 5000.0), (0, -9000.0)):
        x.view(-1)[at] = v
        mgt.mx4_tensor_factor(x, f)
        amax, want = mx4.tensor_factor(np.array([[float(x.view(-1)[at])]]))
        assert f.tolist() == [amax, want]


TAIL = (-84.0, -87.0, -88.0, -89.0, -90.0, -91.0, -91.5, -92.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_silu_far_in_its_negative_tail(fmt):
    """silu(-88) = -88 e^-88 is a normal fp32 number, e^-88 is not. Blocks of one gate each. At -92,
    e^z = 2^-132.7 has 16 bits left: two units for the exponential, half a one for the product with the
    reciprocal make 2.5 * 2^-16.3 of the value, below 2^-14."""
    M, F, up, eps = 32 * len(TAIL), 160, 2.0 ** 100, 2.0 ** -14
    g = torch.tensor(TAIL).repeat_interleave(32).view(-1, 1).expand(M, F)
    uv, da = randn(M, F, seed=1, scale=up).bfloat16(), randn(M, F, seed=2, scale=2.0 ** 20).bfloat16()
    u = torch.cat([g.bfloat16(), uv], 1).contiguous().cuda()
    dg, dup, a = mx4.gated_bwd(np64(da), np64(g), np64(uv), "silu")
    for name, row, want, f in (("at", 0, a.T, 2.0 ** -24), ("dut", 0, dg.T, 2.0 ** -2), ("dut", 256, dup.T, 2.0 ** -104)):
        f = f if fmt == "nvfp4" else 1.0  # (of dgate and dup, 2^100 apart, the one that it is for counts)
        q = operand(fmt, F if name == "at" else 512, M, f=f)
        mgt.mx4_gated_bwd(da.cuda(), u, **{name: q}, act="silu")
        check_near(q.rows_view(row, F), want, f, eps, most=0.01)


@pytest.mark.parametrize("M", [8, 320])
@pytest.mark.parametrize("fmt", FMTS)
def test_gated_product_far_in_the_negative_tail(fmt, M):
    """The same through the products' epilogues, on gates that are sums of a few exact products."""
    F, K, up = 40, 256, 2.0 ** 100 if fmt == "mxfp4" else 2.0 ** 10
    x, w = torch.zeros(M, K), torch.zeros(256, K)
    for m in range(M):  # numbers 6 * 2^k alone in their blocks, which both formats hold
        x[m, 0], x[m, 32], x[m, 64], x[m, 96] = -96, -12, -6, (0, -0.75, -1.5, -3, -6)[m % 5]
        x[m, 128] = 0.75 * (1 + m % 2)
    w[:F, :128] = 0.75
    w[128:128 + F, 128] = up * 1.5 * 0.5 ** (torch.arange(F) % 6)
    X, W = operand(fmt, M, K, x.cuda()), operand(fmt, 256, K, w.cuda())
    gate, upv = (np64(values_of(X) @ values_of(W.rows_view(r, F)).T) for r in (0, 128))
    assert (np.unique(gate) == [-90, -87.75, -86.625, -86.0625, -85.5]).all()
    f = 1.0 if fmt == "mxfp4" else 2.0 ** -117
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = operand(fmt, M, F, f=f)
    mgt.gemm_mx4_gated(X, W, a, st, act="silu")
    check_near(a, mx4.act(gate, "silu")[0] * upv, f, 2.0 ** -14, most=0.01)
    assert int(st) == 0


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", FMTS)
def test_gated_backward_at_huge_gates(fmt, act):
    """Where act' is 0 or 1 to every bit the gradients are 0 or da * up, however large the gate: blocks of
    one gate each. Nearer, at +-10, three fp32 products and an activation: 2^-17, as above."""
    gates = [s * g for g in (10.0, 1e4, 1e13, 1.5e14, 1e19, 1e30) for s in (1, -1)]
    M, F = 32 * len(gates), 70
    g = torch.tensor(gates).repeat_interleave(32).view(-1, 1).expand(M, F).bfloat16()
    uv, da = randn(M, F, seed=1, scale=2.0 ** -40).bfloat16(), randn(M, F, seed=2).bfloat16()
    u = torch.cat([g, uv], 1).contiguous().cuda()
    with np.errstate(over="ignore"):
        dg, dup, a = mx4.gated_bwd(np64(da), np64(g), np64(uv), act)
    fd, fa = (1.0, 1.0) if fmt == "mxfp4" else (2.0 ** -50, 2.0 ** 30)
    du, dut, at = operand(fmt, M, 256, f=fd), operand(fmt, 256, M, f=fd), operand(fmt, F, M, f=fa)
    mgt.mx4_gated_bwd(da.cuda(), u, du, dut, at, act=act)
    for q, want, f in ((du.part(0, M, 0, F), dg, fd), (du.part(0, M, 128, F), dup, fd), (dut.rows_view(0, F), dg.T, fd),
                       (dut.rows_view(128, F), dup.T, fd), (at, a.T, fa)):
        assert torch.isfinite(values_of(q)).all()
        check_near(q, want, f, 2.0 ** -17)


@pytest.mark.parametrize("act,tail", [("gelu", (-11.0, -12.5, -12.875)), ("gelu_tanh", (-9.5, -10.0, -10.0625))])
def test_gelu_far_in_its_negative_tail(act, tail):
    """Both forms as far as their values are normal fp32 numbers (2^-125 at the last gates). The exponent is 88
    there, of three roundings, 2^-16 of the value in all, and what multiplies z has 19 bits left or more:
    2^-14 covers both."""
    M, F, up, eps = 32 * len(tail), 160, 2.0 ** 100, 2.0 ** -14
    g = torch.tensor(tail).repeat_interleave(32).view(-1, 1).expand(M, F)
    uv, da = randn(M, F, seed=1, scale=up).bfloat16(), randn(M, F, seed=2, scale=2.0 ** 20).bfloat16()
    u = torch.cat([g.bfloat16(), uv], 1).contiguous().cuda()
    dg, dup, a = mx4.gated_bwd(np64(da), np64(g), np64(uv), act)
    for name, row, want in (("at", 0, a), ("dut", 0, dg), ("dut", 256, dup)):
        q = operand("mxfp4", F if name == "at" else 512, M)
        mgt.mx4_gated_bwd(da.cuda(), u, **{name: q}, act=act)
        check_near(q.rows_view(row, F), want.T, 1.0, eps, most=0.01)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", FMTS)
def test_gated_backward_carries_nan_gates(fmt, act):
    """A NaN gate makes its block of every result NaN, and no other."""
    M, F = 128, 192
    da, u = randn(M, F, seed=1).bfloat16(), randn(M, 2 * F, seed=2).bfloat16()
    u[70, 100] = float("nan")
    ops = operand(fmt, M, 512), operand(fmt, 512, M), operand(fmt, F, M)
    mgt.mx4_gated_bwd(da.cuda(), u.cuda(), *ops, act=act)
    n = mx4.BLOCK[fmt]
    r, c = slice(70 // n * n, 70 // n * n + n), slice(100 // n * n, 100 // n * n + n)
    for k, q in enumerate((ops[0].part(0, M, 0, F), ops[0].part(0, M, 256, F), ops[1].rows_view(0, F), ops[1].rows_view(256, F),
                           ops[2])):
        want = np.zeros((M, F), bool)
        if k < 2:
            want[70, c] = True
        else:
            want[r, 100] = True
        assert np.array_equal(np.isnan(np64(values_of(q))), want if k < 2 else want.T), k


@pytest.mark.parametrize("fd,ft", [(2.0 ** 90, 2.0 ** -60), (2.0 ** -60, 2.0 ** 90), (2.0 ** 60, 2.0 ** -120),
                                   (2.0 ** -120, 2.0 ** 60), (2.0 ** -10, 2.0 ** -130), (2.0 ** -149, 2.0 ** 120),
                                   (2.0 ** -20, 2.0 ** -14)])
def test_gated_backward_with_factors_far_apart(fd, ft):
    """du and dut each have a factor of their own: each is what it is alone, and saturates or vanishes with
    the right sign where its factor is far off."""
    M, F, act, eps = 70, 150, "silu", 2.0 ** -17
    size = 2.0 ** 8 * max(fd, ft) if max(fd, ft) < 2.0 ** 100 else 2.0 ** 112
    da, u = randn(M, F, seed=1, scale=size).bfloat16(), randn(M, 2 * F, seed=2).bfloat16()
    dad, ud = da.cuda(), u.cuda()
    dg, dup, a = mx4.gated_bwd(np64(da), np64(u[:, :F]), np64(u[:, F:]), act)
    ops = lambda: (operand("nvfp4", M, 512, f=fd), operand("nvfp4", 512, M, f=ft))  # noqa: E731
    (du, dut), (d1, t1), (d2, t2) = ops(), ops(), ops()
    at = operand("nvfp4", F, M, f=2.0 ** -8)
    mgt.mx4_gated_bwd(dad, ud, du, dut, at, act=act)
    mgt.mx4_gated_bwd(dad, ud, du=d1, act=act)
    mgt.mx4_gated_bwd(dad, ud, dut=t1, act=act)
    mgt.mx4_gated_bwd(dad, ud, d2, t2, act=act)
    for q, others, f in ((du, (d1, d2), fd), (dut, (t1, t2), ft)):
        for o in others:
            assert torch.equal(q.codes, o.codes) and torch.equal(q.scales, o.scales)
        for row, want in ((0, dg), (256, dup)):
            part = q.part(0, M, row, F) if q is du else q.rows_view(row, F)
            check_near(part, want if q is du else want.T, f, eps)
    check_near(at, a.T, 2.0 ** -8, eps)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("f", [2.0 ** -149, 2.0 ** -140, 2.0 ** -128, 2.0 ** -127, 2.0 ** -110])
def test_factors_below_the_normal_numbers(f, dtype):
    """A kept factor whose reciprocal is no fp32 number: blocks of zeros stay zeros, small values are
    scaled by it exactly, others saturate."""
    x = randn(70, 200, seed=3, dtype=TYPES[dtype])
    x[:32] *= 2.0 ** -133 if f < 2.0 ** -128 else 2.0 ** -112
    x[5, :64], x[60, :64], x[66:] = 0, 0, 0
    x[8, 3], x[61, 190] = float("inf"), float("nan")
    xd = x.cuda()
    q, t = operand("nvfp4", 70, 200, f=f), operand("nvfp4", 200, 70, f=f)
    t.factor = q.factor
    mgt.mx4_quantize(xd, q, t)
    check_bytes(q, np64(xd), f)
    check_bytes(t, np64(xd).T, f)
    for one in (q, t):
        z = np64(xd) if one is q else np64(xd).T
        for alone in (dict(q=one), dict(qt=one)):
            src = xd if (one is q) == ("q" in alone) else xd.t().contiguous()
            one.codes.fill_(0xCB)
            one.scales.fill_(0xCB)
            mgt.mx4_quantize(src, **alone)
            check_bytes(one, z, f)


@pytest.mark.parametrize("M", [6, 300])
@pytest.mark.parametrize("f", [2.0 ** -149, 2.0 ** -130, 2.0 ** -110])
def test_gated_product_with_a_tiny_factor(f, M):
    """Its result's blocks are zeros where gate or up is, and vanish, fit or saturate elsewhere. The product
    act(gate) * up is subnormal, off by half of 2^-149. The smallest blocks are near 2^-135. With f = 2^-130
    their scale is 2^-8 and the first border between elements 2^-2 of it, 2^-140: half a unit is 2^-10 of
    that. With f = 2^-149 all scales are 448 and the first border is 112 units: half a unit is 2^-7.8 of it."""
    F, K, fx, fw = 150, 128, 2.0 ** -70, 2.0 ** -12
    x, w = randn(M, K, seed=1, scale=2.0 ** -60), randn(512, K, seed=2, scale=2.0 ** -4)
    x[1::3] = 0
    x[2::3] *= 2.0 ** -6
    w[256:] *= 2.0 ** -2
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    X, W = operand("nvfp4", M, K, x.cuda(), fx), operand("nvfp4", 512, K, w.cuda(), fw)
    gate, up = (np64(values_of(X) @ values_of(W.rows_view(r, F)).T) for r in (0, 256))
    a = operand("nvfp4", M, F, f=f)
    mgt.gemm_mx4_gated(X, W, a, st)
    assert (values_of(a)[1::3] == 0).all() and int(st) == 0
    check_near(a, mx4.act(gate, "silu")[0] * up, f, 2.0 ** -7 if f == 2.0 ** -149 else 2.0 ** -9, most=0.2)


def levels(rows, cols, seed, scale=1.0):
    """Random elements times a power of two; every block holds a 6, so that its scale is that power."""
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.tensor(mx4.LEVELS)[torch.randint(8, (rows, cols), generator=g)]
    x[:, ::16] = 6
    x = x * (2.0 * torch.randint(2, (rows, cols), generator=g) - 1)
    return (x * scale).float()


@pytest.mark.parametrize("M", [1, 15, 16, 17, 31, 32, 47, 48, 49, 63, 64, 65, 80])
@pytest.mark.parametrize("fmt", FMTS)
def test_gated_product_at_every_token_tile(fmt, M):
    """Every tile of the few-row kernel's gated form and the first row counts of the other one, sums split
    over eight CTAs. All sums are multiples of 2^-9 below 2^12, so any order gives them exactly: u is
    their rounding, and `a` is off by the activation's 2^-21 + |z| 2^-24 (|z| < 32) and one product."""
    F, K = 300, 2200
    x, w = levels(M, K, M), levels(768, K, 1000 + M, 2.0 ** -7)
    X, W = operand(fmt, M, K, x.cuda(), fill=0xFF), operand(fmt, 768, K, w.cuda())
    assert torch.equal(values_of(X).float(), x.cuda()) and torch.equal(values_of(W).float(), w.cuda())
    gate, up = (x.double() @ w[r:r + F].double().T for r in (0, 384))
    assert gate.abs().max() < 32
    f = 1.0 if fmt == "mxfp4" else 2.0 ** -4
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for pad in (0, 3):  # aligned rows of u and others
        u = torch.full((M + 1, 2 * F + pad), 3.0, dtype=torch.bfloat16, device="cuda")
        a = operand(fmt, M, F, f=f)
        mgt.gemm_mx4_gated(X, W, a, st, u=u[:M, :2 * F])
        assert torch.equal(u[:M, :2 * F].cpu(), torch.cat([gate, up], 1).bfloat16())
        assert (u[M] == 3).all() and (u[:, 2 * F:] == 3).all()
        check_near(a, mx4.act(gate.numpy(), "silu")[0] * up.numpy(), f, 2.0 ** -18, most=0.001)
    assert int(st) == 0


def decoded(q, r0, r1):
    """Rows r0 .. r1 - 1 (r0 a multiple of 128) of an operand of factor 1, by the layout's definition, float64."""
    n, code = mx4.BLOCK[q.fmt], q.codes[r0:r1]
    table = torch.tensor([*mx4.LEVELS, *-mx4.LEVELS], device="cuda")
    v = torch.stack([code & 15, code >> 4], 2).view(r1 - r0, -1)
    tiles = q.scales.view(-1, q.ld // (4 * n), 32, 4, 4)[r0 // 128:(r1 + 127) // 128]
    byte = tiles.permute(0, 3, 2, 1, 4).reshape(-1, q.ld // n)[:r1 - r0].double()
    s = 2.0 ** (byte - 127) if q.fmt == "mxfp4" else 2.0 ** ((byte - 0x38) / 8)  # (powers of two only)
    return (table[v.int()].view(r1 - r0, -1, n) * s.unsqueeze(2)).view(r1 - r0, -1)[:, :q.cols]


@pytest.mark.parametrize("fmt", FMTS)
def test_products_beyond_32_bit_offsets_to_the_bit(fmt):
    """70144 x 65500 elements (2.3 GB of codes) as either operand and as a gated block's weights, every result
    against float64. Elements are random codes, scales 1 or 2: products are multiples of 1/4 up to
    144, sums of them far below 2^22, so that fp32 adds them exactly in any order."""
    F, C, M = 35000, 65500, 300
    P = (F + 127) // 128 * 128
    gen = torch.Generator("cuda").manual_seed(11)

    def filled(rows):
        q = operand(fmt, rows, C)
        q.codes.random_(0, 256, generator=gen)
        q.codes[:, C // 2:] = 0
        one, two = (127, 128) if fmt == "mxfp4" else (0x38, 0x40)
        q.scales.random_(0, 2, generator=gen).mul_(two - one).add_(one)
        return q

    q, v = filled(2 * P), filled(M)
    ref = torch.empty(M, 2 * P, dtype=torch.float64, device="cuda")
    few = decoded(v, 0, M)
    for r0 in range(0, 2 * P, 4096):
        r1 = min(2 * P, r0 + 4096)
        ref[:, r0:r1] = few @ decoded(q, r0, r1).t()
    assert float(ref.abs().max()) < 2.0 ** 20
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for rows in (33, M):  # few rows, and tiles of 256
        V = v.rows_view(0, rows)
        out = torch.empty(rows, 2 * P, device="cuda")
        mgt.gemm_mx4(V, q, out, st)
        assert torch.equal(out.double(), ref[:rows])
        out = torch.empty(2 * P, rows, device="cuda")
        mgt.gemm_mx4(q, V, out, st)
        assert torch.equal(out.double(), ref[:rows].t())
        a, u = operand(fmt, rows, F, f=2.0 ** 10), torch.empty(rows, 2 * F, dtype=torch.bfloat16, device="cuda")
        mgt.gemm_mx4_gated(V, q, a, st, u=u)
        gate, up = ref[:rows, :F], ref[:rows, P:P + F]
        assert torch.equal(u, torch.cat([gate, up], 1).bfloat16())
        # act(gate) is gate or nothing at this size; two roundings of 2^-24 and the activation's 2^-21
        some = slice(0, None, 7)  # (every seventh row: the oracle runs on the CPU)
        check_near(operand_rows(a, some), mx4.act(np64(gate[some]), "silu")[0] * np64(up[some]),
                   1.0 if fmt == "mxfp4" else 2.0 ** 10, 2.0 ** -18, most=0.001)
    assert int(st) == 0


def operand_rows(q, rows):
    """Some rows of an operand, copied into one of their own by way of their values (exact)."""
    y = values_of(q)[rows].float()
    f = float(q.factor[1]) if q.fmt == "nvfp4" else 1.0
    c = operand(q.fmt, *y.shape, f=f)
    n = mx4.BLOCK[q.fmt]
    k = torch.arange(q.rows, device="cuda")[rows]
    c.codes.copy_(q.codes[rows])
    at = lambda r, b: ((r // 128) * (q.ld // (4 * n)) + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4  # noqa: E731
    b = torch.arange(q.ld // n, device="cuda").view(1, -1)
    to = torch.arange(len(k), device="cuda").view(-1, 1)
    c.scales[at(to, b)] = q.scales[at(k.view(-1, 1), b)]
    assert torch.equal(values_of(c).float(), y)
    return c


def check_every(q, exact, err, f=1.0):
    """Each element of q is one that a number within err (elementwise, absolute) of exact rounds to: for the
    scale of its block from the smallest or the largest such maximum, between the roundings of the
    ends."""
    got, n = np64(values_of(q)), mx4.BLOCK[q.fmt]
    low, high = np.maximum(np.abs(exact) - err, 0), np.abs(exact) + err
    fits = np.zeros(got.shape, bool)
    for end in (low, high):
        byte = mx4.quantize(end, q.fmt, f)[1].astype(np.float64)
        if q.fmt == "mxfp4":
            scale = 2.0 ** (byte - 127)
        else:
            e, m = np.floor(byte / 8), byte % 8
            scale = np.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9) * f
        scale = np.repeat(scale, n, 1)[:, :got.shape[1]]
        least, most = (mx4.LEVELS[mx4.e2m1_round(np.where(scale > 0, v / np.where(scale > 0, scale, 1), 0))] * scale
                       for v in (low, high))
        sign = np.where(np.abs(exact) > err, np.sign(exact), np.sign(got))
        fits |= (np.abs(got) >= least) & (np.abs(got) <= most) & ((got == 0) | (np.sign(got) == sign))
    assert fits.all(), np.argwhere(~fits)[:4]


def act_errors(z, act):
    """(h, dh, error of h, error of dh) of the kernels' fp32 activations, from their formulas. e: the
    relative error of sigmoid, Phi or the tanh form's sigmoid."""
    h, dh = mx4.act(z, act)
    a = np.abs(z)
    if act == "silu":  # the exponent's product, ex2.approx, rcp.approx: 2^-21 + |z| 2^-24
        s = 1 / (1 + np.exp(-z))
        e = 2.0 ** -20.5 + a * 2.0 ** -24
        # s (1 + z (1 - s)): s once for itself, once in 1 - s, and roundings of terms up to 1 + |z|
        return h, dh, np.abs(h) * e, s * ((1 + a * (1 - s)) * e + a * s * e + (1 + a) * 2.0 ** -23)
    if act == "gelu":  # arguments with 2^-23 of z^2 / 2 as error; erfcf within four units, expf two
        c, pdf = np.where(z == 0, 0.5, h / np.where(z == 0, 1, z)), np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        e = 2.0 ** -20.5 + z * z * 2.0 ** -23
        return h, dh, np.abs(h) * e, (c + a * pdf) * e
    w = 2 * np.sqrt(2 / np.pi) * a * (1 + 0.044715 * z * z)
    s, inner = 1 / (1 + np.exp(-np.sign(z) * w)), 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * z * z)
    # the exponent is off by four roundings of w + 1.4; 1 / (1 + E) moves by s (1 - s) of that
    e = 2.0 ** -21 + (w + 2) * 2.0 ** -22 * (1 - s)
    return h, dh, np.abs(h) * e, s * ((1 + a * (1 - s) * inner) * e + a * inner * (s * e + 2.0 ** -23) + 2.0 ** -23)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,F", [(130, 260), (40, 1000)])
def test_gated_backward_to_the_last_step(fmt, act, M, F):
    """Every element, the ones next to a border too: products of three bf16 numbers or two and an
    activation round twice more in fp32."""
    da, u = randn(M, F, seed=1, scale=1e-3, dtype=torch.bfloat16), randn(M, 2 * F, seed=2, scale=2.0, dtype=torch.bfloat16)
    P, d = (F + 127) // 128 * 128, np64(da)
    z, up = np64(u[:, :F]), np64(u[:, F:])
    h, dh, eh, edh = act_errors(z, act)
    fd, fa = (1.0, 1.0) if fmt == "mxfp4" else (2.0 ** -18, 2.0 ** -8)
    du, dut, at = operand(fmt, M, 2 * P, f=fd), operand(fmt, 2 * P, M, f=fd), operand(fmt, F, M, f=fa)
    mgt.mx4_gated_bwd(da.cuda(), u.cuda(), du, dut, at, act=act)
    for k, (exact, err) in enumerate(((d * up * dh, np.abs(d * up) * edh), (d * h, np.abs(d) * eh))):
        err = err + np.abs(exact) * 2.0 ** -22
        check_every(du.part(0, M, k * P, F), exact, err, fd)
        check_every(dut.rows_view(k * P, F), exact.T, err.T, fd)
    check_every(at, (h * up).T, (np.abs(up) * eh + np.abs(h * up) * 2.0 ** -22).T, fa)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [3, 48, 300])
def test_gated_product_to_the_last_step(fmt, act, M):
    """Every element of the quantised result, on gates and ups that any order of sums gives exactly."""
    F, K = 300, 600
    x, w = levels(M, K, M), levels(768, K, 1000 + M, 2.0 ** -7)
    X, W = operand(fmt, M, K, x.cuda()), operand(fmt, 768, K, w.cuda())
    gate, up = ((x.double() @ w[r:r + F].double().T).numpy() for r in (0, 384))
    f = 1.0 if fmt == "mxfp4" else 2.0 ** -5
    a, st = operand(fmt, M, F, f=f), torch.zeros(1, dtype=torch.int32, device="cuda")
    mgt.gemm_mx4_gated(X, W, a, st, act=act)
    h, _, eh, _ = act_errors(gate, act)
    check_every(a, h * up, np.abs(up) * eh + np.abs(h * up) * 2.0 ** -23, f)
    assert int(st) == 0


FIRST_CALLS = """
import threading, torch
import tensor_transformer_layer_megatron_b200 as mgt
M, K, F, fmt = 40, 1024, 300, {fmt!r}
dev = dict(device="cuda")
gen = torch.Generator("cuda").manual_seed(1)

class Run:
    def __init__(self, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.x = torch.randn(M, K, generator=g, **dev).bfloat16()
        self.w = torch.randn(768, K, generator=g, **dev) * 0.05
        self.q, self.W, self.a, self.at = (mgt.Mx4(fmt, *n) for n in ((M, K), (768, K), (M, F), (F, M)))
        self.du = mgt.Mx4(fmt, M, 768)
        self.u, self.y = torch.empty(M, 2 * F, dtype=torch.bfloat16, **dev), torch.empty(M, F, **dev)
        self.big = torch.empty(768, 768, **dev)
        self.st = torch.zeros(1, dtype=torch.int32, **dev)

    def go(self, stream=None):
        if fmt == "nvfp4":
            mgt.mx4_tensor_factor(self.x, self.q.factor, stream)
            mgt.mx4_tensor_factor(self.w, self.W.factor, stream)
        mgt.mx4_quantize(self.x, self.q, stream=stream)
        mgt.mx4_quantize(self.w, self.W, stream=stream)
        mgt.gemm_mx4_gated(self.q, self.W, self.a, self.st, u=self.u, stream=stream)
        mgt.mx4_dequantize(self.a, self.y, stream=stream)
        mgt.mx4_gated_bwd(self.y.bfloat16() if stream is None else self.u[:, :F], self.u, self.du, None, self.at, stream=stream)
        mgt.gemm_mx4(self.W, self.W, self.big, self.st, stream=stream)

    def out(self):
        return [t.clone() for t in (self.u, self.y, self.big, self.a.codes, self.du.codes, self.at.codes)]
"""


def run_python(code):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


@pytest.mark.parametrize("fmt", FMTS)
def test_first_calls_of_a_process_may_be_captured(fmt):
    """Nothing has to run eagerly before: a process whose first calls go into a graph."""
    run_python(FIRST_CALLS.format(fmt=fmt) + """
r = Run(1)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    r.go()
g.replay()
torch.cuda.synchronize()
got = r.out()
r.go()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, r.out())) and int(r.st) == 0
print("ok")
""")


@pytest.mark.parametrize("fmt", FMTS)
def test_first_calls_from_two_threads(fmt):
    """Two threads that begin at once, on a stream each."""
    run_python(FIRST_CALLS.format(fmt=fmt) + """
runs, streams = [Run(1), Run(2)], [torch.cuda.Stream() for _ in range(2)]
torch.cuda.synchronize()
errors, gate = [], threading.Barrier(2)
def work(r, s):
    try:
        gate.wait()
        for _ in range(20):
            r.go(s)
    except Exception as e:
        errors.append(e)
threads = [threading.Thread(target=work, args=a) for a in zip(runs, streams)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
got = [r.out() for r in runs]
for r, was, s in zip(runs, got, streams):
    r.go(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(was, r.out())) and int(r.st) == 0
print("ok")
""")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("f", [2.0 ** 100, 2.0 ** 117, 2.0 ** 125, 2.0 ** 127])
def test_factors_near_the_largest_numbers(f, dtype):
    """Scales of up to 2688 f in fp32's range, subnormal reciprocals: every decision as exact arithmetic's."""
    x = randn(70, 200, seed=4, dtype=TYPES[dtype])
    x *= 2.0 ** 98
    x[::2] *= 2.0 ** 25
    x[5], x[6, 7], x[8, :16] = torch.finfo(TYPES[dtype]).max, -torch.finfo(TYPES[dtype]).max, 0
    xd = x.cuda()
    q, t = operand("nvfp4", 70, 200, f=f), operand("nvfp4", 200, 70, f=f)
    t.factor = q.factor
    mgt.mx4_quantize(xd, q, t)
    check_bytes(q, np64(xd), f)
    check_bytes(t, np64(xd).T, f)
