"""What the 4-bit operators refuse, before anything is launched (CPU: no GPU is touched)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import tensor_transformer_layer_megatron_b200 as mgt
from tensor_transformer_layer_megatron_b200.mx4 import _Mx4Operand

OK, EINVAL, EUNSUPPORTED = 0, 1, 2
P = 0x100000  # an address that is never read


@pytest.fixture(scope="module")
def lib():
    return mgt.load_library()


def operand(rows=4, cols=100, ld=None, fmt=0, codes=P, scales=P, factor=P):
    return _Mx4Operand(fmt, rows, cols, (cols + 127) // 128 * 128 if ld is None else ld, codes,
                       scales, factor)


def ref(q):
    return None if q is None else ctypes.addressof(q)


BAD = [  # (changes to a good operand, status)
    (dict(codes=0), EINVAL), (dict(scales=0), EINVAL), (dict(rows=0), EINVAL),
    (dict(cols=0), EINVAL), (dict(cols=-5, ld=128), EINVAL), (dict(ld=100), EINVAL),
    (dict(ld=0), EINVAL), (dict(cols=129, ld=128), EINVAL), (dict(fmt=2), EUNSUPPORTED),
    (dict(fmt=-1), EUNSUPPORTED), (dict(fmt=1, factor=0), EINVAL), (dict(codes=P + 8), EUNSUPPORTED),
    (dict(scales=P + 4), EUNSUPPORTED), (dict(factor=P + 2), EUNSUPPORTED),
    (dict(rows=(1 << 30) + 1), EUNSUPPORTED),
]


def test_sizes(lib):
    ld, a, b = ctypes.c_int64(), ctypes.c_size_t(), ctypes.c_size_t()
    by = [ctypes.byref(v) for v in (ld, a, b)]
    assert lib.mgt_mx4_sizes(0, 129, 130, *by) == OK
    assert (ld.value, a.value, b.value) == (256, 129 * 128, 256 * 8)
    assert lib.mgt_mx4_sizes(1, 1, 1, *by) == OK
    assert (ld.value, a.value, b.value) == (128, 64, 128 * 8)
    assert lib.mgt_mx4_sizes(0, 0, 4, *by) == EINVAL
    assert lib.mgt_mx4_sizes(3, 4, 4, *by) == EUNSUPPORTED
    assert lib.mgt_mx4_sizes(0, 4, 4, None, by[1], by[2]) == EINVAL


@pytest.mark.parametrize("kw,want", BAD)
def test_bad_operands_are_refused_everywhere(lib, kw, want):
    good, bad = operand(), operand(**kw)
    assert lib.mgt_mx4_quantize(1, P, 1 << 20, ref(bad), None, None) == want
    assert lib.mgt_mx4_quantize(1, P, 1 << 20, None, ref(bad), None) == want
    assert lib.mgt_mx4_dequantize(ref(bad), 1, P, 1 << 40, None) == want
    assert lib.mgt_gemm_mx4(ref(bad), ref(good), P, 1, 1 << 20, P, None) == want
    assert lib.mgt_gemm_mx4(ref(good), ref(bad), P, 1, 1 << 40, P, None) == want
    assert lib.mgt_gemm_mx4_gated(ref(bad), ref(good), 0, ref(good), None, 0, P, None) == want
    assert lib.mgt_gemm_mx4_gated(ref(good), ref(bad), 0, ref(good), None, 0, P, None) == want
    assert lib.mgt_gemm_mx4_gated(ref(good), ref(good), 0, ref(bad), None, 0, P, None) == want
    for k in range(3):
        three = [None] * 3
        three[k] = ref(bad)
        assert lib.mgt_mx4_gated_bwd(0, 4, 100, P, 100, P, 200, *three, None) == want


def test_quantize_refusals(lib):
    q, t = operand(4, 100), operand(100, 4)
    call = lambda d=1, x=P, ld=100, q=q, t=t: lib.mgt_mx4_quantize(d, x, ld, ref(q), ref(t), None)  # noqa: E731
    assert call(x=0) == EINVAL
    assert call(q=None, t=None) == EINVAL
    assert call(ld=99) == EINVAL
    assert call(d=2) == EUNSUPPORTED
    assert call(x=P + 1) == EUNSUPPORTED
    assert call(d=0, x=P + 2) == EUNSUPPORTED
    assert call(t=operand(4, 100)) == EINVAL
    assert call(t=operand(100, 4, fmt=1)) == EINVAL
    assert call(q=operand(fmt=1), t=operand(100, 4, fmt=1, factor=P + 16)) == EINVAL
    assert lib.mgt_mx4_tensor_factor(1, 4, 100, P, 99, P, None) == EINVAL
    assert lib.mgt_mx4_tensor_factor(1, 0, 100, P, 100, P, None) == EINVAL
    assert lib.mgt_mx4_tensor_factor(1, 4, 100, P, 100, 0, None) == EINVAL
    assert lib.mgt_mx4_tensor_factor(7, 4, 100, P, 100, P, None) == EUNSUPPORTED


def test_product_refusals(lib):
    a, b = operand(4, 100), operand(7, 100)
    call = lambda a=a, b=b, c=P, d=1, ld=7, st=P: lib.mgt_gemm_mx4(ref(a), ref(b), c, d, ld, st, None)  # noqa: E731
    assert call(a=None) == EINVAL and call(b=None) == EINVAL
    assert call(c=0) == EINVAL and call(st=0) == EINVAL
    assert call(ld=6) == EINVAL
    assert call(b=operand(7, 101)) == EINVAL
    assert call(b=operand(7, 100, fmt=1)) == EINVAL
    assert call(d=2) == EUNSUPPORTED
    assert call(c=P + 1) == EUNSUPPORTED and call(d=0, c=P + 2) == EUNSUPPORTED
    assert lib.mgt_mx4_dequantize(ref(a), 1, P, 99, None) == EINVAL
    assert lib.mgt_mx4_dequantize(ref(a), 1, 0, 100, None) == EINVAL
    assert lib.mgt_mx4_dequantize(ref(a), 5, P, 100, None) == EUNSUPPORTED


def test_gated_refusals(lib):
    x, w, a = operand(4, 100), operand(512, 100), operand(4, 200)
    call = lambda x=x, w=w, act=0, a=a, u=P, ldu=400, st=P: lib.mgt_gemm_mx4_gated(  # noqa: E731
        ref(x), ref(w), act, ref(a), u, ldu, st, None)
    assert call(act=3) == EUNSUPPORTED and call(act=-1) == EUNSUPPORTED
    assert call(ldu=399) == EINVAL
    assert call(u=P + 1) == EUNSUPPORTED
    assert call(w=operand(400, 100)) == EINVAL  # up rows start at a multiple of 128
    assert call(w=operand(512, 101)) == EINVAL
    assert call(a=operand(5, 200)) == EINVAL
    assert call(a=operand(4, 200, fmt=1)) == EINVAL
    assert call(st=0) == EINVAL and call(a=None) == EINVAL
    du, dut, at = operand(4, 512), operand(512, 4), operand(200, 4)
    bwd = lambda act=0, m=4, f=200, da=P, ldd=200, u=P, ldu=400, du=du, dut=dut, at=at: (  # noqa: E731
        lib.mgt_mx4_gated_bwd(act, m, f, da, ldd, u, ldu, ref(du), ref(dut), ref(at), None))
    assert bwd(act=3) == EUNSUPPORTED
    assert bwd(da=0) == EINVAL and bwd(u=0) == EINVAL and bwd(m=0) == EINVAL and bwd(f=0) == EINVAL
    assert bwd(ldd=199) == EINVAL and bwd(ldu=399) == EINVAL
    assert bwd(du=None, dut=None, at=None) == EINVAL
    assert bwd(du=operand(4, 400)) == EINVAL and bwd(dut=operand(400, 4)) == EINVAL
    assert bwd(at=operand(256, 4)) == EINVAL
    assert bwd(at=operand(200, 4, fmt=1)) == EINVAL
    assert bwd(da=P + 1) == EUNSUPPORTED


def test_two_results_in_one_place_are_refused(lib):
    q = operand(128, 128, codes=P)
    for other in (dict(codes=P), dict(scales=P)):  # (codes and scales of `operand` lie at P)
        t = operand(128, 128, **{"codes": P + 65536, "scales": P + 65536, **other})
        assert lib.mgt_mx4_quantize(1, P, 128, ref(q), ref(t), None) == EINVAL
    far = lambda k, r, c: operand(r, c, codes=P + 65536 * k, scales=P + 65536 * k)  # noqa: E731
    three = [far(0, 128, 256), far(1, 256, 128), far(2, 128, 128)]
    for k in range(3):
        for name in ("codes", "scales"):
            bad = list(three)
            bad[k] = operand(bad[k].rows, bad[k].cols, codes=bad[k].codes, scales=bad[k].scales)
            setattr(bad[k], name, getattr(bad[(k + 1) % 3], name))
            assert lib.mgt_mx4_gated_bwd(0, 128, 128, P, 128, P, 256, *map(ref, bad), None) == EINVAL
    x, w, a = far(0, 4, 100), far(1, 512, 100), far(2, 4, 200)
    for other in (x, w):
        b = operand(4, 200, codes=a.codes, scales=other.scales)
        assert lib.mgt_gemm_mx4_gated(ref(x), ref(w), 0, ref(b), None, 0, P, None) == EINVAL


def test_python_operands():
    mk = lambda *a, **k: mgt.Mx4(*a, device="cpu", **k)  # noqa: E731
    q = mk("nvfp4", 300, 200)
    assert q.ld == 256 and q.codes.shape == (300, 128) and q.scales.numel() == 384 * 16
    assert q.factor.tolist() == [1.0, 1.0]
    p = q.part(128, 100, 128, 72)
    assert p._c.codes == q.codes.data_ptr() + (128 * 256 + 128) // 2
    assert p._c.scales == q.scales.data_ptr() + 512 * (1 * 4 + 2)
    assert p.rows_view(0, 10)._c.codes == p._c.codes
    for bad in ((64, 10, 0, 10), (0, 10, 64, 10), (256, 45, 0, 10), (0, 10, 128, 129), (0, 0, 0, 1)):
        with pytest.raises(ValueError):
            q.part(*bad)
    with pytest.raises(ValueError):
        mk("fp4", 1, 1)
    with pytest.raises(ValueError):
        mk("mxfp4", 0, 1)
    with pytest.raises(TypeError):
        mk("mxfp4", 4, 100, codes=torch.empty(4, 64))
    with pytest.raises(TypeError):
        mk("mxfp4", 4, 100, codes=torch.empty(3, 64, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mk("mxfp4", 4, 200, codes=torch.empty(4, 64, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mk("mxfp4", 4, 100, scales=torch.empty(511, dtype=torch.uint8))
    with pytest.raises(TypeError):
        mk("nvfp4", 4, 100, factor=torch.ones(1))


def test_python_checks_types_shapes_and_devices():
    q, x = mgt.Mx4("mxfp4", 4, 100, device="cpu"), torch.zeros(4, 100)
    st = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        mgt.mx4_quantize(x.half(), q)
    with pytest.raises(TypeError):
        mgt.mx4_quantize(x.t(), q)
    with pytest.raises(ValueError):
        mgt.mx4_quantize(x[:3], q)
    with pytest.raises(ValueError):
        mgt.mx4_quantize(x, None, q)
    with pytest.raises(ValueError):
        mgt.mx4_quantize(x, q)  # not on a GPU
    with pytest.raises(ValueError):
        mgt.mx4_dequantize(q, x[:, :99])
    with pytest.raises(ValueError):
        mgt.gemm_mx4(q, q, torch.zeros(4, 5), st)
    with pytest.raises(ValueError):
        mgt.gemm_mx4(q, mgt.Mx4("mxfp4", 5, 101, device="cpu"), torch.zeros(4, 5), st)
    a, u = mgt.Mx4("mxfp4", 4, 60, device="cpu"), torch.zeros(4, 120, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mgt.gemm_mx4_gated(q, q, a, st, act="relu")
    with pytest.raises(TypeError):
        mgt.gemm_mx4_gated(q, q, a, st, u=u.float())
    with pytest.raises(ValueError):
        mgt.gemm_mx4_gated(q, q, a, st, u=u[:, :119])
    with pytest.raises(ValueError):
        mgt.mx4_gated_bwd(u[:, :50], u, a)
    with pytest.raises(TypeError):
        mgt.mx4_gated_bwd(u[:, :60].float(), u, a)


def test_sizes_beyond_int32_are_refused():
    """2^32 + 128 cut to 32 bits is 128: it must not arrive as that. ("meta" tensors have a shape only.)"""
    many, empty = 2 ** 32 + 128, lambda *n, t=torch.uint8: torch.empty(*n, dtype=t, device="meta")  # noqa: E731
    for rows, cols in ((many, 100), (100, many), (2 ** 30 + 1, 1), (1, 2 ** 30 + 1)):
        with pytest.raises(ValueError, match="2\\*\\*30"):
            mgt.Mx4("mxfp4", rows, cols, codes=empty(rows, (cols + 127) // 128 * 64))
    assert mgt.Mx4("mxfp4", 1, 2 ** 30, codes=empty(1, 2 ** 29))._c.cols == 2 ** 30
    f, small = empty(2, t=torch.float32), mgt.Mx4("mxfp4", 128, 128, device="cpu")
    for shape in ((1, many), (many, 1), (2 ** 31, 1), (1, 2 ** 31)):
        x = empty(*shape, t=torch.bfloat16)
        for call in (lambda: mgt.mx4_tensor_factor(x, f), lambda: mgt.mx4_quantize(x, small),
                     lambda: mgt.mx4_dequantize(small, x), lambda: mgt.gemm_mx4(small, small, x, None),
                     lambda: mgt.mx4_gated_bwd(x, x, du=small)):
            with pytest.raises(ValueError, match="2\\*\\*31"):
                call()


def test_an_operand_follows_its_factor_and_keeps_the_rest():
    """The calls take addresses: an assigned factor has to reach them, and nothing else may be assigned."""
    mk = lambda fmt="nvfp4", **k: mgt.Mx4(fmt, 300, 200, device="cpu", **k)  # noqa: E731
    q, t = mk(), torch.ones(2)
    part = q.part(128, 100, 128, 72)
    before = q.factor
    q.factor = t
    assert q.factor is t and q._c.factor == t.data_ptr() and q._addr == ctypes.addressof(q._c)
    assert (q._c.codes, q._c.scales) == (q.codes.data_ptr(), q.scales.data_ptr())
    assert part.factor is before and part._c.factor == before.data_ptr()
    codes, scales = part._c.codes, part._c.scales
    part.factor = t
    assert (part._c.codes, part._c.scales, part._c.factor) == (codes, scales, t.data_ptr())
    assert (part.rows, part.cols, part._c.rows, part._c.cols) == (100, 72, 100, 72)
    for bad, error in ((None, TypeError), (2.0, TypeError), (torch.ones(1), TypeError),
                       (torch.ones(2).double(), TypeError), (torch.ones(4)[::2], TypeError),
                       (torch.ones(2, device="meta"), ValueError)):
        with pytest.raises(error):
            q.factor = bad
        assert q.factor is t and q._c.factor == t.data_ptr()
    for name in ("codes", "scales", "rows", "cols", "ld", "fmt", "device", "index"):
        for operand in (q, part):
            with pytest.raises(AttributeError):
                setattr(operand, name, getattr(operand, name))
    m = mk("mxfp4")
    m.factor = t
    m.factor = None
    assert m._c.factor is None


def host_program(name, tmp_path):
    """Compile tests/host/<name>.cu for the host and run it."""
    nvcc = next((p for p in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc") if p and os.path.exists(p)), None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host", name + ".cu")
    exe = str(tmp_path / name)
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-o", exe, src], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr


def test_resident_clusters_are_kept_by_device(tmp_path):
    host_program("mx4_clusters_check", tmp_path)


def test_launch_shapes_of_the_few_row_product(tmp_path):
    host_program("mx4_shapes_check", tmp_path)
