"""What the block operators refuse, on the host and before any launch (CPU only: no
call here reaches a kernel)."""
import ctypes

import pytest
import torch

import nvfp4_w4a4_gated_b200 as nv

FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced (validation fails first)
BF16, FP32 = nv.DTYPE_BF16, nv.DTYPE_FP32


def fp8(rows=128, cols=256, ld=None, codes=FAKE, scale=FAKE):
    return nv._Fp8(codes, scale, rows, cols, cols if ld is None else ld)


def quantize(x=FAKE, dtype=BF16, rows=128, cols=256, ld=None, out=None):
    t = out if out is not None else fp8(rows, cols)
    return nv.lib().fp8_quantize(x, dtype, rows, cols, cols if ld is None else ld, ctypes.byref(t), None)


@pytest.mark.parametrize("status,kw", [
    (1, dict(x=None)), (1, dict(dtype=7)), (1, dict(rows=0)), (1, dict(cols=0)), (2, dict(cols=24)),
    (2, dict(cols=32768 + 16)), (2, dict(rows=1 << 31)), (1, dict(ld=240)), (3, dict(x=FAKE + 2)), (3, dict(ld=260)),
    (1, dict(out=fp8(128, 272))), (1, dict(out=fp8(127, 256))), (1, dict(out=fp8(codes=0))), (1, dict(out=fp8(scale=0))),
    (3, dict(out=fp8(codes=FAKE + 8))), (3, dict(out=fp8(ld=264))), (1, dict(out=fp8(ld=240))), (3, dict(out=fp8(scale=FAKE + 2))),
])
def test_quantize(status, kw):
    assert quantize(**kw) == status
    assert nv.lib().nvfp4_last_error()


def norm(x=FAKE + 4096, xt=FP32, ld_x=256, r=FAKE, rt=BF16, ld_r=256, w=FAKE, eps=1e-6, rows=128, cols=256, h=FAKE, ld_h=256,
         out=True, n=None, ld_n=256, amax=None):
    t = fp8(rows, cols) if out is True else out
    return nv.lib().add_rmsnorm_quantize(x, xt, ld_x, r, rt, ld_r, w, eps, rows, cols, h, ld_h,
                                         None if t is None else ctypes.byref(t), n, ld_n, amax, None)


@pytest.mark.parametrize("status,kw", [
    (1, dict(x=None)), (1, dict(w=None)), (1, dict(xt=9)), (1, dict(rt=-1)), (1, dict(eps=0.0)), (1, dict(eps=-1.0)),
    (1, dict(eps=float("nan"))), (1, dict(eps=float("inf"))), (1, dict(rows=0)), (1, dict(cols=0)), (2, dict(cols=40)),
    (2, dict(cols=65536, ld_x=65536)), (1, dict(h=None)), (1, dict(r=None)), (1, dict(out=None)), (1, dict(amax=FAKE)),
    (1, dict(ld_x=248)), (1, dict(ld_r=240)), (1, dict(ld_h=240)), (1, dict(n=FAKE + 64, ld_n=240)), (3, dict(x=FAKE + 4)),
    (3, dict(ld_x=258)), (3, dict(r=FAKE + 2)), (3, dict(ld_r=260)), (3, dict(h=FAKE + 8)), (3, dict(w=FAKE + 4)),
    (3, dict(n=FAKE + 2)), (3, dict(n=FAKE + 64, ld_n=260)), (1, dict(n=FAKE)), (1, dict(n=FAKE + 4096)),
    (1, dict(ld_h=264)), (1, dict(x=FAKE, xt=BF16, ld_x=264, r=FAKE + 64)), (1, dict(x=FAKE, r=FAKE + 64)), (1, dict(out=fp8(128, 240))), (3, dict(out=fp8(codes=FAKE + 4))),
])
def test_norm(status, kw):
    assert norm(**kw) == status
    assert nv.lib().nvfp4_last_error()


def epilogue(bias=None, act=0, r=None, rt=BF16, ld_r=64, out=FAKE, ot=BF16, ldc=64):
    return nv._Epilogue(bias, act, r, rt, ld_r, out, ot, ldc)


EPILOGUES = [
    (1, dict(out=None)), (1, dict(ot=3)), (1, dict(act=-1)), (1, dict(act=4)), (1, dict(ldc=63)), (3, dict(out=FAKE + 1)),
    (3, dict(out=FAKE + 2, ot=FP32)), (3, dict(bias=FAKE + 2)), (1, dict(r=FAKE + 64, rt=5)), (1, dict(r=FAKE + 64, ld_r=63)),
    (3, dict(r=FAKE + 1)), (3, dict(r=FAKE + 2, rt=FP32)), (1, dict(r=FAKE, rt=FP32)), (1, dict(r=FAKE, ld_r=65)),
]


@pytest.mark.parametrize("status,kw", EPILOGUES)
def test_w8a8_epilogue(status, kw):
    A, B, e = fp8(8, 256), fp8(64, 256), epilogue(**kw)
    assert nv.lib().w8a8_gemm(ctypes.byref(A), ctypes.byref(B), ctypes.byref(e), None) == status


@pytest.mark.parametrize("status,kw", EPILOGUES)
def test_w4a4_epilogue(status, kw):
    A, B, e = (nv._Tensor(FAKE, FAKE, FAKE, rows, 256) for rows in (8, 64)), None, epilogue(**kw)
    A, B = tuple(A)
    assert nv.lib().w4a4_gemm_fused(ctypes.byref(A), ctypes.byref(B), ctypes.byref(e), None) == status


@pytest.mark.parametrize("status,a,b", [
    (1, fp8(8, 256), fp8(64, 272)), (1, fp8(0, 256), fp8(64, 256)), (2, fp8(8, 24), fp8(64, 24)),
    (1, fp8(8, 256, ld=240), fp8(64, 256)), (3, fp8(8, 256, codes=FAKE + 8), fp8(64, 256)),
    (3, fp8(8, 256), fp8(64, 256, ld=264)), (1, fp8(8, 256, scale=0), fp8(64, 256)), (1, fp8(8, 256), fp8(64, 256, codes=0)),
    (2, fp8(1 << 31, 256), fp8(64, 256)), (2, fp8((1 << 30) + 1, 256), fp8(64, 256)), (2, fp8(8, (1 << 24) + 16), fp8(64, (1 << 24) + 16)),
])
def test_w8a8_operands(status, a, b):
    e = epilogue()
    assert nv.lib().w8a8_gemm(ctypes.byref(a), ctypes.byref(b), ctypes.byref(e), None) == status
    assert nv.lib().nvfp4_last_error()


def test_null_structs():
    L, A, e = nv.lib(), fp8(64, 256), epilogue()
    assert L.w8a8_gemm(None, ctypes.byref(A), ctypes.byref(e), None) == 1
    assert L.w8a8_gemm(ctypes.byref(A), None, ctypes.byref(e), None) == 1
    assert L.w8a8_gemm(ctypes.byref(A), ctypes.byref(A), None, None) == 1
    assert L.fp8_quantize(FAKE, BF16, 64, 256, 256, None, None) == 1


def test_w4a4_operands():
    e = epilogue()
    for status, a, b in ((1, (8, 256), (64, 320)), (2, (8, 96), (64, 96)), (2, ((1 << 30) + 1, 256), (64, 256))):
        A, B = (nv._Tensor(FAKE, FAKE, FAKE, *t) for t in (a, b))
        assert nv.lib().w4a4_gemm_fused(ctypes.byref(A), ctypes.byref(B), ctypes.byref(e), None) == status


def test_host_tensors_are_refused():
    x, w = torch.zeros(4, 64), torch.ones(64)
    q = nv.FP8Matrix(torch.zeros(4, 64).to(torch.float8_e4m3fn), torch.ones(4))
    for call in (lambda: nv.fp8_quantize(x), lambda: nv.add_rmsnorm_quantize(x, w), lambda: nv.w8a8_gemm(q, q)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()


def nvfp4(rows=130, cols=128, codes=None, sf=None, scale=None):
    return nv.NVFP4Matrix(torch.zeros((rows, cols // 2), dtype=torch.uint8) if codes is None else codes,
                          torch.zeros(256 * cols // 16, dtype=torch.uint8) if sf is None else sf,
                          torch.ones(1) if scale is None else scale, rows, cols)


@pytest.mark.parametrize("name,kw", [
    ("codes", dict(codes=torch.zeros((129, 64), dtype=torch.uint8))),
    ("codes", dict(codes=torch.zeros((130, 63), dtype=torch.uint8))),
    ("codes", dict(codes=torch.zeros((130, 80), dtype=torch.uint8)[:, :64])),
    ("codes", dict(codes=torch.zeros((64, 130), dtype=torch.uint8).t())),
    ("codes", dict(codes=torch.zeros((1, 64), dtype=torch.uint8).expand(130, 64))),
    ("codes", dict(codes=torch.zeros((130, 64), dtype=torch.int16))),
    ("sf", dict(sf=torch.zeros(130 * 8, dtype=torch.uint8))),
    ("sf", dict(sf=torch.zeros((256, 16), dtype=torch.uint8)[:, :8])),
    ("sf", dict(sf=torch.zeros(256 * 8, dtype=torch.uint8)[::2])),
    ("scale", dict(scale=torch.ones(1, dtype=torch.float64))),
    ("scale", dict(scale=torch.ones(0))),
])
def test_nvfp4_buffers_that_do_not_hold_the_matrix(name, kw):
    """Refused before the device is looked at, so host tensors show it."""
    good, bad = nvfp4(), nvfp4(**kw)
    for call in (lambda: nv.w4a4_gemm_fused(bad, good), lambda: nv.w4a4_gemm(bad, good, C=torch.zeros(130, 130)),
                 lambda: bad.c()):
        with pytest.raises(ValueError, match=name + ": .* expected"):
            call()
    with pytest.raises(ValueError, match="CUDA tensors"):
        good.c()


def test_words_that_are_not_aligned():
    """A kernel would read or update them as one 32-bit word."""
    assert norm(n=FAKE + 64, amax=FAKE + 2) == 3
    e = epilogue()
    for a, b in ((FAKE + 2, FAKE), (FAKE, FAKE + 1)):
        A, B = nv._Tensor(FAKE, FAKE, a, 8, 256), nv._Tensor(FAKE, FAKE, b, 64, 256)
        assert nv.lib().w4a4_gemm_fused(ctypes.byref(A), ctypes.byref(B), ctypes.byref(e), None) == 3


def test_packed_structures_have_the_c_layout():
    for struct_type, pack, values in ((nv._Tensor, nv._pack_tensor, (1 << 40, 2 << 40, 3 << 40, 64, 5120)),
                                      (nv._Fp8, nv._pack_fp8, (1 << 40, 2 << 40, 64, 5120, 5136)),
                                      (nv._Epilogue, nv._pack_epilogue, (1 << 40, 3, 2 << 40, 1, 77, 3 << 40, 1, 99))):
        assert bytes(struct_type(*values)) == pack(*values)
