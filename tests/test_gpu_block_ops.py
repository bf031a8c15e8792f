"""The block operators on the GPU (residual + RMS norm + E4M3 output, the E4M3 row
quantiser, the W8A8 and NVFP4 products with a fused epilogue) against float64.

Bounds, with u = 2^-24 (half a float32 step, relative):
- h: one float32 addition and one rounding, both to nearest: equal bits.
- n before its rounding: a thread adds at most 32 squares in a row and the partial sums
  meet in at most 10 additions, so the mean square is within 44 u, its division, + eps
  and the root's argument add 2 u; rsqrtf is within 2 units in the last place (4 u); the
  products h w and p rstd add 2 u: (44 + 2) / 2 + 4 + 2 = 29 u.  32 u is used.
- the row scale: that and one division: 34 u.
- a code: half an E4M3 step of n / S, i.e. 2^-4 of its magnitude (2^-10 below 2^-6, where
  the step is 2^-9), and 40 u for n, S, 1 / S and their product.
- a product: each tensor-core step (32 E4M3 or 64 E2M1 products, exact) leaves the
  running float32 sum off by at most 4 u of the sum of magnitudes; split ranges of K and
  the two scales and the bias add 8 more such terms.  The activations' slopes are at most 1.13 and
  their own evaluation is within 8 u of the argument's magnitude.
- an output: half a step of its type (bf16 2^-8, float32 2^-24)."""
import dataclasses
import math
import subprocess
import sys
import threading

import pytest
import torch

import nvfp4_w4a4_gated_b200 as nv

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(shape, seed, dtype=F32, std=1.0, pad=0):
    """Normal values; with ``pad`` the rows are that many elements further apart."""
    rows, cols = shape
    t = (std * torch.randn((rows, cols + pad), generator=gen(seed), device="cuda")).to(dtype)
    return t[:, :cols]


def done():
    torch.cuda.synchronize()
    nv.check_device_error()


# ------------------------------------------------------------- norm, quantiser --
def check_codes(q, n):
    """q holds the float64 rows n."""
    amax = n.abs().amax(1)
    S = torch.where(amax < 2.0 ** -100, torch.ones_like(amax), amax / 448)
    assert torch.all((q.scale.double() - S).abs() <= 34 * U * S)
    v = n / S[:, None]
    off = (q.codes.float().double() - v).abs()
    assert torch.all(off <= torch.clamp(2.0 ** -4 * v.abs(), min=2.0 ** -10) + 40 * U * v.abs())


def over_448(amax):
    """The rounded quotient (a division by a Python number may multiply by its reciprocal)."""
    return torch.div(amax, torch.full_like(amax, 448.0))


def norm_ref(h, w, eps=EPS):
    h = h.double()
    return h * w.double() / torch.sqrt(h.square().mean(1, keepdim=True) + eps)


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (9, 256), (8, 528), (17, 1024), (5, 1040), (1, 5120),
                                       (203, 5120), (149, 4112), (2, 16384), (150, 16400), (3, 32768), (150, 32768)])
@pytest.mark.parametrize("xt,rt", [(F32, BF16), (BF16, BF16), (BF16, F32), (F32, F32), (F32, None), (BF16, None)])
def test_norm(cuda_dev, rows, cols, xt, rt):
    x = rand((rows, cols), 1, xt, 2.0)
    r = None if rt is None else rand((rows, cols), 2, rt, 3.0)
    w = 1 + 0.3 * torch.randn(cols, generator=gen(3), device="cuda")
    h, q, n = nv.add_rmsnorm_quantize(x, w, residual=r, want_norm=True)
    done()
    if r is None:
        assert h is x
    else:
        assert torch.equal(h, (x.float() + r.float()).to(rt))
    ref = norm_ref(h, w)
    assert n.dtype == BF16
    assert torch.all((n.double() - ref).abs() <= (2.0 ** -8 + 33 * U) * ref.abs())
    check_codes(q, ref)


@pytest.mark.parametrize("rows,cols", [(1, 16), (7, 272), (300, 1024), (33, 4096), (150, 5120), (2, 32768)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize(cuda_dev, rows, cols, dtype):
    x = rand((rows, cols), 4, dtype)
    x[0, 0] = 300.0
    q = nv.fp8_quantize(x)
    done()
    check_codes(q, x.double())
    # the definition's float32 operations, to the bit
    S = over_448(x.float().abs().amax(1))
    assert torch.equal(q.scale, S)
    assert torch.equal(q.codes.float(), (x.float() * (1.0 / S)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("cols", [512, 4112])
def test_norm_rows_with_nothing_or_not_finite(cuda_dev, cols):
    """Zero rows, tiny rows, NaN, infinities and sums that overflow, next to ordinary rows."""
    x = rand((9, cols), 5)
    x[1] = 0.0
    x[2] = 1e-35
    x[3, 7] = math.nan
    x[4, 9] = math.inf
    x[5, 11] = -math.inf
    x[6] = 1e30
    w = torch.ones(cols, device="cuda")
    w[5] = -2.0
    r = torch.zeros_like(x)
    h, q, n = nv.add_rmsnorm_quantize(x, w, residual=r, want_norm=True)
    done()
    assert torch.equal(h[6], x[6])
    good = [0, 1, 2, 7, 8]
    bad = [3, 4, 5, 6]
    ref = norm_ref(h[good], w)
    assert torch.all((n[good].double() - ref).abs() <= (2.0 ** -8 + 33 * U) * ref.abs() + 2.0 ** -133)
    assert torch.all(q.scale[1] == 1.0) and torch.all(q.codes[1].float() == 0.0)
    check_codes(nv.FP8Matrix(q.codes[good], q.scale[good]), ref)
    assert torch.all(torch.isnan(q.scale[bad])) and torch.all(torch.isnan(q.codes[bad].float()))
    assert torch.all(torch.isnan(n[bad].float()))
    q = nv.fp8_quantize(x)
    done()
    assert torch.all(torch.isnan(q.scale[[3, 4, 5]])) and torch.all(torch.isnan(q.codes[[3, 4, 5]].float()))
    assert q.scale[1] == 1.0 and torch.all(q.codes[1].float() == 0.0)
    assert q.scale[2] == 1.0   # below 2^-100
    assert torch.equal(q.scale[[0, 6, 7, 8]], over_448(x[[0, 6, 7, 8]].abs().amax(1)))


@pytest.mark.parametrize("cols", [256, 5120])
@pytest.mark.parametrize("rt", [F32, BF16])
def test_norm_strides_in_place_and_untouched_memory(cuda_dev, cols, rt):
    rows, pad = 37, 32
    x = rand((rows, cols), 6, F32, pad=pad)
    r = rand((rows, cols), 7, rt, pad=2 * pad)
    keep = r.clone()
    w = torch.randn(cols, generator=gen(8), device="cuda")
    codes = torch.full((rows + 1, cols + 16), 0x11, dtype=torch.uint8, device="cuda")
    out = nv.FP8Matrix(codes.view(torch.float8_e4m3fn)[:rows, :cols], torch.zeros(rows, device="cuda"))
    n = torch.full((rows + 1, cols + 8), 5.0, dtype=BF16, device="cuda")
    rbase = r._base if r._base is not None else r
    tail = rbase[:, cols:].clone()
    h, q, n_out = nv.add_rmsnorm_quantize(x, w, residual=r, h=r, out=out, norm=n[:rows, :cols])
    done()
    assert h is r and q is out and n_out.data_ptr() == n.data_ptr()
    assert torch.equal(r, (x + keep.float()).to(rt))
    ref = norm_ref(r, w)
    check_codes(out, ref)
    assert torch.all((n_out.double() - ref).abs() <= (2.0 ** -8 + 33 * U) * ref.abs())
    assert torch.all(codes[rows:] == 0x11) and torch.all(codes[:, cols:] == 0x11)
    assert torch.all(n[rows:] == 5.0) and torch.all(n[:, cols:] == 5.0)
    assert torch.equal(rbase[:, cols:], tail)
    # h over x
    x2 = rand((rows, cols), 6, rt)
    r2 = rand((rows, cols), 9, rt)
    want = (x2.float() + r2.float()).to(rt)
    h, q, none = nv.add_rmsnorm_quantize(x2, w, residual=r2, h=x2)
    done()
    assert none is None and torch.equal(x2, want)
    check_codes(q, norm_ref(want, w))


def test_norm_amax_word_feeds_the_nvfp4_quantiser(cuda_dev):
    rows, cols = 77, 1280
    x, r = rand((rows, cols), 10, F32), rand((rows, cols), 11, BF16)
    w = torch.randn(cols, generator=gen(12), device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    h, q, n = nv.add_rmsnorm_quantize(x, w, residual=r, want_fp8=False, want_norm=True, amax_word=ws.view(torch.int32))
    assert q is None
    one = nv.nvfp4_quantize(n, mode=nv.QUANT_FROM_AMAX, workspace=ws)
    two = nv.nvfp4_quantize(n)
    done()
    assert ws.view(torch.float32)[0] == n.float().abs().max()
    for a, b in ((one.codes, two.codes), (one.sf, two.sf), (one.scale, two.scale)):
        assert torch.equal(a, b)


def test_norm_offsets_past_32_bits(cuda_dev):
    """Rows 2^31 elements apart (the third starts 8.6 GB in)."""
    cols, ld = 1040, 2 ** 31
    buf = torch.zeros(2 * ld + cols, dtype=BF16, device="cuda")
    x = buf.as_strided((3, cols), (ld, 1))
    x.copy_(rand((3, cols), 13, BF16))
    out = torch.zeros(2 * ld + cols, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).as_strided((3, cols), (ld, 1))
    w = torch.ones(cols, device="cuda")
    _, q, _ = nv.add_rmsnorm_quantize(x, w, out=nv.FP8Matrix(out, torch.empty(3, device="cuda")))
    done()
    check_codes(nv.FP8Matrix(q.codes.contiguous(), q.scale), norm_ref(x, w))


# --------------------------------------------------------------------- products --
def act64(v, act):
    if act == nv.ACT_SILU:
        return v / (1 + torch.exp(-v))
    if act == nv.ACT_GELU:
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if act == nv.ACT_RELU:
        return v.clamp(min=0)
    return v


def check_product(C, a, b, step, bias, act, r):
    """a, b: float64 operands with their scales; r: the residual as it was before the call."""
    p, mag = a @ b.T, a.abs() @ b.abs().T
    v = p if bias is None else p + bias.double()
    if bias is not None:
        mag = mag + bias.double().abs()
    y = act64(v, act)
    tol = 1.13 * (math.ceil(a.shape[1] / step) + 8) * 4 * U * mag + 8 * U * v.abs()
    if r is not None:
        y = y + r.double()
        tol = tol + U * y.abs()
    tol = tol + HALF[C.dtype] * (y.abs() + tol)
    off = (C.double() - y).abs()
    assert torch.all(off <= tol), float((off / tol).max())


def fp8_pair(M, N, K, seed, pad=0):
    def one(rows, s, std):
        q = nv.fp8_quantize(rand((rows, K), s, F32, std))
        if pad:
            wide = torch.zeros((rows, K + pad), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            wide[:, :K].view(torch.uint8).copy_(q.codes.view(torch.uint8))
            # what lies between the rows must not matter
            wide[:, K:].view(torch.uint8).fill_(0x7F)
            q = nv.FP8Matrix(wide[:, :K], q.scale)
        return q
    return one(M, seed, 1.0), one(N, seed + 1, 0.1)


def value(q):
    return q.codes.float().double() * q.scale.double()[:, None]


# decode, split ranges of K, several token tiles, CTA pairs; sizes of one, odd and ragged
SHAPES = [(1, 1, 16), (1, 128, 128), (1, 5120, 4096), (2, 129, 48), (16, 1000, 1040), (17, 4099, 2064), (32, 256, 4096),
          (33, 640, 512), (64, 12352, 5120), (64, 128, 8192), (65, 130, 144), (128, 512, 1024), (129, 700, 272),
          (500, 333, 640), (257, 12352, 272), (2300, 2311, 208), (2304, 2304, 128), (2100, 2500, 16), (4000, 1300, 1040),
          (1237, 4099, 1040),
          # K in three and in four
          (64, 5120, 2064), (50, 6000, 1552), (128, 2000, 2000), (100, 5003, 1600), (40, 300, 2000), (9, 2000, 2064),
          # last rounds cut into narrow tiles, some of them past the last token
          (1030, 4099, 272), (1537, 1500, 128), (5000, 2000, 48)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_w8a8(cuda_dev, M, N, K, out_dtype):
    A, B = fp8_pair(M, N, K, M + N)
    C = nv.w8a8_gemm(A, B, out_dtype=out_dtype)
    done()
    check_product(C, value(A), value(B), 32, None, nv.ACT_NONE, None)
    again = nv.w8a8_gemm(A, B, out_dtype=out_dtype)
    assert torch.equal(C, again)


@pytest.mark.parametrize("M,N,K", [(2300, 2311, 5120), (1030, 4099, 3856), (200, 7500, 4000), (64, 15000, 3840)])
@pytest.mark.parametrize("act,res", [(nv.ACT_NONE, None), (nv.ACT_SILU, BF16)])
def test_w8a8_long_sums(cuda_dev, M, N, K, act, res):
    """float32 results of long sums: summed in two chains or more."""
    A, B = fp8_pair(M, N, K, 7)
    bias = torch.randn(N, generator=gen(8), device="cuda")
    r = None if res is None else rand((M, N), 9, res)
    C = nv.w8a8_gemm(A, B, bias=bias, act=act, residual=r, out_dtype=F32)
    done()
    # each chain has half the steps: half the bound
    check_product(C, value(A), value(B), 64, bias, act, r)
    stream = rand((M, N), 10, F32, pad=3)
    before = stream.clone()
    nv.w8a8_gemm(A, B, bias=bias, act=act, residual=stream, out=stream)
    done()
    check_product(stream, value(A), value(B), 64, bias, act, before)


@pytest.mark.parametrize("M,N,K", [(1, 515, 256), (40, 1027, 1040), (200, 333, 256), (2300, 2311, 208)])
@pytest.mark.parametrize("act", [nv.ACT_NONE, nv.ACT_SILU, nv.ACT_GELU, nv.ACT_RELU])
@pytest.mark.parametrize("res", [None, F32, BF16])
def test_w8a8_epilogue(cuda_dev, M, N, K, act, res):
    A, B = fp8_pair(M, N, K, 3 * act + M)
    bias = torch.randn(N, generator=gen(5), device="cuda")
    r = None if res is None else rand((M, N), 6, res, 2.0, pad=5)
    for out_dtype in (F32, BF16):
        C = nv.w8a8_gemm(A, B, bias=bias, act=act, residual=r, out_dtype=out_dtype)
        done()
        check_product(C, value(A), value(B), 32, bias, act, r)


@pytest.mark.parametrize("M,N,K", [(3, 130, 272), (70, 257, 528), (2300, 2311, 208)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_w8a8_strides_in_place_and_untouched_memory(cuda_dev, M, N, K, dtype):
    """Padded operands, an odd output pitch and offset, the residual updated in place."""
    A, B = fp8_pair(M, N, K, 21, pad=48)
    wide = rand((M + 1, N + 7), 22, dtype)
    before = wide.clone()
    stream = wide[:M, 3:3 + N]
    out = nv.w8a8_gemm(A, B, residual=stream, out=stream)
    done()
    assert out is stream
    check_product(stream, value(A), value(B), 32, None, nv.ACT_NONE, before[:M, 3:3 + N])
    wide[:M, 3:3 + N] = before[:M, 3:3 + N]
    assert torch.equal(wide, before)


def test_w8a8_rows_that_are_not_finite(cuda_dev):
    """A NaN in one token stays in that token's row, in one weight row in that column."""
    M, N, K = 70, 300, 256
    x, w = rand((M, K), 31), rand((N, K), 32)
    x[5, 3] = math.nan
    w[200, 9] = math.inf
    C = nv.w8a8_gemm(nv.fp8_quantize(x), nv.fp8_quantize(w), act=nv.ACT_RELU, out_dtype=F32)
    done()
    nan = torch.isnan(C)
    assert torch.all(nan[5]) and torch.all(nan[:, 200])
    nan[5] = False
    nan[:, 200] = False
    assert not torch.any(nan)


def test_epilogue_extremes(cuda_dev):
    """Arguments where exp and erf saturate."""
    A = nv.FP8Matrix(torch.ones((1, 16), device="cuda").to(torch.float8_e4m3fn), torch.ones(1, device="cuda"))
    v = torch.tensor([-1e30, -200.0, -89.0, -20.0, -6.0, -1e-3, 0.0, 1e-3, 6.0, 20.0, 89.0, 200.0, 1e30], device="cuda")
    N = v.numel()
    B = nv.FP8Matrix(torch.zeros((N, 16), device="cuda").to(torch.float8_e4m3fn), torch.ones(N, device="cuda"))
    for act in (nv.ACT_SILU, nv.ACT_GELU, nv.ACT_RELU):
        C = nv.w8a8_gemm(A, B, bias=v, act=act, out_dtype=F32)[0].double()
        done()
        # 1 + erf loses what is below half a step of 1: absolute, as a share of the argument
        want = act64(v.double(), act)
        assert torch.all((C - want).abs() <= 8 * U * v.double().abs()), (act, C, want)
        assert torch.all(torch.isfinite(C))
    inf = torch.tensor([math.inf, -math.inf], device="cuda").repeat(7)[:N]
    C = nv.w8a8_gemm(A, B, bias=inf, act=nv.ACT_GELU, out_dtype=F32)[0]
    done()
    assert torch.equal(C, inf.clamp(min=0))


def nvfp4_value(t):
    """float64 values of an NVFP4Matrix."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(t.codes & 15).long()], grid[(t.codes >> 4).long()]], 2).view(t.rows, t.cols // 16, 16)
    sf = t.sf.view(torch.float8_e4m3fn).float().double().view(-1, t.cols // 64, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return (v * sf.reshape(-1, t.cols // 16, 1)[:t.rows]).view(t.rows, t.cols) * t.scale.double()


@pytest.mark.parametrize("M,N,K", [(1, 1, 64), (1, 5120, 4096), (64, 1003, 320), (130, 515, 256), (300, 12352, 192),
                                   (2300, 2311, 448), (1030, 4099, 320), (1537, 1500, 192), (5000, 2000, 64), (100, 3000, 4096),
                                   (64, 5120, 4096), (50, 300, 4160), (9, 2000, 4160)])
@pytest.mark.parametrize("bias,act,res", [(False, nv.ACT_NONE, None), (True, nv.ACT_SILU, F32), (True, nv.ACT_GELU, BF16)])
def test_w4a4_fused(cuda_dev, M, N, K, bias, act, res):
    A = nv.nvfp4_quantize(rand((M, K), 41))
    B = nv.nvfp4_quantize(rand((N, K), 42, std=0.1))
    b = torch.randn(N, generator=gen(43), device="cuda") if bias else None
    r = None if res is None else rand((M, N), 44, res, pad=3)
    for out_dtype in (F32, BF16):
        C = nv.w4a4_gemm_fused(A, B, bias=b, act=act, residual=r, out_dtype=out_dtype)
        done()
        check_product(C, nvfp4_value(A), nvfp4_value(B), 64, b, act, r)
        assert torch.equal(C, nv.w4a4_gemm_fused(A, B, bias=b, act=act, residual=r, out_dtype=out_dtype))


@pytest.mark.parametrize("M,N,K", [(4096, 5120, 5120), (64, 12352, 5120), (300, 3000, 8192)])
def test_w4a4_fused_long_sums(cuda_dev, M, N, K):
    """Scales differ from block to block and from stage to stage (rows and columns of
    very different size): a stage's scales read too early or too late would show.  Runs
    repeat to the bit."""
    size = torch.exp(4 * torch.rand(K, generator=gen(48), device="cuda"))
    A = nv.nvfp4_quantize(rand((M, K), 49) * size)
    B = nv.nvfp4_quantize(rand((N, K), 50) / size.flip(0))
    C = nv.w4a4_gemm_fused(A, B, out_dtype=F32)
    done()
    check_product(C, nvfp4_value(A), nvfp4_value(B), 64, None, nv.ACT_NONE, None)
    for _ in range(5):
        assert torch.equal(C, nv.w4a4_gemm_fused(A, B, out_dtype=F32))
    done()


@pytest.mark.parametrize("M,N,K", [(5, 130, 256), (2300, 2311, 192)])
def test_w4a4_fused_in_place_and_untouched_memory(cuda_dev, M, N, K):
    A, B = nv.nvfp4_quantize(rand((M, K), 45)), nv.nvfp4_quantize(rand((N, K), 46))
    wide = rand((M + 1, N + 7), 47, BF16)
    before = wide.clone()
    stream = wide[:M, 3:3 + N]
    nv.w4a4_gemm_fused(A, B, residual=stream, out=stream)
    done()
    check_product(stream, nvfp4_value(A), nvfp4_value(B), 64, None, nv.ACT_NONE, before[:M, 3:3 + N])
    wide[:M, 3:3 + N] = before[:M, 3:3 + N]
    assert torch.equal(wide, before)


# ------------------------------------------------------------ streams and graphs --
def test_other_stream(cuda_dev):
    M, N, K = 40, 700, 1040
    x, w = rand((M, K), 51), torch.ones(K, device="cuda")
    B = nv.fp8_quantize(rand((N, K), 52))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _, q, _ = nv.add_rmsnorm_quantize(x, w, stream=s)
    C = nv.w8a8_gemm(q, B, stream=s)
    s.synchronize()
    nv.check_device_error()
    _, q2, _ = nv.add_rmsnorm_quantize(x, w)
    assert torch.equal(C, nv.w8a8_gemm(q2, B))


def test_two_graphs_replayed_at_once(cuda_dev):
    """Two captured chains with their own buffers, replayed on two streams together."""
    K, N = 1040, 2000
    B = nv.fp8_quantize(rand((N, K), 61))
    w = torch.randn(K, generator=gen(62), device="cuda")
    chains = []
    for M in (1, 300):
        x, r = torch.zeros((M, K), device="cuda"), torch.zeros((M, K), dtype=BF16, device="cuda")
        def run(x=x, r=r):
            h, q, _ = nv.add_rmsnorm_quantize(x, w, residual=r)
            return h, nv.w8a8_gemm(q, B, act=nv.ACT_SILU)
        run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run()
        chains.append((g, x, r, run, outs, torch.cuda.Stream()))
    for seed in range(3):
        for i, (g, x, r, run, outs, s) in enumerate(chains):
            x.copy_(rand(x.shape, 100 + 10 * seed + i))
            r.copy_(rand(r.shape, 200 + 10 * seed + i))
        torch.cuda.synchronize()
        for g, x, r, run, outs, s in chains:
            with torch.cuda.stream(s):
                g.replay()
        done()
        for g, x, r, run, outs, s in chains:
            for a, b in zip(outs, run()):
                assert torch.equal(a, b)


def test_threads_on_their_own_streams(cuda_dev):
    """Calls that share operands, from several host threads at once."""
    A, B = fp8_pair(300, 3000, 528, 65)
    want = nv.w8a8_gemm(A, B)
    done()
    outs = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                outs[i] = nv.w8a8_gemm(A, B)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(outs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    done()
    assert all(torch.equal(o, want) for o in outs)


FIRST_CALLS = """
import torch
import nvfp4_w4a4_gated_b200 as nv
x, w = torch.randn(300, 512, device="cuda"), torch.ones(512, device="cuda")
r, W = torch.randn(300, 512, device="cuda").bfloat16(), torch.randn(9000, 512, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q = nv.fp8_quantize(W)
    h, a, n = nv.add_rmsnorm_quantize(x, w, residual=r, want_norm=True)
    few = nv.FP8Matrix(a.codes[:3], a.scale[:3])
    C, c = nv.w8a8_gemm(a, q), nv.w8a8_gemm(few, q)
    A4, B4 = nv.nvfp4_quantize(n), nv.nvfp4_quantize(W)
    D = nv.w4a4_gemm_fused(A4, B4, act=nv.ACT_GELU)
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
nv.check_device_error()
assert torch.equal(C, nv.w8a8_gemm(a, q)) and torch.equal(c, nv.w8a8_gemm(few, q))
assert torch.equal(D, nv.w4a4_gemm_fused(A4, B4, act=nv.ACT_GELU))
"""


def test_first_calls_of_a_process_inside_a_capture(cuda_dev):
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# -------------------------------------------------------------------- the block --
@pytest.mark.parametrize("B,T", [(1, 100), (3, 1)])
def test_block_with_8_bit_projections(cuda_dev, B, T):
    """A GDN block with 8-bit projections, as the calls compose: pre-norm, in_proj,
    gates, scan, output gate, out_proj onto the residual stream, MLP product.  Each
    stage against float64 of the stage before."""
    H, dims = 320, nv.GdnDims(2, 4, 64, 64)
    qkv = 2 * dims.Hk * dims.K + dims.Hv * dims.V
    W_in = nv.fp8_quantize(rand((dims.n_in, H), 71, std=0.05))
    W_out = nv.fp8_quantize(rand((H, dims.Hv * dims.V), 72, std=0.05))
    W_up = nv.fp8_quantize(rand((1000, H), 73, std=0.05))
    g1, g2 = (1 + 0.2 * torch.randn(H, generator=gen(s), device="cuda") for s in (74, 75))
    wn = torch.ones(dims.V, device="cuda")
    A_log, dt = torch.zeros(dims.Hv, device="cuda"), torch.zeros(dims.Hv, device="cuda")
    y, stream = rand((B * T, H), 76), rand((B * T, H), 77, BF16)
    start = stream.clone()
    h, x, _ = nv.add_rmsnorm_quantize(y, g1, residual=stream, h=stream)
    assert torch.equal(h, (y + start.float()).to(BF16))
    check_codes(x, norm_ref(h, g1))
    P = nv.w8a8_gemm(x, W_in, out_dtype=F32)
    check_product(P, value(x), value(W_in), 32, None, nv.ACT_NONE, None)
    pad = torch.zeros((B * T, (dims.n_in + 3) // 4 * 4), device="cuda")
    pad[:, :dims.n_in] = P
    q_hat, k_hat, g, beta = nv.gdn_gates(pad, dims, A_log, dt)
    o, _ = nv.gdn_scan(q_hat, k_hat, pad[:, 2 * dims.Hk * dims.K:], g, beta, B, T, dims)
    o = nv.gdn_output_gate(o, pad[:, qkv:], wn)
    flat = o.view(B * T, -1)
    oq = nv.fp8_quantize(flat)
    check_codes(oq, flat.double())
    before = h.clone()
    nv.w8a8_gemm(oq, W_out, residual=h, out=h)
    check_product(h, value(oq), value(W_out), 32, None, nv.ACT_NONE, before)
    _, x2, _ = nv.add_rmsnorm_quantize(h, g2)
    up = nv.w8a8_gemm(x2, W_up, act=nv.ACT_SILU)
    check_product(up, value(x2), value(W_up), 32, None, nv.ACT_SILU, None)
    done()


def test_block_with_nvfp4_projections(cuda_dev):
    """The same calls around the NVFP4 product: the norm in bf16 with its amax, quantised
    in one pass, an up projection with activation, a down projection in place."""
    n, H, F = 100, 320, 640
    W_up, W_down = nv.nvfp4_quantize(rand((F, H), 81, std=0.05)), nv.nvfp4_quantize(rand((H, F), 82, std=0.05))
    g1 = torch.ones(H, device="cuda")
    y, stream = rand((n, H), 83), rand((n, H), 84)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    h, _, x = nv.add_rmsnorm_quantize(y, g1, residual=stream, h=stream, want_fp8=False, want_norm=True,
                                      amax_word=ws.view(torch.int32))
    xq = nv.nvfp4_quantize(x, mode=nv.QUANT_FROM_AMAX, workspace=ws)
    up = nv.w4a4_gemm_fused(xq, W_up, act=nv.ACT_GELU)
    check_product(up, nvfp4_value(xq), nvfp4_value(W_up), 64, None, nv.ACT_GELU, None)
    uq = nv.nvfp4_quantize(up)
    before = h.clone()
    nv.w4a4_gemm_fused(uq, W_down, residual=h, out=h)
    check_product(h, nvfp4_value(uq), nvfp4_value(W_down), 64, None, nv.ACT_NONE, before)
    done()


# ------------------------------------------------------------------ odd arguments --
def test_one_operand_for_both(cuda_dev):
    q = nv.fp8_quantize(rand((300, 272), 91))
    C = nv.w8a8_gemm(q, q, out_dtype=F32)
    done()
    check_product(C, value(q), value(q), 32, None, nv.ACT_NONE, None)


def test_output_offsets_past_32_bits(cuda_dev):
    """An output of 2.4e9 elements, written in place over its residual."""
    M, N, K = 40000, 60000, 16
    A, B = fp8_pair(M, N, K, 92)
    C = torch.ones((M, N), dtype=BF16, device="cuda")
    nv.w8a8_gemm(A, B, residual=C, out=C)
    done()
    rows = torch.tensor([0, 1, 255, 256, 35790, 35791, 35792, 39936, 39999], device="cuda")
    check_product(C[rows], value(A)[rows], value(B), 32, None, nv.ACT_NONE, torch.ones_like(C[rows]))


def test_a_row_whose_stride_says_nothing(cuda_dev):
    """One row of any stride is a matrix with contiguous rows."""
    K = 256
    base = rand((8, K), 93, BF16).contiguous()
    x = base.as_strided((1, K), (7, 1))
    w = torch.ones(K, device="cuda")
    _, q, n = nv.add_rmsnorm_quantize(x, w, residual=x, want_norm=True)
    C = nv.w8a8_gemm(nv.FP8Matrix(q.codes.as_strided((1, K), (3, 1)), q.scale), nv.fp8_quantize(base))
    done()
    check_codes(q, norm_ref((x.float() + x.float()).to(BF16), w))
    assert C.shape == (1, 8)


def test_refused_tensors(cuda_dev):
    x, w = rand((4, 64), 94), torch.ones(64, device="cuda")
    q = nv.fp8_quantize(x)
    wrong = [
        lambda: nv.fp8_quantize(x.t()),
        lambda: nv.fp8_quantize(x.half()),
        lambda: nv.fp8_quantize(x[0]),
        lambda: nv.fp8_quantize(x.cpu()),
        lambda: nv.fp8_quantize(x, out=nv.FP8Matrix.empty(4, 80)),
        lambda: nv.add_rmsnorm_quantize(x, w[:32]),
        lambda: nv.add_rmsnorm_quantize(x, w.bfloat16()),
        lambda: nv.add_rmsnorm_quantize(x, w, residual=x[:3]),
        lambda: nv.add_rmsnorm_quantize(x, w, h=x),
        lambda: nv.add_rmsnorm_quantize(x, w, residual=x, h=x.bfloat16()),
        lambda: nv.add_rmsnorm_quantize(x, w, norm=x),
        lambda: nv.add_rmsnorm_quantize(x, w, want_norm=True, amax_word=torch.zeros(1)),
        lambda: nv.w8a8_gemm(q, nv.FP8Matrix(q.codes, q.scale[:3])),
        lambda: nv.w8a8_gemm(q, nv.FP8Matrix(q.codes.view(torch.uint8), q.scale)),
        lambda: nv.w8a8_gemm(q, q, bias=torch.ones(5, device="cuda")),
        lambda: nv.w8a8_gemm(q, q, out=torch.empty((4, 5), device="cuda")),
        lambda: nv.w8a8_gemm(q, q, out_dtype=torch.float16),
        lambda: nv.w8a8_gemm(q, q, residual=torch.ones((4, 4), device="cuda").half()),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            print("accepted", i)
    refused = [
        lambda: nv.fp8_quantize(torch.empty((0, 64), device="cuda")),
        lambda: nv.fp8_quantize(rand((4, 40), 95)),
        lambda: nv.fp8_quantize(rand((4, 64 + 4), 95)[:, 2:66]),
        lambda: nv.fp8_quantize(x[:1].expand(4, 64)),
        lambda: nv.add_rmsnorm_quantize(x, w, eps=0.0),
        lambda: nv.add_rmsnorm_quantize(x, w, want_fp8=False),
        lambda: nv.add_rmsnorm_quantize(x, w, amax_word=torch.zeros(1, device="cuda")),
        lambda: nv.w8a8_gemm(q, nv.fp8_quantize(rand((4, 80), 96))),
        lambda: nv.w8a8_gemm(q, q, residual=torch.ones((1, 4), device="cuda").expand(4, 4)),
        lambda: nv.w8a8_gemm(q, q, act=9),
    ]
    for call in refused:
        with pytest.raises((nv.NVFP4Error, ValueError)):
            call()
    done()


def test_refused_nvfp4_operands(cuda_dev):
    A, B = nv.nvfp4_quantize(rand((4, 128), 97)), nv.nvfp4_quantize(rand((200, 128), 98))
    def but(m, **kw):
        return dataclasses.replace(m, **kw)
    wrong = [(but(A, rows=8), B), (but(A, cols=256), but(B, cols=256)), (A, but(B, sf=B.sf[:1024])), (A, but(B, codes=B.codes[:128])),
             (A, but(B, codes=B.codes.t())), (but(A, sf=A.sf.cpu()), B), (but(A, scale=A.scale.cpu()), B),
             (A, but(B, codes=B.codes.cpu(), sf=B.sf.cpu(), scale=B.scale.cpu())), (A, but(B, scale=B.scale.double()))]
    for a, b in wrong:
        with pytest.raises(ValueError):
            nv.w4a4_gemm_fused(a, b)
    done()


@pytest.mark.parametrize("M,N,K", [(1, 33, 64), (1, 129, 4096), (30, 131, 2048), (40, 161, 3200), (60, 97, 320), (100, 225, 2048), (100, 1, 8192),
                                   (500, 33, 192), (2300, 2335, 192), (2300, 2305, 4160)])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_a_warp_partly_past_the_last_row(cuda_dev, M, N, K, out_dtype):
    """N cuts a warp's 32 weight rows, in each kernel and split; bias, residual, activation."""
    bias, r = torch.randn(N, generator=gen(101), device="cuda"), rand((M, N), 102, out_dtype, pad=1)
    A, B = fp8_pair(M, N, K, 103)
    C = nv.w8a8_gemm(A, B, bias=bias, act=nv.ACT_SILU, residual=r, out_dtype=out_dtype)
    done()
    check_product(C, value(A), value(B), 32, bias, nv.ACT_SILU, r)
    A, B = nv.nvfp4_quantize(rand((M, K), 104)), nv.nvfp4_quantize(rand((N, K), 105, std=0.1))
    C = nv.w4a4_gemm_fused(A, B, bias=bias, act=nv.ACT_SILU, residual=r, out_dtype=out_dtype)
    done()
    check_product(C, nvfp4_value(A), nvfp4_value(B), 64, bias, nv.ACT_SILU, r)


@pytest.mark.parametrize("cols", [112, 512, 5120, 16400])
def test_norm_rows_that_overflow_are_nan_throughout(cuda_dev, cols):
    """An infinite or NaN weight, h w past float32, a sum of squares past float32, and
    rows just short of it."""
    x = rand((9, cols), 111)
    x[1:] = 0.0
    x[1, 3] = 1.0
    x[2, 3], x[2, 5] = 1e-30, 1e18        # h w = 1e47 at 5
    x[3] = math.sqrt(3.3e38 / cols)       # the sum of squares just fits
    x[4] = math.sqrt(3.5e38 / cols)       # and just does not, while the mean does
    x[5, 8] = 1.0                         # the infinity's column: 0 w too is NaN
    w = torch.ones(cols, device="cuda")
    w[5] = 1e29
    x[0, 5], x[3, 5], x[4, 5] = 0.0, 0.0, 0.0
    word = torch.zeros(1, device="cuda")
    h, q, n = nv.add_rmsnorm_quantize(x, w, residual=torch.zeros_like(x), want_norm=True, amax_word=word)
    done()
    good, bad = [0, 1, 3, 5, 6, 7, 8], [2, 4]
    assert torch.equal(h, x)
    ref = norm_ref(h[good], w)
    assert torch.all((n[good].double() - ref).abs() <= (2.0 ** -8 + 33 * U) * ref.abs() + 2.0 ** -133)
    check_codes(nv.FP8Matrix(q.codes[good], q.scale[good]), ref)
    assert torch.all(torch.isnan(q.scale[bad])) and torch.all(torch.isnan(q.codes[bad].float()))
    assert torch.all(torch.isnan(n[bad].float())) and torch.all(torch.isnan(word))
    for value in (math.inf, -math.inf, math.nan):
        w[5] = value
        _, q, n = nv.add_rmsnorm_quantize(x, w, want_norm=True)
        done()
        assert torch.all(torch.isnan(q.scale)) and torch.all(torch.isnan(q.codes.float())) and torch.all(torch.isnan(n.float()))
    # a tiny mean square and a large weight: n = 1e-18 3e38 / sqrt(1e-36 + 1e-38) = 2.985e38 still fits
    tiny = torch.full((2, cols), 1e-18, device="cuda")
    w.fill_(1.0)
    w[7] = 3e38
    _, q, n = nv.add_rmsnorm_quantize(tiny, w, eps=1e-38, want_norm=True)
    done()
    ref = norm_ref(tiny, w, 1e-38)
    assert torch.all((n.double() - ref).abs() <= (2.0 ** -8 + 33 * U) * ref.abs())
    check_codes(q, ref)
    # alone in its row it is sqrt(cols) times that, while h w = 3e20
    tiny[1] = 0.0
    tiny[1, 7] = 1e-18
    _, q, n = nv.add_rmsnorm_quantize(tiny, w, eps=1e-38, want_norm=True)
    done()
    assert not torch.isnan(q.scale[0]) and torch.isnan(q.scale[1])
    assert torch.all(torch.isnan(n[1].float())) and torch.all(torch.isnan(q.codes[1].float()))


def test_nvfp4_buffers_made_for_more_rows(cuda_dev):
    """The first rows of larger buffers are a matrix of their own."""
    x, B = rand((70, 256), 106), nv.nvfp4_quantize(rand((300, 256), 107))
    large = nv.NVFP4Matrix.empty(500, 256)
    some = dataclasses.replace(large, rows=70)
    nv.nvfp4_quantize(x, out=some)
    C, want = nv.w4a4_gemm_fused(some, B), nv.w4a4_gemm_fused(nv.nvfp4_quantize(x), B)
    done()
    assert torch.equal(C, want)
