"""Sums over long K of the 8-bit product: the tensor cores' float32 accumulation does not
round to nearest, and its error grows with the number of steps, so k-tiles of 128 are
summed in chains of at most 30 for a float32 result, 512 for a bf16 one.

Bounds.  One chain of K values is off by about 1.9e-10 K of the result's norm (activations
with hot channels, where a few terms carry most of the sum): 3840 values, 30 tiles, stay
within 7.5e-7, and the errors of several chains add up like their sums do, as squares.  One
chain of 5120 is off by 9.6e-7, two chains of 11520 / 2 by 1.1e-6, so a product that lost
its chains fails.  Element by element the bounds are those of test_gpu_block_ops.py."""
import pytest
import torch

import nvfp4_w4a4_gated_b200 as nv
from test_gpu_block_ops import BF16, F32, check_product, done, gen, rand, value

pytestmark = pytest.mark.gpu

NORM = 7.5e-7


def operand(rows, K, seed, std=1.0, hot=False):
    """E4M3 rows of any length (the quantiser's rows end at 32768)."""
    x = std * torch.randn((rows, K), generator=gen(seed), device="cuda")
    if hot:
        x *= torch.where(torch.rand(K, generator=gen(seed + 1), device="cuda") < 0.01, 75.0, 1.0)
    scale = x.abs().amax(1) / 448
    return nv.FP8Matrix((x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale)


# CTA pairs (whole and cut tiles), then the split-K kernel: K in 1 (which becomes 2), 2, 3 and 4
PAIRS = [(1024, 4096), (1030, 4099), (257, 12352)]
SPLITS = [(1, 5120), (16, 515), (20, 40000), (40, 12352), (60, 5120), (64, 300), (100, 20000), (128, 2000), (200, 7500)]


@pytest.mark.parametrize("M,N", PAIRS + SPLITS)
@pytest.mark.parametrize("K", [5120, 7680, 11520, 17408, 28672])
def test_float32_sums_by_norm(cuda_dev, M, N, K):
    if (M, N, K) == (20, 40000, 28672):
        N = 20000
    A, B = operand(M, K, 1, hot=True), operand(N, K, 3, std=0.02)
    C = nv.w8a8_gemm(A, B, out_dtype=F32)
    done()
    y = value(A) @ value(B).T
    off = float((C.double() - y).norm() / y.norm())
    assert off <= NORM, off


@pytest.mark.parametrize("M,N,K", [(1030, 4099, 11600), (2300, 2311, 8208), (1, 131, 16400), (30, 1027, 30992), (64, 515, 12304),
                                   (50, 6000, 23056), (100, 5003, 11664), (128, 12352, 8016), (300, 333, 8000), (20, 40000, 7696)])
@pytest.mark.parametrize("act,res", [(nv.ACT_NONE, None), (nv.ACT_SILU, BF16)])
def test_float32_sums_by_element(cuda_dev, M, N, K, act, res):
    A, B = operand(M, K, 5), operand(N, K, 7, std=0.1)
    bias = torch.randn(N, generator=gen(9), device="cuda")
    r = None if res is None else rand((M, N), 10, res, pad=1)
    C = nv.w8a8_gemm(A, B, bias=bias, act=act, residual=r, out_dtype=F32)
    done()
    check_product(C, value(A), value(B), 32, bias, act, r)
    assert torch.equal(C, nv.w8a8_gemm(A, B, bias=bias, act=act, residual=r, out_dtype=F32))
    wide = rand((M + 1, N + 3), 11)
    before = wide.clone()
    stream = wide[:M, 2:2 + N]
    nv.w8a8_gemm(A, B, bias=bias, act=act, residual=stream, out=stream)
    done()
    check_product(stream, value(A), value(B), 32, bias, act, before[:M, 2:2 + N])
    wide[:M, 2:2 + N] = before[:M, 2:2 + N]
    assert torch.equal(wide, before)


@pytest.mark.parametrize("M,N,K", [(1030, 2100, 66048), (300, 200, 65552), (20, 300, 140000), (3, 131, 300000)])
def test_bf16_sums_in_chains(cuda_dev, M, N, K):
    A, B = operand(M, K, 13), operand(N, K, 15, std=0.1)
    C = nv.w8a8_gemm(A, B)
    done()
    assert C.dtype == BF16
    check_product(C, value(A), value(B), 32, None, nv.ACT_NONE, None)
    assert torch.equal(C, nv.w8a8_gemm(A, B))
