"""The bounded-wait failure path on the GPU, made to run out on purpose: one
thread waits on a barrier nothing arrives on, with a ~2 ms budget.  The host
must read NVFP4_ERR_TIMEOUT from nvfp4_check_device_error, the record must be
cleared by that check, and the context must stay usable.  No fault, no hang."""
import pytest
import torch

import nvfp4_w4a4_gated_b200 as nv

pytestmark = pytest.mark.gpu


def test_bounded_wait_expiry_is_reported_and_cleared(cuda_dev):
    nv.check_device_error()                 # start from a clean record
    nv.selftest_wait_timeout(1 << 22)
    with pytest.raises(nv.NVFP4Error) as ei:
        nv.check_device_error()
    assert ei.value.status == 5 and "bounded wait" in str(ei.value)
    nv.check_device_error()                 # the check cleared the record
    # the context still works: a quantisation runs and checks clean
    x = torch.randn((128, 256), device="cuda").to(torch.bfloat16)
    q = nv.nvfp4_quantize(x)
    torch.cuda.synchronize()
    nv.check_device_error()
    assert float(q.scale.item()) > 0


@pytest.mark.parametrize("M,N,K", [(1, 300, 2048), (64, 300, 1552), (128, 40, 2000), (20, 12000, 1024)])
def test_a_split_product_whose_wait_expired_stores_nothing(cuda_dev, M, N, K):
    """One CTA of each cluster gets no operands (K in 4, 3, 3 and 2).  The others, whose sums are
    complete, must not add what it has; the residual that is the output stays as it was."""
    nv.check_device_error()
    A, B = (nv.fp8_quantize(torch.randn((rows, K), device="cuda")) for rows in (M, N))
    stream = torch.randn((M, N), device="cuda")
    before = stream.clone()
    nv.selftest_split_expiry(A, B, residual=stream, out=stream)
    with pytest.raises(nv.NVFP4Error) as ei:
        nv.check_device_error()
    assert ei.value.status == 5
    assert torch.equal(stream, before)
    nv.w8a8_gemm(A, B, residual=stream, out=stream)   # the context still works
    nv.check_device_error()
    want = (A.codes.float() * A.scale[:, None]).double() @ (B.codes.float() * B.scale[:, None]).double().T + before.double()
    assert torch.allclose(stream.double(), want, rtol=1e-4, atol=1e-2)


@pytest.mark.parametrize("M,N,K", [(8, 5120, 128), (4096, 5120, 512)])
def test_the_split_selftest_is_refused_where_nothing_is_split(cuda_dev, M, N, K):
    A, B = (nv.fp8_quantize(torch.randn((rows, K), device="cuda")) for rows in (M, N))
    with pytest.raises(nv.NVFP4Error) as ei:
        nv.selftest_split_expiry(A, B)
    assert ei.value.status == 2
    nv.check_device_error()
