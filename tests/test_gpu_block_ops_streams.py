"""Calls with ``stream=``: their new tensors are ordered with that stream.

A sleep on the current stream keeps work on a freed block pending while the call on the
other stream runs, so results that shared the block would be overwritten by it."""
import pytest
import torch

import nvfp4_w4a4_gated_b200 as nv

pytestmark = pytest.mark.gpu

SLEEP = 200_000_000   # clocks, about 0.1 s


def calls():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((1000, 4096), generator=g, device="cuda")
    r = torch.randn((1000, 4096), generator=g, device="cuda").bfloat16()
    w = torch.randn(4096, generator=g, device="cuda")
    A, B = nv.fp8_quantize(x), nv.fp8_quantize(x + 1)
    A4, B4 = nv.nvfp4_quantize(x), nv.nvfp4_quantize(x + 1)

    def quantize(**kw):
        q = nv.fp8_quantize(x, **kw)
        return q.codes, q.scale

    def norm(**kw):
        h, q, n = nv.add_rmsnorm_quantize(x, w, residual=r, want_norm=True, **kw)
        return h, q.codes, q.scale, n

    def nvfp4(**kw):
        q = nv.nvfp4_quantize(x, **kw)
        return q.codes, q.sf, q.scale

    dims, T = nv.GdnDims(2, 4, 128, 128), 256
    proj = torch.randn((T, dims.n_in), generator=g, device="cuda")
    A_log, dt = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    gates = nv.gdn_gates(proj, dims, A_log, dt)
    v = proj[:, 512:]

    def scan(**kw):   # with a workspace that is dropped when the call returns
        return nv.gdn_scan(gates[0], gates[1], v, gates[2], gates[3], 1, T, dims, algo=nv.SCAN_CHUNKED, **kw)[:1]

    return {"nvfp4": nvfp4, "gemm": lambda **kw: (nv.w4a4_gemm(A4, B4, **kw),), "scan": scan,
            "gates": lambda **kw: nv.gdn_gates(proj, dims, A_log, dt, **kw), "quantize": quantize, "norm": norm, "w8a8": lambda **kw: (nv.w8a8_gemm(A, B, **kw),),
            "w4a4": lambda **kw: (nv.w4a4_gemm_fused(A4, B4, **kw),)}


def equal(a, b):
    return all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b, strict=True))


@pytest.mark.parametrize("name", ["quantize", "norm", "w8a8", "w4a4", "nvfp4", "gemm", "scan", "gates"])
def test_memory_freed_on_the_current_stream(cuda_dev, name):
    call = calls()[name]
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream=s)   # first launches are over
    torch.cuda.synchronize()
    busy = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(SLEEP)
    for t in busy:
        t.view(torch.uint8).fill_(0x35)
    at = {t.data_ptr() for t in busy}
    del busy, t   # free for this stream's next tensors, with the fills still to run
    assert {torch.empty_like(t).data_ptr() for t in want} & at
    got = call(stream=s)
    torch.cuda.synchronize()
    nv.check_device_error()
    assert equal(got, want)


@pytest.mark.parametrize("name", ["quantize", "norm", "w8a8", "w4a4", "nvfp4", "gemm", "scan", "gates"])
def test_result_read_on_the_current_stream_and_dropped(cuda_dev, name):
    call = calls()[name]
    want = call()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(SLEEP)
    kept = [t.clone() for t in got]
    del got
    with torch.cuda.stream(s):   # the stream's next tensors of these sizes
        after = [torch.empty_like(t) for t in want]
        for t in after:
            t.view(torch.uint8).fill_(0x35)
    torch.cuda.synchronize()
    nv.check_device_error()
    assert equal(kept, want)


class Recorder:
    """The library, with the workspace of each nvfp4_quantize noted."""

    def __init__(self, real):
        self.real, self.seen = real, []

    def __getattr__(self, name):
        return getattr(self.real, name)

    def nvfp4_quantize(self, *args):
        self.seen.append(args[7].value)
        return self.real.nvfp4_quantize(*args)


def test_quantisers_on_two_streams_or_in_two_graphs_share_no_amax_word(cuda_dev, monkeypatch):
    x = torch.randn((300, 512), device="cuda")
    want = nv.nvfp4_quantize(x)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    lib = Recorder(nv.lib())
    monkeypatch.setattr(nv, "_lib", lib)
    got = [nv.nvfp4_quantize(x, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert len(set(lib.seen)) == 2
    lib.seen.clear()
    graphs = []
    for _ in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(nv.nvfp4_quantize(x))
        graphs.append(g)
    assert len(set(lib.seen)) == 2
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    nv.check_device_error()
    for q in got:
        assert equal((q.codes, q.sf, q.scale), (want.codes, want.sf, want.scale))
