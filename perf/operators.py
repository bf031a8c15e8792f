"""The block operators around a Gated DeltaNet layer: the residual addition with RMS
norm and 8-bit output, the 8-bit row quantiser, and the W8A8 / W4A4 products with
bias, activation and residual in their epilogue.

``run`` computes them in plain torch operations (``own`` false) or through the
library's entry points (``own`` true), from the same state.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
TINY = 2.0 ** -100
EPS = 1e-6
FLOATS = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2, "none": 0}
ACTS = ("none", "silu", "gelu", "relu")
# most work a drawn case may cost: that of the largest listed one of its kind
NORM_MOST = 32768 * 5120
GEMM_MOST = 8192 * 12352 * 5120


def listed():
    return [
        # the pre-norm of a 32768-token prefill: the layer's fp32 y joins a bf16 residual stream
        {"name": "norm_prefill", "op": "norm", "rows": 32768, "cols": 5120, "x": "fp32", "res": "bf16", "want": "fp8"},
        # one token of one sequence: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 5120, "x": "bf16", "res": "bf16", "want": "fp8"},
        # a ragged batch, fp32 residual stream, the norm kept in bf16 for a W4A4 layer too
        {"name": "norm_ragged", "op": "norm", "rows": 1237, "cols": 4112, "x": "bf16", "res": "fp32", "want": "both"},
        # a fused in_proj weight, quantised once when a model is loaded
        {"name": "quant_weight", "op": "quant", "rows": 12352, "cols": 5120, "x": "fp32"},
        # the scan's output before out_proj, an odd number of tokens
        {"name": "quant_odd", "op": "quant", "rows": 1021, "cols": 4096, "x": "bf16"},
        # in_proj of a long prefill: fp32 for the gates and the scan
        {"name": "w8a8_in_proj", "op": "w8a8", "M": 8192, "N": 12352, "K": 5120, "bias": False, "act": "none",
         "res": "none", "out": "fp32"},
        # out_proj of a 4096-token prefill, added onto the residual stream
        {"name": "w8a8_out_proj", "op": "w8a8", "M": 4096, "N": 5120, "K": 4096, "bias": False, "act": "none",
         "res": "bf16", "out": "bf16"},
        # a batch of 64 decoding sequences: bound by the weight's bytes
        {"name": "w8a8_decode", "op": "w8a8", "M": 64, "N": 12352, "K": 5120, "bias": True, "act": "silu",
         "res": "none", "out": "bf16"},
        # one decoding sequence's out_proj
        {"name": "w8a8_token", "op": "w8a8", "M": 1, "N": 5120, "K": 4096, "bias": True, "act": "none",
         "res": "bf16", "out": "bf16"},
        # odd sizes in every direction
        {"name": "w8a8_ragged", "op": "w8a8", "M": 1237, "N": 4099, "K": 1040, "bias": True, "act": "gelu",
         "res": "fp32", "out": "fp32"},
        # NVFP4 out_proj of a 4096-token prefill onto the residual stream
        {"name": "w4a4_out_proj", "op": "w4a4", "M": 4096, "N": 5120, "K": 4096, "bias": False, "act": "none",
         "res": "bf16", "out": "bf16"},
        # NVFP4 batch of 64 decoding sequences with bias and activation
        {"name": "w4a4_decode", "op": "w4a4", "M": 64, "N": 12352, "K": 5120, "bias": True, "act": "silu",
         "res": "none", "out": "bf16"},
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` between low and high, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "quant", "w8a8", "w8a8", "w4a4"))
    if op in ("norm", "quant"):
        cols = _spread(rng, 64, 16384, 16)
        case = {"op": op, "rows": _spread(rng, 1, min(32768, NORM_MOST // cols)), "cols": cols,
                "x": rng.choice(("fp32", "bf16"))}
        if op == "norm":
            case["res"] = rng.choice(("none", "fp32", "bf16"))
            case["want"] = rng.choice(("fp8", "both"))
        return case
    wide = 16 if op == "w8a8" else 64
    K = _spread(rng, 64, 5120, wide)
    N = _spread(rng, 64, 12352)
    M = _spread(rng, 1, max(1, min(8192, GEMM_MOST // (N * K))))
    out = rng.choice(("fp32", "bf16"))
    return {"op": op, "M": M, "N": N, "K": K, "bias": rng.random() < 0.5, "act": rng.choice(ACTS),
            "res": rng.choice(("none", out)), "out": out}


# ------------------------------------------------------------------- inputs --
def _activations(g, rows, cols):
    """Normal values with about one channel in a hundred 50 to 100 times as large."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    hot = torch.rand(cols, generator=g, device=DEV) < 0.01
    return x * torch.where(hot, 50 + 50 * torch.rand(cols, generator=g, device=DEV), torch.ones((), device=DEV))


def _to_fp8(x):
    """E4M3 codes and one fp32 scale a row."""
    S = x.abs().amax(1) / E4M3_MAX
    return (x / S[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), S


def _to_nvfp4(x):
    """Packed E2M1 codes, E4M3 scales of 16 values in atoms of 128 rows x 4 blocks, one fp32 scale."""
    rows, cols = x.shape
    S = x.abs().amax() / (6 * E4M3_MAX)
    blocks = x.view(rows, cols // 16, 16)
    sf = (blocks.abs().amax(2) / (6 * S)).to(torch.float8_e4m3fn)
    y = blocks / (sf.float() * S).clamp_min(1e-30)[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = (torch.bucketize(y.abs(), edges) + 8 * (y < 0)).to(torch.uint8).view(rows, cols // 2, 2)
    codes = code[:, :, 0] | (code[:, :, 1] << 4)
    pad = -rows % 128
    flat = torch.cat([sf.view(torch.uint8), torch.zeros((pad, cols // 16), dtype=torch.uint8, device=x.device)])
    atoms = flat.view((rows + pad) // 128, 4, 32, cols // 64, 4).permute(0, 3, 2, 1, 4)
    return codes.contiguous(), atoms.reshape(-1).contiguous(), S.reshape(1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] in ("norm", "quant"):
        shape = (case["rows"], case["cols"])
        s["X"] = _activations(g, *shape).to(FLOATS[case["x"]])
        if case["op"] == "norm":
            s["R"] = None if case["res"] == "none" else (
                4 * torch.randn(shape, generator=g, device=DEV)).to(FLOATS[case["res"]])
            s["w"] = 1 + 0.3 * torch.randn(case["cols"], generator=g, device=DEV)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    to = _to_fp8 if case["op"] == "w8a8" else _to_nvfp4
    s["A"] = to(_activations(g, M, K))
    s["B"] = to(0.02 * torch.randn((N, K), generator=g, device=DEV))
    s["b"] = 0.5 * torch.randn(N, generator=g, device=DEV) if case["bias"] else None
    s["R"] = None if case["res"] == "none" else (
        4 * torch.randn((M, N), generator=g, device=DEV)).to(FLOATS[case["res"]])
    return s


# --------------------------------------------------------------- plain forms --
def _plain_quant(x):
    amax = x.abs().amax(1)
    S = torch.where(amax < TINY, torch.ones_like(amax), amax / E4M3_MAX)
    y = (x * (1.0 / S)[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn), S


def _plain_norm(s):
    h = s["X"].float()
    if s["R"] is not None:
        h = (h + s["R"].float()).to(s["R"].dtype)
    f = h.float()
    n = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * s["w"]
    codes, S = _plain_quant(n)
    out = {"codes": codes, "scale": S}
    if s["R"] is not None:
        out["h"] = h
    if s["want"] == "both":
        out["n"] = n.to(torch.bfloat16)
    return out


def _act(y, act):
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "relu":
        return torch.where(y > 0, y, torch.zeros_like(y))
    return y


def _nvfp4_values(codes, sf, rows):
    """code * block scale, without the tensor's scale."""
    cols = 2 * codes.shape[1]
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], 2).view(rows, cols // 16, 16)
    lin = sf.view(torch.float8_e4m3fn).float().view(-1, cols // 64, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return (v * lin.reshape(-1, cols // 16, 1)[:rows]).view(rows, cols)


def _plain_gemm(s):
    if s["op"] == "w8a8":
        (a, sa), (b, sb) = s["A"], s["B"]
        y = (a.float() @ b.float().T) * sa[:, None] * sb
    else:
        a, b = (_nvfp4_values(t[0], t[1], rows) for t, rows in ((s["A"], s["M"]), (s["B"], s["N"])))
        y = (a @ b.T) * (s["A"][2] * s["B"][2])
    if s["b"] is not None:
        y = y + s["b"]
    y = _act(y, s["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(FLOATS[s["out"]])


# ------------------------------------------------------------ library's calls --
def _own(s):
    import nvfp4_w4a4_gated_b200 as nv
    if s["op"] == "quant":
        q = nv.fp8_quantize(s["X"])
        return {"codes": q.codes, "scale": q.scale}
    if s["op"] == "norm":
        h, q, n = nv.add_rmsnorm_quantize(s["X"], s["w"], residual=s["R"], eps=EPS, want_norm=s["want"] == "both")
        out = {"codes": q.codes, "scale": q.scale}
        if s["R"] is not None:
            out["h"] = h
        if n is not None:
            out["n"] = n
        return out
    act = getattr(nv, "ACT_" + s["act"].upper())
    if s["op"] == "w8a8":
        A, B = (nv.FP8Matrix(*t) for t in (s["A"], s["B"]))
        return nv.w8a8_gemm(A, B, bias=s["b"], act=act, residual=s["R"], out_dtype=FLOATS[s["out"]])
    A, B = (nv.NVFP4Matrix(*t, rows, s["K"]) for t, rows in ((s["A"], s["M"]), (s["B"], s["N"])))
    return nv.w4a4_gemm_fused(A, B, bias=s["b"], act=act, residual=s["R"], out_dtype=FLOATS[s["out"]])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm":
        return _plain_norm(state)
    if state["op"] == "quant":
        codes, S = _plain_quant(state["X"].float())
        return {"codes": codes, "scale": S}
    return _plain_gemm(state)


def work(case):
    if case["op"] in ("norm", "quant"):
        size = case["rows"] * case["cols"]
        per = BYTES[case["x"]] + 1
        flops = 3 * size
        if case["op"] == "norm":
            per += 2 * BYTES[case["res"]] + (2 if case["want"] == "both" else 0)
            flops = 7 * size
        return {"bytes": size * per + 4 * case["rows"] + 4 * case["cols"] * (case["op"] == "norm"), "flops": flops}
    M, N, K = case["M"], case["N"], case["K"]
    per = 1.0 if case["op"] == "w8a8" else 0.5 + 1 / 16
    data = (M + N) * K * per + M * N * (BYTES[case["out"]] + BYTES[case["res"]])
    return {"bytes": data + 4 * N * case["bias"] + (4 * (M + N) if case["op"] == "w8a8" else 8), "flops": 2 * M * N * K}


# -------------------------------------------------------------------- 64 bits --
def _exact_rows(n):
    """Values over the row's scale before their rounding to 8 bits, and the scale."""
    top = n.abs().max(dim=1).values
    S = torch.where(top < TINY, torch.ones_like(top), top / E4M3_MAX)
    return n / S.unsqueeze(1), S


def _exact_nvfp4(t, rows, K):
    packed, sf, S = t
    low, high = packed.long() % 16, packed.long() // 16
    idx = torch.stack((low, high), dim=-1).flatten(1)
    mag, half = (idx % 8).double(), idx % 8
    value = torch.where(half < 4, mag / 2, torch.where(half < 6, mag - 2, 2 * mag - 8))
    value = torch.where(idx >= 8, -value, value)
    r = torch.arange(rows, device=packed.device)[:, None]
    j = torch.arange(K // 16, device=packed.device)[None, :]
    at = ((r // 128) * (K // 64) + j // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + j % 4
    scale = sf[at].view(torch.float8_e4m3fn).double()
    return value * scale.repeat_interleave(16, dim=1) * S.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        codes, S = _exact_rows(s["X"].double())
        return {"codes": codes, "scale": S}
    if case["op"] == "norm":
        h = s["X"].double()
        if s["R"] is not None:
            # the sum is rounded once, to the residual stream's type, and that is what is normalised
            h = h + s["R"].double()
            kept = h.to(s["R"].dtype).double()
        else:
            kept = h
        rms = torch.sqrt(kept.square().sum(1, keepdim=True) / case["cols"] + EPS)
        n = s["w"].double() * kept / rms
        codes, S = _exact_rows(n)
        out = {"codes": codes, "scale": S}
        if s["R"] is not None:
            out["h"] = h
        if case["want"] == "both":
            out["n"] = n
        return out
    if case["op"] == "w8a8":
        a, b = (q.double() * sc.double().unsqueeze(1) for q, sc in (s["A"], s["B"]))
    else:
        a, b = _exact_nvfp4(s["A"], case["M"], case["K"]), _exact_nvfp4(s["B"], case["N"], case["K"])
    y = torch.matmul(a, b.t())
    if s["b"] is not None:
        y += s["b"].double()
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif case["act"] == "gelu":
        y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
    elif case["act"] == "relu":
        y = y.clamp(min=0)
    return y if s["R"] is None else y + s["R"].double()
