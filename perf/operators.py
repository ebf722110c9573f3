"""The 8-bit (e4m3) block-scaled operators: what is measured of them, and their plain forms.

Activations are held as e4m3 codes q [n][d] with one fp32 scale per run of 128 columns of a row,
[n][ceil(d / 128)]; weights as codes [out][in] with one fp32 scale per block of 128 x 128,
[ceil(out / 128)][ceil(in / 128)]. A value is code * scale, and a block's scale is
max(max |v|, 2^-100) / 448, so its largest value takes the largest code.

  norm    add_rmsnorm_fp8: x' = x + residual, then the RMSNorm of x' in e4m3
  quant   quantize_fp8: activations in e4m3
  gemm    gemm_fp8: y = W x
  gate_up gemm_fp8_gate_up_silu: h = silu(W_gate x) * (W_up x) in e4m3
  dequant dequant_fp8: packed 4-bit weights (a bfloat16 scale and bias per 64) laid out in e4m3

With `own` false, run() computes them with elementary torch operations in 32 bits.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 128
TOP = 448.0
FLOOR = 2.0 ** -100
EPS = 1e-6


def listed():
    return [
        # one decoded token's residual stream, fp32 as the decode path keeps it: latency
        {"name": "norm_1x4096", "op": "norm", "nb": 1, "dim": 4096, "x": "f32", "res": "f32"},
        # a long prompt's tokens in one call
        {"name": "norm_8192x4096", "op": "norm", "nb": 8192, "dim": 4096, "x": "bf16", "res": "bf16"},
        # an expert's inner width for the tokens of one decode step: latency
        {"name": "quant_16x640", "op": "quant", "nb": 16, "dim": 640, "x": "f16"},
        # a prompt's inner activations
        {"name": "quant_4096x12288", "op": "quant", "nb": 4096, "dim": 12288, "x": "bf16"},
        # one token through the widest layer: the weights are the traffic
        {"name": "gemm_1_4096_12288", "op": "gemm", "nb": 1, "in": 4096, "out": 12288, "y": "f32"},
        # a decode step of several sequences through the long-row layer
        {"name": "gemm_13_12288_4096", "op": "gemm", "nb": 13, "in": 12288, "out": 4096, "y": "f32"},
        # a short prompt through an expert-sized layer with a ragged end
        {"name": "gemm_333_656_2050", "op": "gemm", "nb": 333, "in": 656, "out": 2050, "y": "f16"},
        # a long prompt: a contraction
        {"name": "gemm_8192_4096_12288", "op": "gemm", "nb": 8192, "in": 4096, "out": 12288, "y": "bf16"},
        # the gated half of a layer in a decode step of several sequences
        {"name": "gate_up_8_4096_6144", "op": "gate_up", "nb": 8, "in": 4096, "inter": 6144},
        # the same for a prompt
        {"name": "gate_up_4096_4096_6144", "op": "gate_up", "nb": 4096, "in": 4096, "inter": 6144},
        # one expert's gate and up rows laid out in 8 bits
        {"name": "dequant_1280x2048", "op": "dequant", "out": 1280, "in": 2048},
        # the output head's rows
        {"name": "dequant_151936x4096", "op": "dequant", "out": 151936, "in": 4096},
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "quant", "gemm", "gemm", "gemm", "gate_up", "gate_up", "dequant"))
    if op in ("norm", "quant"):
        c = {"op": op, "nb": _log(rng, 1, 16384), "dim": 16 * _log(rng, 4, 1024), "x": rng.choice(sorted(TYPES))}
        while c["nb"] * c["dim"] > 4096 * 12288:
            c["nb"] = max(1, c["nb"] // 2)
        if op == "norm":
            c["res"] = rng.choice(["none"] + sorted(TYPES))
        return c
    if op == "dequant":
        c = {"op": op, "out": _log(rng, 1, 151936), "in": 64 * _log(rng, 1, 256)}
        while c["out"] * c["in"] > 151936 * 4096:
            c["out"] = max(1, c["out"] // 2)
        return c
    c = {"op": op, "nb": _log(rng, 1, 8192), "in": 16 * _log(rng, 4, 1024)}
    if op == "gemm":
        c["out"] = _log(rng, 1, 32768)
        c["y"] = rng.choice(sorted(TYPES))
        rows = "out"
        most = 8192 * 12288 * 4096
    else:
        c["inter"] = BLOCK * _log(rng, 1, 96)
        rows = "inter"
        most = 8192 * 6144 * 4096
    while c["nb"] * c["in"] * c[rows] > most:
        c["nb"] = max(1, c["nb"] // 2)
    return c


# ---- inputs ----------------------------------------------------------------------------------


def _spread(gen, rows, cols, std):
    """fp32 values whose columns differ in size, with a few outlier columns, as a network's
    activations do."""
    size = torch.exp(0.3 * torch.randn(cols, device="cuda", generator=gen))
    size[:: 257] *= 20.0
    return torch.randn(rows, cols, device="cuda", generator=gen) * size * std


def _rows_in_8_bits(v):
    """Codes and scales per 128 columns of a row, in the type's own arithmetic."""
    n, d = v.shape
    kb = -(-d // BLOCK)
    p = torch.nn.functional.pad(v, (0, kb * BLOCK - d)).view(n, kb, BLOCK)
    scale = p.abs().amax(dim=2).clamp_min(FLOOR) / TOP
    q = (p / scale.unsqueeze(2)).to(F8)
    return q.view(n, kb * BLOCK)[:, :d].contiguous(), scale


def _blocks_in_8_bits(v):
    """Codes and scales per block of 128 x 128."""
    n, d = v.shape
    nbk, kb = -(-n // BLOCK), -(-d // BLOCK)
    p = torch.nn.functional.pad(v, (0, kb * BLOCK - d, 0, nbk * BLOCK - n)).view(nbk, BLOCK, kb, BLOCK)
    scale = p.abs().amax(dim=(1, 3)).clamp_min(FLOOR) / TOP
    q = (p / scale.view(nbk, 1, kb, 1)).to(F8)
    return q.view(nbk * BLOCK, kb * BLOCK)[:n, :d].contiguous(), scale


def _weights(gen, rows, cols):
    """Weights N(0, 1 / sqrt(cols)) whose rows differ in size, in 8-bit blocks."""
    size = torch.exp(0.5 * torch.randn(rows, 1, device="cuda", generator=gen))
    return _blocks_in_8_bits(torch.randn(rows, cols, device="cuda", generator=gen) * size / math.sqrt(cols))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"op": case["op"]}
    if case["op"] in ("norm", "quant"):
        nb, dim = case["nb"], case["dim"]
        st["x"] = _spread(gen, nb, dim, 0.5).to(TYPES[case["x"]])
        if case["op"] == "norm":
            st["w"] = (1.0 + 0.05 * torch.randn(dim, device="cuda", generator=gen)).to(torch.bfloat16)
            st["res"] = None
            if case["res"] != "none":
                st["res"] = _spread(gen, nb, dim, 2.0).to(TYPES[case["res"]])
    elif case["op"] in ("gemm", "gate_up"):
        rows = case["out"] if case["op"] == "gemm" else 2 * case["inter"]
        st["w"], st["ws"] = _weights(gen, rows, case["in"])
        st["x"], st["xs"] = _rows_in_8_bits(_spread(gen, case["nb"], case["in"], 1.0))
        st["y"] = TYPES[case["y"]] if case["op"] == "gemm" else None
    else:
        rows, cols = case["out"], case["in"]
        st["w"] = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
        st["s"] = (0.02 * torch.randn(rows, cols // 64, device="cuda", generator=gen)).abs().to(torch.bfloat16)
        st["b"] = (-0.08 * torch.randn(rows, cols // 64, device="cuda", generator=gen)).to(torch.bfloat16)
    return st


# ---- one pass ----------------------------------------------------------------------------------


def _run_own(st):
    import affine_q4_dequant_gb300 as q4a

    if st["op"] == "norm":
        q, scale, x_new = q4a.add_rmsnorm_fp8(st["x"], st["w"], residual=st["res"], eps=EPS)
        return {"q": q, "scale": scale, "x_new": x_new}
    if st["op"] == "quant":
        q, scale = q4a.quantize_fp8(st["x"])
        return {"q": q, "scale": scale}
    if st["op"] == "gemm":
        return {"y": q4a.gemm_fp8(st["w"], st["ws"], st["x"], st["xs"], out_dtype=st["y"])}
    if st["op"] == "gate_up":
        q, scale = q4a.gemm_fp8_gate_up_silu(st["w"], st["ws"], st["x"], st["xs"])
        return {"q": q, "scale": scale}
    q, scale = q4a.dequant_fp8(st["w"], st["s"], st["b"])
    return {"q": q, "scale": scale}


def _values_of_rows(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK, dim=1)[:, : q.shape[1]]


def _values_of_blocks(q, scale):
    by_row = scale.repeat_interleave(BLOCK, dim=0)[: q.shape[0]]
    return q.float() * by_row.repeat_interleave(BLOCK, dim=1)[:, : q.shape[1]]


def run(state):
    st = state
    if own:
        return _run_own(st)
    if st["op"] == "norm":
        v, x_new = st["x"].float(), None
        if st["res"] is not None:
            x_new = (v + st["res"].float()).to(st["res"].dtype)
            v = x_new.float()
        n = v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS) * st["w"].float()
        q, scale = _rows_in_8_bits(n)
        return {"q": q, "scale": scale, "x_new": x_new}
    if st["op"] == "quant":
        q, scale = _rows_in_8_bits(st["x"].float())
        return {"q": q, "scale": scale}
    if st["op"] == "gemm":
        y = _values_of_rows(st["x"], st["xs"]) @ _values_of_blocks(st["w"], st["ws"]).t()
        return {"y": y.to(st["y"])}
    if st["op"] == "gate_up":
        gu = _values_of_rows(st["x"], st["xs"]) @ _values_of_blocks(st["w"], st["ws"]).t()
        gate, up = gu.chunk(2, dim=1)
        q, scale = _rows_in_8_bits(gate / (1.0 + torch.exp(-gate)) * up)
        return {"q": q, "scale": scale}
    codes = torch.stack((st["w"] & 15, st["w"] >> 4), dim=2).view(st["w"].shape[0], -1, 64).float()
    v = codes * st["s"].float().unsqueeze(2) + st["b"].float().unsqueeze(2)
    q, scale = _blocks_in_8_bits(v.view(codes.shape[0], -1))
    return {"q": q, "scale": scale}


# ---- in 64 bits --------------------------------------------------------------------------------


def _exact_product(st):
    """W x block by block in 64 bits: the codes' product of a block, then its two scales."""
    x, w = st["x"], st["w"]
    y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    row_block = torch.arange(w.shape[0], device="cuda") // BLOCK
    for k in range(st["xs"].shape[1]):
        at = slice(k * BLOCK, min((k + 1) * BLOCK, x.shape[1]))
        part = x[:, at].double() @ w[:, at].double().t()
        part *= st["xs"][:, k].double().unsqueeze(1)
        part *= st["ws"][row_block, k].double().unsqueeze(0)
        y += part
    return y


def _exact_rows(v):
    """What the codes of the rows of v stand for before they are rounded, and the scales."""
    scales, codes = [], []
    for part in v.split(BLOCK, dim=1):
        top = part.abs().max(dim=1, keepdim=True).values
        scale = torch.where(top > FLOOR, top, torch.full_like(top, FLOOR)) / TOP
        scales.append(scale)
        codes.append(part / scale)
    return torch.cat(codes, dim=1), torch.cat(scales, dim=1)


def exact(case, seed):
    """The operators in 64 bits. Codes are given as the numbers that they round."""
    st = prepare(case, seed)
    if st["op"] == "norm":
        v, x_new = st["x"].double(), None
        if st["res"] is not None:
            x_new = v + st["res"].double()
            v = x_new.to(st["res"].dtype).double()   # the norm reads the stream as it is stored
        root = torch.sqrt((v * v).sum(dim=1, keepdim=True) / v.shape[1] + EPS)
        q, scale = _exact_rows(v / root * st["w"].double())
        return {"q": q, "scale": scale, "x_new": x_new}
    if st["op"] == "quant":
        q, scale = _exact_rows(st["x"].double())
        return {"q": q, "scale": scale}
    if st["op"] == "gemm":
        return {"y": _exact_product(st)}
    if st["op"] == "gate_up":
        gu = _exact_product(st)
        half = gu.shape[1] // 2
        q, scale = _exact_rows(gu[:, :half] * torch.sigmoid(gu[:, :half]) * gu[:, half:])
        return {"q": q, "scale": scale}
    rows, cols = case["out"], case["in"]
    q = torch.empty(rows, cols, dtype=torch.float64, device="cuda")
    scale = torch.empty(-(-rows // BLOCK), -(-cols // BLOCK), dtype=torch.float64, device="cuda")
    for r in range(scale.shape[0]):
        at = slice(r * BLOCK, min((r + 1) * BLOCK, rows))
        s, b = st["s"][at].double(), st["b"][at].double()
        v = torch.empty(s.shape[0], cols, dtype=torch.float64, device="cuda")
        v[:, 0::2] = (st["w"][at] % 16).double()
        v[:, 1::2] = (st["w"][at] // 16).double()
        v *= s.repeat_interleave(64, dim=1)
        v += b.repeat_interleave(64, dim=1)
        pad = torch.nn.functional.pad(v, (0, scale.shape[1] * BLOCK - cols))
        top = pad.abs().view(v.shape[0], -1, BLOCK).amax(dim=(0, 2)).clamp_min(FLOOR)
        scale[r] = top / TOP
        q[at] = v / scale[r].repeat_interleave(BLOCK)[:cols]
    return {"q": q, "scale": scale}


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    size = {"f32": 4, "f16": 2, "bf16": 2, "none": 0}
    op = case["op"]
    if op in ("norm", "quant"):
        nb, dim = case["nb"], case["dim"]
        n = nb * dim * (size[case["x"]] + 1) + 4 * nb * -(-dim // BLOCK)
        if op == "norm":
            n += 2 * nb * dim * size[case["res"]] + 2 * dim
        return {"bytes": n, "flops": nb * dim * (8 if op == "norm" else 3)}
    if op == "dequant":
        rows, cols = case["out"], case["in"]
        n = rows * cols // 2 + rows * cols // 16 + rows * cols + 4 * -(-rows // BLOCK) * -(-cols // BLOCK)
        return {"bytes": n, "flops": 4 * rows * cols}
    rows = case["out"] if op == "gemm" else 2 * case["inter"]
    nb, cols = case["nb"], case["in"]
    kb = -(-cols // BLOCK)
    n = rows * cols + nb * cols + 4 * kb * (nb + -(-rows // BLOCK))
    n += nb * rows * size[case["y"]] if op == "gemm" else nb * case["inter"] + 4 * nb * (case["inter"] // BLOCK)
    return {"bytes": n, "flops": 2 * nb * rows * cols}
