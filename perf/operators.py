"""The 8-bit projection path of a linear-attention layer, as measured work:

  add_rms_norm_i8  h = x + residual, rounded to the residual's type; RMS norm
                   of h with a weight; the row in 8-bit integers with one scale
  quantize_i8      rows in 8-bit integers with one scale a row (activations by
                   token, weights by output channel)
  linear_i8        y = (x w^T) * x_scale[m] * w_scale[n], 8-bit integers in,
                   exact integer sums, fp32 or bf16 out

Rows are quantised symmetrically: with m the largest |a| of the row,
q = round-half-even(127 a / m) and scale = m / 127 (divided by the row's
root mean square where a norm stands before it; a = fp32(h * weight)). The
integers are whole numbers that the definition decides exactly, so they are
returned as such, with the scales beside them.

With `own` false every case runs as elementary torch operations; with `own`
true through this repository's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}

# Largest work of a drawn case of each operator: the largest listed one's.
MOST_MACS = 16384 * 8192 * 2048
MOST_LINEAR_BYTES = 16384 * 8192 * 4
MOST_ROW_ELEMENTS = 16384 * 4096


def listed():
    return [
        # One sequence decodes one token through the qkv projection: the
        # weights' 16 MB are all the work, latency counts.
        {"name": "linear_decode_1", "op": "linear", "M": 1, "N": 8192, "K": 2048, "out": "fp32"},
        # 64 sequences decode one token through the output-gate projection.
        {"name": "linear_decode_64", "op": "linear", "M": 64, "N": 4096, "K": 2048, "out": "fp32"},
        # The beta / decay projection has 64 outputs, here for the two-token
        # verification of 128 sequences: little work, few output tiles.
        {"name": "linear_thin_256", "op": "linear", "M": 256, "N": 64, "K": 2048, "out": "fp32"},
        # A ragged prompt through a projection whose sizes fit no tile.
        {"name": "linear_ragged_777", "op": "linear", "M": 777, "N": 2050, "K": 1040, "out": "bf16"},
        # The output projection over one prompt of 4096 tokens, bf16 out.
        {"name": "linear_out_4096", "op": "linear", "M": 4096, "N": 2048, "K": 4096, "out": "bf16"},
        # The qkv projection over 4 prompts of 4096 tokens, the largest.
        {"name": "linear_qkv_16384", "op": "linear", "M": 16384, "N": 8192, "K": 2048, "out": "fp32"},
        # Before a layer's projections, one token: latency only.
        {"name": "norm_decode_1", "op": "norm", "M": 1, "D": 2048, "x": "fp32", "residual": "bf16"},
        # The first layer of a stack has no residual yet; a ragged batch.
        {"name": "norm_ragged_509", "op": "norm", "M": 509, "D": 4112, "x": "bf16", "residual": "none"},
        # Between two layers over 4 prompts of 4096 tokens, fp32 stream.
        {"name": "norm_prefill_16384", "op": "norm", "M": 16384, "D": 2048, "x": "fp32", "residual": "fp32"},
        # The recurrent layer's output for 64 decoded sequences (32 heads of
        # 128), before the output projection.
        {"name": "quantize_decode_64", "op": "quantize", "M": 64, "D": 4096, "x": "fp32"},
        # Weights of the qkv projection, one scale an output channel.
        {"name": "quantize_weights_8192", "op": "quantize", "M": 8192, "D": 2048, "x": "bf16"},
        # The recurrent layer's output over 4 prompts of 4096 tokens.
        {"name": "quantize_prefill_16384", "op": "quantize", "M": 16384, "D": 4096, "x": "fp32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "quantize"])
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 16384), _log(rng, 1, 8192), 16 * _log(rng, 1, 512)
            if M * N * K <= MOST_MACS and M * K + N * K + 4 * M * N <= MOST_LINEAR_BYTES:
                return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["fp32", "bf16"])}
    while True:
        M, D = _log(rng, 1, 16384), 16 * _log(rng, 1, 1024)
        if M * D <= MOST_ROW_ELEMENTS // 2:
            break
    x = rng.choice(["fp32", "bf16"])
    if op == "quantize":
        return {"op": op, "M": M, "D": D, "x": x}
    return {"op": op, "M": M, "D": D, "x": x, "residual": rng.choice(["none", "fp32", "bf16"])}


def _activations(g, M, D, device):
    """Rows of a residual stream: normal, token by token of another size, a
    few channels far larger than the rest."""
    x = torch.randn(M, D, generator=g, device=device)
    x *= torch.exp(0.3 * torch.randn(M, 1, generator=g, device=device))
    big = torch.rand(1, D, generator=g, device=device) < 0.01
    return torch.where(big, 8.0 * x, x)


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=device).manual_seed(seed)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s = {"op": "linear", "out": TYPES[case["out"]]}
        for name, rows in (("x", M), ("w", N)):
            a = torch.randn(rows, K, generator=g, device=device)
            m = a.abs().amax(1, keepdim=True)
            s[name] = torch.round(a * (127.0 / m)).clamp_(-127, 127).to(torch.int8)
            s[name + "_scale"] = (m[:, 0] / 127.0 / (math.sqrt(K) if name == "w" else 1.0)).contiguous()
        s["y"] = torch.empty(M, N, dtype=s["out"], device=device)
        return s
    M, D = case["M"], case["D"]
    s = {"op": case["op"], "x": _activations(g, M, D, device).to(TYPES[case["x"]])}
    s["q"] = torch.empty(M, D, dtype=torch.int8, device=device)
    s["scale"] = torch.empty(M, dtype=torch.float32, device=device)
    if case["op"] == "norm":
        s["weight"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=device)
        s["residual"] = s["residual_out"] = None
        if case["residual"] != "none":
            t = TYPES[case["residual"]]
            s["residual"] = (4.0 * _activations(g, M, D, device)).to(t)
            s["residual_out"] = torch.empty(M, D, dtype=t, device=device)
    return s


def _round_rows(a):
    """Integers of the rows of `a` (fp32) and their largest magnitudes; in 64
    bits, so that values next to a border fall on their own side of it."""
    m = a.abs().amax(1, keepdim=True).double()
    t = 127.0 * a.double() / torch.where(m > 0, m, torch.ones_like(m))
    return torch.round(t).to(torch.int8), m


def run(s):
    if own:
        from linear_attention_recurrence_04_b200 import gdn
        if s["op"] == "linear":
            return gdn.linear_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["y"])
        if s["op"] == "quantize":
            return gdn.quantize_i8(s["x"], s["q"], s["scale"])
        q, scale, h = gdn.add_rms_norm_i8(s["x"], s["weight"], s["residual"], s["residual_out"],
                                          s["q"], s["scale"], eps=EPS)
        return (q, scale) if h is None else (q, scale, h)
    if s["op"] == "linear":
        y = torch.matmul(s["x"].float(), s["w"].float().t())
        y = y * s["x_scale"][:, None] * s["w_scale"][None, :]
        return y.to(s["out"])
    if s["op"] == "quantize":
        q, m = _round_rows(s["x"].float())
        return q, (m / 127.0).float()[:, 0]
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(s["residual"].dtype)
    hf = h.float()
    q, m = _round_rows(hf * s["weight"])
    rms = torch.sqrt(hf.double().square().mean(1, keepdim=True) + EPS)
    scale = (m / (127.0 * rms)).float()[:, 0]
    return (q, scale) if s["residual"] is None else (q, scale, h)


def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        size = 4 if case["out"] == "fp32" else 2
        return {"bytes": M * K + N * K + 4 * (M + N) + size * M * N, "flops": 2 * M * N * K}
    M, D = case["M"], case["D"]
    n = M * D
    bytes_ = n * (4 if case["x"] == "fp32" else 2) + n + 4 * M
    if case["op"] == "quantize":
        return {"bytes": bytes_, "flops": 3 * n}
    if case["residual"] != "none":
        bytes_ += 2 * n * (4 if case["residual"] == "fp32" else 2)
    return {"bytes": bytes_ + 4 * D, "flops": 7 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        # the integer sums are below 2^53: exact in 64 bits in any order
        acc = torch.einsum("mk,nk->mn", s["x"].double(), s["w"].double())
        acc *= s["x_scale"].double().unsqueeze(1)
        acc *= s["w_scale"].double().unsqueeze(0)
        return acc
    a = s["x"].double()
    rms = 1.0
    if case["op"] == "norm":
        if s["residual"] is not None:
            # the definition's roundings: the sum in fp32, then the stored type
            a = (a + s["residual"].double()).float().to(s["residual"].dtype).double()
        h = a
        rms = ((h * h).sum(1) / case["D"] + EPS).sqrt()
        a = (h * s["weight"].double()).float().double()
    top = a.abs().max(1).values
    q = (a * 127.0 / top.clamp(min=1e-300).unsqueeze(1)).round().to(torch.int8)
    scale = top / 127.0 / rms
    if case["op"] == "quantize" or s["residual"] is None:
        return q, scale
    return q, scale, h
