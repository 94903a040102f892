"""Measured cases of the operators over the block-128 FP8 store (fp8b128): the activation
quantizer, the 8-bit product, the gated feed-forward product, and the backward passes of the
two products.

A store holds E4M3 codes [out][in] and one fp32 scale per 128 x 128 block; activations hold
E4M3 codes [T][in] and one fp32 scale per token and 128 inputs. The last block of a row or a
column may be a part of one.

With ``own`` false, ``run`` computes an operator by elementary torch operations in fp32 (the
plain form); with ``own`` true it calls the package. Both take what ``prepare`` made.
"""

import math

import torch

own = False

BLOCK = 128
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0

# The largest listed product in flops: 2 * 8192 tokens * 5120 inputs * 7168 outputs.
MAX_GEMM = 2 * 8192 * 5120 * 7168
MAX_GATED = 2 * 8192 * 5120 * 4096
MAX_GEMM_BWD = 4 * 8192 * 5120 * 1536
MAX_GATED_BWD = 6 * 4096 * 5120 * 4096
MAX_QUANT = 8192 * 5120


def listed():
    """5120 inputs, 1,536 gate and up outputs (768 intermediate channels) and chunks of 8,192
    tokens are the repository's shared expert and prefill chunk; the others are generic."""
    return [
        # one decode batch of 64 tokens entering the shared expert
        {"name": "quantize decode", "op": "quantize", "T": 64, "n": 5120},
        # one prefill chunk
        {"name": "quantize prefill", "op": "quantize", "T": 8192, "n": 5120},
        # a single token through the shared expert's gate and up projections: latency
        {"name": "gemm one token", "op": "gemm", "T": 1, "n": 5120, "out": 1536, "y": "f32"},
        # a decode batch whose sizes end inside a block on every side
        {"name": "gemm ragged batch", "op": "gemm", "T": 77, "n": 2000, "out": 2640, "y": "bf16"},
        # a prefill chunk through a large dense projection: the matrix cores' rate
        {"name": "gemm prefill", "op": "gemm", "T": 8192, "n": 5120, "out": 7168, "y": "bf16"},
        # single-token serving of the shared expert's gated product
        {"name": "gated one token", "op": "gated", "T": 1, "n": 5120, "out": 1536},
        # a decode batch through the shared expert's gated product
        {"name": "gated decode batch", "op": "gated", "T": 128, "n": 5120, "out": 1536},
        # a prefill chunk through a dense layer's gated product
        {"name": "gated prefill", "op": "gated", "T": 8192, "n": 5120, "out": 4096},
        # the gradients of a short, odd batch
        {"name": "gemm backward short", "op": "gemm_backward", "T": 333, "n": 768, "out": 5120},
        # the gradients of a whole chunk through the shared expert's projections
        {"name": "gemm backward chunk", "op": "gemm_backward", "T": 8192, "n": 5120, "out": 1536},
        # the gated block's gradients at an odd batch whose sizes end inside blocks
        {"name": "gated backward ragged", "op": "gated_backward", "T": 201, "n": 2576, "out": 1440},
        # a training step's gated block
        {"name": "gated backward chunk", "op": "gated_backward", "T": 4096, "n": 5120, "out": 4096},
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    """Tokens 1 .. 8,192 and widths 64 .. 7,168 (multiples of 16, every residue of 128 among
    them), over their logarithms; as many tokens as keep it within the largest listed case."""
    op = rng.choice(["quantize", "gemm", "gemm", "gated", "gemm_backward", "gated_backward"])
    T = max(1, round(_log(rng, 1, 8192)))
    n = 16 * round(_log(rng, 16, 448))
    if op == "quantize":
        return {"op": op, "T": max(1, min(T, MAX_QUANT // n)), "n": n}
    out = 32 * round(_log(rng, 2, 224)) if op.startswith("gated") else 16 * round(_log(rng, 4, 448))
    most, per = {"gemm": (MAX_GEMM, 2), "gated": (MAX_GATED, 2),
                 "gemm_backward": (MAX_GEMM_BWD, 4),
                 "gated_backward": (MAX_GATED_BWD, 6)}[op]
    case = {"op": op, "T": max(1, min(T, most // (per * n * out))), "n": n, "out": out}
    if op == "gemm":
        case["y"] = rng.choice(["f32", "bf16"])
    return case


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---- inputs ------------------------------------------------------------------------------
def _activations(gen, T, n):
    """bf16 rows of hidden states: unit normal values, a few channels far larger than the
    rest, tokens of different norms, and a zero row (a padded token) where there are several."""
    x = torch.randn((T, n), generator=gen, device="cuda")
    x[:, :: 97] *= 12.0
    x *= torch.exp(0.5 * torch.randn((T, 1), generator=gen, device="cuda"))
    if T > 8:
        x[T // 2] = 0
    return x.bfloat16()


def _codes_of(x):
    """E4M3 codes and power-of-two scales of bf16 rows, for the operators that start from
    quantized activations."""
    T, n = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _blocks(n) * BLOCK - n)).view(T, -1, BLOCK)
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    k = torch.where(amax > 0, k, torch.zeros_like(k)).int()
    scale = ((k + 127) << 23).view(torch.float32)
    inverse = ((127 - k) << 23).view(torch.float32)
    codes = (v * inverse[..., None]).to(E4M3).view(T, -1)[:, :n].contiguous()
    return codes, scale.contiguous()


def _weights(gen, out, n):
    """A projection as such checkpoints hold it: normal weights, each 128 x 128 block scaled
    so that its largest magnitude is 448."""
    ob, nb = _blocks(out), _blocks(n)
    w = torch.randn((ob * BLOCK, nb * BLOCK), generator=gen, device="cuda") / math.sqrt(n)
    w *= torch.exp(0.3 * torch.randn((ob * BLOCK, 1), generator=gen, device="cuda"))
    w[out:] = 0
    w[:, n:] = 0
    b = w.view(ob, BLOCK, nb, BLOCK)
    scale = b.abs().amax((1, 3)) / E4M3_MAX
    codes = (b / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    codes = codes.view(ob * BLOCK, nb * BLOCK)[:out, :n].contiguous()
    return codes, scale.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"], "y": case.get("y")}
    T, n = case["T"], case["n"]
    x = _activations(gen, T, n)
    if case["op"] == "quantize":
        s["x"] = x
        return s
    s["xc"], s["xs"] = _codes_of(x)
    s["wc"], s["ws"] = _weights(gen, case["out"], n)
    if case["op"] == "gemm_backward":
        s["dy"] = (0.1 * torch.randn((T, case["out"]), generator=gen, device="cuda")).bfloat16()
    if case["op"] == "gated_backward":
        dh = torch.randn((T, case["out"] // 2), generator=gen, device="cuda")
        s["dh"] = (0.1 * dh).bfloat16()
    return s


# ---- the operators -----------------------------------------------------------------------
def _run_own(s):
    from trellis_quantized_moe_amd import ops
    if s["op"] == "quantize":
        codes, scales = ops.fp8b128_quantize(s["x"])
        return {"codes": codes.view(E4M3), "scales": scales}
    layer = ops.Fp8b128Layer(s["wc"], s["ws"])
    if s["op"] == "gemm":
        flags = ops.TQ_OUT_BF16 if s["y"] == "bf16" else 0
        return {"y": ops.fp8b128_gemm(layer, s["xc"], s["xs"], flags=flags)}
    if s["op"] == "gated":
        return {"h": ops.fp8b128_gated(layer, s["xc"], s["xs"])}
    if s["op"] == "gemm_backward":
        dx, dw = ops.fp8b128_gemm_backward(layer, s["xc"], s["xs"], s["dy"])
    else:
        dx, dw = ops.fp8b128_gated_backward(layer, s["xc"], s["xs"], s["dh"])
    return {"dx": dx, "dw": dw}


def _wide_x(s):
    """The activations' values in fp32: a code times its block's scale."""
    x = s["xc"].float()
    return x * s["xs"].repeat_interleave(BLOCK, 1)[:, :x.shape[1]]


def _wide_w(s):
    """The weights' values in fp32 (one rounding: a 4-bit code times a 24-bit scale)."""
    w = s["wc"].float()
    rows = s["ws"].repeat_interleave(BLOCK, 1)[:, :w.shape[1]]
    return w * rows.repeat_interleave(BLOCK, 0)[:w.shape[0]]


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "quantize":
        codes, scales = _codes_of(s["x"])
        return {"codes": codes, "scales": scales}
    x, w = _wide_x(s), _wide_w(s)
    if s["op"] == "gemm":
        y = x @ w.t()
        return {"y": y if s["y"] == "f32" else y.bfloat16()}
    if s["op"] == "gemm_backward":
        dy = s["dy"].float()
        return {"dx": (dy @ w).bfloat16(), "dw": (dy.t() @ x).bfloat16()}
    half = w.shape[0] // 2
    gu = x @ w.t()
    g, u = gu[:, :half], gu[:, half:]
    sig = 1 / (1 + torch.exp(-g))
    if s["op"] == "gated":
        return {"h": (g * sig * u).bfloat16()}
    dh = s["dh"].float()
    d = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)
    return {"dx": (d @ w).bfloat16(), "dw": (d.t() @ x).bfloat16()}


# ---- bounds ------------------------------------------------------------------------------
def work(case):
    T, n = case["T"], case["n"]
    nb = _blocks(n)
    xq = T * n + 4 * T * nb
    if case["op"] == "quantize":
        return {"bytes": 2 * T * n + xq, "flops": 3 * T * n}
    out = case["out"]
    read = xq + out * n + 4 * _blocks(out) * nb
    if case["op"] == "gemm":
        return {"bytes": read + T * out * (4 if case["y"] == "f32" else 2), "flops": 2 * T * n * out}
    if case["op"] == "gated":
        return {"bytes": read + T * out, "flops": 2 * T * n * out}
    grads = 2 * T * n + 2 * out * n
    if case["op"] == "gemm_backward":
        return {"bytes": read + 2 * T * out + grads, "flops": 4 * T * n * out}
    return {"bytes": read + T * out + grads, "flops": 6 * T * n * out}


# ---- the definition in 64 bits -----------------------------------------------------------
def _exact_codes(x):
    """Nearest E4M3 value, ties to even, of x / s, with s the smallest power of two that
    brings the block's largest magnitude to 448 or less: by arithmetic, not by a cast."""
    T, n = x.shape
    nb = _blocks(n)
    v = torch.zeros((T, nb * BLOCK), dtype=torch.float64, device=x.device)
    v[:, :n] = x.double()
    v = v.reshape(T, nb, BLOCK)
    top = v.abs().max(dim=2).values
    some = torch.where(top > 0, top, torch.full_like(top, E4M3_MAX))
    k = torch.ceil(torch.log2(some / E4M3_MAX))
    k = torch.where(some > E4M3_MAX * torch.exp2(k), k + 1, k)
    k = torch.where(some <= E4M3_MAX * torch.exp2(k - 1), k - 1, k)
    scale = torch.exp2(k.clamp(min=-126))
    q = v / scale[:, :, None]
    size = q.abs().clamp(min=2.0 ** -30)
    step = torch.exp2(torch.floor(torch.log2(size)).clamp(min=-6) - 3)
    q = torch.round(q / step) * step
    return q.reshape(T, -1)[:, :n].contiguous(), scale


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        codes, scales = _exact_codes(s["x"])
        return {"codes": codes, "scales": scales}
    n, out = case["n"], case["out"]
    col = torch.arange(n, device="cuda") // BLOCK
    row = torch.arange(out, device="cuda") // BLOCK
    x = s["xc"].double().mul_(s["xs"].double()[:, col])
    w = s["wc"].double().mul_(s["ws"].double()[row][:, col])
    if s["op"] == "gemm":
        return {"y": torch.matmul(x, w.transpose(0, 1))}
    if s["op"] == "gemm_backward":
        d = s["dy"].double()
    else:
        g = torch.matmul(x, w[:out // 2].transpose(0, 1))
        u = torch.matmul(x, w[out // 2:].transpose(0, 1))
        sig = torch.sigmoid(g)
        if s["op"] == "gated":
            return {"h": g * sig * u}
        dh = s["dh"].double()
        slope = sig + g * sig * (1 - sig)
        d = torch.cat((dh * u * slope, dh * (g * sig)), dim=1)
    return {"dx": torch.matmul(d, w), "dw": torch.matmul(d.transpose(0, 1), x)}
