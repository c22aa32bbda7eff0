"""The 8-bit linear layers of a decoder and the matrix product's epilogue, as cases to measure: RMSNorm (after
the residual's addition) with an e4m3 output and a scale per row, rows quantised the same way, the product of
two such matrices with bias, activation and residual in its epilogue, and the bf16 product with that epilogue.

A row v of n values is held as e4m3 numbers y and one 32-bit scale s = max(max|v| / 448, 2^-126), y = e4m3(v / s).
A product is C = act(z) + residual with z = (A W^T) + bias, A's and W's rows times their scales; with "swiglu",
W's rows come in blocks of 16 gate rows and then the 16 up rows of the same features, and act gives
silu(gate) * up, half as many columns.
"""
import math
import random

import torch

own = False

DEV = "cuda"
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu")
TOP = 448.0            # the largest e4m3 number
LEAST = 2.0 ** -126    # the least scale
BLOCK = 16             # features of a block of gate (then up) rows


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the norm before a layer's projections, one decode step of 64 sequences: latency counts
        dict(name="norm step of 64", op="norm", M=64, H=4096, residual=True),
        # the same over a whole prompt of the 8192-token workload
        dict(name="norm prompt of 8192", op="norm", M=8192, H=4096, residual=True),
        # the first layer's norm (nothing to add) of a ragged batch, a width that is no power of two
        dict(name="norm 1999 of 1040", op="norm", M=1999, H=1040, residual=False),
        # the attention output of a decode step, on its way to the output projection
        dict(name="quantise step of 64", op="quant", M=64, K=4096),
        # the feed-forward product of a prompt, on its way to the down projection
        dict(name="quantise prompt of 8192", op="quant", M=8192, K=14336),
        # the query/key/value projection of a small decode step, with a bias: the weight's bytes count
        dict(name="q8 qkv step of 16", op="q8", M=16, N=6144, K=4096, act="none", bias=True, residual=False),
        # the gate/up projection of a decode step of 64, SwiGLU in its epilogue
        dict(name="q8 gate up step of 64", op="q8", M=64, N=28672, K=4096, act="swiglu", bias=False, residual=False),
        # the same of a whole prompt: the tensor cores' rate counts
        dict(name="q8 gate up prompt of 8192", op="q8", M=8192, N=28672, K=4096, act="swiglu", bias=False,
             residual=False),
        # a feed-forward layer with GELU of a ragged batch, every size odd in units of a tile
        dict(name="q8 gelu 333", op="q8", M=333, N=1000, K=1136, act="gelu", bias=True, residual=True),
        # the output projection of a small decode step in bf16, the residual stream added to it
        dict(name="bf16 output step of 16", op="bf16", M=16, N=4096, K=4096, act="none", bias=False, residual=True),
        # the down projection of a prompt chunk, the residual stream added to it
        dict(name="bf16 down chunk of 2048", op="bf16", M=2048, N=4096, K=14336, act="none", bias=False,
             residual=True),
        # a biased feed-forward layer of a ragged batch
        dict(name="bf16 gelu 777", op="bf16", M=777, N=2056, K=1000, act="gelu_tanh", bias=True, residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng: random.Random):
    op = rng.choice(("norm", "quant", "q8", "q8", "bf16", "bf16"))
    if op in ("norm", "quant"):
        wide = 16 * _log(rng, 4, 1024)
        rows = _log(rng, 1, min(32768, 8192 * 4096 // wide))
        if op == "norm":
            return dict(op=op, M=rows, H=wide, residual=rng.random() < 0.5)
        return dict(op=op, M=rows, K=wide)
    act = rng.choice(ACTS)
    n = 32 * _log(rng, 2, 896) if act == "swiglu" else 8 * _log(rng, 4, 3584)
    k = 16 * _log(rng, 4, 896) if op == "q8" else 8 * _log(rng, 8, 1792)
    most = 8192 * 28672 * 4096 if op == "q8" else 2048 * 4096 * 14336
    return dict(op=op, M=_log(rng, 1, min(8192, most // (n * k))), N=n, K=k, act=act, bias=rng.random() < 0.5,
                residual=rng.random() < 0.5)


def _columns(case):
    return case["N"] // 2 if case["act"] == "swiglu" else case["N"]


# -------------------------------------------------------------- preparation
def _stream_rows(shape, g):
    """bf16 rows as a residual stream holds them: channels of unlike size, a few ten times the others, and
    tokens of unlike size."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(0.8 * torch.randn((shape[1],), generator=g, device=DEV))
    x *= torch.exp(0.5 * torch.randn((shape[0], 1), generator=g, device=DEV))
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        s["x"] = _stream_rows((M, H), g)
        s["w"] = (1.0 + 0.2 * torch.randn((H,), generator=g, device=DEV)).to(torch.bfloat16)
        if case["residual"]:
            s["r"] = _stream_rows((M, H), g)
            s["h"] = torch.empty((M, H), dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "quant":
        s["x"] = _stream_rows((case["M"], case["K"]), g)
    if case["op"] in ("norm", "quant"):
        s["y"] = torch.empty(s["x"].shape, dtype=torch.float8_e4m3fn, device=DEV)
        s["scale"] = torch.empty((case["M"],), dtype=torch.float32, device=DEV)
        return s
    M, N, K, n = case["M"], case["N"], case["K"], _columns(case)
    a = _stream_rows((M, K), g)
    w = (torch.randn((N, K), generator=g, device=DEV) * (1.0 / math.sqrt(K))).to(torch.bfloat16)
    if case["op"] == "q8":
        s["a"], s["sa"] = _quantise(a.float())
        s["w"], s["sw"] = _quantise(w.float())
    else:
        s["a"], s["w"] = a, w
    s["b"] = s["r"] = None
    if case["bias"]:
        s["b"] = (0.1 * torch.randn((N,), generator=g, device=DEV)).to(torch.bfloat16)
    if case["residual"]:
        s["r"] = _stream_rows((M, n), g)
    s["c"] = torch.empty((M, n), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------- plain forms
def _quantise(v):
    scale = (v.abs().amax(1) / TOP).clamp(min=LEAST)
    return (v / scale[:, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"]:
        h = (h + s["r"].float()).to(torch.bfloat16)
        s["h"].copy_(h)
        h = h.float()
    v = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-5) * s["w"].float()
    return _quantise(v)


def _plain_product(s):
    z = s["a"].float() @ s["w"].float().T
    if s["op"] == "q8":
        z = z * s["sa"][:, None] * s["sw"]
    if s["b"] is not None:
        z = z + s["b"].float()
    act = s["act"]
    if act == "relu":
        z = torch.where(z > 0, z, 0.0)
    elif act == "gelu":
        z = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    elif act == "silu":
        z = z / (1.0 + torch.exp(-z))
    elif act == "swiglu":
        z = z.view(z.shape[0], -1, 2, BLOCK)
        z = (z[:, :, 0] / (1.0 + torch.exp(-z[:, :, 0])) * z[:, :, 1]).flatten(1)
    if s["r"] is not None:
        z = z + s["r"].float()
    return z.to(torch.bfloat16)


def run(state):
    s = state
    if own:
        import invariant_bi_rmsnorm_02_gb300 as bi
        if s["op"] == "norm":
            if s["residual"]:
                bi.bi_add_rmsnorm_q8(s["x"], s["r"], s["w"], s["h"], s["y"], s["scale"], 1e-5)
                return {"y": s["y"], "scale": s["scale"], "h": s["h"]}
            bi.bi_rmsnorm_q8(s["x"], s["w"], s["y"], s["scale"], 1e-5)
            return {"y": s["y"], "scale": s["scale"]}
        if s["op"] == "quant":
            bi.bi_quantize_q8(s["x"], s["y"], s["scale"])
            return {"y": s["y"], "scale": s["scale"]}
        act = getattr(bi, "ACT_" + s["act"].upper())
        if s["op"] == "q8":
            bi.bi_gemm_q8(s["a"], s["sa"], s["w"], s["sw"], s["c"], bias=s["b"], residual=s["r"], activation=act)
        else:
            bi.bi_gemm_epilogue(s["a"], s["w"], s["c"], bias=s["b"], residual=s["r"], activation=act)
        return s["c"]
    if s["op"] == "norm":
        y, scale = _plain_norm(s)
        return {"y": y, "scale": scale, "h": s["h"]} if s["residual"] else {"y": y, "scale": scale}
    if s["op"] == "quant":
        y, scale = _quantise(s["x"].float())
        return {"y": y, "scale": scale}
    return _plain_product(s)


# --------------------------------------------------------- bytes and flops
def work(case):
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        return {"bytes": M * (H * (7 if case["residual"] else 3) + 4) + 2 * H, "flops": 8 * M * H}
    if case["op"] == "quant":
        return {"bytes": case["M"] * (3 * case["K"] + 4), "flops": 3 * case["M"] * case["K"]}
    M, N, K, n = case["M"], case["N"], case["K"], _columns(case)
    wide = 1 if case["op"] == "q8" else 2
    moved = wide * (M + N) * K + 2 * M * n
    if case["op"] == "q8":
        moved += 4 * (M + N)
    if case["bias"]:
        moved += 2 * N
    if case["residual"]:
        moved += 2 * M * n
    return {"bytes": moved, "flops": 2 * M * N * K}


# --------------------------------------------- the definitions in 64 bits
def _exact_e4m3(x):
    """x to the nearest of the e4m3 numbers, ties to an even last digit."""
    digit = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / digit) * digit).clamp(-TOP, TOP)


def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] in ("norm", "quant"):
        v = s["x"].to(f8)
        out = {}
        if case["op"] == "norm":
            if case["residual"]:
                out["h"] = v + s["r"].to(f8)
                v = out["h"].to(torch.bfloat16).to(f8)  # the stream is held in bf16
            v = s["w"].to(f8) * v / torch.sqrt((v * v).sum(1, keepdim=True) / case["H"] + 1e-5)
        top = torch.maximum(v.amax(1), -v.amin(1))
        out["scale"] = torch.clamp(top / TOP, min=LEAST)
        out["y"] = _exact_e4m3(v / out["scale"][:, None])
        return out
    a, w = s["a"].to(f8), s["w"].to(f8)
    if case["op"] == "q8":
        a, w = a * s["sa"].to(f8)[:, None], w * s["sw"].to(f8)[:, None]
    z = torch.matmul(a, w.t())
    del a, w
    if case["bias"]:
        z += s["b"].to(f8)[None, :]
    if case["act"] == "relu":
        z = z.clamp(min=0.0)
    elif case["act"] == "gelu":
        z = z * torch.special.erfc(-z / math.sqrt(2.0)) / 2.0
    elif case["act"] == "gelu_tanh":
        z = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
    elif case["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif case["act"] == "swiglu":
        column = torch.arange(case["N"] // 2, device=DEV)
        gate = column // BLOCK * (2 * BLOCK) + column % BLOCK
        z = z[:, gate] * torch.sigmoid(z[:, gate]) * z[:, gate + BLOCK]
    if case["residual"]:
        z = z + s["r"].to(f8)
    return z
