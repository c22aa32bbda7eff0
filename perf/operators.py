"""The quantised-cache path of a long-context decoder, as cases to measure: rotary positions with
scaled frequencies, K/V rows quantised to e4m3 as they are written into the paged cache, the pages read
back as bf16, and decode attention over the quantised pages.

A page record of one kv head holds K[16][D] e4m3, V[16][D] e4m3, then 16 scale bytes of K and 16 of V
(32 D + 32 bytes); a scale byte c stands for 2^(c - 127), one per row.  A row's scale is the least power
of two, kept within 2^-124 .. 2^7, that brings its largest magnitude to 448 or less; a row with an
infinity or a NaN is stored as zeros under scale byte 135 and reads back as NaN.
"""
import math
import random

import torch

own = False

PAGE = 16
DEV = "cuda"
PAIRS = ((4, 2), (32, 8), (8, 8), (16, 1), (24, 8), (16, 2), (7, 1))  # query heads, kv heads


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch of 64: a few microseconds of work, launch latency counts
        dict(name="rope step of 64", op="rope", T=64, hq=32, hkv=8, d=128, rot=128, inter=False,
             scaling="llama3", theta=500000.0, far=131072),
        # a whole prompt chunk of the 8192-token workload, frequencies stretched for long contexts
        dict(name="rope chunk of 8192", op="rope", T=8192, hq=32, hkv=8, d=128, rot=128, inter=False,
             scaling="yarn", theta=10000.0, far=131072),
        # interleaved pairs over a quarter of the head, an odd number of tokens
        dict(name="rope 2047 part of the head", op="rope", T=2047, hq=16, hkv=16, d=128, rot=32,
             inter=True, scaling="linear", theta=10000.0, far=32768),
        # one new token for each of 64 sequences
        dict(name="write step of 64", op="write", n=64, seqs=64, hkv=8, d=128, longest=512),
        # an odd count of rows of half the width, many sequences
        dict(name="write 999 of 37", op="write", n=999, seqs=37, hkv=2, d=64, longest=512),
        # a prompt of 8192 tokens written at once
        dict(name="write prompt of 8192", op="write", n=8192, seqs=1, hkv=8, d=128, longest=8192),
        # the prefix of one chunked prompt, read for the prefill of its next chunk
        dict(name="read prompt of 8192", op="read", seqs=1, hkv=8, d=128, shortest=8192,
             longest=8192, empty=0),
        # 64 ragged sequences read back
        dict(name="read 64 ragged", op="read", seqs=64, hkv=8, d=128, shortest=1, longest=32768,
             empty=0),
        # a tiny decoder's step: 8 short sequences, one slot idle
        dict(name="decode 8 short", op="decode", seqs=8, hq=4, hkv=2, d=64, shortest=1, longest=512,
             split=64, empty=1),
        # the serving workload: 64 requests, lengths log-uniform to 32768
        dict(name="decode 64 ragged", op="decode", seqs=64, hq=32, hkv=8, d=128, shortest=1,
             longest=32768, split=256, empty=0),
        # one request with a long context: few rows, the long axis has to be split
        dict(name="decode one of 131072", op="decode", seqs=1, hq=32, hkv=8, d=128,
             shortest=131072, longest=131072, split=256, empty=0),
        # all query heads on one kv head, more sequences than one plan slab, mid lengths
        dict(name="decode 160 on one kv head", op="decode", seqs=160, hq=16, hkv=1, d=128,
             shortest=256, longest=4096, split=256, empty=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(("rope", "write", "read", "decode", "decode"))
    hq, hkv = rng.choice(PAIRS)
    d = rng.choice((64, 128))
    if op == "rope":
        d = rng.choice((64, 128, 80, 256))
        most = 8192 * 48 * 128 // ((hq + 2 * hkv) * d)
        rot = rng.choice((d, d // 2, d // 4, 6))
        return dict(op=op, T=_log(rng, 1, min(8192, most)), hq=hq, hkv=hkv, d=d, rot=rot,
                    inter=rng.random() < 0.5,
                    scaling=rng.choice(("none", "linear", "ntk", "yarn", "llama3")),
                    theta=rng.choice((10000.0, 500000.0)), far=_log(rng, 64, 1 << 20))
    if op == "write":
        n = _log(rng, 1, 8192)
        seqs = _log(rng, 1, min(n, 128))
        return dict(op=op, n=n, seqs=seqs, hkv=hkv, d=d,
                    longest=max(-(-n // seqs), _log(rng, 64, 1024)))
    seqs = _log(rng, 1, 200)
    longest = _log(rng, 1, min(131072, 64 * 32768 // seqs))
    shortest = max(1, _log(rng, 1, longest))
    empty = rng.randrange(0, max(1, seqs // 4) + 1) if seqs > 2 else 0
    if op == "read":
        return dict(op=op, seqs=seqs, hkv=hkv, d=d, shortest=shortest, longest=longest, empty=empty)
    return dict(op=op, seqs=seqs, hq=hq, hkv=hkv, d=d, shortest=shortest, longest=longest,
                split=rng.choice((64, 256, 512)), empty=empty)


# -------------------------------------------------------------- preparation
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(case):
    """Lengths spread evenly over the logarithm of [shortest, longest], the `empty` smallest ones 0."""
    n, lo, hi = case["seqs"], case["shortest"], case["longest"]
    lens = [round(hi * (lo / hi) ** (i / max(1, n - 1))) for i in range(n)]
    return lens[:n - case["empty"]] + [0] * case["empty"]


def _tables(blocks, g):
    """Page tables of sequences with `blocks` pages each, out of one shuffled pool; unused entries are 0."""
    total = int(blocks.sum())
    perm = torch.randperm(max(total, 1), generator=g, device=DEV).to(torch.int32)
    first = torch.cumsum(blocks, 0) - blocks
    j = torch.arange(max(int(blocks.max()), 1), device=DEV)
    at = first[:, None] + j[None, :]
    table = perm[at.clamp(max=perm.numel() - 1)]
    return torch.where(j[None, :] < blocks[:, None], table, 0).to(torch.int32).contiguous(), max(total, 1)


def _rows(shape, g, keys):
    """bf16 rows as a decoder makes them: keys have channels of unlike size (a few are ten times the
    others) and both have tokens of unlike size."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))
    if keys:
        x *= torch.exp(0.8 * torch.randn((shape[-1],), generator=g, device=DEV))
    return x.to(torch.bfloat16)


def _frequencies(case):
    """Rotation frequencies in 64 bits and the factor on cosine and sine, for each way of stretching the
    positions of a model trained on 8192 tokens to eight times that."""
    r, theta, kind, factor, trained = case["rot"], case["theta"], case["scaling"], 8.0, 8192
    if kind == "ntk":
        theta = theta * factor ** (r / (r - 2))
    f = [theta ** (-2.0 * i / r) for i in range(r // 2)]
    m = 1.0
    if kind == "linear":
        f = [x / factor for x in f]
    elif kind == "llama3":
        low, high = 1.0, 4.0
        def stretch(x):
            turns = trained * x / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            return (1 - keep) * x / factor + keep * x
        f = [stretch(x) for x in f]
    elif kind == "yarn":
        def pair_of(turns):
            return r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(theta))
        first = max(math.floor(pair_of(32.0)), 0)
        last = min(math.ceil(pair_of(1.0)), r - 1)
        width = max(last - first, 0.001)
        keep = [1 - min(1.0, max(0.0, (i - first) / width)) for i in range(r // 2)]
        f = [(1 - w) * x / factor + w * x for x, w in zip(f, keep)]
        m = 0.1 * math.log(factor) + 1.0
    return f, m


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "rope":
        T, hq, hkv, d = case["T"], case["hq"], case["hkv"], case["d"]
        s["qkv"] = torch.randn((T, (hq + 2 * hkv) * d), generator=g, device=DEV).to(torch.bfloat16)
        s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
        f, s["m"] = _frequencies(case)
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        s["q"], s["k"], s["v"] = (torch.empty((T, h, d), dtype=torch.bfloat16, device=DEV)
                                  for h in (hq, hkv, hkv))
        return s
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "write":
        n, seqs = case["n"], case["seqs"]
        blocks = torch.full((seqs,), -(-case["longest"] // PAGE), device=DEV)
        s["table"], pages = _tables(blocks, g)
        # each sequence's new tokens are consecutive, from a place of its own on
        per = -(-n // seqs)
        start = (torch.rand(seqs, generator=g, device=DEV) * (case["longest"] - per + 1)).to(torch.int32)
        i = torch.arange(n, device=DEV, dtype=torch.int32)
        s["seq"] = i // per
        s["pos"] = (start[(i // per).long()] + i % per).to(torch.int32)
        s["k"], s["v"] = _rows((n, hkv, d), g, True), _rows((n, hkv, d), g, False)
        s["k"][n // 2] = 0  # a row of zeros
        s["cache"] = torch.zeros((pages, hkv, 32 * d + 32), dtype=torch.uint8, device=DEV)
        return s
    # the same lengths for every seed, in an order of the seed's
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    s["lens"] = lens[torch.randperm(case["seqs"], generator=g, device=DEV)].contiguous()
    s["table"], pages = _tables((s["lens"].long() + PAGE - 1) // PAGE, g)
    cache = torch.zeros((pages, hkv, 32 * d + 32), dtype=torch.uint8, device=DEV)
    for at in (0, 1):  # K rows, V rows
        data, scale = _quantise(_rows((pages, hkv, PAGE, d), g, at == 0))
        cache[:, :, at * PAGE * d:(at + 1) * PAGE * d] = data.view(torch.uint8).flatten(2)
        cache[:, :, 32 * d + at * PAGE:32 * d + (at + 1) * PAGE] = scale
    s["cache"] = cache
    if case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.zeros((pages, hkv, PAGE, d), dtype=torch.bfloat16, device=DEV)
                                  for _ in range(2))
    else:
        s["q"] = torch.randn((case["seqs"], case["hq"], d), generator=g, device=DEV).to(torch.bfloat16)
    return s


# ------------------------------------------------------------- plain forms
def _quantise(x):
    """(e4m3 values, scale bytes) of rows of x along its last axis."""
    x = x.float()
    fine = torch.isfinite(x).all(-1)
    x = torch.where(fine[..., None], x, 0.0)
    part, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(part <= 0.875, e - 9, e - 8)  # 448 = 0.875 * 2^9
    e = torch.where(part == 0, -124, e).clamp(-124, 7)
    shrink = ((127 - e) << 23).view(torch.float32)  # 2^-e
    data = (x * shrink[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return data, torch.where(fine, e + 127, 135).to(torch.uint8)


def _values(cache, d):
    """K and V of records [..., 32 d + 32] in 32 bits, [..., 16, d] each."""
    data = cache[..., :32 * d].view(torch.float8_e4m3fn).float().unflatten(-1, (2, PAGE, d))
    code = cache[..., 32 * d:].to(torch.int32).unflatten(-1, (2, PAGE))
    scale = torch.where(code == 135, float("nan"), (code << 23).view(torch.float32))
    x = data * scale[..., None]
    return x.select(-3, 0), x.select(-3, 1)


def _plain_rope(s):
    T, hq, hkv, d, r = s["T"], s["hq"], s["hkv"], s["d"], s["rot"]
    x = s["qkv"].view(T, hq + 2 * hkv, d)
    angle = s["pos"].double()[:, None] * s["freqs"]
    c = (s["m"] * torch.cos(angle)).float()[:, None]
    t = (s["m"] * torch.sin(angle)).float()[:, None]
    y = x[:, :hq + hkv].float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if s["inter"] else (y[..., :r // 2], y[..., r // 2:r])
    rotated = (a * c - b * t, b * c + a * t)
    y = torch.cat((torch.stack(rotated, -1).flatten(-2) if s["inter"] else torch.cat(rotated, -1), y[..., r:]), -1)
    y = y.to(torch.bfloat16)
    return {"q": y[:, :hq].contiguous(), "k": y[:, hq:].contiguous(), "v": x[:, hq + hkv:].contiguous()}


def _plain_write(s):
    d = s["d"]
    page = s["table"][s["seq"].long(), (s["pos"] // PAGE).long()].long()
    slot = (s["pos"] % PAGE).long()
    for at, x in ((0, s["k"]), (1, s["v"])):
        data, scale = _quantise(x)
        rows = s["cache"][..., :32 * d].unflatten(-1, (2, PAGE, d))[:, :, at]
        rows[page, :, slot] = data.view(torch.uint8)
        s["cache"][..., 32 * d + at * PAGE:32 * d + (at + 1) * PAGE][page, :, slot] = scale


def _plain_read(s):
    j = torch.arange(s["table"].shape[1] * PAGE, device=DEV)
    seq, pos = torch.nonzero(j[None, :] < s["lens"][:, None], as_tuple=True)
    page, slot = s["table"][seq, pos // PAGE].long(), pos % PAGE
    k, v = _values(s["cache"], s["d"])
    s["k_out"][page, :, slot] = k[page, :, slot].to(torch.bfloat16)
    s["v_out"][page, :, slot] = v[page, :, slot].to(torch.bfloat16)


def _plain_decode(s):
    b, hq, hkv, d = s["seqs"], s["hq"], s["hkv"], s["d"]
    k, v = _values(s["cache"][s["table"].long()], d)          # [b, blocks, hkv, 16, d]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))  # [b, hkv, keys, d]
    seen = torch.arange(k.shape[2], device=DEV)[None, :] < s["lens"][:, None]
    v = torch.where(seen[:, None, :, None], v, 0.0)
    score = (s["q"].float().view(b, hkv, hq // hkv, d) @ k.transpose(2, 3)) * d ** -0.5
    score = torch.where(seen[:, None, None, :], score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    return o.view(b, hq, d).to(torch.bfloat16)


def _stored(s):
    """A cache's records as the values they stand for: e4m3 rows and power-of-two scales."""
    n = 32 * s["d"]
    return {"rows": s["cache"][..., :n].view(torch.float8_e4m3fn),
            "scales": s["cache"][..., n:].view(torch.float8_e8m0fnu)}


def run(state):
    s = state
    if own:
        import invariant_bi_rmsnorm_02_gb300 as bi
        if s["op"] == "rope":
            bi.bi_rope_qkv_scaled(s["qkv"], s["pos"], s["hq"], s["hkv"], s["d"], s["freqs"], s["q"],
                                  s["k"], s["v"], interleaved=s["inter"], attn_scale=s["m"])
            return {"q": s["q"], "k": s["k"], "v": s["v"]}
        if s["op"] == "write":
            bi.bi_kv_write_q8(s["k"], s["v"], s["seq"], s["pos"], s["cache"], s["table"])
            return _stored(s)
        if s["op"] == "read":
            bi.bi_kv_read_q8(s["cache"], s["table"], s["lens"], s["k_out"], s["v_out"], s["table"],
                             max_kv_len=s["longest"])
            return {"k": s["k_out"], "v": s["v_out"]}
        return bi.attn_decode_q8(s["q"], s["cache"], s["table"], s["lens"], max_kv_len=s["longest"],
                                 split_size=s["split"])
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "write":
        _plain_write(s)
        return _stored(s)
    if s["op"] == "read":
        _plain_read(s)
        return {"k": s["k_out"], "v": s["v_out"]}
    return _plain_decode(s)


# --------------------------------------------------------- bytes and flops
def work(case):
    if case["op"] == "rope":
        row = (case["hq"] + 2 * case["hkv"]) * case["d"]
        return {"bytes": case["T"] * (4 * row + 4) + 4 * case["rot"],
                "flops": case["T"] * (case["hq"] + case["hkv"]) * case["rot"] * 3}
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "write":
        return {"bytes": case["n"] * (hkv * (4 * d + 2 * d + 2) + 12), "flops": case["n"] * hkv * d * 4}
    tokens = sum(_lengths(case))
    if case["op"] == "read":
        return {"bytes": tokens * (hkv * (2 * d + 2 + 4 * d) + 0.25), "flops": tokens * hkv * 2 * d}
    return {"bytes": tokens * (hkv * (2 * d + 2) + 0.25) + case["seqs"] * (4 * case["hq"] * d + 4),
            "flops": tokens * case["hq"] * 4 * d}


# --------------------------------------------- the definitions in 64 bits
def _exact_row_scale(x):
    """The least e with max|x| 2^-e <= 448 in [-124, 7], by trying exponents around the logarithm."""
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)) + 1
    for _ in range(3):
        e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    return e.clamp(-124, 7)


def _exact_e4m3(x):
    """x to the nearest of the e4m3 numbers, ties to an even last digit, in 64 bits."""
    size = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / size) * size).clamp(-448.0, 448.0)


def _exact_decoded(cache, d):
    code = cache[..., :32 * d].to(torch.int64)
    exponent, digits = (code >> 3) & 15, (code & 7).double()
    x = torch.where(exponent == 0, digits * 2.0 ** -9,
                    (1 + digits / 8) * torch.exp2((exponent - 7).double()))
    x = torch.where(code >= 128, -x, x).unflatten(-1, (2, PAGE, d))
    return x * torch.exp2(cache[..., 32 * d:].double() - 127).unflatten(-1, (2, PAGE))[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "rope":
        T, hq, hkv, r = case["T"], case["hq"], case["hkv"], case["rot"]
        x = s["qkv"].double().view(T, hq + 2 * hkv, d)
        turn = torch.polar(torch.full((T, r // 2), s["m"], dtype=torch.float64, device=DEV),
                           s["pos"].double()[:, None] * s["freqs"][None, :])[:, None, :]
        y = x[:, :hq + hkv].clone()
        i = torch.arange(r // 2, device=DEV)
        first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + r // 2)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return {"q": y[:, :hq], "k": y[:, hq:], "v": x[:, hq + hkv:]}
    if case["op"] == "write":
        rows = torch.zeros(s["cache"].shape[:2] + (32 * d,), dtype=torch.float64, device=DEV)
        scales = torch.full(s["cache"].shape[:2] + (32,), 2.0 ** -127, dtype=torch.float64, device=DEV)
        where = (s["table"][s["seq"].long(), (s["pos"] // PAGE).long()].long(), slice(None))
        slot = (s["pos"] % PAGE).long()
        for at, x in ((0, s["k"].double()), (1, s["v"].double())):
            e = _exact_row_scale(x)
            rows.unflatten(-1, (2, PAGE, d))[where + (at, slot)] = _exact_e4m3(x / torch.exp2(e)[..., None])
            scales.unflatten(-1, (2, PAGE))[where + (at, slot)] = torch.exp2(e)
        return {"rows": rows, "scales": scales}
    lens = s["lens"].tolist()
    out = {"k": torch.zeros(s["cache"].shape[:2] + (PAGE, d), dtype=torch.float64, device=DEV)}
    out["v"] = torch.zeros_like(out["k"])
    if case["op"] == "read":
        for b, n in enumerate(lens):
            pages = s["table"][b, :-(-n // PAGE)].long()
            x = _exact_decoded(s["cache"][pages], d)
            seen = (torch.arange(pages.numel() * PAGE, device=DEV) < n).view(-1, 1, PAGE, 1)
            out["k"][pages], out["v"][pages] = x[:, :, 0] * seen, x[:, :, 1] * seen
        return out
    group = case["hq"] // case["hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        x = _exact_decoded(s["cache"][s["table"][b, :-(-n // PAGE)].long()], d)
        k, v = (x[:, :, at].transpose(0, 1).flatten(1, 2)[:, :n] for at in (0, 1))
        for h in range(case["hkv"]):
            q = s["q"][b, h * group:(h + 1) * group].double()
            o[b, h * group:(h + 1) * group] = torch.softmax(q @ k[h].T / math.sqrt(d), -1) @ v[h]
    return o
