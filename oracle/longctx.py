"""Plain fp64 definitions of the quantised KV cache and of scaled rotary
positions.  Test infrastructure only, numpy alone: the e4m3 numbers are a
table, rounding is a search for the nearest of them, and rotation is complex
multiplication, so nothing here shares a method with the kernels.

bf16 inputs are uint16 arrays of bit patterns (``bits_of`` takes a tensor).
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 16
NON_FINITE = 135


def bits_of(t) -> np.ndarray:
    import torch
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def bf16_to_f64(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


def _positive_e4m3() -> np.ndarray:
    """The values of codes 0 .. 0x7e in increasing order."""
    codes = np.arange(0x7f)
    e, f = codes >> 3, (codes & 7) / 8.0
    return np.where(e == 0, f * 2.0 ** -6, (1.0 + f) * 2.0 ** (e - 7.0))


E4M3 = _positive_e4m3()


def e4m3_codes(x) -> np.ndarray:
    """Codes of the e4m3 numbers nearest to x (ties to the even code, which has
    the even last digit; magnitudes above 448 give 448; -0 keeps its sign)."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 0x7e)
    lo = np.clip(hi - 1, 0, 0x7e)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(a >= 448.0, 0x7e, np.where(up, hi, lo))
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def quantise_rows(bits):
    """(codes, scale bytes) of rows along the last axis of bf16 bit patterns."""
    x = bf16_to_f64(bits)
    finite = np.isfinite(x).all(-1)
    x = np.where(finite[..., None], x, 0.0)
    amax = np.abs(x).max(-1)
    e = np.full(amax.shape, 7)
    for k in range(6, -125, -1):          # the least exponent that still fits
        e = np.where(amax <= 448.0 * 2.0 ** k, k, e)
    codes = e4m3_codes(x * 2.0 ** -e[..., None].astype(np.float64))
    codes = np.where(finite[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(finite, e + 127, NON_FINITE).astype(np.uint8)


def values(codes, scales) -> np.ndarray:
    """What stored rows stand for, fp64."""
    v = np.where(codes >= 0x80, -1.0, 1.0) * np.append(E4M3, np.nan)[codes & 0x7f]
    v = v * 2.0 ** (scales.astype(np.float64) - 127)[..., None]
    return np.where((scales == NON_FINITE)[..., None], np.nan, v)


def record_views(cache, D):
    """Views of an array [pages, Hkv, 32 D + 32]: rows [pages, Hkv, 2, 16, D]
    (K, V) and scales [pages, Hkv, 2, 16]."""
    P, H, _ = cache.shape
    rows = cache[..., :32 * D].reshape(P, H, 2, PAGE, D)
    return rows, cache[..., 32 * D:].reshape(P, H, 2, PAGE)


def write(cache, k_bits, v_bits, seq, pos, table):
    """The cache (a new array) after K/V rows [n, Hkv, D] are written."""
    D = k_bits.shape[-1]
    rows, scales = (a.copy() for a in record_views(cache, D))
    for kind, bits in enumerate((k_bits, v_bits)):
        codes, c = quantise_rows(bits)
        for i in range(len(seq)):
            page, slot = table[seq[i], pos[i] // PAGE], pos[i] % PAGE
            rows[page, :, kind, slot] = codes[i]
            scales[page, :, kind, slot] = c[i]
    return np.concatenate([rows.reshape(*cache.shape[:2], 32 * D),
                           scales.reshape(*cache.shape[:2], 32)], -1)


def pages(cache, D):
    """K and V of every page, fp64 [pages, Hkv, 16, D] each."""
    v = values(*record_views(cache, D))
    return v[:, :, 0], v[:, :, 1]


def frequencies(rot, theta, kind="none", factor=1.0, trained=8192.0, low=1.0, high=4.0):
    """(freqs, factor on cosine and sine) of the named way of scaling."""
    i = np.arange(rot // 2, dtype=np.float64)
    if kind == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = 1.0 / theta ** (2 * i / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "llama3":
        wavelength = 2 * math.pi / f
        smooth = np.clip((trained / wavelength - low) / (high - low), 0, 1)
        return (1 - smooth) * f / factor + smooth * f, 1.0
    if kind == "yarn":
        dim = lambda turns: rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(theta))
        a, b = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
        ramp = np.clip((i - a) / max(b - a, 0.001), 0, 1)
        return ramp * f / factor + (1 - ramp) * f, 0.1 * math.log(factor) + 1
    return f, 1.0


def rope(x, pos, freqs, interleaved, attn_scale):
    """Rotated heads: x fp64 [T, heads, D], the first 2 len(freqs) elements."""
    n = len(freqs)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    # whole turns are taken out exactly (fmod); the turns made are fp64, so a far
    # position is off by 2^-52 of them
    turns = np.array([[math.fmod(float(p) * (f / (2 * math.pi)), 1.0) for f in freqs] for p in pos])
    w = attn_scale * np.exp(2j * math.pi * turns)[:, None, :]
    z = (x[..., a] + 1j * x[..., b]) * w
    y = x.copy()
    y[..., a], y[..., b] = z.real, z.imag
    return y
