"""Scaled rotary positions on the GPU: how far off an angle may be at the last
int32 positions, against integer arithmetic of 200 bits, and heads of many
counts and widths against the fp64 definition."""
import math
from decimal import Decimal, localcontext

import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
from invariant_bi_rmsnorm_02_gb300 import synth
from test_gpu_rope_scaled import check

pytestmark = pytest.mark.gpu
BITS = 200


def turns_per_position(f):
    """f / (2 pi) in units of 2^-BITS (an int)."""
    with localcontext() as c:
        c.prec = 90
        pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628")
        return int(Decimal(f) / (2 * pi) * 2 ** BITS)


def reduced(f, pos):
    """pos * f less its whole turns, in radians, and its distance from the
    nearest odd quarter turn: both to the full precision of a float."""
    n = turns_per_position(f) * pos % 2 ** BITS
    quarter = 2 ** (BITS - 2)
    k = 1 if n < 2 * quarter else 3
    return 2 * math.pi * (n / 2 ** BITS), 2 * math.pi * ((n - k * quarter) / 2 ** BITS), k


@pytest.mark.parametrize("f", [1.0, 0.8145833435, 500000.0 ** (-2 / 128), 500000.0 ** (-10 / 128),
                               10000.0 ** (-14 / 64)])
def test_angles_of_far_positions_stay_within_their_bound(cuda, f):
    # near an odd quarter turn the cosine is the angle's distance from it, so
    # that a bf16 number shows an error far below one of bf16's at 1
    far = [p for p in range(2 ** 31 - 60000, 2 ** 31, 3)]
    far.sort(key=lambda p: abs(reduced(f, p)[1]))
    pos = far[:40] + [-p for p in far[:20]]
    T, D = len(pos), 16
    qkv = torch.zeros(T, 3 * D, dtype=torch.bfloat16, device=cuda)
    qkv[:, 0:D:2] = 1.0                              # x0 = 1, x1 = 0: y0 = cos, y1 = sin
    freqs = torch.full((D // 2,), f, dtype=torch.float64, device=cuda)
    q, _, _ = bi.rope_qkv_scaled(qkv, torch.tensor(pos, dtype=torch.int32, device=cuda), 1, 1, D,
                                 freqs, True)
    got = q[:, 0, 0].cpu().double().numpy()
    for p, y in zip(pos, got):
        _, d, k = reduced(f, abs(p))
        want = math.sin(-d) if k == 1 else math.sin(d)
        # the stated bound of the angle, its rounding to fp32 (half a unit of 24
        # bits at an angle below pi), 2 ulp of the cosine, half a step of bf16
        bound = abs(p) * (f * 2.0 ** -52 + 2.0 ** -62) + math.pi * 2.0 ** -24 + \
            2.0 ** -8 * abs(want)
        assert abs(y - want) <= bound, (p, y, want)


@pytest.mark.parametrize("Hq,Hkv,D,rot", [(24, 8, 80, 80), (32, 8, 80, 40), (40, 8, 128, 128),
                                          (28, 4, 128, 128), (64, 8, 128, 64), (16, 16, 256, 256),
                                          (1, 1, 16, 16), (7, 1, 128, 6), (100, 7, 112, 112)])
def test_heads_of_many_counts_and_widths(cuda, Hq, Hkv, D, rot):
    # blocks of either size, steps of several tokens and tokens of several
    # chunks, with a last step that is not whole
    freqs, m = bi.rope_frequencies(rot, 10000.0)
    for T in (1, 2, 1203):
        qkv = synth.normal_bf16((T, (Hq + 2 * Hkv) * D), 34000 + T, device=cuda)
        pos = synth.uniform_int(T, 0, 131072, 34001 + T).to(torch.int32)
        for inter in (False, True):
            q, k, v = bi.rope_qkv_scaled(qkv, pos.to(cuda), Hq, Hkv, D, freqs, inter, m)
            check(q, k, v, qkv, pos.tolist(), Hq, Hkv, D, freqs.cpu().numpy(), inter, m, 131072)
    assert bi.bi_check_device_errors() == bi.OK
