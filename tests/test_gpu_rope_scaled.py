"""Rotary positions with scaled frequencies, both pair arrangements and part
of the head, on the GPU against the fp64 definition."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
from invariant_bi_rmsnorm_02_gb300 import synth
from oracle import longctx
from gpu_util import bf16_half_ulp, check_close, f64, same_bytes

pytestmark = pytest.mark.gpu
KINDS = {"none": bi.ROPE_NONE, "linear": bi.ROPE_LINEAR, "ntk": bi.ROPE_NTK,
         "llama3": bi.ROPE_LLAMA3, "yarn": bi.ROPE_YARN}


def check(q, k, v, qkv, pos, Hq, Hkv, D, freqs, inter, m, far):
    T = len(pos)
    x = f64(qkv).reshape(T, Hq + 2 * Hkv, D)
    n = len(freqs)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + n)
    y = longctx.rope(x[:, :Hq + Hkv], pos, freqs, inter, m)
    both = np.zeros_like(y)           # |x0| + |x1| of each element's pair
    both[..., a] = both[..., b] = np.abs(x[:, :Hq + Hkv][..., a]) + np.abs(x[:, :Hq + Hkv][..., b])
    got = np.concatenate([f64(q), f64(k)], 1)
    # fp32: the turn rounded to 24 bits (an angle off by at most pi 2^-24),
    # cosine and sine 2 ulp each, the factor, two products and a sum: below
    # 2^-21 of m (|x0| + |x1|); far positions add the fp64 oracle's own
    # rounding of pos * freq, 2^-53 of the turns made
    slack = m * both * (2.0 ** -21 + 2 * np.pi * far * 2.0 ** -52)
    # half a bf16 step at the larger of the two magnitudes, then the slack
    bound = np.maximum(bf16_half_ulp(got), bf16_half_ulp(y)) + slack + 1e-40
    check_close(got, y, bound, "rope")
    assert np.array_equal(got[..., 2 * n:], x[:, :Hq + Hkv, 2 * n:])
    assert np.array_equal(f64(v), x[:, Hq + Hkv:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", [(1, 32, 8, 128, 128), (37, 4, 2, 64, 64),
                                            (5, 16, 16, 128, 32), (3, 7, 1, 80, 20),
                                            (9, 2, 1, 256, 6), (2, 1, 1, 16, 2),
                                            (33, 3, 2, 80, 80), (6, 8, 8, 128, 8),
                                            (4, 2, 2, 1024, 1024), (130, 24, 8, 64, 48)])
def test_rope_matches_the_definition(cuda, T, Hq, Hkv, D, rot, inter):
    freqs, m = bi.rope_frequencies(rot, 10000.0)
    qkv = synth.normal_bf16((T, (Hq + 2 * Hkv) * D), 30000 + T + D, device=cuda)
    pos = synth.uniform_int(T, 0, 131072, 30001 + T).to(torch.int32)
    pos[0] = 0 if T > 1 else 77
    q, k, v = bi.rope_qkv_scaled(qkv, pos.to(cuda), Hq, Hkv, D, freqs, inter, m)
    assert bi.bi_check_device_errors() == bi.OK
    check(q, k, v, qkv, pos.tolist(), Hq, Hkv, D, freqs.cpu().numpy(), inter, m, 131072)
    if T > 1:
        assert np.array_equal(f64(q)[0], f64(qkv)[0, :Hq * D].reshape(Hq, D))


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_rope_scalings_far_and_negative_positions(cuda, kind):
    T, Hq, Hkv, D, rot = 12, 4, 2, 128, 128
    want, wm = longctx.frequencies(rot, 500000.0, kind, 8.0, 8192.0, 1.0, 32.0)
    freqs, m = bi.rope_frequencies(rot, 500000.0, KINDS[kind], 8.0, 8192.0, 1.0, 32.0)
    f = freqs.cpu().numpy()
    assert (np.abs(f - want) <= 2.0 ** -46 * want).all() and abs(m - wm) < 2.0 ** -23 * wm
    pos = [0, 1, 2, 8191, 8192, 65535, 1 << 20, (1 << 31) - 1, -1, -8192, -(1 << 31), 12345]
    qkv = synth.normal_bf16((T, (Hq + 2 * Hkv) * D), 31000, device=cuda)
    for inter in (False, True):
        q, k, v = bi.rope_qkv_scaled(qkv, torch.tensor(pos, dtype=torch.int32, device=cuda), Hq,
                                     Hkv, D, freqs, inter, m)
        assert bi.bi_check_device_errors() == bi.OK
        check(q, k, v, qkv, pos, Hq, Hkv, D, f, inter, m, 2.0 ** 31)


def test_rope_small_angles_keep_their_precision(cuda):
    # a pair that turns by 2^-30 a position: y1 = x1 + x0 sin has to show it
    D = 16
    freqs = torch.tensor([2.0 ** -30], dtype=torch.float64, device=cuda)
    qkv = torch.zeros(1, 3 * D, dtype=torch.bfloat16, device=cuda)
    qkv[0, 0] = qkv[0, D] = 1.0
    q, k, _ = bi.rope_qkv_scaled(qkv, torch.tensor([3], dtype=torch.int32, device=cuda), 1, 1, D,
                                 freqs)
    want = np.sin(3 * 2.0 ** -30)
    assert abs(f64(q)[0, 0, 1] - want) <= 2.0 ** -8 * want
    assert abs(f64(k)[0, 0, 1] - want) <= 2.0 ** -8 * want


@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (128, 64, True), (80, 20, False)])
def test_rope_rows_do_not_depend_on_the_batch(cuda, D, rot, inter):
    T, Hq, Hkv = 333, 8, 2
    freqs, m = bi.rope_frequencies(rot, 10000.0, bi.ROPE_YARN, 4.0, 8192, 1.0, 32.0)
    qkv = synth.normal_bf16((T, (Hq + 2 * Hkv) * D), 32000, device=cuda)
    pos = synth.uniform_int(T, 0, 40000, 32001).to(torch.int32).to(cuda)
    whole = bi.rope_qkv_scaled(qkv, pos, Hq, Hkv, D, freqs, inter, m)
    for a, b in ((0, 1), (1, 8), (100, 333)):
        part = bi.rope_qkv_scaled(qkv[a:b].contiguous(), pos[a:b].contiguous(), Hq, Hkv, D, freqs,
                                  inter, m)
        for x, y in zip(whole, part):
            assert same_bytes(x[a:b].contiguous(), y)


def test_rope_non_finite_frequencies_and_inputs_stay_in_their_pairs(cuda):
    D, T = 64, 2
    freqs = torch.full((D // 2,), 0.25, dtype=torch.float64, device=cuda)
    freqs[3] = float("inf")
    qkv = synth.normal_bf16((T, 3 * D), 33000, device=cuda)
    qkv[1, 5] = float("nan")
    q, k, v = bi.rope_qkv_scaled(qkv, torch.tensor([4, 9], dtype=torch.int32, device=cuda), 1, 1,
                                 D, freqs)
    bad = torch.isnan(q[:, 0])
    want = torch.zeros(T, D, dtype=torch.bool, device=cuda)
    want[:, 3] = want[:, 3 + D // 2] = True
    want[1, 5] = want[1, 5 + D // 2] = True
    assert torch.equal(bad, want) and not torch.isnan(v).any()
    want[1, 5] = want[1, 5 + D // 2] = False
    assert torch.equal(torch.isnan(k[:, 0]), want)
