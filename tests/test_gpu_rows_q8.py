"""Rows held as e4m3 with a scale each, on the GPU: quantised bf16 rows have
the definition's bytes, the norm's have the bytes of quantising bi_rmsnorm's
fp32 values, rows that hold nothing, infinities or NaN, invariance over the
batch, in-place residuals, other streams and captured graphs."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
import oracle
from invariant_bi_rmsnorm_02_gb300 import synth
from oracle import linear8, longctx
from gpu_util import f64, same_bytes

pytestmark = pytest.mark.gpu

# one warp a row (one and two vectors a thread), blocks of one to eight vectors
# a thread, widths that are no power of two
WIDTHS = [16, 64, 256, 272, 512, 528, 1040, 2032, 2048, 4096, 14336, 32768, 40016, 65536]


def codes(y):
    return y.cpu().view(torch.uint8).numpy()


def stream_rows(M, H, seed, dev):
    """Rows of unlike size with a few large channels, in bf16."""
    x = synth.normal_bf16((M, H), seed).float()
    x *= torch.exp(0.8 * synth.normal_bf16((H,), seed + 1).float())
    x *= torch.exp2(synth.uniform_int(M, -30, 30, seed + 2).float())[:, None]
    return x.to(torch.bfloat16).to(dev)


@pytest.mark.parametrize("K", WIDTHS)
def test_quantised_rows_have_the_definitions_bytes(cuda, K):
    M = 11
    x = stream_rows(M, K, 100 + K, cuda)
    x[3] = 0
    x[4, 1:] = 0
    x[5] = -0.0
    x[6] = x[6].abs()
    y, s = bi.quantize_q8(x)
    assert bi.bi_check_device_errors() == bi.OK
    want, scale = linear8.quantise(f64(x))
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(codes(y), want)


def test_rows_of_every_magnitude(cuda):
    """Largest elements from subnormal bf16 numbers to the largest finite one."""
    e = torch.arange(-133, 128)
    x = synth.normal_bf16((len(e), 256), 7).double()
    x = x / x.abs().amax(1, keepdim=True) * torch.exp2(e.double())[:, None]
    x = x.to(torch.bfloat16).to(cuda)
    y, s = bi.quantize_q8(x)
    want, scale = linear8.quantise(f64(x))
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(codes(y), want)
    top = torch.full((1, 64), 3.3895313892515355e38, dtype=torch.bfloat16, device=cuda)
    y, s = bi.quantize_q8(top)
    assert (codes(y) == 0x7e).all() and torch.isfinite(s).all()


@pytest.mark.parametrize("K", [64, 1040, 4096])
def test_rows_with_infinities_or_nan(cuda, K):
    x = synth.normal_bf16((6, K), 9, device=cuda)
    x[1, 0] = float("inf")
    x[2, K - 1] = -float("inf")
    x[3, K // 2] = float("nan")
    x[4, 3], x[4, 4] = float("nan"), float("inf")
    y, s = bi.quantize_q8(x)
    want, scale = linear8.quantise(f64(x))
    assert np.array_equal(s.cpu().numpy(), scale, equal_nan=True)
    assert np.array_equal(codes(y), want)
    w = torch.ones(K, dtype=torch.bfloat16, device=cuda)
    y, s = bi.rmsnorm_q8(x, w)
    assert torch.isnan(s).cpu().tolist() == [False, True, True, True, True, False]
    assert (codes(y)[1:5] == 0).all()


def as_kernel_rounds(v32):
    """codes and scale of fp32 rows: v times 448 / t, the quotient and the
    product each rounded once to fp32."""
    v = v32.cpu().numpy()
    t = np.maximum(np.abs(v).max(1, keepdims=True), np.float32(linear8.LEAST_TOP))
    q = v * (np.float32(448.0) / t)
    return longctx.e4m3_codes(q.astype(np.float64)), (t[:, 0] / np.float32(448.0))


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("add", [False, True])
def test_norm_rows_have_the_bytes_of_quantising_the_norm(cuda, H, add):
    M = 9
    x, r = stream_rows(M, H, 300 + H, cuda), stream_rows(M, H, 400 + H, cuda)
    w = synth.normal_bf16((H,), 500 + H, std=0.2, mean=1.0, device=cuda)
    if add:
        want_h = r.clone()
        _, v = bi.add_rmsnorm(x, want_h, w, 1e-5, want_f32=True)
        y, s = bi.add_rmsnorm_q8(x, r, w, 1e-5)
        assert same_bytes(r, want_h)
    else:
        _, v = bi.rmsnorm(x, w, 1e-5, want_f32=True)
        y, s = bi.rmsnorm_q8(x, w, 1e-5)
    assert bi.bi_check_device_errors() == bi.OK
    want, scale = as_kernel_rounds(v)
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(codes(y), want)


@pytest.mark.parametrize("M,H", [(5, 64), (7, 1040), (3, 4096)])
def test_norm_rows_match_the_formula(cuda, M, H):
    x, r = stream_rows(M, H, 600, cuda), stream_rows(M, H, 700, cuda)
    w = synth.normal_bf16((H,), 800, std=0.2, mean=1.0, device=cuda)
    h_bits, v = oracle.add_rmsnorm(x.cpu(), r.cpu(), w.cpu(), 1e-5)
    h = torch.empty_like(x)
    y, s = (torch.empty(M, H, dtype=torch.float8_e4m3fn, device=cuda),
            torch.empty(M, dtype=torch.float32, device=cuda))
    bi.bi_add_rmsnorm_q8(x, r, w, h, y, s, 1e-5)
    assert np.array_equal(longctx.bits_of(h), h_bits)
    # v in fp32: the sum of squares is off by H 2^-24 of itself at most, which
    # the root halves; the mean, rsqrtf (2 units) and two products add 6 units
    ev = (H / 2 + 6) * 2.0 ** -24
    scale = np.abs(v).max(1) / 448.0
    g = s.cpu().numpy().astype(np.float64)
    assert (np.abs(g - scale) <= (ev + 2.0 ** -23) * scale).all()
    got = linear8.numbers(codes(y)) * g[:, None]
    # half an e4m3 step: 2^-4 of the value, 2^-10 of the scale where subnormal;
    # the scale's and the quotient's roundings beside it
    bound = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * g[:, None]) * (1 + 2.0 ** -10) + \
        (2 * ev + 2.0 ** -21) * np.abs(v)
    assert (np.abs(got - v) <= bound).all()


@pytest.mark.parametrize("H", [512, 4096])
def test_a_row_does_not_depend_on_its_batch(cuda, H):
    M = 517
    x, r = stream_rows(M, H, 31, cuda), stream_rows(M, H, 32, cuda)
    w = synth.normal_bf16((H,), 33, std=0.2, mean=1.0, device=cuda)
    idx = torch.tensor([516, 0, 77, 300], device=cuda)
    for call in (lambda i: bi.quantize_q8(x[i].contiguous()),
                 lambda i: bi.rmsnorm_q8(x[i].contiguous(), w),
                 lambda i: bi.add_rmsnorm_q8(x[i].contiguous(), r[i].contiguous(), w)):
        y, s = call(torch.arange(M, device=cuda))
        for sel in (torch.arange(1, device=cuda), torch.arange(9, device=cuda), idx):
            ys, ss = call(sel)
            assert same_bytes(ys, y[sel]) and same_bytes(ss, s[sel])


def test_blocks_that_take_several_rows(cuda):
    """More rows of more than 8192 elements than blocks: the same bytes as few."""
    M, K = 700, 12304
    x = stream_rows(M, K, 61, cuda)
    x[311, 5] = float("nan")
    y, s = bi.quantize_q8(x)
    for at in range(0, M, 100):
        ys, ss = bi.quantize_q8(x[at:at + 100].contiguous())
        assert same_bytes(ys, y[at:at + 100])
        assert same_bytes(ss, s[at:at + 100])
    want, scale = linear8.quantise(f64(x[300:320]))
    assert np.array_equal(codes(y[300:320]), want)
    assert np.array_equal(s[300:320].cpu().numpy(), scale, equal_nan=True)


def test_rows_past_32_bits(cuda):
    """2.3e9 elements: rows at both ends as a small call gives them."""
    M, H = 140000, 16400
    x = torch.empty(M, H, dtype=torch.bfloat16, device=cuda)
    part = stream_rows(7, H, 71, cuda)
    x[:] = part[0]
    x[M - 7:] = part
    x[M // 2:M // 2 + 7] = part.flip(0)
    w = synth.normal_bf16((H,), 72, device=cuda)
    for call in (bi.quantize_q8, lambda t: bi.rmsnorm_q8(t, w),
                 lambda t: bi.add_rmsnorm_q8(t, t.clone(), w)):
        y, s = call(x)
        for at in (0, M // 2, M - 7):
            ys, ss = call(x[at:at + 7].contiguous())
            assert same_bytes(ys, y[at:at + 7]) and same_bytes(ss, s[at:at + 7])


def test_in_place_streams_and_what_lies_behind_the_last_row(cuda):
    M, H, more = 13, 1040, 3
    x, r = stream_rows(M, H, 41, cuda), stream_rows(M, H, 42, cuda)
    w = synth.normal_bf16((H,), 43, device=cuda)
    h = torch.empty_like(x)
    y = torch.full((M + more, H), 0x55, dtype=torch.uint8, device=cuda).view(torch.float8_e4m3fn)
    s = torch.full((M + more,), 7.0, device=cuda)
    bi.bi_add_rmsnorm_q8(x, r, w, h, y[:M], s[:M], 1e-6)
    assert (y[M:].view(torch.uint8) == 0x55).all() and (s[M:] == 7.0).all()
    for over in ("r", "x"):
        t = {"x": x.clone(), "r": r.clone()}
        y2, s2 = torch.empty_like(y[:M]), torch.empty_like(s[:M])
        bi.bi_add_rmsnorm_q8(t["x"], t["r"], w, t[over], y2, s2, 1e-6)
        assert same_bytes(t[over], h) and same_bytes(y2, y[:M]) and same_bytes(s2, s[:M])
    assert bi.bi_check_device_errors() == bi.OK


def test_empty_calls(cuda):
    w = torch.ones(64, dtype=torch.bfloat16, device=cuda)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=cuda)
    for y, s in (bi.quantize_q8(x), bi.rmsnorm_q8(x, w), bi.add_rmsnorm_q8(x, x.clone(), w)):
        assert y.shape == (0, 64) and s.shape == (0,)


def test_refusals_of_the_binding(cuda):
    x = synth.normal_bf16((4, 64), 1, device=cuda)
    y = torch.empty(4, 64, dtype=torch.float8_e4m3fn, device=cuda)
    s = torch.empty(4, dtype=torch.float32, device=cuda)
    with pytest.raises(TypeError):
        bi.bi_quantize_q8(x.cpu(), y, s)
    with pytest.raises(TypeError):
        bi.bi_quantize_q8(x.half(), y, s)
    with pytest.raises(TypeError):
        bi.bi_quantize_q8(x, y.view(torch.uint8), s)
    with pytest.raises(ValueError):
        bi.bi_quantize_q8(synth.normal_bf16((4, 128), 1, device=cuda)[:, ::2], y, s)
    with pytest.raises(bi.BiError):
        bi.quantize_q8(synth.normal_bf16((4, 24), 1, device=cuda))


def test_other_streams_and_graphs(cuda):
    M, H = 40, 4096
    x, r = stream_rows(M, H, 51, cuda), stream_rows(M, H, 52, cuda)
    w = synth.normal_bf16((H,), 53, device=cuda)
    want = bi.add_rmsnorm_q8(x, r.clone(), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2 = r.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = bi.add_rmsnorm_q8(x, r2, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(same_bytes(a, b) for a, b in zip(got, want))
    h = torch.empty_like(r)
    y, s = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bi.bi_add_rmsnorm_q8(x, r, w, h, y, s, 1e-6)
    for _ in range(2):
        y.view(torch.uint8).zero_()
        s.zero_()
        g.replay()
    assert same_bytes(y, want[0]) and same_bytes(s, want[1]) and same_bytes(h, r2)
    assert bi.bi_check_device_errors() == bi.OK
