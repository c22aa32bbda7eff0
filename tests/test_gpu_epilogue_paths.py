"""Paths of the products with an epilogue that few shapes or calls reach: pairs of
CTAs whose warps come to their common barriers from work of single lanes, small
inputs that the call before writes, gates and scales past fp32's range, stages that
K does not fill, and operands whose tiles are walked in groups."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
from invariant_bi_rmsnorm_02_gb300 import synth
from oracle import linear8
from gpu_util import check_close, f64, first_divergence, same_bytes

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "q8"]


class Operands:
    """A and W of one product in either type, with their values in 64 bits."""

    def __init__(self, kind, M, N, K, dev, seed):
        self.kind = kind
        a = synth.normal_bf16((M, K), seed, device=dev)
        w = synth.normal_bf16((N, K), seed + 1, std=K ** -0.5, device=dev)
        self.b = synth.normal_bf16((N,), seed + 2, device=dev)
        if kind == "q8":
            self.a, self.w = bi.quantize_q8(a), bi.quantize_q8(w)
        else:
            self.a, self.w = (a,), (w,)

    def run(self, rows=slice(None), act=bi.ACT_NONE):
        a = tuple(t[rows] for t in self.a)
        call = bi.gemm_q8 if self.kind == "q8" else bi.gemm_epilogue
        return call(*a, *self.w, self.b, None, act)

    def values(self, side, rows):
        t = [x[rows] for x in side]
        if self.kind == "q8":
            return linear8.numbers(t[0].cpu().view(torch.uint8).numpy()) * f64(t[1])[:, None]
        return f64(t[0])

    def check(self, got, rows, act="none"):
        args = (self.values(self.a, rows), self.values(self.w, slice(None)), f64(self.b), None, act)
        check_close(f64(got[rows]), linear8.product(*args), linear8.product_bound(*args), act)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(130, 4096, 4096),      # 64 rows a CTA, the last CTA without any
                                   (200, 6144, 4096),
                                   (275, 392, 12864)])     # 128 rows a CTA, few tiles
def test_pairs_meet_at_their_start_and_end(cuda, kind, M, N, K):
    """A pair's CTAs meet after one thread has set the barriers up, and again
    after elected threads have copied, multiplied and stored: many short calls
    behind one another, each with the bytes of single-CTA calls."""
    c = Operands(kind, M, N, K, cuda, 100 + M)
    want = torch.cat([c.run(slice(at, min(at + 64, M))) for at in range(0, M, 64)])
    got = [c.run() for _ in range(60)]
    assert bi.bi_check_device_errors() == bi.OK
    for g in got:
        assert same_bytes(g, want), first_divergence(g, want)


def test_small_inputs_written_by_the_call_before(cuda):
    """The norm's weight, both scales and the bias, each written anew by the call
    right before the one that reads it: queued without a pause they give what they
    give with the device idle between them."""
    M, N, H = 200, 2048, 512
    bf = dict(dtype=torch.bfloat16, device=cuda)
    f8 = dict(dtype=torch.float8_e4m3fn, device=cuda)
    f32 = dict(dtype=torch.float32, device=cuda)
    x = synth.normal_bf16((M, H), 11, device=cuda)
    ws = [synth.normal_bf16((N, H), 12 + i, std=(i + 1) * H ** -0.5, device=cuda) for i in range(3)]
    ones = [synth.normal_bf16((1, 64), 20 + i, device=cuda) for i in range(3)]
    to_h = synth.normal_bf16((H, 64), 30, std=0.125, device=cuda)
    to_n = synth.normal_bf16((N, 64), 31, std=0.125, device=cuda)

    def rounds(pause):
        g, b = torch.empty(1, H, **bf), torch.empty(1, N, **bf)
        y8, ys = torch.empty(M, H, **f8), torch.empty(M, **f32)
        w8, sw = torch.empty(N, H, **f8), torch.empty(N, **f32)
        outs = [torch.empty(M, N, **bf) for _ in range(30)]
        torch.cuda.synchronize()
        for i, out in enumerate(outs):
            bi.bi_gemm_epilogue(ones[i % 3], to_h, g)                # the norm's weight
            pause()
            bi.bi_rmsnorm_q8(x, g.view(H), y8, ys, 1e-6)
            pause()
            bi.bi_gemm_epilogue(ones[(i + 1) % 3], to_n, b)          # the bias
            pause()
            bi.bi_quantize_q8(ws[(i // 2) % 3], w8, sw)              # the weight's scales
            pause()
            bi.bi_gemm_q8(y8, ys, w8, sw, out, bias=b.view(N))
            pause()
            bi.bi_gemm_epilogue(ones[i % 3], to_n, b)                # the bias right before
            pause()
            bi.bi_gemm_q8(y8, ys, w8, sw, out, bias=b.view(N), residual=out)
            pause()
            bi.bi_quantize_q8(x, y8, ys)                             # the rows' scales
            pause()
            bi.bi_gemm_q8(y8, ys, w8, sw, out, residual=out)
            pause()
        torch.cuda.synchronize()
        return outs

    want, got = rounds(torch.cuda.synchronize), rounds(lambda: None)
    assert not same_bytes(want[0], want[1])
    for a, b in zip(got, want):
        assert same_bytes(a, b), first_divergence(a, b)
    assert bi.bi_check_device_errors() == bi.OK


def test_swiglu_of_far_gates_under_large_ups(cuda):
    """silu(g) u to 2^-14 of its value and 2^-119 max(|u|, 1): gates where exp(-g)
    leaves fp32's range, under ups of every size.  (Without the factor |u| the
    second term does not hold: a gate of -88.5 under 1e30 gives 0 for -3e-7.)"""
    g = [-60.0, -80.0, -86.0, -87.0, -87.5, -88.5, -90.0, -95.0, -100.0, -200.0, -1e30, 0.0, 3.0, 88.0]
    u = [1e38, -1e30, 1e12, 1.0, -3.0, 1e-6, 1e-30, 0.0]
    A = torch.zeros(len(g) * len(u), 32)
    A[:, 0] = torch.tensor(g).repeat_interleave(len(u))
    A[:, 1] = torch.tensor(u).repeat(len(g))
    W = torch.zeros(32, 32)
    W[0, 0] = W[16, 1] = 1.0       # column 0's gate and up; each sum has one term
    A = A.to(torch.bfloat16)
    gv, uv = f64(A[:, 0]), f64(A[:, 1])
    got = f64(bi.gemm_epilogue(A.to(cuda), W.to(torch.bfloat16).to(cuda),
                               activation=bi.ACT_SWIGLU)[:, 0])
    assert bi.bi_check_device_errors() == bi.OK
    want = linear8.activation(gv, "silu") * uv
    over = np.abs(want) > 3.389e38            # (88 times 1e38: past bf16)
    assert np.isinf(got[over]).all()
    got, want, uv = got[~over], want[~over], uv[~over]

    def bound(least):                         # then one rounding to bf16
        e = 2.0 ** -14 * np.abs(want) + least
        return e + 2.0 ** -8 * (np.abs(want) + e) + 2.0 ** -134

    check_close(got, want, bound(2.0 ** -119 * np.maximum(np.abs(uv), 1.0)), "swiglu")
    assert (np.abs(got - want) > bound(2.0 ** -119)).any()


def test_infinite_scales(cuda):
    """A scale of infinity gives its row (A) or column (W) the sum's sign: relu
    leaves +inf, 0 and, where the sum is 0, NaN; the rest keeps its bytes."""
    M, N, K = 40, 96, 128
    c = Operands("q8", M, N, K, cuda, 7000)
    (a, sa), (w, sw) = c.a, c.w
    a.view(torch.uint8)[9, 1:] = 0            # row 9: one element, so that some
    w.view(torch.uint8)[40:44, 0] = 0         # sums are exactly 0
    a.view(torch.uint8)[12] = 0               # and, in column 17, a row of zeros
    want = bi.gemm_q8(a, sa, w, sw, activation=bi.ACT_RELU)
    sums = torch.from_numpy(linear8.numbers(a.cpu().view(torch.uint8).numpy())
                            @ linear8.numbers(w.cpu().view(torch.uint8).numpy()).T)
    sa[9], sw[17] = float("inf"), float("inf")
    got = bi.gemm_q8(a, sa, w, sw, activation=bi.ACT_RELU).cpu()
    assert bi.bi_check_device_errors() == bi.OK
    for rows, cols in ((9, slice(None)), (slice(None), 17)):
        s, g = sums[rows, cols], got[rows, cols]
        assert ((s > 0).sum() > 5 and (s < 0).sum() > 5 and (s == 0).any())
        assert (g[s > 0] == float("inf")).all()
        assert (g[s < 0] == 0).all()
        assert torch.isnan(g[s == 0]).all()
    rows = [i for i in range(M) if i != 9]
    cols = [j for j in range(N) if j != 17]
    assert same_bytes(got[rows][:, cols], want.cpu()[rows][:, cols])


def check_rows(c, got, rows):
    """Rows of A W^T + bias against 64-bit sums (on the device: long rows of many
    columns), within linear8.product_bound's terms for no activation."""
    def held(side, pick):
        v = side[0][pick].to(torch.float32).double()
        return v * side[1][pick].double()[:, None] if len(side) == 2 else v
    a, w, b = held(c.a, rows), held(c.w, slice(None)), c.b.double()
    want, mag = a @ w.T + b, a.abs() @ w.abs().T + b.abs()
    e = (a.shape[1] + 3) * 2.0 ** -23 * mag
    check_close(f64(got[rows]), f64(want), f64(e + 2.0 ** -8 * (want.abs() + e) + 2.0 ** -118),
                "%s %s" % (c.kind, tuple(got.shape)))


@pytest.mark.parametrize("kind,M,N,K", [
    # one copy for several k-blocks of rows that are whole k-blocks, some left over
    # at the end: five in fours and in twos, seven in fours
    ("q8", 16, 6144, 640), ("q8", 100, 1000, 640), ("q8", 16, 4096, 896),
    ("bf16", 16, 6144, 320), ("bf16", 100, 1000, 320), ("bf16", 16, 4096, 448),
    # pairs of 64 rows a CTA: two k-blocks a stage, an odd number of them; one a stage
    ("q8", 146, 5752, 10320), ("bf16", 146, 5752, 5160),
    ("q8", 159, 7808, 13296), ("bf16", 159, 7808, 6648),
    # pairs of 128 rows a CTA, two k-blocks a stage, an odd number of them
    ("bf16", 275, 392, 12864), ("q8", 275, 392, 25728)])
def test_stages_that_k_does_not_fill(cuda, kind, M, N, K):
    c = Operands(kind, M, N, K, cuda, 200 + M)
    got = c.run()
    check_rows(c, got, torch.tensor([0, 1, 7, M // 2, M - 1], device=cuda))
    for at in range(0, M, 50):                   # up to 64 rows: another form
        part = c.run(slice(at, min(at + 50, M)))
        assert same_bytes(got[at:at + 50], part), (at, first_divergence(got[at:at + 50], part))
    one = c.run(slice(M - 1, M))
    assert same_bytes(got[M - 1:], one)
    assert bi.bi_check_device_errors() == bi.OK


@pytest.mark.parametrize("kind,M,N,K", [("q8", 5400, 5600, 16384), ("q8", 5600, 5400, 16384),
                                        ("bf16", 5400, 6000, 8192), ("bf16", 6000, 5400, 8192),
                                        ("q8", 4400, 4600, 16000), ("q8", 4600, 4400, 16000)])
def test_operands_larger_than_the_cache_share(cuda, kind, M, N, K):
    """Both operands above 60 MiB: the smaller one's tiles are walked in two even
    groups, or in three, the last smaller.  Every row as calls of 1000 rows, in one
    group, give it."""
    c = Operands(kind, M, N, K, cuda, 300)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=cuda)
    if kind == "q8":
        bi.bi_gemm_q8(*c.a, *c.w, out, c.b)
    else:
        bi.bi_gemm_epilogue(*c.a, *c.w, out, c.b)
    assert bi.bi_check_device_errors() == bi.OK
    check_rows(c, out, torch.tensor([0, M // 2, M - 1], device=cuda))
    for at in range(0, M, 1000):
        part = c.run(slice(at, min(at + 1000, M)))
        assert same_bytes(out[at:at + 1000], part), (at, first_divergence(out[at:at + 1000], part))
