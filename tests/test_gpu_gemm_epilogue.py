"""The GEMM with bias, activation and residual in its epilogue, on bf16 and on
e4m3 operands: against the 64-bit definition, the plain GEMM's bytes without
an epilogue, rows that do not depend on the batch whatever tiles serve them,
residuals in place, ragged sizes, and a run of the 8-bit layer's calls."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
from invariant_bi_rmsnorm_02_gb300 import synth
from oracle import linear8, longctx
from gpu_util import check_close, f64, first_divergence, same_bytes

pytestmark = pytest.mark.gpu

ACTS = {"none": bi.ACT_NONE, "relu": bi.ACT_RELU, "gelu": bi.ACT_GELU,
        "gelu_tanh": bi.ACT_GELU_TANH, "silu": bi.ACT_SILU, "swiglu": bi.ACT_SWIGLU}


class Case:
    """Operands of one product, and their values in 64 bits."""

    def __init__(self, kind, M, N, K, dev, seed, act="none", bias=True, residual=True, spread=1.0):
        self.kind, self.act = kind, ACTS[act]
        a = synth.normal_bf16((M, K), seed, std=spread)
        w = synth.normal_bf16((N, K), seed + 1, std=K ** -0.5)
        n = N // 2 if act == "swiglu" else N
        self.b = synth.normal_bf16((N,), seed + 2).to(dev) if bias else None
        self.r = synth.normal_bf16((M, n), seed + 3).to(dev) if residual else None
        if kind == "q8":
            (self.a, self.sa), (self.w, self.sw) = (bi.quantize_q8(t.to(dev)) for t in (a, w))
            self.va, self.vw = (linear8.numbers(t.cpu().view(torch.uint8).numpy()) *
                                f64(s)[:, None] for t, s in ((self.a, self.sa), (self.w, self.sw)))
        else:
            self.a, self.w = a.to(dev), w.to(dev)
            self.va, self.vw = f64(a), f64(w)
        self.vb = None if self.b is None else f64(self.b)
        self.vr = None if self.r is None else f64(self.r)
        self.name = act

    def run(self, rows=slice(None)):
        r = None if self.r is None else self.r[rows].contiguous()
        if self.kind == "q8":
            return bi.gemm_q8(self.a.view(torch.uint8)[rows].contiguous()
                              .view(torch.float8_e4m3fn), self.sa[rows].contiguous(), self.w,
                              self.sw, self.b, r, self.act)
        return bi.gemm_epilogue(self.a[rows].contiguous(), self.w, self.b, r, self.act)

    def check(self):
        got = f64(self.run())
        assert bi.bi_check_device_errors() == bi.OK
        args = (self.va, self.vw, self.vb, self.vr, self.name)
        check_close(got, linear8.product(*args), linear8.product_bound(*args),
                    "%s %s %s" % (self.kind, self.name, got.shape))


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("kind,M,N,K", [("bf16", 1, 32, 8), ("bf16", 33, 96, 72),
                                        ("bf16", 130, 2080, 1000), ("bf16", 64, 736, 512),
                                        ("q8", 1, 32, 16), ("q8", 33, 96, 144),
                                        ("q8", 130, 2080, 1136), ("q8", 64, 736, 512)])
def test_products_match_the_definition(cuda, act, kind, M, N, K):
    # (a spread that takes the activations into both tails)
    Case(kind, M, N, K, cuda, 1000 + M, act, spread=4.0).check()


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_each_part_of_the_epilogue_is_optional(cuda, kind, bias, residual):
    for act in ("none", "gelu", "swiglu"):
        Case(kind, 70, 224, 272, cuda, 2000, act, bias, residual).check()


@pytest.mark.parametrize("N", [8, 16, 24, 40, 248, 264, 520, 1000])
@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_widths_that_end_inside_a_tile(cuda, kind, N):
    for M in (1, 65, 129):
        c = Case(kind, M, N, 128, cuda, 3000 + N, "silu")
        c.check()
        # nothing is written past the last row
        n = c.r.shape[1]
        out = torch.full((M + 2, n), 5.0, dtype=torch.bfloat16, device=cuda)
        if kind == "q8":
            bi.bi_gemm_q8(c.a, c.sa, c.w, c.sw, out[:M], c.b, c.r, c.act)
        else:
            bi.bi_gemm_epilogue(c.a, c.w, out[:M], c.b, c.r, c.act)
        assert same_bytes(out[:M], c.run()) and (out[M:] == 5.0).all()


@pytest.mark.parametrize("M,N,K", [(1, 6144, 4096), (16, 4096, 4096), (48, 520, 200),
                                   (128, 14336, 512), (200, 2056, 1000), (700, 6144, 256),
                                   (1025, 4104, 136)])
def test_without_an_epilogue_it_has_the_plain_gemms_bytes(cuda, M, N, K):
    A = synth.normal_bf16((M, K), 4000 + M, device=cuda)
    W = synth.normal_bf16((N, K), 4001 + N, std=0.05, device=cuda)
    got, want = bi.gemm_epilogue(A, W), bi.gemm(A, W)
    assert bi.bi_check_device_errors() == bi.OK
    assert same_bytes(got, want), first_divergence(got, want)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("N,K,act", [(6144, 1024, "none"), (4096, 2048, "gelu"),
                                     (2080, 272, "swiglu"), (512, 4096, "none")])
def test_rows_do_not_depend_on_the_batch(cuda, kind, N, K, act):
    """Every tile width and operand ring that a batch size leads to gives a row
    the same bytes."""
    c = Case(kind, 2100, N, K, cuda, 5000 + N, act)
    full = c.run()
    for M in (1, 2, 17, 32, 33, 64, 65, 128, 129, 256, 300, 513, 1024):
        got = c.run(slice(0, M))
        assert same_bytes(got, full[:M]), (M, first_divergence(got, full[:M]))
    idx = torch.tensor([2099, 3, 130, 1000, 64], device=cuda)
    assert same_bytes(c.run(idx), full[idx])
    assert bi.bi_check_device_errors() == bi.OK


@pytest.mark.parametrize("kind,M,N,K,act", [("bf16", 5, 4096, 512, "none"),
                                            ("bf16", 300, 1000, 512, "gelu"),
                                            ("q8", 5, 4096, 512, "none"),
                                            ("q8", 300, 2080, 512, "swiglu")])
def test_the_residual_in_place(cuda, kind, M, N, K, act):
    c = Case(kind, M, N, K, cuda, 6000 + M, act)
    want = c.run()
    for _ in range(3):
        h = c.r.clone()
        if kind == "q8":
            bi.bi_gemm_q8(c.a, c.sa, c.w, c.sw, h, c.b, h, c.act)
        else:
            bi.bi_gemm_epilogue(c.a, c.w, h, c.b, h, c.act)
        assert same_bytes(h, want)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_values_that_are_not_finite_stay_in_their_row(cuda, kind):
    M, N, K = 40, 96, 128
    c = Case(kind, M, N, K, cuda, 7000, "relu", bias=False, residual=False)
    want = c.run()
    if kind == "q8":
        c.sa[7], c.sa[9] = float("nan"), float("inf")
    else:
        c.a[7, 5], c.a[9, :] = float("nan"), float("inf")
    got = c.run()
    rows = [i for i in range(M) if i not in (7, 9)]
    assert same_bytes(got[rows], want[rows])
    assert torch.isnan(got[7]).all()
    assert not torch.isfinite(got[9]).any() or kind == "q8"
    c = Case(kind, M, N, K, cuda, 7000, "none", bias=True, residual=False)
    want = c.run()
    c.b[11] = float("-inf")
    got = c.run()
    assert (got[:, 11] == float("-inf")).all()
    cols = [j for j in range(N) if j != 11]
    assert same_bytes(got[:, cols].contiguous(), want[:, cols].contiguous())


def test_e4m3_nan_bytes(cuda):
    for M in (5, 200):
        c = Case("q8", M, 96, 144, cuda, 7100 + M, "silu", residual=False)
        want = c.run()
        c.a.view(torch.uint8)[3, 100] = 0x7f
        c.w.view(torch.uint8)[50, 7] = 0xff
        got = c.run()
        assert torch.isnan(got[3]).all() and torch.isnan(got[:, 50]).all()
        rows = [i for i in range(M) if i != 3]
        cols = [j for j in range(96) if j != 50]
        assert same_bytes(got[rows][:, cols].contiguous(), want[rows][:, cols].contiguous())


def test_activations_at_their_ends(cuda):
    """z far into both tails, both infinities and NaN, through a product with an
    identity."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 2.0 ** -120, 0.5, -0.5, 5.0, -5.0, -12.0, -30.0, -87.0,
                      -88.5, -100.0, -1e4, -3e38, 12.0, 30.0, 1e4, 3e38, float("inf"),
                      -float("inf"), float("nan")])
    A = torch.zeros(len(z), 32)
    A[:, 0] = z
    W = torch.zeros(32, 32)
    W[0, 0] = 1.0        # column 0 is z, the others 0 (0 times inf or NaN: NaN)
    A, W = A.to(torch.bfloat16).to(cuda), W.to(torch.bfloat16).to(cuda)
    zb = A[:, 0].double().cpu().numpy()
    inf = np.inf
    ends = {"none": (inf, -inf), "relu": (inf, 0.0), "gelu": (inf, 0.0), "gelu_tanh": (inf, None),
            "silu": (inf, None)}
    for act, (hi, lo) in ends.items():
        got = bi.gemm_epilogue(A, W, activation=ACTS[act])[:, 0].double().cpu().numpy()
        fin = np.isfinite(zb)
        want = linear8.activation(zb[fin], act)
        bound = 2.0 ** -14 * np.abs(want) + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -118
        assert (np.abs(got[fin] - want) <= bound).all(), (act, got, want)
        assert got[20] == hi and (np.isnan(got[21]) if lo is None else got[21] == lo), act
        assert np.isnan(got[22]), act


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_operands_on_16_byte_boundaries(cuda, kind):
    """Every pointer 16 bytes past a 256-byte boundary, rows of no whole k-block."""
    def off(t):
        n = t.numel() * t.element_size()
        b = torch.zeros(n + 272, dtype=torch.uint8, device=cuda)
        at = (-b.data_ptr()) % 256 + 16
        v = b[at:at + n].view(t.dtype).view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v
    for M in (3, 65, 300):
        c = Case(kind, M, 328, 208, cuda, 9000 + M, "gelu")
        want = c.run()
        out = off(torch.zeros_like(want))
        b, r = off(c.b), off(c.r)
        if kind == "q8":
            bi.bi_gemm_q8(off(c.a), off(c.sa), off(c.w), off(c.sw), out, b, r, c.act)
        else:
            bi.bi_gemm_epilogue(off(c.a), off(c.w), out, b, r, c.act)
        assert same_bytes(out, want)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_outputs_past_32_bits(cuda, kind):
    """C of 2.3e9 elements with a residual: rows at both ends as a small call
    gives them."""
    M, N, K = 70016, 32768, 64
    A = synth.normal_bf16((M, K), 41, device=cuda)
    W = synth.normal_bf16((N, K), 42, std=0.1, device=cuda)
    b = synth.normal_bf16((N,), 43, device=cuda)
    h = torch.full((M, N), 0.5, dtype=torch.bfloat16, device=cuda)
    if kind == "q8":
        (a, sa), (w, sw) = bi.quantize_q8(A), bi.quantize_q8(W)
        bi.bi_gemm_q8(a, sa, w, sw, h, b, h, bi.ACT_SILU)
        few = lambda i: bi.gemm_q8(a[i].contiguous(), sa[i].contiguous(), w, sw, b,
                                   torch.full((i.stop - i.start, N), 0.5, dtype=torch.bfloat16,
                                              device=cuda), bi.ACT_SILU)
    else:
        bi.bi_gemm_epilogue(A, W, h, b, h, bi.ACT_SILU)
        few = lambda i: bi.gemm_epilogue(A[i].contiguous(), W, b,
                                         torch.full((i.stop - i.start, N), 0.5,
                                                    dtype=torch.bfloat16, device=cuda), bi.ACT_SILU)
    for i in (slice(0, 5), slice(M // 2 - 3, M // 2 + 3), slice(65530, 65540), slice(M - 130, M)):
        assert same_bytes(h[i], few(i))
    assert bi.bi_check_device_errors() == bi.OK


def test_e4m3_sums_are_exact_where_fp32_holds_them(cuda):
    """Operands whose products and partial sums are integers below 2^24: every
    output is the integer sum rounded once."""
    M, N, K = 150, 264, 2048
    rng = np.random.default_rng(8)
    a = torch.from_numpy(rng.integers(-8, 9, (M, K)).astype(np.float32))
    w = torch.from_numpy(rng.integers(-8, 9, (N, K)).astype(np.float32))
    one = lambda n: torch.ones(n, dtype=torch.float32, device=cuda)
    got = bi.gemm_q8(a.to(torch.float8_e4m3fn).to(cuda), one(M), w.to(torch.float8_e4m3fn).to(cuda),
                     one(N))
    want = (a.double() @ w.double().T).to(torch.bfloat16)
    assert same_bytes(got.cpu(), want)
    # scales: (sum * a_scale) * w_scale, each product rounded once
    sa = torch.from_numpy(np.exp2(rng.normal(size=M)).astype(np.float32))
    sw = torch.from_numpy(np.exp2(rng.normal(size=N)).astype(np.float32))
    got = bi.gemm_q8(a.to(torch.float8_e4m3fn).to(cuda), sa.to(cuda),
                     w.to(torch.float8_e4m3fn).to(cuda), sw.to(cuda))
    want = ((a.double() @ w.double().T).float() * sa[:, None] * sw).to(torch.bfloat16)
    assert same_bytes(got.cpu(), want)


def test_empty_calls_and_refusals(cuda):
    c = Case("q8", 4, 32, 64, cuda, 1)
    none = torch.empty(0, 64, dtype=torch.bfloat16, device=cuda)
    assert bi.gemm_epilogue(none, synth.normal_bf16((32, 64), 1, device=cuda)).shape == (0, 32)
    assert bi.gemm_q8(c.a[:0], c.sa[:0], c.w, c.sw).shape == (0, 32)
    with pytest.raises(TypeError):
        bi.gemm_q8(c.a.view(torch.uint8), c.sa, c.w, c.sw)
    with pytest.raises(TypeError):
        bi.gemm_q8(c.a, c.sa.double(), c.w, c.sw)
    with pytest.raises(TypeError):
        bi.gemm_epilogue(none.float(), none)
    with pytest.raises(bi.BiError):
        bi.gemm_q8(c.a, c.sa, c.w, c.sw, activation=9)
    with pytest.raises(bi.BiError):
        bi.gemm_epilogue(synth.normal_bf16((4, 60), 1, device=cuda),
                         synth.normal_bf16((32, 60), 1, device=cuda))


def test_two_at_once_on_two_streams(cuda):
    cs = [Case("q8", 200, 1040, 512, cuda, 8000 + i, "gelu") for i in range(2)]
    want = [c.run() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = [bi.gemm_q8(c.a, c.sa, c.w, c.sw, c.b, c.r, c.act, stream=s)
               for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        assert all(same_bytes(a, b) for a, b in zip(got, want))
    assert bi.bi_check_device_errors() == bi.OK


def test_an_8_bit_feed_forward_layer(cuda):
    """norm -> gate/up with SwiGLU -> quantise -> down onto the residual
    stream, eagerly and from a captured graph, against its definition stage by
    stage."""
    M, H, F = 37, 512, 1040
    h0 = synth.normal_bf16((M, H), 91, device=cuda)
    g = synth.normal_bf16((H,), 92, std=0.1, mean=1.0, device=cuda)
    wgu = synth.normal_bf16((2 * F, H), 93, std=H ** -0.5, device=cuda)
    wd = synth.normal_bf16((H, F), 94, std=F ** -0.5, device=cuda)
    perm = torch.from_numpy(bi.swiglu_interleave(F, 16)).long().to(cuda)
    wgu8, sgu = bi.quantize_q8(wgu[perm].contiguous())
    wd8, sd = bi.quantize_q8(wd)
    f8 = dict(dtype=torch.float8_e4m3fn, device=cuda)
    f32 = dict(dtype=torch.float32, device=cuda)
    y8, ys = torch.empty(M, H, **f8), torch.empty(M, **f32)
    a8, as_ = torch.empty(M, F, **f8), torch.empty(M, **f32)
    act = torch.empty(M, F, dtype=torch.bfloat16, device=cuda)

    def layer(h):
        bi.bi_rmsnorm_q8(h, g, y8, ys, 1e-5)
        bi.bi_gemm_q8(y8, ys, wgu8, sgu, act, activation=bi.ACT_SWIGLU)
        bi.bi_quantize_q8(act, a8, as_)
        bi.bi_gemm_q8(a8, as_, wd8, sd, h, residual=h)

    h = h0.clone()
    layer(h)
    values = lambda q, s: linear8.numbers(q.cpu().view(torch.uint8).numpy()) * f64(s)[:, None]
    args = (values(y8, ys), values(wgu8, sgu), None, None, "swiglu")
    check_close(f64(act), linear8.product(*args), linear8.product_bound(*args), "gate/up")
    want, scale = linear8.quantise(f64(act))
    assert np.array_equal(as_.cpu().numpy(), scale)
    assert np.array_equal(a8.cpu().view(torch.uint8).numpy(), want)
    args = (values(a8, as_), values(wd8, sd), None, f64(h0), "none")
    check_close(f64(h), linear8.product(*args), linear8.product_bound(*args), "down")
    # the whole against the bf16 layer's definition: 8 bits keep about 2^-4 of
    # each operand, whose errors add up like noise
    v = f64(h0)
    v = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-5) * f64(g)
    z = v @ f64(wgu).T
    ref = linear8.activation(z[:, :F], "silu") * z[:, F:] @ f64(wd).T
    got = f64(h) - f64(h0)
    assert np.linalg.norm(got - ref) < 0.12 * np.linalg.norm(ref)
    hg = h0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(hg)
    for _ in range(2):
        hg.copy_(h0)
        graph.replay()
    assert same_bytes(hg, h)
    assert bi.bi_check_device_errors() == bi.OK


def test_the_longest_rows(cuda):
    """The largest K there is: a tile's sum lasts more than a second."""
    M, N, K = 1, 8, 2 ** 31 - 1024
    a = torch.zeros(M, K, dtype=torch.float8_e4m3fn, device=cuda)
    w = torch.zeros(N, K, dtype=torch.float8_e4m3fn, device=cuda)
    at = torch.tensor([0, 127, 2 ** 30, 2 ** 31 - 2048, K - 1], device=cuda)
    one = 0x38  # e4m3
    a.view(torch.uint8)[0, at] = one
    for n in range(N):
        w.view(torch.uint8)[n, at[:n % 6]] = one
    scale = torch.ones(N, dtype=torch.float32, device=cuda)
    got = bi.gemm_q8(a, scale[:1], w, scale)
    assert bi.bi_check_device_errors() == bi.OK
    assert got[0].tolist() == [float(n % 6) for n in range(N)]


def chain(x8, sx, w, sw, act, a8, sa, wd, sd, h):
    """Four calls, each of which reads what the one before it wrote."""
    bi.bi_quantize_q8(h, x8, sx)
    bi.bi_gemm_q8(x8, sx, w, sw, act, activation=bi.ACT_GELU_TANH)
    bi.bi_quantize_q8(act, a8, sa)
    bi.bi_gemm_q8(a8, sa, wd, sd, h, residual=h)


@pytest.mark.parametrize("M", [3, 100, 300, 2048])
def test_calls_that_follow_one_another(cuda, M):
    """The feed-forward calls thirty times over the same buffers, with nothing
    between them: queued at once, from a graph, and from two graphs on two
    streams they give what they give with the device idle between them."""
    H, F = 512, 1104
    f8 = dict(dtype=torch.float8_e4m3fn, device=cuda)
    w, sw = bi.quantize_q8(synth.normal_bf16((F, H), 61, std=H ** -0.5, device=cuda))
    wd, sd = bi.quantize_q8(synth.normal_bf16((H, F), 62, std=F ** -0.5, device=cuda))
    starts = [synth.normal_bf16((M, H), 63 + i, device=cuda) for i in range(2)]

    def buffers():
        return (torch.empty(M, H, **f8), torch.empty(M, dtype=torch.float32, device=cuda), w, sw,
                torch.empty(M, F, dtype=torch.bfloat16, device=cuda), torch.empty(M, F, **f8),
                torch.empty(M, dtype=torch.float32, device=cuda), wd, sd)

    want = []
    for h0 in starts:
        h, b = h0.clone(), buffers()
        for _ in range(30):
            bi.bi_quantize_q8(h, b[0], b[1])
            torch.cuda.synchronize()
            bi.bi_gemm_q8(*b[:5], activation=bi.ACT_GELU_TANH)
            torch.cuda.synchronize()
            bi.bi_quantize_q8(b[4], b[5], b[6])
            torch.cuda.synchronize()
            bi.bi_gemm_q8(*b[5:], h, residual=h)
            torch.cuda.synchronize()
        want.append(h)
    assert torch.isfinite(want[0]).all() and not same_bytes(want[0], starts[0])
    h, b = starts[0].clone(), buffers()
    for _ in range(30):
        chain(*b, h)
    assert same_bytes(h, want[0])
    hs, graphs = [torch.empty_like(h) for h in starts], []
    for i in range(2):
        b = buffers()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(30):
                chain(*b, hs[i])
        graphs.append((g, b))
    streams = [torch.cuda.Stream() for _ in starts]
    for _ in range(2):
        for i in range(2):
            hs[i].copy_(starts[i])
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert same_bytes(hs[i], want[i]), first_divergence(hs[i], want[i])
    assert bi.bi_check_device_errors() == bi.OK


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("N,K,act", [(6144, 4096, "none"), (4104, 8192, "gelu"),
                                     (6176, 4096, "swiglu")])
def test_rows_of_a_few_hundred_and_a_long_k(cuda, kind, N, K, act):
    """Batches that pairs of 64 rows a CTA take, their columns in two halves of
    the accumulator's lanes: the bytes of small and of large batches, and the
    64-bit definition."""
    c = Case(kind, 1100, N, K, cuda, 7000 + N, act)
    full = c.run()
    for M in (40, 64, 128, 130, 200, 256, 300, 384, 520, 777):
        got = c.run(slice(0, M))
        assert same_bytes(got, full[:M]), (M, first_divergence(got, full[:M]))
    rows = slice(120, 320)
    args = (c.va[rows], c.vw, c.vb, c.vr[rows], c.name)
    check_close(f64(c.run(rows)), linear8.product(*args), linear8.product_bound(*args),
                "%s %s" % (kind, act))
    assert bi.bi_check_device_errors() == bi.OK
