"""Host-side checks of the 8-bit linear layers' entry points and pins of their
fp64 definitions; no GPU."""
import math

import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
from oracle import linear8

P = 1 << 20   # a 16-byte aligned fake address: never dereferenced on these paths
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return bi.load()


def _norm(lib, **kw):
    a = dict(x=P, w=2 * P, y=3 * P, s=4 * P, M=4, H=64, eps=1e-6)
    a.update(kw)
    return lib.bi_rmsnorm_q8(a["x"], a["w"], a["y"], a["s"], a["M"], a["H"], a["eps"], None)


def _add(lib, **kw):
    a = dict(x=P, r=2 * P, w=3 * P, h=4 * P, y=5 * P, s=6 * P, M=4, H=64, eps=1e-6)
    a.update(kw)
    return lib.bi_add_rmsnorm_q8(a["x"], a["r"], a["w"], a["h"], a["y"], a["s"], a["M"], a["H"],
                                 a["eps"], None)


def _quant(lib, **kw):
    a = dict(x=P, y=2 * P, s=3 * P, M=4, H=64)
    a.update(kw)
    return lib.bi_quantize_q8(a["x"], a["y"], a["s"], a["M"], a["H"], None)


@pytest.mark.parametrize("call", [_norm, _add, _quant])
def test_row_calls_refuse_shapes_and_pointers(lib, call):
    for bad in (dict(H=8), dict(H=72), dict(H=65552), dict(M=1 << 31)):
        assert call(lib, **bad) == bi.ERR_UNSUPPORTED, bad
    for bad in (dict(M=-1), dict(H=0), dict(x=None), dict(y=None), dict(s=None), dict(x=P + 8),
                dict(y=7 * P + 8), dict(s=7 * P + 2), dict(y=P), dict(y=P + 256), dict(s=P + 16),
                dict(y=7 * P, s=7 * P + 252)):
        assert call(lib, **bad) == bi.ERR_INVALID_ARG, bad
    assert call(lib, M=0, x=None) == bi.OK


def test_norms_refuse_their_own_arguments(lib):
    for call in (_norm, _add):
        for bad in (dict(w=None), dict(w=7 * P + 8), dict(eps=-1.0), dict(eps=NAN),
                    dict(y=7 * P, w=7 * P + 240), dict(s=7 * P, w=7 * P)):
            assert call(lib, **bad) == bi.ERR_INVALID_ARG, bad
    for bad in (dict(r=None), dict(h=None), dict(r=7 * P + 8), dict(h=7 * P + 8), dict(h=P + 16),
                dict(h=2 * P + 256), dict(h=3 * P + 64), dict(y=2 * P), dict(h=7 * P, y=7 * P),
                dict(h=7 * P, s=7 * P + 64), dict(s=2 * P + 64)):
        assert _add(lib, **bad) == bi.ERR_INVALID_ARG, bad


def _bf16(lib, **kw):
    a = dict(A=P, W=2 * P, b=3 * P, r=4 * P, C=5 * P, M=4, N=64, K=64, act=0)
    a.update(kw)
    return lib.bi_gemm_epilogue(a["A"], a["W"], a["b"], a["r"], a["C"], a["M"], a["N"], a["K"],
                                a["act"], None)


def _q8(lib, **kw):
    a = dict(A=P, sa=6 * P, W=2 * P, sw=7 * P, b=3 * P, r=4 * P, C=5 * P, M=4, N=64, K=64, act=0)
    a.update(kw)
    return lib.bi_gemm_q8(a["A"], a["sa"], a["W"], a["sw"], a["b"], a["r"], a["C"], a["M"],
                          a["N"], a["K"], a["act"], None)


@pytest.mark.parametrize("call", [_bf16, _q8])
def test_products_refuse_shapes_and_pointers(lib, call):
    for bad in (dict(N=12), dict(K=12), dict(N=48, act=bi.ACT_SWIGLU), dict(M=(1 << 31) - 1023),
                dict(N=(1 << 31) - 992), dict(K=(1 << 31) - 1008)):
        assert call(lib, **bad) == bi.ERR_UNSUPPORTED, bad
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(act=6), dict(act=-1), dict(A=None),
                dict(W=None), dict(C=None), dict(A=P + 8), dict(W=2 * P + 8), dict(b=3 * P + 8),
                dict(r=4 * P + 8), dict(C=5 * P + 8), dict(C=P), dict(C=2 * P + 64),
                dict(C=3 * P + 16), dict(C=4 * P + 16), dict(C=4 * P - 16)):
        assert call(lib, **bad) == bi.ERR_INVALID_ARG, bad
    assert call(lib, M=0, A=None) == bi.OK


def test_products_refuse_their_own_arguments(lib):
    assert _q8(lib, K=72) == bi.ERR_UNSUPPORTED          # rows of 72 bytes
    assert _bf16(lib, K=1 << 30) == bi.ERR_UNSUPPORTED   # rows of 2^31 bytes
    for bad in (dict(sa=None), dict(sw=None), dict(sa=6 * P + 2), dict(sw=7 * P + 4),
                dict(C=6 * P), dict(C=7 * P)):
        assert _q8(lib, **bad) == bi.ERR_INVALID_ARG, bad


def test_binding_refuses_wrong_shapes_before_any_device_call():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    q = lambda *s: z(*s, dt=torch.float8_e4m3fn)
    f = lambda *s: z(*s, dt=torch.float32)
    for bad in (lambda: bi.bi_rmsnorm_q8(z(2, 64), z(64), q(2, 32), f(2), 1e-6),
                lambda: bi.bi_rmsnorm_q8(z(2, 64), z(32), q(2, 64), f(2), 1e-6),
                lambda: bi.bi_add_rmsnorm_q8(z(2, 64), z(2, 64), z(64), z(1, 64), q(2, 64), f(2),
                                             1e-6),
                lambda: bi.bi_quantize_q8(z(2, 64), q(2, 64), f(3)),
                lambda: bi.bi_gemm_epilogue(z(2, 64), z(32, 32), z(2, 32)),
                lambda: bi.bi_gemm_epilogue(z(2, 64), z(32, 64), z(2, 32),
                                            activation=bi.ACT_SWIGLU),
                lambda: bi.bi_gemm_epilogue(z(2, 64), z(32, 64), z(2, 32), bias=z(16)),
                lambda: bi.bi_gemm_epilogue(z(2, 64), z(32, 64), z(2, 32), residual=z(1, 32)),
                lambda: bi.bi_gemm_q8(q(2, 64), f(1), q(32, 64), f(32), z(2, 32)),
                lambda: bi.bi_gemm_q8(q(2, 64), f(2), q(32, 64), f(2), z(2, 32))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("F,block", [(32, 16), (16, 16), (256, 128)])
def test_swiglu_interleave_blocks(F, block):
    perm = bi.swiglu_interleave(F, block)
    assert sorted(perm.tolist()) == list(range(2 * F))
    for r, src in enumerate(perm):
        feature = r // (2 * block) * block + r % block
        assert src == (feature if r % (2 * block) < block else F + feature)
    with pytest.raises(ValueError):
        bi.swiglu_interleave(F + 8, block)


# -------------------------------------------------------- the definitions
def test_row_definition():
    v = np.array([[448.0, -448.0, 1.0, 0.0], [0.0, 0.0, 0.0, -0.0], [7.0, 3.5, -1.75, 7.0],
                  [1.0, np.nan, 2.0, 3.0], [np.inf, 1.0, 1.0, 1.0]])
    codes, scale = linear8.quantise(v)
    assert scale[0] == 1.0 and scale[1] == 2.0 ** -126 and scale[2] == 2.0 ** -6
    assert np.isnan(scale[3:]).all() and (codes[3:] == 0).all()
    assert np.array_equal(linear8.numbers(codes[0]), v[0])
    assert codes[1].tolist() == [0, 0, 0, 0x80]
    assert np.array_equal(linear8.numbers(codes[2]) * scale[2], v[2])


def test_bf16_rows_are_never_within_rounding_of_a_tie_they_are_not_on():
    """448 v / t of two bf16 numbers is midway between two e4m3 numbers, or at
    least 2^-14 of itself away: forming it with one fp32 rounding gives the code
    of the exact quotient."""
    mid = (linear8.E4M3[1:] + linear8.E4M3[:-1]) / 2
    mid = mid[mid > 8]   # a binade or two stand for the rest: all scale by two
    for t in range(128, 256):
        v = np.arange(1, 2 * t + 1) / 2.0     # integers and halves up to t
        q = 448.0 * v / t
        d = np.abs(q[:, None] / mid - 1.0)
        assert ((d == 0) | (d > 2.0 ** -14)).all(), t


def test_activations_against_torch():
    z = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    f = torch.nn.functional
    for act, want in (("relu", f.relu(z)), ("gelu", f.gelu(z)), ("silu", f.silu(z)),
                      ("gelu_tanh", f.gelu(z, approximate="tanh")), ("none", z)):
        assert np.abs(linear8.activation(z.numpy(), act) - want.numpy()).max() < 1e-14, act
    slope = np.abs(np.gradient(linear8.activation(z.numpy(), "gelu"), z.numpy())).max()
    assert 1.12 < slope < 1.13


def test_product_definition():
    rng = np.random.default_rng(3)
    a, w = rng.normal(size=(3, 16)), rng.normal(size=(64, 16))
    b, r = rng.normal(size=64), rng.normal(size=(3, 32))
    got = linear8.product(a, w, b, r, "swiglu")
    for i in range(3):
        for j in range(32):
            g = a[i] @ w[32 * (j // 16) + j % 16] + b[32 * (j // 16) + j % 16]
            u = a[i] @ w[32 * (j // 16) + 16 + j % 16] + b[32 * (j // 16) + 16 + j % 16]
            assert math.isclose(got[i, j], g / (1 + math.exp(-g)) * u + r[i, j], rel_tol=1e-12)


# ------------------------------------------------------- the decoder's options
def test_the_decoders_configuration():
    import dataclasses

    from invariant_bi_rmsnorm_02_gb300.decoder import TINY, DecoderWeights, _rows_in_blocks_of_16
    with pytest.raises(ValueError):
        dataclasses.replace(TINY, linear="fp8")
    with pytest.raises(ValueError):
        dataclasses.replace(TINY, linear="e4m3", ffn=192)
    with pytest.raises(ValueError):
        dataclasses.replace(TINY, linear="e4m3", hidden=264)
    a = DecoderWeights(TINY, 3, "cpu")
    b = DecoderWeights(dataclasses.replace(TINY, linear="e4m3", qkv_bias=True), 3, "cpu")
    for k in ("wqkv", "wo", "wgu", "wdown"):   # the same numbers, whatever holds them
        assert all(torch.equal(x, y) for x, y in zip(getattr(a, k), getattr(b, k)))
    assert a.bqkv == [None] * TINY.layers and b.bqkv[1].shape == (TINY.qkv_dim,)
    rows = _rows_in_blocks_of_16(256, "cpu").tolist()
    perm = bi.swiglu_interleave(256, 128).tolist()      # row -> row of [gate; up]
    assert [perm[r] for r in rows] == bi.swiglu_interleave(256, 16).tolist()
