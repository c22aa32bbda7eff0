"""Host-side checks of the quantised cache's and the scaled rotary positions'
entry points, and pins of their fp64 definitions; no GPU."""
import ctypes
import math

import numpy as np
import pytest

import invariant_bi_rmsnorm_02_gb300 as bi
from oracle import longctx

P = 1 << 20   # a 16-byte aligned fake address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    return bi.load()


def _write(lib, **kw):
    a = dict(k=P, v=P, seq=P, pos=P, n=4, cache=P, bt=P, seqs=2, Hkv=2, D=64, page=16, npages=8,
             maxblk=4)
    a.update(kw)
    return lib.bi_kv_write_q8(a["k"], a["v"], a["seq"], a["pos"], a["n"], a["cache"], a["bt"],
                              a["seqs"], a["Hkv"], a["D"], a["page"], a["npages"], a["maxblk"],
                              None)


def test_write_argument_checks(lib):
    for D in (16, 80, 96, 256):
        assert _write(lib, D=D) == bi.ERR_UNSUPPORTED
    assert _write(lib, page=32) == bi.ERR_UNSUPPORTED
    assert _write(lib, npages=1 << 31) == bi.ERR_UNSUPPORTED
    assert _write(lib, npages=(1 << 26)) == bi.ERR_UNSUPPORTED     # rows of the pool >= 2^31
    assert _write(lib, n=1 << 30) == bi.ERR_UNSUPPORTED
    for bad in (dict(n=-1), dict(seqs=-1), dict(Hkv=0), dict(npages=0), dict(maxblk=0),
                dict(k=None), dict(v=None), dict(seq=None), dict(pos=None), dict(cache=None),
                dict(bt=None), dict(k=P + 8), dict(cache=P + 4)):
        assert _write(lib, **bad) == bi.ERR_INVALID_ARG, bad
    assert _write(lib, n=0, k=None) == bi.OK


def _read(lib, **kw):
    a = dict(cache=P, bt=P, kl=P, B=2, Hkv=2, D=64, page=16, npages=8, maxblk=4, maxkv=64,
             ko=2 * P, vo=3 * P, ot=P, nout=8, outblk=4)
    a.update(kw)
    return lib.bi_kv_read_q8(a["cache"], a["bt"], a["kl"], a["B"], a["Hkv"], a["D"], a["page"],
                             a["npages"], a["maxblk"], a["maxkv"], a["ko"], a["vo"], a["ot"],
                             a["nout"], a["outblk"], None)


def test_read_argument_checks(lib):
    assert _read(lib, D=96) == bi.ERR_UNSUPPORTED
    assert _read(lib, page=8) == bi.ERR_UNSUPPORTED
    assert _read(lib, B=65536) == bi.ERR_UNSUPPORTED
    assert _read(lib, nout=1 << 26) == bi.ERR_UNSUPPORTED
    for bad in (dict(B=-1), dict(maxkv=-1), dict(nout=0), dict(outblk=0), dict(cache=None),
                dict(bt=None), dict(kl=None), dict(ko=None), dict(vo=None), dict(ot=None),
                dict(ko=2 * P + 2), dict(ko=2 * P + 16), dict(vo=3 * P + 16),
                dict(cache=P + 8), dict(vo=2 * P), dict(ko=P), dict(vo=2 * P + 32)):
        assert _read(lib, **bad) == bi.ERR_INVALID_ARG, bad
    assert _read(lib, B=0, cache=None) == bi.OK
    assert _read(lib, maxkv=0, cache=None) == bi.OK


def _decode(lib, **kw):
    a = dict(q=P, cache=P, bt=P, kl=P, out=P, o32=None, B=2, Hq=4, Hkv=2, D=64, page=16, npages=8,
             maxblk=4, maxkv=64, S=64, scale=0.125, mode=0, vs=0, ws=P, wsb=1 << 20)
    a.update(kw)
    return lib.bi_attn_decode_q8(a["q"], a["cache"], a["bt"], a["kl"], a["out"], a["o32"], a["B"],
                                 a["Hq"], a["Hkv"], a["D"], a["page"], a["npages"], a["maxblk"],
                                 a["maxkv"], a["S"], a["scale"], a["mode"], a["vs"], a["ws"],
                                 a["wsb"], None)


def test_decode_argument_checks(lib):
    for bad in (dict(D=96), dict(Hq=6, Hkv=4), dict(Hq=34, Hkv=2), dict(page=32), dict(S=100),
                dict(npages=1 << 27), dict(B=65536)):
        assert _decode(lib, **bad) == bi.ERR_UNSUPPORTED, bad
    for bad in (dict(q=None), dict(cache=None), dict(bt=None), dict(kl=None), dict(out=None),
                dict(out=P + 4), dict(cache=P + 8), dict(o32=P + 4), dict(npages=0), dict(B=-1),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(mode=2)):
        assert _decode(lib, **bad) == bi.ERR_INVALID_ARG, bad
    for bad in (dict(ws=None), dict(wsb=64), dict(ws=P + 4)):
        assert _decode(lib, **bad) == bi.ERR_WORKSPACE, bad
    assert _decode(lib, B=0) == bi.OK


def _rope(lib, **kw):
    a = dict(qkv=P, pos=P, T=4, Hq=4, Hkv=2, D=64, rot=64, inter=0, f=P, m=1.0, q=2 * P, k=3 * P,
             v=4 * P)
    a.update(kw)
    return lib.bi_rope_qkv_scaled(a["qkv"], a["pos"], a["T"], a["Hq"], a["Hkv"], a["D"], a["rot"],
                                  a["inter"], a["f"], a["m"], a["q"], a["k"], a["v"], None)


def test_rope_argument_checks(lib):
    for bad in (dict(D=72, rot=8), dict(D=2048), dict(rot=7), dict(Hq=65000, Hkv=500),
                dict(T=1 << 31)):
        assert _rope(lib, **bad) == bi.ERR_UNSUPPORTED, bad
    for bad in (dict(T=-1), dict(rot=0), dict(rot=66), dict(inter=2), dict(m=0.0),
                dict(m=float("nan")), dict(m=float("inf")), dict(qkv=None), dict(pos=None),
                dict(f=None), dict(q=None), dict(k=None), dict(v=None), dict(q=2 * P + 2),
                dict(f=P + 8), dict(q=P), dict(k=P + 512), dict(v=3 * P), dict(k=2 * P + 1024)):
        assert _rope(lib, **bad) == bi.ERR_INVALID_ARG, bad
    assert _rope(lib, T=0, qkv=None) == bi.OK


def test_frequency_argument_checks(lib):
    f = (ctypes.c_double * 64)()
    m = ctypes.c_float()

    def call(rot=128, theta=1e4, kind=bi.ROPE_YARN, factor=4.0, trained=8192.0, low=1.0, high=32.0,
             out=f):
        return lib.bi_rope_frequencies(rot, theta, kind, factor, trained, low, high, out, m)

    assert call() == bi.OK
    for bad in (dict(rot=7), dict(rot=2048), dict(rot=2, kind=bi.ROPE_NTK)):
        assert call(**bad) == bi.ERR_UNSUPPORTED, bad
    nan = float("nan")
    for bad in (dict(rot=0), dict(theta=1.0), dict(theta=nan), dict(kind=5), dict(kind=-1),
                dict(factor=0.5), dict(factor=nan), dict(trained=0.0), dict(trained=nan),
                dict(low=0.0), dict(high=1.0), dict(high=nan), dict(out=None)):
        assert call(**bad) == bi.ERR_INVALID_ARG, bad
    # what a kind does not read is not checked
    assert call(kind=bi.ROPE_NONE, factor=nan, trained=nan, low=nan, high=nan) == bi.OK
    assert call(kind=bi.ROPE_NTK, trained=nan, low=nan, high=nan) == bi.OK


@pytest.mark.parametrize("rot,theta", [(128, 500000.0), (64, 10000.0), (20, 10000.0), (4, 1e6)])
@pytest.mark.parametrize("kind", ["none", "linear", "ntk", "llama3", "yarn"])
def test_frequencies_match_their_formulas(kind, rot, theta):
    code = {"none": bi.ROPE_NONE, "linear": bi.ROPE_LINEAR, "ntk": bi.ROPE_NTK,
            "llama3": bi.ROPE_LLAMA3, "yarn": bi.ROPE_YARN}[kind]
    f, m = bi.rope_frequencies(rot, theta, code, 8.0, 8192, 1.0, 4.0, device="cpu")
    want, wm = longctx.frequencies(rot, theta, kind, 8.0, 8192.0, 1.0, 4.0)
    # a power by pow and one by a quotient: a few roundings apart
    assert (np.abs(f.numpy() - want) <= 2.0 ** -46 * want).all()
    assert abs(m - wm) <= 2.0 ** -23 * wm
    if kind == "none":
        assert f[0] == 1.0
    if kind in ("llama3", "yarn"):   # the fastest pairs are kept, the slowest divided
        plain = longctx.frequencies(rot, theta)[0]
        assert f[0] == plain[0]
        assert abs(f[-1] - plain[-1] / 8) < 1e-12 * plain[-1] or rot < 20


def test_the_library_refuses_a_frequency_array_of_another_kind():
    for bad in (np.empty(64, np.float32), np.empty(63), np.empty(128)[::2], [0.0] * 64):
        with pytest.raises(TypeError):
            bi.bi_rope_frequencies(128, 1e4, bi.ROPE_NONE, 1, 1, 1, 2, bad)


def test_binding_refuses_wrong_shapes_before_any_device_call():
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    rec = z(3, 2, bi.kv_q8_record_bytes(64), dt=torch.uint8)
    with pytest.raises(ValueError):
        bi.bi_kv_write_q8(z(4, 2, 64), z(4, 2, 64), i(3), i(4), rec, i(1, 3))
    with pytest.raises(ValueError):
        bi.bi_kv_write_q8(z(4, 2, 128), z(4, 2, 128), i(4), i(4), rec, i(1, 3))
    with pytest.raises(ValueError):
        bi.bi_kv_read_q8(rec, i(2, 3), i(1), z(3, 2, 16, 64), z(3, 2, 16, 64), i(1, 3),
                         max_kv_len=16)
    with pytest.raises(ValueError):
        bi.bi_attn_decode_q8(z(2, 4, 64), rec, i(1, 3), i(2), z(2, 4, 64), max_kv_len=16,
                             split_size=64, sm_scale=0.1)
    with pytest.raises(ValueError):
        bi.bi_rope_qkv_scaled(z(2, 512), i(2), 4, 2, 64, z(32, dt=torch.float64), z(2, 4, 64),
                              z(2, 1, 64), z(2, 2, 64))


# -------------------------------------------------------- the definitions
def test_e4m3_table_and_rounding():
    assert longctx.E4M3[0] == 0 and longctx.E4M3[1] == 2.0 ** -9 and longctx.E4M3[-1] == 448
    assert (np.diff(longctx.E4M3) > 0).all()
    codes = longctx.e4m3_codes(longctx.E4M3)
    assert np.array_equal(codes, np.arange(0x7f))
    assert longctx.e4m3_codes(np.array([-0.0, -448.0, 1e9, 272.0, 304.0, 2.0 ** -10,
                                        3 * 2.0 ** -10])).tolist() == \
        [0x80, 0xfe, 0x7e, 0x78, 0x7a, 0, 2]


def test_e4m3_codes_match_torch():
    import torch
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1)).double() * 60
    x = torch.cat([x, x * 1e-3, torch.tensor([0.0, -0.0, 448.0, -448.0])]).clamp(-448, 448)
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(longctx.e4m3_codes(x.float().double().numpy()), want)


def test_scale_is_the_least_that_fits():
    import torch
    for amax, e in ((448.0, 0), (450.0, 1), (224.0, -1), (226.0, 0), (57344.0, 7), (1e38, 7),
                    (0.0, -124), (2.0 ** -130, -124), (1.0, -8)):
        row = torch.zeros(1, 64)
        row[0, 7] = amax
        _, s = longctx.quantise_rows(longctx.bits_of(row.bfloat16()))
        assert int(s[0]) == e + 127, amax
    for bad in (math.inf, -math.inf, math.nan):
        row = torch.ones(1, 64)
        row[0, 9] = bad
        c, s = longctx.quantise_rows(longctx.bits_of(row.bfloat16()))
        assert int(s[0]) == 135 and (c == 0).all() and np.isnan(longctx.values(c, s)).all()
