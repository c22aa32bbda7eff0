"""The decoder with one-byte projections on the GPU: every stored activation of
a small model against its definition, logits that depend neither on the chunking
nor on the attention kernel, tokens identical under every batch mix, captured
steps beside eager ones, a bias on the query, key and value projection."""
import dataclasses

import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
import oracle
from invariant_bi_rmsnorm_02_gb300.decoder import TINY, Decoder, DecoderWeights
from invariant_bi_rmsnorm_02_gb300.serving import assert_reproducible, synthetic_requests
from oracle import linear8
from gpu_util import check_close, f64, same_bytes
from test_gpu_decoder import chunk_plan, decode_plan, serve

pytestmark = pytest.mark.gpu

VARIANTS = {
    "e4m3": dict(linear="e4m3"),
    "e4m3-bias": dict(linear="e4m3", qkv_bias=True),
    "e4m3-all": dict(linear="e4m3", kv_cache="e4m3", rope_scaling="llama3", rope_factor=8.0),
    "bf16-bias": dict(qkv_bias=True),
}


def config(name):
    return dataclasses.replace(TINY, **VARIANTS[name])


def values(q, s):
    return linear8.numbers(q.cpu().view(torch.uint8).numpy()) * f64(s)[:, None]


def held(t):
    """The values of a bf16 matrix's rows once held as e4m3."""
    codes, scale = linear8.quantise(f64(t))
    return linear8.numbers(codes) * scale.astype(np.float64)[:, None]


def blocks_of_16(ffn):
    """Row of a gate/up weight in blocks of 128 features, in order of blocks of 16."""
    r = np.arange(2 * ffn)
    f = r // 32 * 16 + r % 16
    return f // 128 * 256 + f % 128 + np.where(r % 32 < 16, 0, 128)


@pytest.mark.parametrize("name", ["e4m3", "e4m3-bias"])
def test_every_stage_matches_its_definition(cuda, name):
    cfg = config(name)
    w, plain = DecoderWeights(cfg, 51, cuda, gen_device="cpu"), DecoderWeights(cfg, 51, "cpu")
    T, mb = 75, 8
    prompt = np.random.default_rng(52).integers(0, cfg.vocab, T).astype(np.int32)
    table = np.random.default_rng(53).permutation(mb).astype(np.int32)
    dec = Decoder(cfg, w, num_pages=mb, max_tokens=128, max_seqs=128, max_blocks=mb, device=cuda)
    dec.capture = []
    dec.step(chunk_plan(prompt, 0, T, table))
    assert bi.bi_check_device_errors() == bi.OK
    st = {(layer, what): t.cpu() for layer, what, t in dec.capture}
    order = blocks_of_16(cfg.ffn)
    for layer in range(cfg.layers):
        # the weights are the plain ones held as e4m3, gate and up rows re-ordered
        rows = {"wqkv": plain.wqkv[layer], "wo": plain.wo[layer], "wgu": plain.wgu[layer][order],
                "wdown": plain.wdown[layer]}
        wv = {k: held(t) for k, t in rows.items()}
        for k, v in wv.items():
            assert np.array_equal(values(*getattr(w, k)[layer]), v), k
        h = st[(layer, "h")]
        for what, src, norm in (("y8_attn", h, plain.attn_norm),
                                ("y8_mlp", st[(layer, "h_mid")], plain.mlp_norm)):
            v = oracle.rmsnorm(src, norm[layer], cfg.eps)
            got = values(st[(layer, what)], st[(layer, what + "_scale")])
            s = f64(st[(layer, what + "_scale")])[:, None]
            # v in fp32 (H/2 + 6 units: the sum of squares, the root, two
            # products), then half an e4m3 step, 2^-4 or 2^-10 of the scale
            ev = (cfg.hidden / 2 + 6) * 2.0 ** -24
            bound = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s) * (1 + 2.0 ** -10) + \
                (2 * ev + 2.0 ** -21) * np.abs(v)
            check_close(got, v, bound, what)
        y = values(st[(layer, "y8_attn")], st[(layer, "y8_attn_scale")])
        b = f64(plain.bqkv[layer]) if cfg.qkv_bias else None
        args = (y, wv["wqkv"], b, None, "none")
        check_close(f64(st[(layer, "qkv")]), linear8.product(*args), linear8.product_bound(*args),
                    "qkv")
        a = held(st[(layer, "att")].reshape(T, -1))
        args = (a, wv["wo"], None, f64(h), "none")
        check_close(f64(st[(layer, "h_mid")]), linear8.product(*args),
                    linear8.product_bound(*args), "output projection")
        y = values(st[(layer, "y8_mlp")], st[(layer, "y8_mlp_scale")])
        args = (y, wv["wgu"], None, None, "swiglu")
        check_close(f64(st[(layer, "act")]), linear8.product(*args),
                    linear8.product_bound(*args), "gate/up")
        nxt = st[(layer + 1, "h")] if layer + 1 < cfg.layers else st[(-1, "h")]
        args = (held(st[(layer, "act")]), wv["wdown"], None, f64(st[(layer, "h_mid")]), "none")
        check_close(f64(nxt), linear8.product(*args), linear8.product_bound(*args),
                    "down projection")


def test_the_bias_of_bf16_projections(cuda):
    cfg = config("bf16-bias")
    w = DecoderWeights(cfg, 54, cuda, gen_device="cpu")
    T, mb = 40, 4
    prompt = np.random.default_rng(55).integers(0, cfg.vocab, T).astype(np.int32)
    dec = Decoder(cfg, w, num_pages=mb, max_tokens=64, max_seqs=64, max_blocks=mb, device=cuda)
    dec.capture = []
    dec.step(chunk_plan(prompt, 0, T, np.arange(mb, dtype=np.int32)))
    st = {(layer, what): t for layer, what, t in dec.capture}
    for layer in range(cfg.layers):
        args = (f64(st[(layer, "y_attn")]), f64(w.wqkv[layer]), f64(w.bqkv[layer]), None, "none")
        check_close(f64(st[(layer, "qkv")]), linear8.product(*args), linear8.product_bound(*args),
                    "qkv")


@pytest.mark.parametrize("name", ["e4m3-bias", "e4m3-all", "bf16-bias"])
def test_logits_do_not_depend_on_chunking_or_on_the_kernel(cuda, name):
    cfg = config(name)
    w = DecoderWeights(cfg, 61, cuda, gen_device="cpu")
    T, mb = 150, 12
    prompt = np.random.default_rng(62).integers(0, cfg.vocab, T).astype(np.int32)
    table = np.random.default_rng(63).permutation(mb).astype(np.int32)

    def decoder():
        return Decoder(cfg, w, num_pages=mb, max_tokens=160, max_seqs=160, max_blocks=mb,
                       device=cuda)
    whole = decoder()
    whole.step(chunk_plan(prompt, 0, T, table))
    parts, dec = [], decoder()
    for at, n in ((0, 40), (40, 1), (41, 60), (101, 3)):
        dec.step(chunk_plan(prompt, at, n, table))
        parts.append(dec.logits[:n].clone())
    for p in range(104, T):
        dec.step(decode_plan(prompt[p], p, table))
        parts.append(dec.logits[:1].clone())
    assert bi.bi_check_device_errors() == bi.OK
    assert same_bytes(torch.cat(parts), whole.logits[:T])


def test_tokens_identical_under_every_batch_mix(cuda):
    cfg = config("e4m3-bias")
    w = DecoderWeights(cfg, 71, cuda)
    kw = dict(num_pages=400, max_tokens=512, max_seqs=16, max_blocks=32, device=cuda)
    dec = Decoder(cfg, w, **kw)
    reqs = synthetic_requests(12, 16, 200, 24, cfg.vocab, seed=72, mean_gap=2.0)
    burst = [dataclasses.replace(r, arrival=0) for r in reqs]
    runs = {}
    for name, rq, mix in (("alone", reqs, dict(max_seqs=1, token_budget=16)),
                          ("4 slots", reqs, dict(max_seqs=4, token_budget=64, prefill_chunk=32)),
                          ("burst", burst, dict(max_seqs=16, token_budget=512))):
        runs[name], _ = serve(dec, cfg, rq, **mix)
    gdec = Decoder(cfg, w, use_graphs=True, graph_kv_bucket=64, **kw)
    runs["graphs"], _ = serve(gdec, cfg, reqs, max_seqs=4, token_budget=64)
    assert gdec.graph_replays > 20
    assert_reproducible(runs)
    assert len({t for r in runs["alone"].values() for t in r}) > 12


def test_no_batch_variant_form(cuda):
    cfg = config("e4m3")
    dec = Decoder(cfg, DecoderWeights(cfg, 81, cuda), num_pages=4, max_tokens=8, max_seqs=8,
                  max_blocks=4, device=cuda, mode=bi.VARIANT)
    with pytest.raises(ValueError):
        dec.step(decode_plan(1, 0, np.arange(4, dtype=np.int32)))
