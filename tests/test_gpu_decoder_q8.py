"""The decoder with a one-byte K/V cache and scaled rotary positions on the
GPU: the four operators in a run together.  Every stored activation of a small
model against its definition, the same bytes whichever kernel (prefill over
the pages read back, or decode over the records) serves a position, tokens
identical under every batch mix, and a captured step beside an eager one."""
import dataclasses

import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
import oracle
from invariant_bi_rmsnorm_02_gb300 import synth
from invariant_bi_rmsnorm_02_gb300.decoder import TINY, Decoder, DecoderWeights
from invariant_bi_rmsnorm_02_gb300.serving import (Scheduler, assert_reproducible,
                                                   synthetic_requests)
from oracle import longctx
from gpu_util import bf16_half_ulp, check_close, f64, same_bytes
from test_gpu_decoder import chunk_plan, decode_plan, serve

pytestmark = pytest.mark.gpu

VARIANTS = {
    "e4m3": dict(kv_cache="e4m3"),
    "llama3": dict(rope_scaling="llama3", rope_factor=8.0, rope_trained_len=64),
    "e4m3-yarn-part": dict(kv_cache="e4m3", rope_scaling="yarn", rope_factor=4.0, rope_dim=32,
                           rope_trained_len=128, rope_high_turns=32.0),
    "e4m3-linear-pairs": dict(kv_cache="e4m3", rope_scaling="linear", rope_factor=2.0,
                              rope_interleaved=True),
}


def config(name):
    return dataclasses.replace(TINY, **VARIANTS[name])


def quantised_values(bits):
    """bf16 bit patterns of the values an e4m3 cache holds for K or V rows."""
    v = longctx.values(*longctx.quantise_rows(bits))
    return longctx.bits_of(torch.from_numpy(v).to(torch.bfloat16))   # exact


@pytest.mark.parametrize("name", sorted(VARIANTS))
def test_every_stage_of_attention_matches_its_definition(cuda, name):
    cfg = config(name)
    w = DecoderWeights(cfg, 51, cuda, gen_device="cpu")
    T, mb = 75, 8
    prompt = np.random.default_rng(52).integers(0, cfg.vocab, T).astype(np.int32)
    table = np.random.default_rng(53).permutation(mb).astype(np.int32)
    dec = Decoder(cfg, w, num_pages=mb, max_tokens=128, max_seqs=128, max_blocks=mb, device=cuda)
    dec.capture = []
    dec.step(chunk_plan(prompt, 0, T, table))
    assert bi.bi_check_device_errors() == bi.OK
    st = {(layer, what): t.cpu() for layer, what, t in dec.capture}
    Hq, Hkv, D, P = cfg.heads, cfg.kv_heads, cfg.head_dim, cfg.page_size
    freqs, m = longctx.frequencies(cfg.rope_dim or D, cfg.rope_theta, cfg.rope_scaling,
                                   cfg.rope_factor, cfg.rope_trained_len, cfg.rope_low_turns,
                                   cfg.rope_high_turns)
    n = len(freqs)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if cfg.rope_interleaved else (i, i + n)
    npages = -(-T // P)
    for layer in range(cfg.layers):
        x = f64(st[(layer, "qkv")]).reshape(T, Hq + 2 * Hkv, D)
        y = longctx.rope(x[:, :Hq + Hkv], range(T), freqs, cfg.rope_interleaved, m)
        pair = np.zeros_like(y)
        pair[..., a] = pair[..., b] = np.abs(x[:, :Hq + Hkv][..., a]) + \
            np.abs(x[:, :Hq + Hkv][..., b])
        got = np.concatenate([f64(st[(layer, "q")]), f64(st[(layer, "k")])], 1)
        bound = np.maximum(bf16_half_ulp(got), bf16_half_ulp(y)) + m * 2.0 ** -20 * pair + 1e-30
        check_close(got, y, bound, "%s layer %d rope" % (name, layer))
        # attention of the stored q over the cache's values of the stored k, v
        rows = [longctx.bits_of(st[(layer, c)]) for c in "kv"]
        if cfg.kv_cache == "e4m3":
            rows = [quantised_values(r) for r in rows]
        pages = []
        for r in rows:
            c = np.zeros((npages * P, Hkv, D), np.uint16)
            c[:T] = r
            pages.append(np.ascontiguousarray(c.reshape(npages, P, Hkv, D).transpose(0, 2, 1, 3)))
        ra = oracle.attention(longctx.bits_of(st[(layer, "q")]), np.zeros(T, np.int32),
                              np.arange(T) + 1, *pages, np.arange(npages, dtype=np.int32)[None],
                              D ** -0.5)
        g = f64(st[(layer, "att")])
        check_close(g, ra.reshape(g.shape), bf16_half_ulp(g) + 2e-3, "%s attention" % name)


@pytest.mark.parametrize("name", ["e4m3", "e4m3-yarn-part"])
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
    cfg = config("e4m3-linear-pairs")
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


def test_a_run_of_the_operators_on_another_stream_and_in_graphs(cuda):
    """rope -> write -> decode, eagerly on a side stream, and captured twice
    with a workspace each and replayed in turn: the same bytes."""
    B, Hq, Hkv, D, L = 5, 8, 2, 128, 130
    lens = torch.tensor([L, 1, 64, 17, L - 1], dtype=torch.int32, device=cuda)
    pages = -(-L // 16)
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(4)) \
        .to(torch.int32).view(B, pages).to(cuda)
    freqs, m = bi.rope_frequencies(64, 10000.0, bi.ROPE_LLAMA3, 8.0, 64)
    base = bi.kv_cache_q8(B * pages, Hkv, D, cuda)
    old = synth.normal_bf16((B * L, Hkv, D), 81, device=cuda)
    bi.kv_write_q8(old, old.flip(0).contiguous(),
                   torch.arange(B, dtype=torch.int32, device=cuda).repeat_interleave(L),
                   torch.arange(L, dtype=torch.int32, device=cuda).repeat(B), base, table)
    qkv = synth.normal_bf16((B, (Hq + 2 * Hkv) * D), 82, device=cuda)
    seq = torch.arange(B, dtype=torch.int32, device=cuda)
    nbytes = bi.bi_attn_decode_workspace_size(B, Hq, Hkv, D, L, 64)

    class Run:
        def __init__(self):
            self.cache, self.pos = base.clone(), (lens - 1).contiguous()
            self.q = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=cuda)
            self.k, self.v = (torch.empty(B, Hkv, D, dtype=torch.bfloat16, device=cuda)
                              for _ in range(2))
            self.out = torch.empty_like(self.q)
            self.ws = torch.empty(nbytes // 4 + 4, dtype=torch.float32, device=cuda)

        def go(self):
            bi.bi_rope_qkv_scaled(qkv, self.pos, Hq, Hkv, D, freqs, self.q, self.k, self.v,
                                  attn_scale=m)
            bi.bi_kv_write_q8(self.k, self.v, seq, self.pos, self.cache, table)
            bi.bi_attn_decode_q8(self.q, self.cache, table, lens, self.out, max_kv_len=L,
                                 split_size=64, sm_scale=D ** -0.5, workspace=self.ws)

    eager = Run()
    eager.go()
    side, there = torch.cuda.Stream(), Run()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there.go()
    torch.cuda.current_stream().wait_stream(side)
    # the helpers with a stream given: outputs and workspace belong to it
    given = bi.attn_decode_q8(eager.q, eager.cache, table, lens, max_kv_len=L, split_size=64,
                              stream=side)
    torch.cuda.synchronize()
    assert same_bytes(there.out, eager.out) and torch.equal(there.cache, eager.cache)
    assert same_bytes(given, eager.out)
    runs, graphs = [Run(), Run()], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.go()
        graphs.append(g)
    for _ in range(3):
        for r, g in zip(runs, graphs):
            r.out.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert bi.bi_check_device_errors() == bi.OK
    for r in runs:
        assert same_bytes(r.out, eager.out) and torch.equal(r.cache, eager.cache)


def test_two_decodes_at_once_with_a_workspace_each(cuda):
    B, Hq, Hkv, D = 16, 32, 8, 128
    lens = synth.loguniform_int(B, 1, 3000, 91).tolist()
    kv = synth.paged_kv(lens, Hkv, D, 16, 92, device=cuda)
    rows = lambda t: t.transpose(1, 2).reshape(-1, Hkv, D).contiguous()
    P = kv.num_pages
    rec = bi.kv_cache_q8(P, Hkv, D, cuda)
    bi.kv_write_q8(rows(kv.k_cache), rows(kv.v_cache),
                   torch.arange(P, dtype=torch.int32, device=cuda).repeat_interleave(16),
                   torch.arange(16, dtype=torch.int32, device=cuda).repeat(P), rec,
                   torch.arange(P, dtype=torch.int32, device=cuda).view(P, 1))
    qs = [synth.normal_bf16((B, Hq, D), 93 + i, device=cuda) for i in range(2)]
    call = lambda q, s=None: bi.attn_decode_q8(q, rec, kv.block_table, kv.kv_lens,
                                               max_kv_len=3000, split_size=256, stream=s)
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [call(q, s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert same_bytes(x, y)
    assert bi.bi_check_device_errors() == bi.OK
