"""Decode attention where scale bytes, scores or values are out of the
ordinary, on the GPU through the C ABI: scales that change from tile to tile,
splits that no key of reaches the softmax, keys and values that are not
finite.  The bf16 decode, the decode over the quantised records and the
prefill chunk give the same bytes there too."""
import math

import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
from invariant_bi_rmsnorm_02_gb300 import synth
from oracle import longctx
from gpu_util import first_divergence, same_bytes

pytestmark = pytest.mark.gpu
PAGE = 16


def i32(v, dev):
    return torch.as_tensor(v, dtype=torch.int32).to(dev)


def records(kv, D, dev):
    """The quantised cache of a bf16 paged one, page by page through the write call."""
    P, H = kv.k_cache.shape[:2]
    rec = bi.kv_cache_q8(P, H, D, dev)
    rows = lambda t: t.to(dev).transpose(1, 2).reshape(P * PAGE, H, D).contiguous()
    i = torch.arange(P * PAGE, dtype=torch.int32, device=dev)
    ident = torch.arange(P, dtype=torch.int32, device=dev).view(P, 1)
    bi.kv_write_q8(rows(kv.k_cache), rows(kv.v_cache), i // PAGE, i % PAGE, rec, ident)
    return rec


def test_every_tile_takes_its_own_scales(cuda):
    # the scale bytes of one lane's copies are read by the other lanes: every
    # row's scale differs from that of the same row in the tiles before it, so
    # that a scale left from another tile would show
    for D, Hq, Hkv in ((64, 4, 2), (128, 32, 8), (128, 16, 1), (64, 16, 1)):
        lens = [2048, 1111, 64, 65]
        kv = synth.paged_kv(lens, Hkv, D, PAGE, 24000 + D)
        # a page's place in its sequence is not its place in the pool, so the
        # exponent goes by both page and row
        page = torch.arange(kv.num_pages).view(-1, 1, 1, 1)
        row = torch.arange(PAGE).view(1, 1, -1, 1)
        kv.k_cache.mul_(torch.exp2(((7 * page + 3 * row) % 11 - 8).float()).bfloat16())
        kv.v_cache.mul_(torch.exp2(((5 * page + 7 * row) % 13 - 6).float()).bfloat16())
        rec = records(kv, D, cuda)
        bt, lens = kv.block_table.to(cuda), kv.kv_lens.to(cuda)
        q = synth.normal_bf16((4, Hq, D), 24001 + D, device=cuda)
        k, v = bi.kv_read_q8(rec, D, bt, lens, max_kv_len=2048)
        _, ref = bi.attn_decode(q, k, v, bt, lens, max_kv_len=2048, split_size=512, want_f32=True)
        for _ in range(20):
            _, out = bi.attn_decode_q8(q, rec, bt, lens, max_kv_len=2048, split_size=512,
                                       want_f32=True)
            assert same_bytes(out, ref), (D, Hq, Hkv, first_divergence(out, ref))
    assert bi.bi_check_device_errors() == bi.OK
