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


def masked_case(lens, empty, Hq, Hkv, D, split, seed, lowest=-57344.0):
    """A cache whose keys in the splits that ``empty`` names (per sequence)
    score below every finite number for every query: the queries' first
    channel holds 2^125 and those keys' first channel ``lowest``, the other
    keys' first channel 0.  Returns the cache, the queries and, per sequence,
    the mask of its ordinary keys."""
    kv = synth.paged_kv(lens, Hkv, D, PAGE, seed)
    kv.k_cache[..., 0] = 0
    keep = []
    for b, n in enumerate(lens):
        j = torch.arange(n)
        gone = torch.zeros(n, dtype=torch.bool)
        for s in empty[b]:
            gone |= j // split == s
        page = kv.block_table[b, j // PAGE].long()
        kv.k_cache[page[gone], :, (j % PAGE)[gone], 0] = lowest
        keep.append(~gone)
    q = synth.normal_bf16((len(lens), Hq, D), seed + 9)
    q[..., 0] = 2.0 ** 125
    return kv, q, keep


def definition(q, k_cache, v_cache, block_table, keep):
    """Softmax attention in 64 bits over each sequence's ordinary keys, zeros
    where there is none.  Their first channel is 0, so that of q drops out."""
    q = q.cpu().double().clone()
    q[..., 0] = 0
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    for b in range(B):
        j = torch.nonzero(keep[b])[:, 0]
        if not len(j):
            continue
        page = block_table[b].cpu()[j // PAGE].long()
        k, v = (t.cpu()[page, :, j % PAGE].double() for t in (k_cache, v_cache))
        qg = q[b].view(Hkv, Hq // Hkv, D)
        p = torch.softmax(torch.einsum("hgd,khd->hgk", qg, k) / math.sqrt(D), -1)
        o[b] = torch.einsum("hgk,khd->hgd", p, v).reshape(Hq, D)
    return o


def weight_bound(v):
    """An output is off by the weights' error times the largest value: below
    2^-14 for P's two truncated bf16 parts, 2^-21 for ex2, 2^-19 for a score
    rounded at a magnitude below 2^5, and 2^-24 for each of up to 128 splits
    folded in; 2^-13 covers their sum."""
    return 2.0 ** -13 * float(v.abs().max())


# splits without a reachable key: none, some, whole chunks of 32 and more at
# the head of a row, a chunk in the middle, single ones, all of them
EMPTY = [(), range(3), range(31), range(32), range(33), range(64), range(95), range(32, 64),
         (0, 33, 64), range(1, 99), range(100)]


@pytest.mark.parametrize("Hq,Hkv,D,copies", [(4, 2, 64, 1), (8, 1, 128, 1), (16, 1, 64, 2),
                                             (32, 8, 128, 1), (12, 4, 128, 3)])
def test_splits_without_a_reachable_key(cuda, Hq, Hkv, D, copies):
    # 100 splits a row; few rows and many take the merge's different forms
    S = 64
    empty = [e for e in EMPTY for _ in range(copies)]
    lens = [100 * S - 7 * (i % 3) for i in range(len(empty))]
    kv, q, keep = masked_case(lens, empty, Hq, Hkv, D, S, 24100 + Hq)
    bt, kl, qc = kv.block_table.to(cuda), kv.kv_lens.to(cuda), q.to(cuda)
    out, out32 = bi.attn_decode(qc, kv.k_cache.to(cuda), kv.v_cache.to(cuda), bt, kl,
                                max_kv_len=100 * S, split_size=S, want_f32=True)
    want = definition(q, kv.k_cache, kv.v_cache, kv.block_table, keep)
    err = (out32.cpu().double() - want).abs().amax((1, 2))
    assert (err <= weight_bound(kv.v_cache)).all(), err
    assert (out32[torch.tensor([len(e) == 100 for e in empty])] == 0).all()
    assert same_bytes(out, out32.to(torch.bfloat16))
    # each sequence alone: the merge's few-rows form gives the same bytes
    for b in range(0, len(empty), copies):
        one = bi.attn_decode(qc[b:b + 1], kv.k_cache.to(cuda), kv.v_cache.to(cuda), bt[b:b + 1],
                             kl[b:b + 1], max_kv_len=100 * S, split_size=S)
        assert same_bytes(one, out[b:b + 1].contiguous()), empty[b]
    assert bi.bi_check_device_errors() == bi.OK


@pytest.mark.parametrize("Hq,Hkv,D,copies", [(4, 2, 64, 1), (32, 8, 128, 1), (16, 1, 64, 2)])
def test_splits_without_a_reachable_key_of_a_quantised_cache(cuda, Hq, Hkv, D, copies):
    S = 64
    empty = [e for e in EMPTY for _ in range(copies)]
    lens = [100 * S - 7 * (i % 3) for i in range(len(empty))]
    kv, q, keep = masked_case(lens, empty, Hq, Hkv, D, S, 24200 + Hq)
    rec = records(kv, D, cuda)
    bt, kl, qc = kv.block_table.to(cuda), kv.kv_lens.to(cuda), q.to(cuda)
    k, v = bi.kv_read_q8(rec, D, bt, kl, max_kv_len=100 * S)
    out, out32 = bi.attn_decode_q8(qc, rec, bt, kl, max_kv_len=100 * S, split_size=S,
                                   want_f32=True)
    want = definition(q, k, v, kv.block_table, keep)
    err = (out32.cpu().double() - want).abs().amax((1, 2))
    assert (err <= weight_bound(v)).all(), err
    ref, ref32 = bi.attn_decode(qc, k, v, bt, kl, max_kv_len=100 * S, split_size=S, want_f32=True)
    assert same_bytes(out32, ref32), first_divergence(out32, ref32)
    assert same_bytes(out, ref)
    assert bi.bi_check_device_errors() == bi.OK


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (32, 8, 128), (16, 1, 128), (12, 4, 64)])
def test_prefill_of_splits_without_a_reachable_key(cuda, Hq, Hkv, D):
    # the last positions of each sequence, and a whole prompt whose first keys
    # are out of reach: the bytes of the decode at every position, zeros where
    # a query reaches no key
    S = 64
    lens = [100 * S - 7 * (i % 3) for i in range(len(EMPTY))]
    kv, _, keep = masked_case(lens, EMPTY, Hq, Hkv, D, S, 24300 + Hq)
    kc, vc, bt, kl = (t.to(cuda) for t in (kv.k_cache, kv.v_cache, kv.block_table, kv.kv_lens))
    n = 5
    q = synth.normal_bf16((n * len(lens), Hq, D), 24301 + Hq)
    q[..., 0] = 2.0 ** 125
    qc = q.to(cuda)
    cu = i32([n * b for b in range(len(lens) + 1)], cuda)
    pre, pre32 = bi.attn_prefill_chunk(qc, cu, kl - n, kc, vc, bt, kl, max_q_len=n,
                                       max_kv_len=100 * S, split_size=S, want_f32=True)
    at = (kl[:, None] - n + 1 + torch.arange(n, device=cuda)[None, :]).to(torch.int32).flatten()
    rows = bt.repeat_interleave(n, 0).contiguous()
    each, each32 = bi.attn_decode(qc, kc, vc, rows, at.contiguous(), max_kv_len=100 * S,
                                  split_size=S, want_f32=True)
    assert same_bytes(pre32, each32), first_divergence(pre32, each32)
    assert same_bytes(pre, each)
    assert (pre32[-n:] == 0).all() and torch.isfinite(pre32).all()

    L = 400                                    # splits 0, 1, 2 and 5 of a prompt out of reach
    kv, _, keep = masked_case([L], [(0, 1, 2, 5)], Hq, Hkv, D, S, 24400 + Hq)
    kc, vc, bt, kl = (t.to(cuda) for t in (kv.k_cache, kv.v_cache, kv.block_table, kv.kv_lens))
    q = synth.normal_bf16((L, Hq, D), 24401 + Hq)
    q[..., 0] = 2.0 ** 125
    qc = q.to(cuda)
    _, pre32 = bi.attn_prefill_chunk(qc, i32([0, L], cuda), i32([0], cuda), kc, vc, bt, kl,
                                     max_q_len=L, max_kv_len=L, split_size=S, want_f32=True)
    _, each32 = bi.attn_decode(qc, kc, vc, bt.expand(L, -1).contiguous(),
                               i32(range(1, L + 1), cuda), max_kv_len=L, split_size=S,
                               want_f32=True)
    assert same_bytes(pre32, each32), first_divergence(pre32, each32)
    assert (pre32[:3 * S] == 0).all()
    want = definition(q[L - 1:], kv.k_cache, kv.v_cache, kv.block_table, keep)
    assert (pre32[L - 1:].cpu().double() - want).abs().max() <= weight_bound(kv.v_cache)
    assert bi.bi_check_device_errors() == bi.OK


def nan_agree(a, b):
    """The same elements NaN and the same bytes elsewhere."""
    nan = torch.isnan(a)
    return torch.equal(nan, torch.isnan(b)) and same_bytes(a[~nan], b[~nan])


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 4, 64), (16, 4, 128), (48, 4, 128), (64, 4, 64)])
@pytest.mark.parametrize("split", [64, 512])
def test_a_key_that_is_not_finite_is_not_hidden(cuda, Hq, Hkv, D, split):
    # a NaN or an infinite key (NaN in a quantised cache) makes its head's
    # whole output NaN in its own sequence, and nothing else: one split or
    # several, decode and prefill
    G = Hq // Hkv
    lens = [100, 300, 200]
    for bad in (float("nan"), float("inf"), float("-inf")):
        kv = synth.paged_kv(lens, Hkv, D, PAGE, 24500 + Hq)
        page = int(kv.block_table[1, 2])
        kv.k_cache[page, 1, 3, 17] = bad                # key 35 of sequence 1, kv head 1
        kc, vc, bt, kl = (t.to(cuda) for t in (kv.k_cache, kv.v_cache, kv.block_table,
                                               kv.kv_lens))
        rec = records(kv, D, cuda)
        kb, vb = bi.kv_read_q8(rec, D, bt, kl, max_kv_len=300)
        assert torch.isnan(kb[page, 1, 3]).all()
        q = synth.normal_bf16((3, Hq, D), 24501 + Hq, device=cuda)
        args = dict(max_kv_len=300, split_size=split, want_f32=True)
        want = torch.zeros(3, Hkv, G, D, dtype=torch.bool, device=cuda)
        want[1, 1] = True
        out, out32 = bi.attn_decode_q8(q, rec, bt, kl, **args)
        assert torch.equal(torch.isnan(out32), want.view(3, Hq, D))
        assert torch.equal(torch.isnan(out), want.view(3, Hq, D))
        _, ref32 = bi.attn_decode(q, kb, vb, bt, kl, **args)
        assert nan_agree(out32, ref32)
        if math.isnan(bad):                             # an infinite key scores +-inf there
            _, raw32 = bi.attn_decode(q, kc, vc, bt, kl, **args)
            assert torch.equal(torch.isnan(raw32), want.view(3, Hq, D))
        # positions 20 .. 299 of sequence 1: finite up to the key, NaN from it on
        qp = synth.normal_bf16((280, Hq, D), 24502 + Hq, device=cuda)
        _, pre32 = bi.attn_prefill_chunk(qp, i32([0, 280], cuda), i32([20], cuda), kb, vb,
                                         bt[1:2], kl[1:2], max_q_len=280, **args)
        _, each32 = bi.attn_decode_q8(qp, rec, bt[1:2].expand(280, -1).contiguous(),
                                      i32(range(21, 301), cuda), **args)
        nan = torch.isnan(pre32).view(280, Hkv, G, D)
        assert nan[15:, 1].all() and not nan[:15].any() and not nan[:, [0, 2, 3]].any()
        assert nan_agree(pre32, each32)
    assert bi.bi_check_device_errors() == bi.OK


def test_a_query_that_is_not_finite_is_not_hidden(cuda):
    for D, Hq, Hkv in ((64, 4, 2), (128, 32, 8), (128, 16, 1)):
        lens = [50, 700, 64]
        kv = synth.paged_kv(lens, Hkv, D, PAGE, 24600 + Hq)
        rec = records(kv, D, cuda)
        bt, kl = kv.block_table.to(cuda), kv.kv_lens.to(cuda)
        kb, vb = bi.kv_read_q8(rec, D, bt, kl, max_kv_len=700)
        q = synth.normal_bf16((3, Hq, D), 24601 + Hq, device=cuda)
        q[0, 1, 5] = q[1, 2, 7] = float("nan")
        want = torch.zeros(3, Hq, D, dtype=torch.bool, device=cuda)
        want[0, 1] = want[1, 2] = True
        for split in (64, 256, 1024):
            args = dict(max_kv_len=700, split_size=split, want_f32=True)
            _, out32 = bi.attn_decode_q8(q, rec, bt, kl, **args)
            _, ref32 = bi.attn_decode(q, kb, vb, bt, kl, **args)
            _, pre32 = bi.attn_prefill_chunk(q, i32([0, 1, 2, 3], cuda), kl - 1, kb, vb, bt, kl,
                                             max_q_len=1, **args)
            assert torch.equal(torch.isnan(out32), want)
            assert nan_agree(out32, ref32) and nan_agree(pre32, ref32)
    assert bi.bi_check_device_errors() == bi.OK


def test_bounds_at_the_ends_of_their_ranges(cuda):
    # the largest bound on the lengths and the largest split size are those of
    # a call with no split and the sequence's own length
    D, Hq, Hkv = 64, 4, 2
    lens = [300, 1, 0, 129]
    kv = synth.paged_kv(lens, Hkv, D, PAGE, 24700)
    rec = records(kv, D, cuda)
    bt, kl = kv.block_table.to(cuda), kv.kv_lens.to(cuda)
    q = synth.normal_bf16((4, Hq, D), 24701, device=cuda)
    top, whole = 2 ** 31 - 1, 2 ** 31 - 64
    kb, vb = bi.kv_read_q8(rec, D, bt, kl, max_kv_len=300)
    k2, v2 = bi.kv_read_q8(rec, D, bt, kl, max_kv_len=top)
    assert same_bytes(kb, k2) and same_bytes(vb, v2)
    cu, start = i32([0, 1, 1, 1, 2], cuda), i32([299, 0, 0, 128], cuda)
    qp = q[:2].contiguous()
    for mode in (bi.INVARIANT, bi.VARIANT):
        # the variant mode's plan goes by the bound itself, so it keeps it
        bound = top if mode == bi.INVARIANT else 300
        args = dict(split_size=320, max_kv_len=300, mode=mode)
        wide = dict(split_size=whole, max_kv_len=bound, mode=mode)
        a = bi.attn_decode_q8(q, rec, bt, kl, **args)
        assert same_bytes(a, bi.attn_decode_q8(q, rec, bt, kl, **wide))
        b = bi.attn_decode(q, kb, vb, bt, kl, **args)
        assert same_bytes(b, bi.attn_decode(q, kb, vb, bt, kl, **wide))
        c = bi.attn_prefill_chunk(qp, cu, start, kb, vb, bt, kl, max_q_len=1, **args)
        d = bi.attn_prefill_chunk(qp, cu, start, kb, vb, bt, kl, max_q_len=1, **wide)
        assert same_bytes(c, d)
    assert bi.bi_check_device_errors() == bi.OK


def test_prefill_refuses_a_start_whose_end_passes_32_bits(cuda):
    D, Hq, Hkv, n = 64, 4, 2, 200
    kv = synth.paged_kv([300, 300], Hkv, D, PAGE, 24800)
    kc, vc, bt, kl = (t.to(cuda) for t in (kv.k_cache, kv.v_cache, kv.block_table, kv.kv_lens))
    q = synth.normal_bf16((2 * n, Hq, D), 24801, device=cuda)
    cu = i32([0, n, 2 * n], cuda)
    want = bi.attn_prefill_chunk(q, cu, i32([100, 100], cuda), kc, vc, bt, kl, max_q_len=n,
                                 max_kv_len=300, split_size=64)
    for start in (101, 2 ** 31 - 1, 2 ** 31 - n, 2 ** 31 - 100, -1):
        out = torch.full_like(q, 7.0)
        bi.bi_attn_prefill_chunk(q, cu, i32([100, start], cuda), kc, vc, bt, kl, out,
                                 max_q_len=n, max_kv_len=300, split_size=64, sm_scale=D ** -0.5)
        assert bi.bi_check_device_errors() == bi.ERR_DEVICE_BOUNDS, start
        assert same_bytes(out[:n], want[:n]) and (out[n:] == 7.0).all(), start


def spread_values(D, Hkv, lens, lo, hi, seed):
    """A cache whose V rows have magnitudes from 2^lo to 2^hi, row by row in a
    shuffled order; the upper half of the columns is zero in every row above
    the middle of that range, so that only small rows reach those columns."""
    kv = synth.paged_kv(lens, Hkv, D, PAGE, seed)
    rows = kv.num_pages * PAGE
    order = torch.randperm(rows, generator=torch.Generator().manual_seed(seed))
    e = (lo + (hi - lo) * order.double() / (rows - 1)).round().view(-1, 1, PAGE, 1)
    v = kv.v_cache.double()
    v = v / v.abs().amax(-1, keepdim=True) * torch.exp2(e)
    v[..., D // 2:] = torch.where(e > (lo + hi) / 2, 0.0, v[..., D // 2:])
    kv.v_cache.copy_(v.to(torch.bfloat16))
    return kv


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 16, 1), (64, 4, 4)])
def test_values_of_unlike_scales_give_the_bf16_bytes(cuda, D, Hq, Hkv):
    # scores below 2^3 in magnitude (weights above 2^-8 of the largest) and V
    # rows 2^72 apart: every part of a sum is above 2^-72 - 8 - 9 (the least
    # e4m3 number beside the largest of its row) = 2^-89 of the largest value
    lens = [700, 64, 130]
    kv = spread_values(D, Hkv, lens, -60, 12, 24900 + D)
    rec = records(kv, D, cuda)
    bt, kl = kv.block_table.to(cuda), kv.kv_lens.to(cuda)
    kb, vb = bi.kv_read_q8(rec, D, bt, kl, max_kv_len=700)
    q = synth.normal_bf16((3, Hq, D), 24901 + D, std=0.3, device=cuda)
    for split in (64, 1024):
        out = bi.attn_decode_q8(q, rec, bt, kl, max_kv_len=700, split_size=split, want_f32=True)
        ref = bi.attn_decode(q, kb, vb, bt, kl, max_kv_len=700, split_size=split, want_f32=True)
        assert same_bytes(out[1], ref[1]), first_divergence(out[1], ref[1])
        assert same_bytes(out[0], ref[0])
    assert bi.bi_check_device_errors() == bi.OK


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 16, 1)])
def test_values_over_the_whole_range_of_scales(cuda, D, Hq, Hkv):
    # from the least scale to the largest: beyond the range of equal bytes, but
    # off by no more than the weights' error in each column's own values and
    # 2^-120 of the largest value
    lens = [700, 64, 130]
    kv = spread_values(D, Hkv, lens, -115, 15, 25000 + D)
    rec = records(kv, D, cuda)
    bt, kl = kv.block_table.to(cuda), kv.kv_lens.to(cuda)
    kb, vb = bi.kv_read_q8(rec, D, bt, kl, max_kv_len=700)
    scale = rec[..., 32 * D + PAGE:]
    assert int(scale.min()) <= 4 and int(scale.max()) == 134
    q = synth.normal_bf16((3, Hq, D), 25001 + D, std=0.3, device=cuda)
    keep = [torch.ones(n, dtype=torch.bool) for n in lens]
    q[..., 0] = 0                                # as the definition takes it
    want = definition(q, kb, vb, kv.block_table, keep).view(3, Hkv, Hq // Hkv, D)
    for split in (64, 1024):
        _, out = bi.attn_decode_q8(q, rec, bt, kl, max_kv_len=700, split_size=split,
                                   want_f32=True)
        got = out.cpu().double().view(3, Hkv, Hq // Hkv, D)
        for b, n in enumerate(lens):
            page = kv.block_table[b, torch.arange(n) // PAGE].long()
            v = vb.cpu().double()[page, :, torch.arange(n) % PAGE]          # [n, Hkv, D]
            bound = 2.0 ** -13 * v.abs().amax(0) + 2.0 ** -120 * v.abs().max()
            assert ((got[b] - want[b]).abs() <= bound[:, None]).all(), (b, split)
    assert bi.bi_check_device_errors() == bi.OK


def test_rows_without_a_reachable_key_are_plus_zero(cuda):
    # every value negative: weights of 0 must not leave -0, one split or many
    for D, Hq, Hkv in ((64, 4, 2), (128, 32, 8), (128, 16, 1)):
        lens = [1, 64, 130, 700]
        kv, q, _ = masked_case(lens, [range(11)] * 4, Hq, Hkv, D, 64, 25100 + Hq)
        kv.v_cache.copy_(-kv.v_cache.abs())
        rec = records(kv, D, cuda)
        kc, vc, bt, kl, qc = (t.to(cuda) for t in (kv.k_cache, kv.v_cache, kv.block_table,
                                                   kv.kv_lens, q))
        for split in (64, 128, 704):
            args = dict(max_kv_len=704, split_size=split, want_f32=True)
            outs = [bi.attn_decode(qc, kc, vc, bt, kl, **args),
                    bi.attn_decode_q8(qc, rec, bt, kl, **args),
                    bi.attn_prefill_chunk(qc, i32(range(5), cuda), kl - 1, kc, vc, bt, kl,
                                          max_q_len=1, **args)]
            for out, out32 in outs:
                assert same_bytes(out, torch.zeros_like(out)), (D, split)
                assert same_bytes(out32, torch.zeros_like(out32)), (D, split)
    assert bi.bi_check_device_errors() == bi.OK


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (16, 1, 128), (4, 2, 64), (64, 4, 64)])
@pytest.mark.parametrize("what", ["values", "keys", "queries"])
def test_small_elements_give_the_bf16_bytes(cuda, what, Hq, Hkv, D):
    # elements that the stored or converted types hold as subnormal numbers:
    # their products must be aligned as the bf16 kernel's are.  Columns of V,
    # or of K under queries too wide for fp16, that are e4m3 subnormals in every
    # row; queries whose elements are 2^29 to 2^32 below their largest
    g = torch.Generator().manual_seed(25200 + D)
    lens = torch.cat([torch.arange(48), torch.randint(48, 700, (80,), generator=g)]).tolist()
    kv = synth.paged_kv(lens, Hkv, D, PAGE, 25201 + Hq)
    q = synth.normal_bf16((len(lens), Hq, D), 25202 + Hq)
    small = torch.arange(D) >= D // 2
    if what == "values":
        kv.v_cache[..., small] *= 2.0 ** -15
    else:
        # the scores come from the small elements; one large element of q in
        # each row meets a zero in every key
        kv.k_cache[..., 1] = 0
        if what == "keys":
            kv.k_cache[..., small] *= 2.0 ** -15
            q[..., ~small] *= 2.0 ** -20
            q[..., 1] = 2.0 ** 30
            q[..., small] *= 2.0 ** 9
        else:
            q = ((2 + 14 * torch.rand(q.shape, generator=g)) * q.float().sign()).bfloat16()
            q[..., 1] = 2.0 ** 33
    rec = records(kv, D, cuda)
    if what != "queries":
        rows, _ = longctx.record_views(rec.cpu().numpy(), D)
        kind = 1 if what == "values" else 0
        codes = rows[:, :, kind, :, D // 2:] & 0x7f
        assert (codes < 8).mean() > 0.9 and (codes > 0).mean() > 0.5
    bt, kl, qc = kv.block_table.to(cuda), kv.kv_lens.to(cuda), q.to(cuda)
    kb, vb = bi.kv_read_q8(rec, D, bt, kl, max_kv_len=700)
    for split in (64, 1024):
        args = dict(max_kv_len=700, split_size=split, want_f32=True)
        out = bi.attn_decode_q8(qc, rec, bt, kl, **args)
        ref = bi.attn_decode(qc, kb, vb, bt, kl, **args)
        assert torch.isfinite(ref[1]).all()
        assert same_bytes(out[1], ref[1]), int((out[1] != ref[1]).sum())
        assert same_bytes(out[0], ref[0])
    assert bi.bi_check_device_errors() == bi.OK
