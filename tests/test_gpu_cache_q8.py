"""The quantised KV cache on the GPU through the C ABI: rows quantised as they
are written (byte for byte against the fp64 definition), pages read back
(exactly), and decode attention over the records (byte for byte the bf16
decode on the pages read back, and within 2e-3 of the fp64 oracle)."""
import numpy as np
import pytest
import torch

import invariant_bi_rmsnorm_02_gb300 as bi
import oracle
from invariant_bi_rmsnorm_02_gb300 import synth
from oracle import longctx
from gpu_util import check_close, f64, first_divergence, same_bytes

pytestmark = pytest.mark.gpu
PAGE = 16
ATOL = 2e-3   # the attention tests' bound on the fp32 result


def i32(v, dev):
    return torch.as_tensor(v, dtype=torch.int32).to(dev)


def quantised(kv, D):
    """The records of a bf16 paged cache, by the definition (CPU uint8)."""
    recs = []
    for t in (kv.k_cache, kv.v_cache):
        recs.append(longctx.quantise_rows(longctx.bits_of(t)))
    P, H = kv.k_cache.shape[:2]
    parts = [c.reshape(P, H, -1) for c, _ in recs] + [s.reshape(P, H, -1) for _, s in recs]
    return torch.from_numpy(np.concatenate(parts, -1))


def table_for(lens, extra=0, seed=0):
    need = [-(-(n + extra) // PAGE) for n in lens]
    perm = torch.randperm(max(sum(need), 1), generator=torch.Generator().manual_seed(seed))
    bt = torch.zeros(len(lens), max(need + [1]), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, max(sum(need), 1)


# ------------------------------------------------------------------- write
@pytest.mark.parametrize("n,seqs,Hkv,D", [(1, 1, 1, 64), (1, 1, 8, 128), (37, 5, 3, 64),
                                          (200, 7, 8, 128), (33, 33, 2, 128)])
def test_write_stores_the_defined_bytes(cuda, n, seqs, Hkv, D):
    per = -(-n // seqs)
    bt, pages = table_for([per + 5] * seqs, seed=n)
    k = synth.normal_bf16((n, Hkv, D), 20000 + n)
    v = synth.normal_bf16((n, Hkv, D), 20001 + n)
    k *= torch.exp2(torch.linspace(-20, 12, n)).to(torch.bfloat16)[:, None, None]
    seq = np.arange(n) // per
    pos = np.arange(n) % per + seq % 4
    before = torch.randint(0, 256, (pages, Hkv, bi.kv_q8_record_bytes(D)), dtype=torch.uint8,
                           generator=torch.Generator().manual_seed(n))
    cache = before.to(cuda)
    bi.kv_write_q8(k.to(cuda), v.to(cuda), i32(seq, cuda), i32(pos, cuda), cache, bt.to(cuda))
    assert bi.bi_check_device_errors() == bi.OK
    want = longctx.write(before.numpy(), longctx.bits_of(k), longctx.bits_of(v), seq, pos,
                         bt.numpy())
    assert np.array_equal(cache.cpu().numpy(), want)


def special_rows(D):
    """Rows whose scale or rounding is at an edge, as bf16 bit patterns."""
    r = np.zeros((14, D), np.uint16)
    top = lambda i, x: r.__setitem__((i, 3), longctx.bits_of(torch.tensor([x]).bfloat16())[0])
    r[1, :] = 0x8000                            # -0 throughout
    r[2, 5], r[2, 6] = 0x0001, 0x8003           # subnormals only
    for i, x in ((3, 448.0), (4, 450.0), (5, 224.0), (6, 57344.0), (7, 57600.0), (8, 3e38),
                 (9, 2.0 ** -115)):
        r[i] = longctx.bits_of(synth.normal_bf16((D,), 90 + i))
        r[i] = longctx.bits_of((torch.from_numpy(longctx.bf16_to_f64(r[i])) * x / 8).bfloat16())
        top(i, x)
    r[10, 1], r[10, 2] = 0x3f80, 0x7f80         # 1 and +inf
    r[11, 1], r[11, 2] = 0x3f80, 0xff80         # 1 and -inf
    r[12, 0], r[12, 1] = 0x7fc0, 0x3f80         # NaN and 1
    # halfway cases of e4m3 at scale 1 (17 / 16 and 19 / 16 of 256), and of its
    # smallest step: 2^-10 is half of 2^-9
    r[13, :6] = longctx.bits_of(torch.tensor([272.0, 304.0, 2.0 ** -10, 3 * 2.0 ** -10, -272.0,
                                              256.0]).bfloat16())
    return r


@pytest.mark.parametrize("D", [64, 128])
def test_write_and_read_special_rows(cuda, D):
    rows = special_rows(D)
    n = len(rows)
    k = torch.from_numpy(rows.view(np.int16)).view(torch.bfloat16).view(n, 1, D)
    v = k.flip(0).contiguous()
    bt = torch.zeros(1, 1, dtype=torch.int32)
    cache = bi.kv_cache_q8(1, 1, D, cuda)
    bi.kv_write_q8(k.to(cuda), v.to(cuda), i32([0] * n, cuda), i32(range(n), cuda), cache,
                   bt.to(cuda))
    want = longctx.write(np.zeros((1, 1, 32 * D + 32), np.uint8), longctx.bits_of(k),
                         longctx.bits_of(v), [0] * n, list(range(n)), bt.numpy())
    assert np.array_equal(cache.cpu().numpy(), want)
    gk, gv = bi.kv_read_q8(cache, D, bt.to(cuda), i32([n], cuda), max_kv_len=n)
    assert bi.bi_check_device_errors() == bi.OK
    wk, wv = longctx.pages(want, D)
    for got, ref in ((gk, wk), (gv, wv)):
        got = f64(got)
        assert np.array_equal(got[0, 0, :n], ref[0, 0, :n], equal_nan=True)
        assert (got[0, 0, n:] == 0).all()
    nan = np.isnan(f64(gk)[0, 0])
    assert nan[10:13].all() and not nan[:10].any() and not nan[13:].any()
    # an element is off by at most half a step: 2^-4 of it or half of 2^(e-9)
    x = longctx.bf16_to_f64(rows)
    e = want[0, 0, 32 * D:32 * D + n].astype(float) - 127
    for i in list(range(7)) + [9, 13]:
        bound = np.maximum(np.abs(x[i]) * 2.0 ** -4, 2.0 ** (e[i] - 10))
        assert (np.abs(f64(gk)[0, 0, i] - x[i]) <= bound).all(), i


def test_write_skips_and_records_what_is_out_of_range(cuda):
    D, Hkv = 64, 2
    bt = i32([[0, 5], [1, 2]], cuda)           # page 5 is outside the pool of 3
    k = synth.normal_bf16((6, Hkv, D), 20500, device=cuda)
    cache = bi.kv_cache_q8(3, Hkv, D, cuda)
    seq, pos = i32([0, 0, 2, -1, 1, 1], cuda), i32([3, 17, 0, 0, 32, -1], cuda)
    bi.kv_write_q8(k, k, seq, pos, cache, bt)
    assert bi.bi_check_device_errors() == bi.ERR_DEVICE_BOUNDS
    one = bi.kv_cache_q8(3, Hkv, D, cuda)
    bi.kv_write_q8(k[:1].contiguous(), k[:1].contiguous(), seq[:1], pos[:1], one, bt)
    assert bi.bi_check_device_errors() == bi.OK
    assert torch.equal(cache, one) and int((one != 0).sum()) > 0


def test_write_rows_do_not_depend_on_the_batch(cuda):
    n, Hkv, D = 300, 8, 128
    bt, pages = table_for([n], seed=3)
    bt = bt.to(cuda)
    k = synth.normal_bf16((n, Hkv, D), 20600, device=cuda)
    v = synth.normal_bf16((n, Hkv, D), 20601, device=cuda)
    whole = bi.kv_cache_q8(pages, Hkv, D, cuda)
    bi.kv_write_q8(k, v, i32([0] * n, cuda), i32(range(n), cuda), whole, bt)
    parts = bi.kv_cache_q8(pages, Hkv, D, cuda)
    for a, b in ((0, 1), (1, 100), (100, 300)):
        bi.kv_write_q8(k[a:b].contiguous(), v[a:b].contiguous(), i32([0] * (b - a), cuda),
                       i32(range(a, b), cuda), parts, bt)
    assert torch.equal(whole, parts)


# -------------------------------------------------------------------- read
@pytest.mark.parametrize("lens,Hkv,D", [([0, 1, 15, 16, 17, 100], 2, 64), ([33], 8, 128),
                                        ([0], 1, 64), (list(range(0, 140, 2)), 1, 128)])
def test_read_gives_the_stored_values_and_leaves_the_rest(cuda, lens, Hkv, D):
    kv = synth.paged_kv(lens, Hkv, D, PAGE, 21000 + len(lens))
    rec = quantised(kv, D)
    P = rec.shape[0]
    # pages go to other ids of a larger pool, through a wider table
    g = torch.Generator().manual_seed(7)
    out_pages = P + 3
    perm = torch.randperm(out_pages, generator=g).to(torch.int32)
    ot = torch.full((len(lens), kv.max_blocks + 2), -1, dtype=torch.int32)
    ot[:, :kv.max_blocks] = perm[kv.block_table.long()]
    ko = torch.full((out_pages, Hkv, PAGE, D), 7.0, dtype=torch.bfloat16, device=cuda)
    vo = torch.full_like(ko, 9.0)
    bi.bi_kv_read_q8(rec.to(cuda), kv.block_table.to(cuda), kv.kv_lens.to(cuda), ko, vo,
                     ot.to(cuda), max_kv_len=max(lens + [1]))
    assert bi.bi_check_device_errors() == bi.OK
    wk, wv = longctx.pages(rec.numpy(), D)
    for got, ref, fill in ((ko, wk, 7.0), (vo, wv, 9.0)):
        want = np.full(got.shape, fill)
        for b, n in enumerate(lens):
            for t in range(n):
                want[int(ot[b, t // PAGE]), :, t % PAGE] = \
                    ref[int(kv.block_table[b, t // PAGE]), :, t % PAGE]
        assert np.array_equal(f64(got), want)


def test_read_records_bad_pages_and_lengths(cuda):
    D, Hkv = 128, 1
    kv = synth.paged_kv([32, 32, 32], Hkv, D, PAGE, 21100)
    rec = quantised(kv, D).to(cuda)
    bt = kv.block_table.clone()
    bt[0, 1] = 99
    lens = i32([32, 33, 32], cuda)             # 33 is past the table
    ko = torch.zeros(6, Hkv, PAGE, D, dtype=torch.bfloat16, device=cuda)
    vo = torch.zeros_like(ko)
    bi.bi_kv_read_q8(rec, bt.to(cuda), lens, ko, vo, bt.to(cuda), max_kv_len=64)
    assert bi.bi_check_device_errors() == bi.ERR_DEVICE_BOUNDS
    wk, wv = longctx.pages(rec.cpu().numpy(), D)
    done = {int(bt[0, 0]), int(bt[2, 0]), int(bt[2, 1])}
    for p in range(6):
        assert np.array_equal(f64(ko[p]), wk[p] if p in done else np.zeros_like(wk[p]))
        assert np.array_equal(f64(vo[p]), wv[p] if p in done else np.zeros_like(wv[p]))


# ------------------------------------------------------------------ decode
def both_decodes(q, rec, bt, lens, D, max_len, S, mode=bi.INVARIANT, splits=0):
    """decode over the records, and the bf16 decode on the pages read back."""
    out, out32 = bi.attn_decode_q8(q, rec, bt, lens, max_kv_len=max_len, split_size=S, mode=mode,
                                   variant_splits=splits, want_f32=True)
    k, v = bi.kv_read_q8(rec, D, bt, lens, max_kv_len=max_len)
    ref, ref32 = bi.attn_decode(q, k, v, bt, lens, max_kv_len=max_len, split_size=S,
                                want_f32=True)
    return out, out32, ref, ref32, k, v


@pytest.mark.parametrize("Hq,Hkv,D,S", [(4, 2, 64, 64), (32, 8, 128, 256), (8, 8, 128, 64),
                                        (16, 1, 128, 256), (16, 1, 64, 512), (9, 1, 64, 64),
                                        (7, 1, 128, 128), (16, 2, 64, 2048)])
def test_decode_equals_bf16_decode_on_the_pages_read_back(cuda, Hq, Hkv, D, S):
    lens = [1, 0, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 511, 1000]
    kv = synth.paged_kv(lens, Hkv, D, PAGE, 22000 + Hq + D)
    kv.k_cache *= torch.exp(0.8 * torch.randn(D, generator=torch.Generator().manual_seed(2)))
    rec = quantised(kv, D)
    q = synth.normal_bf16((len(lens), Hq, D), 22500 + Hq + D)
    out, out32, ref, ref32, k, v = both_decodes(q.to(cuda), rec.to(cuda),
                                                kv.block_table.to(cuda), kv.kv_lens.to(cuda), D,
                                                1024, S)
    assert bi.bi_check_device_errors() == bi.OK
    assert same_bytes(out32, ref32), first_divergence(out32, ref32)
    assert same_bytes(out, ref) and same_bytes(out, out32.to(torch.bfloat16))
    want = oracle.decode_attention(q, k.cpu(), v.cpu(), kv.block_table, kv.kv_lens, D ** -0.5)
    check_close(f64(out32), want, np.full(want.shape, ATOL), "decode q8")
    assert (out32[1] == 0).all()
    # the batch-variant plan: the same values up to the order of the sums
    var, var32 = bi.attn_decode_q8(q.to(cuda), rec.to(cuda), kv.block_table.to(cuda),
                                   kv.kv_lens.to(cuda), max_kv_len=1024, split_size=S,
                                   mode=bi.VARIANT, want_f32=True)
    assert bi.bi_check_device_errors() == bi.OK
    check_close(f64(var32), want, np.full(want.shape, ATOL), "decode q8 variant")


def test_decode_with_extreme_scales_is_still_the_bf16_decode(cuda):
    # rows from the least scale (2^-124) to the largest (2^7), and zeros
    D, Hkv, L = 128, 2, 200
    kv = synth.paged_kv([L], Hkv, D, PAGE, 22700)
    e = torch.linspace(-130, 12, PAGE)[None, None, :, None]
    kv.k_cache.copy_((kv.k_cache.double() * torch.exp2(e.double())).bfloat16())
    kv.v_cache.copy_((kv.v_cache.double() * torch.exp2(-e.double().clamp(min=-12))).bfloat16())
    kv.k_cache[:, :, 5] = 0
    rec = quantised(kv, D)
    q = synth.normal_bf16((1, 8, D), 22701) * 1e-3
    out, out32, ref, ref32, _, _ = both_decodes(q.to(cuda), rec.to(cuda), kv.block_table.to(cuda),
                                                kv.kv_lens.to(cuda), D, L, 64)
    assert same_bytes(out32, ref32) and same_bytes(out, ref)
    assert torch.isfinite(out32).all()


def test_decode_reads_nothing_behind_the_last_token(cuda):
    # slots past the length hold every kind of bits: all-ones bytes, scale
    # bytes of non-finite rows and beyond
    for D, L in ((64, 5), (128, 77), (128, 129)):
        kv = synth.paged_kv([L], 2, D, PAGE, 22800 + L)
        rec = quantised(kv, D)
        q = synth.normal_bf16((1, 8, D), 22801 + L, device=cuda)
        bt, lens = kv.block_table.to(cuda), kv.kv_lens.to(cuda)
        a, a32 = bi.attn_decode_q8(q, rec.to(cuda), bt, lens, max_kv_len=256, split_size=64,
                                   want_f32=True)
        rows, scales = longctx.record_views(rec.numpy(), D)
        for fill_row, fill_scale in ((0xff, 135), (0x7f, 255), (0x80, 0)):
            r, s = rows.copy(), scales.copy()
            page = int(kv.block_table[0, L // PAGE])
            r[page, :, :, L % PAGE:] = fill_row
            s[page, :, :, L % PAGE:] = fill_scale
            bad = torch.from_numpy(np.concatenate([r.reshape(*rec.shape[:2], -1),
                                                   s.reshape(*rec.shape[:2], -1)], -1))
            b, b32 = bi.attn_decode_q8(q, bad.to(cuda), bt, lens, max_kv_len=256, split_size=64,
                                       want_f32=True)
            assert same_bytes(a32, b32) and same_bytes(a, b)
    assert bi.bi_check_device_errors() == bi.OK


def test_decode_non_finite_rows_reach_their_own_heads_only(cuda):
    D, Hkv, lens = 128, 4, [100, 300]
    kv = synth.paged_kv(lens, Hkv, D, PAGE, 22900)
    page = int(kv.block_table[1, 2])
    kv.k_cache[page, 1, 3, 17] = float("nan")      # a key of sequence 1, head 1
    kv.v_cache[page, 2, 4, 9] = float("-inf")      # a value of sequence 1, head 2
    rec = quantised(kv, D).to(cuda)
    q = synth.normal_bf16((2, 16, D), 22901, device=cuda)
    out, out32 = bi.attn_decode_q8(q, rec, kv.block_table.to(cuda), kv.kv_lens.to(cuda),
                                   max_kv_len=300, split_size=64, want_f32=True)
    nan = torch.isnan(out32).view(2, Hkv, 4, D)
    # the value's whole row is NaN, so every column of its heads is
    assert nan[1, 2].all() and not nan[0].any() and not nan[1, 0].any() and not nan[1, 3].any()
    # a NaN score's behaviour is the bf16 kernel's on the pages read back
    k, v = bi.kv_read_q8(rec, D, kv.block_table.to(cuda), kv.kv_lens.to(cuda), max_kv_len=300)
    _, ref32 = bi.attn_decode(q, k, v, kv.block_table.to(cuda), kv.kv_lens.to(cuda),
                              max_kv_len=300, split_size=64, want_f32=True)
    assert torch.equal(torch.isnan(ref32), torch.isnan(out32))


def test_decode_bad_pages_zero_their_sequence_and_are_recorded(cuda):
    D, lens = 64, [40, 200, 40]
    kv = synth.paged_kv(lens, 2, D, PAGE, 23000)
    rec = quantised(kv, D).to(cuda)
    q = synth.normal_bf16((3, 4, D), 23001, device=cuda)
    good = bi.attn_decode_q8(q, rec, kv.block_table.to(cuda), kv.kv_lens.to(cuda),
                             max_kv_len=256, split_size=64)
    for bad in (-1, rec.shape[0]):
        bt = kv.block_table.clone()
        bt[1, 5] = bad
        out = bi.attn_decode_q8(q, rec, bt.to(cuda), kv.kv_lens.to(cuda), max_kv_len=256,
                                split_size=64)
        assert bi.bi_check_device_errors() == bi.ERR_DEVICE_BOUNDS
        assert (out[1] == 0).all() and same_bytes(out[::2].contiguous(), good[::2].contiguous())
    too_long = i32([40, 257, 40], cuda)
    out = bi.attn_decode_q8(q, rec, kv.block_table.to(cuda), too_long, max_kv_len=256,
                            split_size=64)
    assert bi.bi_check_device_errors() == bi.ERR_DEVICE_BOUNDS
    assert (out[1] == 0).all() and same_bytes(out[::2].contiguous(), good[::2].contiguous())


def test_decode_batch_invariance_and_large_batches(cuda):
    # one request alone, among 8, and among 200 (the plan kernel's range)
    D, Hq, Hkv, S = 128, 32, 8, 256
    lens = (synth.loguniform_int(200, 1, 700, 23100)).tolist()
    lens[0] = 700
    kv = synth.paged_kv(lens, Hkv, D, PAGE, 23101, device=cuda)
    kq = bi.kv_cache_q8(kv.num_pages, Hkv, D, cuda)
    # fill the records through the write call: every page's rows
    P = kv.num_pages
    seq = torch.arange(P, dtype=torch.int32, device=cuda).repeat_interleave(PAGE)
    pos = torch.arange(PAGE, dtype=torch.int32, device=cuda).repeat(P)
    ident = torch.arange(P, dtype=torch.int32, device=cuda).view(P, 1)
    rows = lambda t: t.transpose(1, 2).reshape(P * PAGE, Hkv, D).contiguous()
    bi.kv_write_q8(rows(kv.k_cache), rows(kv.v_cache), seq, pos, kq, ident)
    q = synth.normal_bf16((200, Hq, D), 23102, device=cuda)
    out = bi.attn_decode_q8(q, kq, kv.block_table, kv.kv_lens, max_kv_len=704, split_size=S)
    assert bi.bi_check_device_errors() == bi.OK
    for n in (1, 8, 129):
        got = bi.attn_decode_q8(q[:n].contiguous(), kq, kv.block_table[:n].contiguous(),
                                kv.kv_lens[:n].contiguous(), max_kv_len=704, split_size=S)
        assert same_bytes(got, out[:n]), n
    perm = torch.randperm(200, generator=torch.Generator().manual_seed(5)).to(cuda)
    got = bi.attn_decode_q8(q[perm].contiguous(), kq, kv.block_table[perm].contiguous(),
                            kv.kv_lens[perm].contiguous(), max_kv_len=704, split_size=S)
    assert same_bytes(got, out[perm].contiguous())
    # a prompt chunk on the pages read back gives the bytes of the decode at
    # every one of its positions
    k, v = bi.kv_read_q8(kq, D, kv.block_table, kv.kv_lens, max_kv_len=704)
    qp = synth.normal_bf16((60, Hq, D), 23103, device=cuda)
    pre = bi.attn_prefill_chunk(qp, i32([0, 60], cuda), i32([640], cuda), k, v,
                                kv.block_table[:1].contiguous(), kv.kv_lens[:1].contiguous(),
                                max_q_len=60, max_kv_len=704, split_size=S)
    each = bi.attn_decode_q8(qp, kq, kv.block_table[:1].expand(60, -1).contiguous(),
                             i32(range(641, 701), cuda), max_kv_len=704, split_size=S)
    assert same_bytes(pre, each), first_divergence(pre, each)


@pytest.mark.parametrize("mode", [bi.INVARIANT, bi.VARIANT])
@pytest.mark.parametrize("B", [31, 32, 33, 128, 129, 1024, 1025])
def test_decode_plans_of_every_batch_size(cuda, B, mode):
    # the plan worked out in the kernel (32 slabs of 32 sequences at most) and
    # the plan kernel behind it, with idle slots and lengths out of range
    D, Hq, Hkv = 64, 4, 2
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 200, (B,), generator=g)
    lens[B // 2:B // 2 + 8] = 0
    pool = 40
    kv = synth.paged_kv([pool * PAGE], Hkv, D, PAGE, 23200)
    rec = quantised(kv, D).to(cuda)
    bt = torch.randint(0, pool, (B, 13), generator=g, dtype=torch.int32).to(cuda)
    q = synth.normal_bf16((B, Hq, D), 23201 + B, device=cuda)
    kl = lens.to(torch.int32).to(cuda)
    out, out32 = bi.attn_decode_q8(q, rec, bt, kl, max_kv_len=208, split_size=64, mode=mode,
                                   want_f32=True)
    assert bi.bi_check_device_errors() == bi.OK
    k, v = bi.kv_read_q8(rec, D, torch.arange(pool, dtype=torch.int32, device=cuda).view(1, -1),
                         i32([pool * PAGE], cuda), max_kv_len=pool * PAGE)
    ref, ref32 = bi.attn_decode(q, k, v, bt, kl, max_kv_len=208, split_size=64, want_f32=True)
    if mode == bi.INVARIANT:
        assert same_bytes(out32, ref32) and same_bytes(out, ref)
    else:
        check_close(f64(out32), f64(ref32), np.full(out32.shape, 2 * ATOL), "variant")
    assert (out32[lens == 0] == 0).all()
    kl[1], kl[B - 1] = -5, 209
    bad = bi.attn_decode_q8(q, rec, bt, kl, max_kv_len=208, split_size=64, mode=mode)
    assert bi.bi_check_device_errors() == bi.ERR_DEVICE_BOUNDS
    assert (bad[1] == 0).all() and (bad[B - 1] == 0).all()
    if mode == bi.INVARIANT:
        assert same_bytes(bad[2:B - 1].contiguous(), out[2:B - 1].contiguous())


def test_decode_queries_of_every_range(cuda):
    # rows of q whose elements do not all fit fp16 beside their largest one
    # take the bf16 form of the scores: the same bytes again
    D, Hq, Hkv, L = 128, 16, 4, 300
    kv = synth.paged_kv([L], Hkv, D, PAGE, 23300)
    rec = quantised(kv, D).to(cuda)
    q = synth.normal_bf16((1, Hq, D), 23301)
    q[0, 0] = 0                                        # all zeros
    q[0, 1, 1:] = 0                                    # one element
    q[0, 2, 0], q[0, 2, 1] = 2.0 ** 20, 2.0 ** -12     # 2^32 apart: still exact
    q[0, 4, 0], q[0, 4, 1] = 2.0 ** 20, 1.5 * 2.0 ** -13   # further apart
    q[0, 5] *= 2.0 ** -120
    q[0, 8, 3] = 2.0 ** -133                           # the least bf16 number
    q[0, 9] *= 2.0 ** 40                               # scores beyond any softmax's range
    q[0, 12] *= 2.0 ** 70
    q[0, 13] *= 2.0 ** -20
    q[0, 13, 5] = 2.0 ** 66
    q[0, 14, 2] = float("nan")
    q[0, 15, 2] = float("inf")
    args = (kv.block_table.to(cuda), kv.kv_lens.to(cuda), D, L, 64)
    out, out32, ref, ref32, _, _ = both_decodes(q.to(cuda), rec, *args)
    assert bi.bi_check_device_errors() == bi.OK
    fine = ~torch.isnan(ref32)
    assert torch.equal(torch.isnan(out32), ~fine)
    assert fine[0, :9].all()
    assert torch.equal(out32[fine], ref32[fine])
    # groups of four heads share a unit: the same with each head's q alone in
    # an otherwise ordinary group
    for h in range(14):
        q1 = synth.normal_bf16((1, Hq, D), 23302 + h)
        q1[0, h] = q[0, h]
        out, out32, ref, ref32, _, _ = both_decodes(q1.to(cuda), rec, *args)
        nan = torch.isnan(ref32)      # scores past the softmax's range, rows 9 and on
        assert torch.equal(torch.isnan(out32), nan), h
        assert torch.equal(out32[~nan], ref32[~nan]), h
        assert not nan.any() or h >= 9


def test_offsets_beyond_32_bits(cuda):
    # a pool of 4.6 GB of records (and 9 GB of pages read back) whose last
    # pages hold the sequence
    D, Hkv, Hq, L = 128, 8, 32, 200
    P = 140000
    n = -(-L // PAGE)
    k = synth.normal_bf16((L, Hkv, D), 23400, device=cuda)
    v = synth.normal_bf16((L, Hkv, D), 23401, device=cuda)
    q = synth.normal_bf16((1, Hq, D), 23402, device=cuda)
    seq, pos = i32([0] * L, cuda), i32(range(L), cuda)
    outs = []
    for pages, first in ((n, 0), (P, P - n)):
        cache = torch.zeros(pages, Hkv, bi.kv_q8_record_bytes(D), dtype=torch.uint8, device=cuda)
        bt = torch.arange(first, first + n, dtype=torch.int32, device=cuda).view(1, n)
        bi.kv_write_q8(k, v, seq, pos, cache, bt)
        ko, vo = bi.kv_read_q8(cache, D, bt, i32([L], cuda), max_kv_len=L)
        outs.append((cache[first:].clone(), ko[first:].clone(), vo[first:].clone(),
                     bi.attn_decode_q8(q, cache, bt, i32([L], cuda), max_kv_len=L,
                                       split_size=64)))
        del cache, ko, vo
        torch.cuda.empty_cache()
    assert bi.bi_check_device_errors() == bi.OK
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_the_binding_refuses_what_the_library_cannot_take(cuda):
    D, Hkv = 64, 2
    rec = bi.kv_cache_q8(4, Hkv, D, cuda)
    k = synth.normal_bf16((3, Hkv, D), 23500, device=cuda)
    seq, pos = i32([0, 0, 0], cuda), i32([0, 1, 2], cuda)
    bt = i32([[0, 1]], cuda)
    bi.kv_write_q8(k, k, seq, pos, rec, bt)
    with pytest.raises(TypeError):
        bi.kv_write_q8(k.float(), k, seq, pos, rec, bt)
    with pytest.raises(TypeError):
        bi.kv_write_q8(k, k, seq.long(), pos, rec, bt)
    with pytest.raises(TypeError):
        bi.kv_write_q8(k, k, seq, pos, rec.view(torch.int8), bt)
    with pytest.raises(TypeError):
        bi.kv_write_q8(k.cpu(), k, seq, pos, rec, bt)
    with pytest.raises(ValueError):
        bi.kv_write_q8(k.transpose(0, 1).contiguous().transpose(0, 1), k, seq, pos, rec, bt)
    with pytest.raises(ValueError):
        bi.kv_write_q8(k, k, seq[:2], pos, rec, bt)
    with pytest.raises(ValueError):
        bi.kv_write_q8(k, k, seq, pos, rec[:, :1], bt)
    odd = torch.zeros(4 * Hkv * PAGE * D + 8, dtype=torch.bfloat16, device=cuda)
    off = odd[8:].view(4, Hkv, PAGE, D)                # 16- but not 32-byte aligned
    with pytest.raises(bi.BiError):
        bi.bi_kv_read_q8(rec, bt, i32([3], cuda), off, off, bt, max_kv_len=3)
    q = synth.normal_bf16((1, 4, D), 23501, device=cuda)
    with pytest.raises(bi.BiError) as e:
        bi.bi_attn_decode_q8(q, rec, bt, i32([3], cuda), torch.empty_like(q), max_kv_len=3,
                             split_size=64, sm_scale=0.1)
    assert e.value.status == bi.ERR_WORKSPACE
    assert bi.bi_check_device_errors() == bi.OK


@pytest.mark.parametrize("mode", [bi.INVARIANT, bi.VARIANT])
def test_decode_units_of_more_pages_than_a_warp_holds(cuda, mode):
    # splits of 2048 keys: 128 pages a unit, past the 64 ids kept in registers
    D, Hq, Hkv, lens = 64, 8, 2, [3001, 1025, 2048, 1040, 7]
    kv = synth.paged_kv(lens, Hkv, D, PAGE, 23600)
    rec = quantised(kv, D).to(cuda)
    q = synth.normal_bf16((len(lens), Hq, D), 23601, device=cuda)
    bt = kv.block_table.to(cuda)
    args = (q, rec, bt, kv.kv_lens.to(cuda), D, 3008, 2048, mode, 1)
    out, out32, ref, ref32, _, _ = both_decodes(*args)
    assert bi.bi_check_device_errors() == bi.OK
    if mode == bi.INVARIANT:
        assert same_bytes(out32, ref32) and same_bytes(out, ref)
    else:
        check_close(f64(out32), f64(ref32), np.full(out32.shape, 2 * ATOL), "variant")
    bad = bt.clone()
    bad[0, 100] = rec.shape[0]                 # a page of the unit past the first 64
    got = bi.attn_decode_q8(q, rec, bad, kv.kv_lens.to(cuda), max_kv_len=3008, split_size=2048,
                            mode=mode, variant_splits=1)
    assert bi.bi_check_device_errors() == bi.ERR_DEVICE_BOUNDS
    assert (got[0] == 0).all()
    if mode == bi.INVARIANT:
        assert same_bytes(got[1:].contiguous(), out[1:].contiguous())


@pytest.mark.parametrize("D", [64, 128])
def test_decode_of_a_cache_on_a_16_byte_boundary_with_shared_pages(cuda, D):
    # the least alignment the cache may have; two sequences that share pages
    Hq, Hkv, lens = 8, 2, [77, 64, 1, 16]
    kv = synth.paged_kv(lens, Hkv, D, PAGE, 23700)
    rec = quantised(kv, D).to(cuda)
    q = synth.normal_bf16((len(lens) + 1, Hq, D), 23701, device=cuda)
    bt = torch.cat([kv.block_table, kv.block_table[:1]]).to(cuda)
    L = i32(lens + [70], cuda)
    raw = torch.zeros(rec.numel() + 16, dtype=torch.uint8, device=cuda)
    off = raw[16:].view(rec.shape)
    off.copy_(rec)
    assert off.data_ptr() % 32 == 16
    want = both_decodes(q, rec, bt, L, D, 77, 64)
    got = bi.attn_decode_q8(q, off, bt, L, max_kv_len=77, split_size=64)
    assert bi.bi_check_device_errors() == bi.OK
    assert same_bytes(got, want[0]) and same_bytes(got, want[2])


def test_empty_calls(cuda):
    D, Hq, Hkv = 64, 4, 2
    cache = torch.full((3, Hkv, bi.kv_q8_record_bytes(D)), 0x55, dtype=torch.uint8, device=cuda)
    before = cache.clone()
    bt = torch.zeros(2, 1, dtype=torch.int32, device=cuda)
    zero = i32([0, 0], cuda)
    q = synth.normal_bf16((2, Hq, D), 23702, device=cuda)
    for most in (0, 16):                       # every length zero: rows of zeros
        out, out32 = bi.attn_decode_q8(q, cache, bt, zero, max_kv_len=most, split_size=64,
                                       want_f32=True)
        assert (out == 0).all() and (out32 == 0).all()
        k, v = bi.kv_read_q8(cache, D, bt, zero, max_kv_len=most)
        assert (k == 0).all() and (v == 0).all()
    none = bi.attn_decode_q8(q[:0], cache, bt[:0], zero[:0], max_kv_len=16, split_size=64)
    assert none.shape == (0, Hq, D)
    rows = q[:0, :Hkv].contiguous()
    bi.kv_write_q8(rows, rows, zero[:0], zero[:0], cache, bt)
    assert bi.bi_check_device_errors() == bi.OK
    assert torch.equal(cache, before)
