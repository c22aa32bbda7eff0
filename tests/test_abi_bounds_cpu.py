"""The attention calls' host bounds at the ends of their ranges; no GPU."""
import pytest

import invariant_bi_rmsnorm_02_gb300 as bi

P = 1 << 20              # a 16-byte aligned fake address: never dereferenced on these paths
INT_MAX = 2 ** 31 - 1
LARGEST_SPLIT = 2 ** 31 - 64


def up(x, to):
    return -(-x // to) * to


@pytest.mark.parametrize("max_kv_len", [1, 64, 65, 2 ** 30, INT_MAX - 62, INT_MAX])
@pytest.mark.parametrize("split", [64, 256, 2 ** 30, LARGEST_SPLIT])
def test_decode_workspace_size_of_every_bound(max_kv_len, split):
    B, Hq, D = 3, 4, 64
    s = -(-max_kv_len // split)
    want = 256 + up(16 * B * s, 256) + up(8 * B * Hq * up(s, 2), 256) + 4 * B * Hq * s * D
    assert bi.bi_attn_decode_workspace_size(B, Hq, 2, D, max_kv_len, split, bi.INVARIANT, 0) == want


@pytest.mark.parametrize("name", ["bi_attn_decode", "bi_attn_decode_q8"])
@pytest.mark.parametrize("max_kv_len,split", [(INT_MAX, 64), (INT_MAX - 62, 64), (INT_MAX, 2 ** 30),
                                              (64, LARGEST_SPLIT), (INT_MAX, LARGEST_SPLIT)])
def test_decode_asks_for_its_workspace_at_every_bound(name, max_kv_len, split):
    lib = bi.load()
    caches = (P, P) if name == "bi_attn_decode" else (P,)
    for ws in ((None, 0), (P, 256)):
        assert getattr(lib, name)(P, *caches, P, P, P, None, 2, 4, 2, 64, 16, 8, 4, max_kv_len,
                                  split, 0.125, bi.INVARIANT, 0, *ws, None) == bi.ERR_WORKSPACE
