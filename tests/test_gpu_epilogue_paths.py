"""Paths of the products with an epilogue that few shapes reach: pairs of CTAs
whose warps come to their common barriers from work of single lanes."""
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
