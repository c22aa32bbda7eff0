"""The ramps of scaled rotary positions that a caller gets without naming
them; no GPU."""
import dataclasses

import numpy as np
import pytest

import invariant_bi_rmsnorm_02_gb300 as bi
from invariant_bi_rmsnorm_02_gb300.decoder import LLAMA3_8B, TINY
from oracle import longctx

PUBLISHED = {"llama3": (bi.ROPE_LLAMA3, 4.0), "yarn": (bi.ROPE_YARN, 32.0)}


@pytest.mark.parametrize("kind", sorted(PUBLISHED))
@pytest.mark.parametrize("rot,theta", [(128, 500000.0), (64, 10000.0)])
def test_default_ramp_is_the_published_one(kind, rot, theta):
    code, high = PUBLISHED[kind]
    f, m = bi.rope_frequencies(rot, theta, code, 8.0, 8192, device="cpu")
    want, wm = longctx.frequencies(rot, theta, kind, 8.0, 8192.0, 1.0, high)
    assert (np.abs(f.numpy() - want) <= 2.0 ** -46 * want).all()
    assert abs(m - wm) <= 2.0 ** -23 * wm
    # the two published ramps are told apart by these sizes
    other = longctx.frequencies(rot, theta, kind, 8.0, 8192.0, 1.0, 36.0 - high)[0]
    assert (np.abs(f.numpy() - other) > 1e-3 * other).any()


@pytest.mark.parametrize("base", [LLAMA3_8B, TINY])
def test_configuration_takes_the_published_ramp(base):
    for kind, (_, high) in PUBLISHED.items():
        cfg = dataclasses.replace(base, rope_scaling=kind, rope_factor=8.0)
        assert cfg.rope_high_turns == high and cfg.rope_low_turns == 1.0
        assert dataclasses.replace(cfg, layers=1).rope_high_turns == high
        given = dataclasses.replace(base, rope_scaling=kind, rope_high_turns=6.0)
        assert given.rope_high_turns == 6.0
    for kind in ("none", "linear", "ntk"):      # no ramp, nothing to settle
        cfg = dataclasses.replace(base, rope_scaling=kind, rope_factor=8.0)
        assert dataclasses.replace(cfg, rope_scaling="yarn").rope_high_turns == 32.0


def test_configuration_refuses_a_width_that_is_no_part_of_a_head():
    for bad in (0, -2, 7, TINY.head_dim + 2):
        with pytest.raises(ValueError):
            dataclasses.replace(TINY, rope_dim=bad)
    for good in (None, 2, TINY.head_dim):
        assert dataclasses.replace(TINY, rope_dim=good).rope_dim == good
