"""Latent rows and queries of the rotated append: 16 query heads a warp (rows enough that 8 are
not needed to fill the GPU; a plan for one SM has them at sizes that the oracle can follow) and
positions of several axes."""
import pytest

import rope_helpers as rh
from test_gpu_rope_append import check

pytestmark = pytest.mark.gpu


def latent(seed, **kw):
    return rh.make(seed=seed, layout="mla", **{"kv_dtype": "fp8_e4m3", "rot": 64, **kw})


@pytest.mark.parametrize("kv_dtype", ["int8", "fp8_e4m3"])
@pytest.mark.parametrize("kw", [dict(), dict(in_place=True), dict(q=False), dict(pad=8)])
def test_many_rows(kv_dtype, kw):
    check(latent(40, seq_lens=[290, 0, 9], seq_lens_kv=[13, 3, 64], kv_dtype=kv_dtype), sms=1, **kw)


@pytest.mark.parametrize("sms", [None, 1])
@pytest.mark.parametrize("order", ["turns", "runs", "odd"])
@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("rot", [64, 48])
def test_axes(rot, pairs, axes, order, sms):
    n = rot // 2
    of = {"turns": [i % axes for i in range(n)], "runs": [i * axes // n for i in range(n)],
          "odd": [min(axes - 1, i // 7) for i in range(n)]}[order]
    check(latent(41, seq_lens=[9, 1, 120 if sms else 3], seq_lens_kv=[2, 200, 61], rot=rot, pairs=pairs, axes=axes, pair_axis=of,
                 table_rows=300), sms=sms)


@pytest.mark.parametrize("sms", [None, 1])
def test_positions_handed_over_on_one_axis(sms):
    check(latent(42, seq_lens=[130], seq_lens_kv=[7], kv_dtype="int8", given=True, table_rows=1000), sms=sms)
