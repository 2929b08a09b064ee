"""Zeros in rows of the rotated append: E4M3 keeps the sign of a zero, as pa_cache_append does."""
import numpy as np
import pytest

import rope_helpers as rh
from oracle import kv4
from test_gpu_rope_append import check, launch

pytestmark = pytest.mark.gpu


def with_zeros(seed, **kw):
    """Rows with zeros of both signs strewn in, rows of nothing else among them."""
    p = rh.make(seed=seed, **kw)
    r = np.random.default_rng(seed)
    for n in ("q_new", "k_new", "v_new"):
        x = getattr(p, n)
        if x is None:
            continue
        x = x.copy()
        zero = np.where(r.random(x.shape) < 0.5, np.uint16(0x8000), np.uint16(0))
        x = np.where(r.random(x.shape) < 0.2, zero, x)
        x[3::7] = zero[3::7]
        setattr(p, n, x)
    return p


@pytest.mark.parametrize("sms", [None, 1])
@pytest.mark.parametrize("kv_dtype", ["int8", "fp8_e4m3"])
@pytest.mark.parametrize("scale_kind", ["per_kv_head", "per_channel", "global"])
@pytest.mark.parametrize("rot, pairs", [(128, "halves"), (64, "adjacent")])
def test_zeros(rot, pairs, scale_kind, kv_dtype, sms):
    check(with_zeros(30, seq_lens=[70, 9], seq_lens_kv=[30, 0], kv_dtype=kv_dtype, scale_kind=scale_kind, rot=rot, pairs=pairs),
          sms=sms)


@pytest.mark.parametrize("kv_dtype", ["int8", "fp8_e4m3"])
def test_zeros_of_latent_rows(kv_dtype):
    check(with_zeros(31, seq_lens=[17, 2], seq_lens_kv=[60, 0], layout="mla", kv_dtype=kv_dtype, rot=64))


@pytest.mark.parametrize("sms", [None, 1])
@pytest.mark.parametrize("scale_kind", ["per_kv_head", "per_channel"])
@pytest.mark.parametrize("kv_dtype", ["int4", "fp4_e2m1"])
def test_zeros_of_four_bits(kv_dtype, scale_kind, sms):
    """The stored values (a zero's code may have either sign) and block scales."""
    p = with_zeros(32, seq_lens=[70, 9], seq_lens_kv=[30, 0], kv_dtype=kv_dtype, scale_kind=scale_kind)
    got, want = launch(p, sms=sms)[1:3], rh.expected(p)[1:]
    table = kv4.code_table(kv_dtype)
    for unpack, a, b in zip((kv4.unpack_k, kv4.unpack_v), got, want):
        (ca, sa), (cb, sb) = unpack(a), unpack(b)
        assert (table[ca] == table[cb]).all() and (sa == sb).all()
