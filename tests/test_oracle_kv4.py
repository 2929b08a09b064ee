"""CPU pins of the 4-bit oracle: code values, slab layout, quantisation and
attention against closed forms."""
import math

import numpy as np
import pytest

from oracle import kv4
from kv4_helpers import KINDS, make, reference, seen_mask


def test_code_values():
    assert [kv4.fp4_value(c) for c in range(8)] == [0, .5, 1, 1.5, 2, 3, 4, 6]
    assert [kv4.fp4_value(c) for c in range(9, 16)] == [-.5, -1, -1.5, -2, -3, -4, -6]
    assert kv4.code_table("int4").tolist() == [0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1]


def test_slab_layout_by_hand():
    codes, scales = np.zeros((64, 128), np.uint8), np.zeros((64, 8), np.uint8)
    codes[33, 5], scales[33, 7] = 9, 0x38
    k, v = kv4.pack_k(codes, scales), kv4.pack_v(codes, scales)
    assert k.shape == v.shape == (4608,)
    assert k[2304 + 1 * 64 + 2] == 9 << 4 and k[2304 + 2048 + 1 * 8 + 7] == 0x38 and (k != 0).sum() == 2
    assert v[2304 + 5 * 16 + 0] == 9 << 4 and v[2304 + 2048 + 7 * 32 + 1] == 0x38 and (v != 0).sum() == 2


def test_pack_inverts_unpack():
    r = np.random.default_rng(1)
    s = r.integers(0, 256, (3, 2, 4608)).astype(np.uint8)
    assert np.array_equal(kv4.pack_k(*kv4.unpack_k(s)), s)
    assert np.array_equal(kv4.pack_v(*kv4.unpack_v(s)), s)


@pytest.mark.parametrize("kind", KINDS)
def test_values_on_the_grid_are_stored_exactly(kind):
    """Multiples that a block scale of 0.5 represents come back as they were."""
    top = 6.0 if kind == "fp4_e2m1" else 7.0
    table = kv4.code_table(kind)
    table = table[np.abs(table) <= top]
    x = np.zeros((1, 128), np.float32)
    x[0, :16] = np.resize(table, 16) * 0.5
    x[0, 0] = top * 0.5
    codes, sb = kv4.quantise_rows(x, np.ones(128, np.float32), kind)
    assert kv4.E4M3[sb[0, 0]] == 0.5
    assert np.array_equal(kv4.code_table(kind)[codes[0]] * np.repeat(kv4.E4M3[sb[0]], 16), x[0])
    assert (sb[0, 1:] == 0).all() and (codes[0, 16:] == 0).all()


def test_ties_go_to_even_and_saturate():
    x = np.zeros((1, 128), np.float32)
    x[0, :8] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5]
    x[0, 16:20] = [np.inf, -np.inf, np.nan, 1]
    c, s = kv4.quantise_rows(x, np.ones(128, np.float32), "fp4_e2m1")
    assert kv4.code_table("fp4_e2m1")[c[0, :8]].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]
    assert kv4.E4M3[s[0, 1]] == 448 and kv4.code_table("fp4_e2m1")[c[0, 16:20]].tolist() == [6, -6, 0, 0]
    x[0, :8] = [7, .5, 1.5, 2.5, -.5, -1.5, -2.5, 6.5]
    c, _ = kv4.quantise_rows(x, np.ones(128, np.float32), "int4")
    assert kv4.code_table("int4")[c[0, :8]].tolist() == [7, 0, 2, 2, 0, -2, -2, 6]


@pytest.mark.parametrize("kind", KINDS)
def test_one_visible_position_returns_its_value(kind):
    p = make(3, seq_lens=[1, 1], seq_lens_kv=[0, 0], q_heads=4, kv_heads=2, kv_dtype=kind)
    out, lse, _, _ = reference(p)
    for b in range(2):
        for h in range(4):
            assert np.allclose(out[b, h], kv4.rows(p, "v", b, h // 2, 1)[0], rtol=1e-14)


def test_attention_against_a_plain_loop():
    p = make(4, seq_lens=[3, 2], seq_lens_kv=[70, 5], q_heads=4, kv_heads=2, scale_kind="per_channel")
    out, lse, _, _ = reference(p)
    for b, i, h in [(0, 0, 0), (0, 2, 3), (1, 1, 2)]:
        n = int(p.seq_lens_kv[b]) + i + 1
        K, V = kv4.rows(p, "k", b, h // 2, n), kv4.rows(p, "v", b, h // 2, n)
        t = int(p.cu_seqlens_q[b]) + i
        q = kv4.bf16_to_f64(p.q_bits[t, h * 128:(h + 1) * 128])
        s = [sum(q[d] * K[j, d] for d in range(128)) * p.sm_scale for j in range(n)]
        z = sum(math.exp(x) for x in s)
        assert abs(lse[t, h] - math.log(z)) < 1e-10
        assert np.allclose(out[t, h], sum(math.exp(x) / z * V[j] for j, x in enumerate(s)), atol=1e-10)


def test_cross_attention_sees_the_states_and_nothing_else():
    p = make(5, seq_lens=[2, 3, 1], seq_lens_kv=[5, 0, 64], q_heads=2, kv_heads=1, causal=False, cross=True)
    assert seen_mask(p, 0).shape == (2, 5) and seen_mask(p, 0).all()
    out, lse, _, _ = reference(p)
    assert (out[2:5] == 0).all() and np.isneginf(lse[2:5]).all() and np.isfinite(lse[[0, 1, 5]]).all()
