"""What pa_rope_append refuses, before any GPU work (CPU)."""
import numpy as np
import pytest

import rope_helpers as rh


@pytest.fixture(scope="module")
def pa():
    import paged_quantized_kv_gqa_gb300 as m
    return m


def call(pa, *, layout="gqa", kv_dtype="int8", cross=False, rope=None, **kw):
    """Addresses are never followed: every call here is refused on the host."""
    p = rh.make(seq_lens=[2], seq_lens_kv=[3], layout=layout, kv_dtype=kv_dtype)
    plan = pa.pa_plan(pa.make_problem(**{k: getattr(p, k) for k in (
        "bsz", "q_heads", "kv_heads", "head_dim_qk", "head_dim_v", "block_size", "max_blocks_per_seq", "num_pages", "kv_dtype",
        "scale_kind", "layout", "chunk_size", "sm_scale", "q_stride")}, causal=not cross, cross=cross), p.seq_lens,
        p.seq_lens_kv, p.cu_seqlens_q, 152)
    args = pa.make_args(q=None, cache_k=1 << 20, cache_v=1 << 20, k_scale=1 << 20, v_scale=1 << 20, block_table=1 << 20,
                        out=None, seq_lens=1 << 20, seq_lens_kv=1 << 20, cu_seqlens_q=1 << 20)
    r = dict(cos_sin=1 << 20, table_rows=8, rot_dim=64)
    r.update(rope or {})
    width = p.q_heads * (192 if layout == "mla" else 128)
    a = dict(q_new=1 << 20, q_stride=width, q_out=1 << 21, q_out_stride=width, k_new=1 << 20, v_new=1 << 20,
             kv_stride=p.kv_heads * p.head_dim_qk, workspace=1 << 20)
    a.update(kw)
    pa.pa_rope_append(plan, args, pa.make_rope(**r), a["q_new"], a["q_stride"], a["q_out"], a["q_out_stride"], a["k_new"],
                      a["v_new"], a["kv_stride"], a["workspace"], stream=0)


@pytest.mark.parametrize("kw, text", [
    (dict(rope=dict(cos_sin=None)), "cos_sin"),
    (dict(rope=dict(cos_sin=(1 << 20) + 8)), "aligned"),
    (dict(rope=dict(rot_dim=24)), "rot_dim"),
    (dict(rope=dict(rot_dim=0)), "rot_dim"),
    (dict(rope=dict(rot_dim=96), layout="mla", kv_dtype="fp8_e4m3"), "rot_dim"),
    (dict(rope=dict(table_rows=0)), "table_rows"),
    (dict(rope=dict(pairs=2)), "pairs"),
    (dict(rope=dict(axes=5, positions=1 << 20)), "axes"),
    (dict(rope=dict(axes=2)), "positions"),
    (dict(rope=dict(axes=2, positions=1 << 20, pair_axes=[2] + [0] * 31)), "pair_axis"),
    (dict(rope=dict(positions=(1 << 20) + 2)), "aligned"),
    (dict(q_new=None), "together"),
    (dict(q_out=None), "together"),
    (dict(q_stride=504), "stride"),
    (dict(q_out_stride=8), "stride"),
    (dict(q_out=1 << 20, q_out_stride=1024), "in place"),
    (dict(q_new=(1 << 20) + 2), "aligned"),
    (dict(q_stride=513), "aligned"),
    (dict(k_new=(1 << 20) + 8), "aligned"),
    (dict(v_new=(1 << 20) + 8), "aligned"),
    (dict(kv_stride=257), "aligned"),
    (dict(kv_stride=128), "kv_stride"),
    (dict(k_new=None), "null"),
    (dict(v_new=None), "null"),
    (dict(workspace=None), "null"),
    (dict(cross=True), "cross"),
])
def test_refusals(pa, kw, text):
    with pytest.raises(pa.PaError, match=text) as e:
        call(pa, **kw)
    assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_make_rope_wants_an_axis_for_every_pair(pa):
    for axes in ([0] * 31, [0] * 33, [-1] + [0] * 31):
        with pytest.raises(ValueError):
            pa.make_rope(cos_sin=1 << 20, table_rows=4, rot_dim=64, pair_axes=axes)


def test_the_struct_is_the_headers(pa):
    import ctypes
    r = pa.make_rope(cos_sin=16, table_rows=3, rot_dim=128, pairs="adjacent", positions=32, axes=2,
                     pair_axes=[0] * 32 + [1] * 32)
    raw = bytes(r)
    assert ctypes.sizeof(pa.PaRope) == 2 * 8 + 4 * 4 + 64
    assert np.frombuffer(raw[:16], np.uint64).tolist() == [16, 32]
    assert np.frombuffer(raw[16:32], np.int32).tolist() == [3, 128, 1, 2]
    assert raw[32:] == bytes([0] * 32 + [1] * 32)
