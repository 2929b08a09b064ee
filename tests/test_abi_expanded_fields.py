"""Fields of pa_problem that plans of expanded rows do not use (CPU)."""
import pytest


@pytest.fixture(scope="module")
def pa():
    import paged_quantized_kv_gqa_gb300 as m
    return m


def problem(pa, **kw):
    p = pa.make_problem(bsz=2, q_heads=4, kv_heads=4, head_dim_qk=192, head_dim_v=128, kv_dtype="bf16", layout="mla_expanded",
                        causal=True, chunk_size=-1, sm_scale=0.07, q_stride=4 * 192)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw", [dict(max_blocks_per_seq=0, num_pages=0), dict(num_pages=-1), dict(scale_kind=9),
                                dict(max_blocks_per_seq=0, num_pages=0, scale_kind=0)])
def test_fields_of_a_cache_may_hold_anything(pa, kw):
    want = pa.pa_plan(problem(pa), [300, 5], [70, 9], [0, 300, 305], 152).describe()
    got = pa.pa_plan(problem(pa, **kw), [300, 5], [70, 9], [0, 300, 305], 152).describe()
    assert (got["items"] == want["items"]).all() and got["max_chunks"] == want["max_chunks"]


@pytest.mark.parametrize("field", ["max_blocks_per_seq", "num_pages"])
def test_a_cache_needs_them(pa, field):
    p = pa.make_problem(bsz=1, q_heads=4, kv_heads=4, head_dim_qk=128, head_dim_v=128, max_blocks_per_seq=1, num_pages=1,
                        kv_dtype="int8", scale_kind="global", layout="gqa", causal=True, chunk_size=0, sm_scale=0.1, q_stride=512)
    setattr(p, field, 0)
    with pytest.raises(pa.PaError) as e:
        pa.pa_plan(p, [5], [3], [0, 5], 152)
    assert e.value.status == pa.PA_ERR_INVALID_ARG
