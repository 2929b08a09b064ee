"""Refusals of pa_merge before any launch (CPU)."""
import pytest


def test_mla_merge_refuses_an_unaligned_out():
    """As pa_run does: its rows leave as 8-byte stores."""
    import paged_quantized_kv_gqa_gb300 as pa
    prob = pa.make_problem(bsz=1, q_heads=128, kv_heads=1, head_dim_qk=576, head_dim_v=512, block_size=64,
                           max_blocks_per_seq=64, num_pages=64, kv_dtype="fp8_e4m3", scale_kind="global",
                           layout="mla", causal=True, chunk_size=-1, sm_scale=0.1, q_stride=128 * 576)
    pl = pa.pa_plan(prob, [1], [4000], [0, 1], 152)
    assert len(pl.describe()["merge_tokens"])
    for call in (pa.pa_run, pa.pa_merge):
        args = pa.make_args(q=256, cache_k=256, cache_v=256, k_scale=256, v_scale=256, block_table=256, out=264)
        with pytest.raises(pa.PaError) as e:
            call(pl, args, 256, 0)
        assert e.value.status == pa.PA_ERR_INVALID_ARG and "aligned" in str(e.value)
