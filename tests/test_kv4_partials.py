"""Partial rows of plans over a 4-bit cache: the workspace holds as many as the plan
has chunks, whatever the lengths beside each other (CPU)."""
import numpy as np
import pytest

from kv4_helpers import make, problem

ROW = 128 * 4 + 8        # an fp32 partial row, its maximum and its sum


@pytest.fixture(scope="module")
def pa():
    import paged_quantized_kv_gqa_gb300 as m
    return m


def plan(pa, p, sms=152):
    return pa.pa_plan(problem(pa, p), p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, sms)


def lengths(q, kv, heads, kv_heads, **kw):
    """A problem without its cache: plans take lengths alone."""
    p = make(1, seq_lens=[1], seq_lens_kv=[1], q_heads=heads, kv_heads=kv_heads, garbage=False, **kw)
    p.seq_lens, p.seq_lens_kv = np.asarray(q, np.int32), np.asarray(kv, np.int32)
    p.bsz = len(q)
    p.cu_seqlens_q = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    p.max_blocks_per_seq = int(max(-(-(a + b) // 64) for a, b in zip(q, kv)))
    p.num_pages = int(sum(-(-(a + b) // 64) for a, b in zip(q, kv)))
    return p


def partial_bytes(d, q_heads):
    n = d["nch_token"].astype(np.int64)
    return int(n[n > 1].sum()) * q_heads * ROW


@pytest.mark.parametrize("q,kv,heads,kv_heads,kw", [
    ([1] * 256, [131071] + [500] * 255, 64, 8, {}),
    ([1] * 64, [500] * 63 + [131071], 64, 8, {}),
    ([1] * 256, [131071] + [512] * 255, 16, 1, {}),
    ([2] * 40, [60000] + [700] * 39, 32, 4, {}),                      # 16 rows
    ([6] * 32, [60000] + [1200] * 31, 64, 8, {}),                     # 48 rows
    ([65] + [3] * 20, [30000] + [100] * 20, 8, 2, dict(chunk_size=512)),   # append
])
@pytest.mark.parametrize("kind", ["int4", "fp4_e2m1"])
def test_workspace_holds_the_plans_chunks_and_no_more(pa, q, kv, heads, kv_heads, kw, kind):
    pl = plan(pa, lengths(q, kv, heads, kv_heads, kv_dtype=kind, **kw))
    d = pl.describe()
    assert d["max_chunks"] > 8 and d["nch_token"].min() * 4 < d["max_chunks"]
    need = partial_bytes(d, heads)
    assert need <= pl.workspace_size <= need + d["plan_bytes"] + 5 * 256
    assert d["workspace_bytes"] == pl.workspace_size


def test_a_long_sequence_beside_short_ones_fits_the_built_in_workspace(pa):
    pl = plan(pa, lengths([1] * 64, [131071] + [500] * 63, 64, 8))
    assert pl.workspace_size < 32 << 20


def test_plans_without_split_rows_need_no_partial_rows(pa):
    pl = plan(pa, lengths([1] * 9, [400] * 9, 8, 2))
    d = pl.describe()
    assert d["max_chunks"] == 1 and pl.workspace_size <= d["plan_bytes"] + 2 * 256


@pytest.mark.parametrize("q,kv,cross,kind", [
    ([1, 1], [5000, 30], False, "int4"), ([6], [9000], False, "fp4_e2m1"),
    ([1, 2], [0, 0], True, "int4"), ([70, 3], [0, 100], True, "fp4_e2m1"), ([1, 1], [0, 100], True, "int8"),
])
def test_plans_made_without_chunks_leave_nothing_to_merge(pa, q, kv, cross, kind):
    """chunk_size 0 promises final rows after pa_run: pa_merge does nothing (here it
    would fail, there being no device memory behind the arguments)."""
    p = make(1, seq_lens=q, seq_lens_kv=kv, q_heads=16, kv_heads=2, causal=not cross, cross=cross, garbage=False)
    p.kv_dtype = kind
    pl = plan(pa, p)
    assert len(pl.describe()["merge_tokens"])
    a = dict(q=256, cache_k=256, cache_v=256, k_scale=256, v_scale=256, block_table=256, out=256)
    pa.pa_merge(pl, pa.make_args(**a), 256, 0)


@pytest.mark.parametrize("q,G,workers", [(1, 8, 16), (2, 8, 8), (3, 4, 8), (2, 5, 8), (1, 16, 8), (1, 4, 16)])
def test_decode_is_cut_for_the_warps_that_a_cta_has(pa, q, G, workers):
    """Pieces: one for every tile and head, and one cut for every worker at most (16
    warps a CTA up to 8 rows, 8 warps up to 16)."""
    r = np.random.default_rng(q * G)
    d = plan(pa, lengths([q] * 32, r.integers(2048, 8192, 32), 8 * G, 8)).describe()
    assert 152 * workers * 0.9 < d["num_items"] <= 152 * workers + 32 * 8
