"""CPU checks of the 4-bit cache's and cross attention's entry points: plans
equal to the oracle planner's, sizes, and refusals before any launch."""
import numpy as np
import pytest

import synth
from oracle import planner as op
from kv4_helpers import KINDS, make, problem


@pytest.fixture(scope="module")
def pa():
    import paged_quantized_kv_gqa_gb300 as m
    return m


def plan(pa, p, sms=152):
    return pa.pa_plan(problem(pa, p), p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, sms)


def same_plan(got, want):
    for key in ("family", "chunk", "tokens_per_tile", "num_ctas", "max_chunks"):
        assert got[key] == want[key], key
    for key in ("items", "work_indptr", "nch_token", "merge_tokens"):
        assert np.array_equal(got[key], want[key]), key


@pytest.mark.parametrize("seed", range(30))
def test_cross_planner_matches_oracle(pa, seed):
    r = np.random.default_rng(seed)
    bsz = int(r.integers(1, 7))
    kvh = int(r.choice([1, 2, 8]))
    q = r.integers(0, 4, bsz) if seed % 2 else r.integers(0, 150, bsz)
    kv = np.where(r.random(bsz) < 0.3, 0, r.integers(0, 3000, bsz))
    p = make(seed, seq_lens=q, seq_lens_kv=kv, q_heads=kvh * int(r.choice([1, 3, 4])), kv_heads=kvh,
             causal=False, cross=True, chunk_size=int(r.choice([0, 64, 512, -1])), garbage=False)
    sms = int(r.choice([1, 8, 152]))
    got = plan(pa, p, sms).describe()
    same_plan(got, op.plan(p, sms))
    pairs = sum(int(a) * int(b) for a, b in zip(q, kv))
    assert got["flops"] == pairs * p.q_heads * 512
    pages = sum(-(-int(b) // 64) for a, b in zip(q, kv) if a > 0)
    assert got["kv_bytes"] == pages * 2 * 4608 * kvh
    assert not got["fused_merge"]


def test_cross_rows_without_states_are_merge_tokens(pa):
    p = make(1, seq_lens=[2, 1, 3], seq_lens_kv=[0, 100, 0], q_heads=4, kv_heads=2, causal=False, cross=True)
    d = plan(pa, p).describe()
    assert d["nch_token"].tolist() == [0, 0, 1, 0, 0, 0] and d["merge_tokens"].tolist() == [0, 1, 3, 4, 5]
    assert len(d["items"]) == 2 and d["max_chunks"] == 1
    p = make(1, seq_lens=[2], seq_lens_kv=[0], q_heads=4, kv_heads=2, causal=False, cross=True, chunk_size=-1)
    d = plan(pa, p).describe()
    assert d["num_ctas"] == 0 and d["merge_tokens"].tolist() == [0, 1]


def test_cross_sequence_longer_than_its_query_needs_no_page_for_it(pa):
    """The query tokens are not in the cache: 64 states and 70 tokens fit one page."""
    p = make(1, seq_lens=[70], seq_lens_kv=[64], q_heads=1, kv_heads=1, causal=False, cross=True)
    assert p.max_blocks_per_seq == 1
    plan(pa, p)


def test_single_launch_option_is_not_taken_with_empty_rows_or_4_bits(pa):
    def fused(kind, lens):
        p = make(1, seq_lens=[1, 1], seq_lens_kv=lens, q_heads=4, kv_heads=2, causal=False, cross=True, chunk_size=64)
        p.kv_dtype = kind
        return plan(pa, p).describe()["fused_merge"]
    pa.pa_set_fused_merge(True)
    try:
        assert fused("int8", [200, 70])
        assert not fused("int8", [200, 0]) and not fused("int4", [200, 70])
    finally:
        pa.pa_set_fused_merge(False)


@pytest.mark.parametrize("seed", range(30))
def test_four_bit_plans_match_oracle(pa, seed):
    """Every family; decode takes equal shares of the pages."""
    r = np.random.default_rng(100 + seed)
    bsz, kvh, G = int(r.integers(1, 7)), int(r.choice([1, 3, 8])), int(r.choice([1, 4, 5, 16]))
    q = r.integers(0, max(1, 16 // G) + 1, bsz) if seed % 3 else r.integers(0, 90, bsz)
    p = make(seed, seq_lens=q, seq_lens_kv=r.integers(0, 4000, bsz), q_heads=kvh * G, kv_heads=kvh,
             kv_dtype=KINDS[seed % 2], chunk_size=int(r.choice([0, 64, 512, -1, -1])), causal=bool(r.random() < 0.7),
             garbage=False)
    sms = int(r.choice([1, 8, 152]))
    d = plan(pa, p, sms).describe()
    same_plan(d, op.plan(p, sms))
    assert d["kv_bytes"] == sum(-(-int(n) // 64) for n, a in zip(p.held, q) if a) * 2 * 4608 * kvh


@pytest.mark.parametrize("G", [4, 9])
@pytest.mark.parametrize("chunk", [-1, 128])
def test_decode_shares_cover_every_position_once(pa, chunk, G):
    p = make(3, seq_lens=[1, 2, 1, 1], seq_lens_kv=[5000, 63, 0, 777], q_heads=3 * G, kv_heads=3, chunk_size=chunk,
             garbage=False)
    d = plan(pa, p, 20).describe()
    pieces = {}
    for b, h, tok, n, base, lo, hi, c in d["items"].tolist():
        pieces.setdefault((b, h), []).append((lo, hi, c & 0xFFFF, c >> 16))
        assert lo < hi
    for b in range(4):
        for h in range(3):
            got = sorted(pieces[b, h])
            assert [x[0] for x in got] == [0] + [x[1] for x in got[:-1]] and got[-1][1] == p.held[b]
            assert [x[2] for x in got] == list(range(len(got))) and all(x[3] == len(got) for x in got)
            assert (d["nch_token"][p.cu_seqlens_q[b]:p.cu_seqlens_q[b + 1]] == len(got)).all()


def test_cache_bytes(pa):
    p = make(2, seq_lens=[3], seq_lens_kv=[70], q_heads=8, kv_heads=2)
    assert pa.pa_cache_bytes(problem(pa, p)) == (p.cache_k.size, p.cache_v.size)
    c = synth.make_case(name="b", seed=1, seq_lens=[3], seq_lens_kv=[70], q_heads=8, kv_heads=2)
    assert pa.pa_cache_bytes(pa.problem_of(c)) == (c.cache_k.size, c.cache_v.size)
    with pytest.raises(pa.PaError):
        prob = problem(pa, p)
        prob.num_pages = 0
        pa.pa_cache_bytes(prob)


@pytest.mark.parametrize("field,value,status", [
    ("kv_dtype", 4, 1), ("kv_dtype", -1, 1), ("causal", 3, 1), ("causal", -1, 1), ("head_dim_qk", 64, 2),
    ("block_size", 32, 1), ("layout", 1, 2), ("num_pages", 1 << 24, 2), ("chunk_size", 96, 1),
])
def test_invalid_problems_rejected(pa, field, value, status):
    p = make(1, seq_lens=[2], seq_lens_kv=[10], q_heads=8, kv_heads=2)
    prob = problem(pa, p)
    if field == "block_size":
        prob.chunk_size = 48
    setattr(prob, field, value)
    with pytest.raises(pa.PaError) as e:
        pa.pa_plan(prob, p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, 152)
    assert e.value.status == status


def test_pools_up_to_the_tma_row_limit(pa):
    """72 rows of 64 bytes a slab; 8-bit caches 128."""
    p = make(1, seq_lens=[2], seq_lens_kv=[10], q_heads=8, kv_heads=2)
    prob = problem(pa, p)
    prob.num_pages = ((1 << 31) - 1) // (2 * 72)
    pa.pa_plan(prob, p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, 152)
    prob.num_pages += 1
    with pytest.raises(pa.PaError):
        pa.pa_plan(prob, p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, 152)
    prob.num_pages, prob.kv_dtype = (1 << 31) // (2 * 128), pa.KV_DTYPES["int8"]
    with pytest.raises(pa.PaError):
        pa.pa_plan(prob, p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, 152)


def test_single_launch_plans_refuse_an_unaligned_out(pa):
    """The in-kernel merge stores four elements at once (8-bit plans with split rows)."""
    c = synth.make_case(name="f", seed=1, seq_lens=[1], seq_lens_kv=[300], q_heads=8, kv_heads=2, chunk_size=64)
    pa.pa_set_fused_merge(True)
    try:
        pl = pa.pa_plan(pa.problem_of(c), c.seq_lens, c.seq_lens_kv, c.cu_seqlens_q, 152)
    finally:
        pa.pa_set_fused_merge(False)
    assert pl.describe()["fused_merge"]
    for out in (258, 260):
        with pytest.raises(pa.PaError) as e:
            pa.pa_run(pl, fake_args(pa, out=out), 256, None)
        assert e.value.status == pa.PA_ERR_INVALID_ARG and "aligned" in str(e.value)


def test_mla_refuses_four_bits_and_cross(pa):
    kw = dict(bsz=1, q_heads=128, kv_heads=1, head_dim_qk=576, head_dim_v=512, block_size=64, max_blocks_per_seq=1,
              num_pages=1, scale_kind="global", layout="mla", chunk_size=0, sm_scale=0.1, q_stride=128 * 576)
    for extra in (dict(kv_dtype="int4", causal=True), dict(kv_dtype="int8", causal=False, cross=True)):
        with pytest.raises(pa.PaError) as e:
            pa.pa_plan(pa.make_problem(**kw, **extra), [1], [5], [0, 1], 152)
        assert e.value.status == pa.PA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        pa.make_problem(**kw, kv_dtype="int8", causal=True, cross=True)


def fake_args(pa, **kw):
    a = dict(q=256, cache_k=256, cache_v=256, k_scale=256, v_scale=256, block_table=256, out=256, seq_lens=256,
             seq_lens_kv=256, cu_seqlens_q=256)
    return pa.make_args(**{**a, **kw})


def test_run_rejects_bad_arguments_before_launch(pa):
    p = make(1, seq_lens=[1], seq_lens_kv=[10], q_heads=8, kv_heads=2)
    pl = plan(pa, p)
    for kw in (dict(q=None), dict(cache_k=None), dict(k_scale=None), dict(cache_v=264), dict(q=8), dict(out=None),
               dict(block_table=None)):
        with pytest.raises(pa.PaError) as e:
            pa.pa_run(pl, fake_args(pa, **kw), 256, None)
        assert e.value.status == pa.PA_ERR_INVALID_ARG, kw
    # a tree mask needs the causal decode family
    x = make(1, seq_lens=[2], seq_lens_kv=[10], q_heads=8, kv_heads=2, causal=False, cross=True)
    with pytest.raises(pa.PaError) as e:
        pa.pa_run(plan(pa, x), fake_args(pa, attn_mask=256), 256, None)
    assert e.value.status == pa.PA_ERR_INVALID_ARG
    with pytest.raises(pa.PaError) as e:
        pa.pa_run(pl, fake_args(pa, k_scale=257), 256, None)
    assert e.value.status == pa.PA_ERR_INVALID_ARG
    z = make(1, seq_lens=[40], seq_lens_kv=[10], q_heads=8, kv_heads=2, scale_kind="per_channel")
    with pytest.raises(pa.PaError) as e:
        pa.pa_run(plan(pa, z), fake_args(pa, k_scale=264), 256, None)
    assert e.value.status == pa.PA_ERR_INVALID_ARG and "per-channel" in pa.pa_last_error()
    y = make(1, seq_lens=[40], seq_lens_kv=[10], q_heads=8, kv_heads=2)
    with pytest.raises(pa.PaError) as e:
        pa.pa_run(plan(pa, y), fake_args(pa, attn_mask=256), 256, None)
    assert e.value.status == pa.PA_ERR_UNSUPPORTED
    with pytest.raises(pa.PaError) as e:     # the append family stores 16-byte pieces
        pa.pa_run(plan(pa, y), fake_args(pa, out=258), 256, None)
    assert e.value.status == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", ["pa_cache_append", "pa_cache_read"])
def test_row_calls_reject_bad_arguments_before_launch(pa, call):
    f = getattr(pa, call)
    p = make(1, seq_lens=[1], seq_lens_kv=[10], q_heads=8, kv_heads=2)
    pl = plan(pa, p)
    bad = [dict(v_scale=255), dict(cache_k=None), dict(cache_v=None), dict(k_scale=None), dict(v_scale=None), dict(block_table=None),
           dict(seq_lens=None), dict(seq_lens_kv=None), dict(cu_seqlens_q=None), dict(cache_k=264)]
    for kw in bad:
        with pytest.raises(pa.PaError) as e:
            f(pl, fake_args(pa, **kw), 256, 256, 256, 256, None)
        assert e.value.status == pa.PA_ERR_INVALID_ARG, kw
    for rows in ((None, 256, 256, 256), (256, None, 256, 256), (257, 256, 256, 256), (256, 256, 255, 256),
                 (256, 256, 256, None)):
        with pytest.raises(pa.PaError) as e:
            f(pl, fake_args(pa), *rows, None)
        assert e.value.status == pa.PA_ERR_INVALID_ARG, rows
    x = make(1, seq_lens=[1], seq_lens_kv=[10], q_heads=8, kv_heads=2, causal=False, cross=True)
    with pytest.raises(pa.PaError) as e:
        f(plan(pa, x), fake_args(pa), 256, 256, 256, 256, None)
    assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_raw_gather_refuses_four_bit_caches(pa):
    p = make(1, seq_lens=[1], seq_lens_kv=[10], q_heads=8, kv_heads=2)
    with pytest.raises(pa.PaError) as e:
        pa.pa_debug_gather(problem(pa, p), fake_args(pa), 0, 0, 0, 1, 256, 256, None)
    assert e.value.status == pa.PA_ERR_UNSUPPORTED
