"""GPU parity of long sequences beside many short ones over the 4-bit cache."""
import numpy as np
import pytest

from kv4_helpers import KINDS, args_of, bf16_bits, check, device, make, plan_of, reference, run, workspace

pytestmark = pytest.mark.gpu

MIXED = [
    dict(seq_lens=[1] * 40, seq_lens_kv=[90 + 13 * i for i in range(39)] + [20000], q_heads=8, kv_heads=2),
    dict(seq_lens=[1] * 12, seq_lens_kv=[20000, 0, 511, 512, 700] + [1200] * 7, q_heads=10, kv_heads=2),
    dict(seq_lens=[3, 1, 2, 0, 3], seq_lens_kv=[12000, 40, 513, 9, 600], q_heads=12, kv_heads=3),       # 12 rows
    dict(seq_lens=[6, 5, 1, 6], seq_lens_kv=[200, 12000, 1500, 0], q_heads=16, kv_heads=2),             # 48 rows
    dict(seq_lens=[70, 1, 3], seq_lens_kv=[500, 3000, 5], q_heads=8, kv_heads=2, chunk_size=256),       # append
    dict(seq_lens=[1, 2, 1], seq_lens_kv=[0, 9000, 800], q_heads=4, kv_heads=4, causal=False, cross=True),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", MIXED)
def test_long_beside_short(kw, kind):
    p = make(71, kv_dtype=kind, **kw)
    out, lse, _, plan = run(p)
    check(p, out, lse)
    n = plan.describe()["nch_token"]
    assert n.max() > 8 and n.min() <= 2


def test_long_beside_short_in_the_built_in_workspace():
    """131k positions beside 63 of 500: 5.8 MB of partial rows are written."""
    import paged_quantized_kv_gqa_gb300 as pa
    p = make(72, seq_lens=[1] * 64, seq_lens_kv=[131071] + [500] * 63, q_heads=8, kv_heads=1, kv_dtype="int4")
    d = device(p)
    pa.pa_run_static(plan_of(pa, p), args_of(pa, d), check=True)
    check(p, d["out"].float().cpu().numpy().astype(np.float64), d["lse"].cpu().numpy().astype(np.float64))


@pytest.mark.parametrize("G", [3, 8, 20])
def test_rows_of_every_chunk_count_are_merged_together(G):
    """From no chunk at all to more than 128, so that rows taking 1 to 32 warps of the
    merge stand beside each other.  3 heads: all rows fit the GPU with the longest one's
    warps; 8 and 20 heads: each gets its own.  20 rows are the tensor-memory kernel's."""
    kv = [700, 30000, 0, 1500, 7000, 100, 14000, 3000]
    p = make(73, seq_lens=[1] * 44, seq_lens_kv=kv + [600 + 5 * i for i in range(36)], q_heads=G, kv_heads=1,
             causal=False, cross=True)
    out, lse, _, plan = run(p)
    check(p, out, lse)
    n = plan.describe()["nch_token"]
    warps = 1 << sum(int(n.max()) > x for x in (8, 16, 32, 64, 128))
    assert n[2] == 0 and n[5] == 1 and n[0] > 1
    assert (int((n != 1).sum()) * G * warps > 32 * 152) == (G > 3)
    if G < 20:
        assert {sum(int(x) > y for y in (8, 16, 32, 64, 128)) for x in n} == set(range(6))


def without_merge(pa, p):
    """Plan, upload, pa_run alone; then pa_merge, which must leave the rows alone."""
    d = device(p)
    plan = plan_of(pa, p)
    ws, args = workspace(plan), args_of(pa, d)
    pa.pa_plan_upload(plan, ws)
    pa.pa_run(plan, args, ws)
    assert pa.pa_check(plan, ws)[0] == 0
    assert len(plan.describe()["merge_tokens"])
    got = d["out"].float().cpu().numpy().astype(np.float64), d["lse"].cpu().numpy().astype(np.float64)
    d["out"].fill_(7)
    pa.pa_merge(plan, args, ws)
    assert pa.pa_check(plan, ws)[0] == 0 and bool((d["out"] == 7).all())
    assert bool((d["out_all"][-1] == 7).all()) and bool((d["lse_all"][-1] == 7).all())
    return got


@pytest.mark.parametrize("kw", [
    dict(seq_lens=[1, 1, 2], seq_lens_kv=[5000, 30, 700], q_heads=8, kv_heads=2),
    dict(seq_lens=[6, 1], seq_lens_kv=[4000, 9], q_heads=16, kv_heads=2),
    dict(seq_lens=[1, 2, 1], seq_lens_kv=[0, 3000, 5], q_heads=4, kv_heads=2, causal=False, cross=True),
    dict(seq_lens=[2, 1], seq_lens_kv=[0, 0], q_heads=4, kv_heads=2, causal=False, cross=True),
    dict(seq_lens=[70, 3, 9], seq_lens_kv=[0, 100, 0], q_heads=4, kv_heads=2, causal=False, cross=True),
])
def test_rows_of_plans_without_chunks_are_final_after_pa_run(kw):
    """A program that never splits (chunk_size 0) and does not call pa_merge."""
    import paged_quantized_kv_gqa_gb300 as pa
    p = make(74, kv_dtype="int4", chunk_size=0, **kw)
    check(p, *without_merge(pa, p))


def test_8_bit_cross_rows_without_chunks_are_final_after_pa_run():
    import types
    import synth
    from oracle import attention as oa
    import paged_quantized_kv_gqa_gb300 as pa
    c = synth.make_case(name="z", seed=75, kv_dtype="int8", causal=False, seq_lens=[1, 2, 1], seq_lens_kv=[0, 200, 64],
                        q_heads=8, kv_heads=2, chunk_size=0)
    p = types.SimpleNamespace(**{n: getattr(c, n) for n in (
        "q_heads", "kv_heads", "kv_dtype", "scale_kind", "layout", "causal", "chunk_size", "sm_scale", "q_stride",
        "seq_lens", "seq_lens_kv", "bsz", "cu_seqlens_q", "total_q", "num_pages", "max_blocks_per_seq", "block_table",
        "cache_k", "cache_v", "k_scale", "v_scale", "q_bits")})
    c.cross = p.cross = True
    p.held = c.seq_lens_kv
    ref = reference(p, rows=lambda w, b, h, n: oa.dequant_kv(c, b, h, n)[w == "v"])
    check(p, *without_merge(pa, p), ref)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", [dict(seq_lens=[4, 2], seq_lens_kv=[61, 1150], q_heads=4, kv_heads=2),      # 8 rows
                                dict(seq_lens=[4, 2], seq_lens_kv=[61, 1150], q_heads=8, kv_heads=2),      # 16
                                dict(seq_lens=[3, 2], seq_lens_kv=[127, 1500], q_heads=14, kv_heads=2),    # 21
                                dict(seq_lens=[6, 5], seq_lens_kv=[1021, 63], q_heads=16, kv_heads=2),     # 48
                                dict(seq_lens=[8, 5], seq_lens_kv=[900, 0], q_heads=16, kv_heads=2)])      # 64
def test_tree_masks_over_per_channel_scales(kw, kind):
    p = make(76, kv_dtype=kind, scale_kind="per_channel", **kw)
    M = int(p.seq_lens.max())
    r = np.random.default_rng(6)
    p.attn_mask = np.tril(r.integers(0, 2, (p.bsz, M, M)), -1).astype(np.uint8) + np.eye(M, dtype=np.uint8)[None]
    out, lse, *_ = run(p)
    check(p, out, lse)


def test_a_plan_without_chunks_captured_alone_and_in_the_built_in_workspace():
    """pa_run alone (attention and the merge it enqueues) as a graph that is replayed with
    other queries, on a side stream; then the same plan through pa_run_static."""
    import torch
    import paged_quantized_kv_gqa_gb300 as pa
    p = make(77, seq_lens=[1, 2, 1], seq_lens_kv=[6000, 700, 3], q_heads=8, kv_heads=2, kv_dtype="int4", chunk_size=0)
    d = device(p)
    plan = plan_of(pa, p)
    ws, args = workspace(plan), args_of(pa, d)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        pa.pa_plan_upload(plan, ws)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pa.pa_run(plan, args, ws)
        p.q_bits = bf16_bits(np.random.default_rng(8).standard_normal(p.q_bits.shape))
        d["q"].copy_(torch.from_numpy(p.q_bits.view(np.int16)).view(torch.bfloat16))
        for _ in range(2):
            g.replay()
        assert pa.pa_check(plan, ws)[0] == 0
    host = lambda: [d[n].float().cpu().numpy().astype(np.float64) for n in ("out", "lse")]  # noqa: E731
    check(p, *host())
    d["out"].fill_(7)
    pa.pa_run_static(plan, args, check=True)
    check(p, *host())
