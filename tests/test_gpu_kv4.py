"""GPU parity of the 4-bit cache with the float64 oracle: attention of every
family, cross attention, quantise-and-write, and reading back."""
import importlib.util
import os
import subprocess
import sys
import types

import numpy as np
import pytest
import torch

import synth
from oracle import attention as oa
from oracle import kv4
from oracle.formats import decode_table
from synth.device import to_device
from kv4_helpers import (KINDS, SCALES, args_of, bf16_bits, check, device, make, plan_of, problem, reference, run,
                         workspace)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pa():
    import paged_quantized_kv_gqa_gb300 as m
    return m


# ---------------------------------------------------------------- attention
DECODE = [
    dict(seq_lens=[1], seq_lens_kv=[0], q_heads=1, kv_heads=1),                        # one position
    dict(seq_lens=[1, 1], seq_lens_kv=[100, 37], q_heads=4, kv_heads=1),
    dict(seq_lens=[1] * 6, seq_lens_kv=[30, 31, 32, 62, 63, 64], q_heads=8, kv_heads=2),
    dict(seq_lens=[1, 0, 1], seq_lens_kv=[1000, 9, 511], q_heads=10, kv_heads=2, chunk_size=128),
    dict(seq_lens=[2, 1, 2], seq_lens_kv=[300, 0, 64], q_heads=14, kv_heads=2, chunk_size=64),
    dict(seq_lens=[4, 1], seq_lens_kv=[700, 129], q_heads=8, kv_heads=2, chunk_size=-1),
    dict(seq_lens=[1] * 3, seq_lens_kv=[2100, 5, 800], q_heads=32, kv_heads=2),        # 16 rows, 33 pages
]
VERIFY = [
    dict(seq_lens=[6, 6, 2], seq_lens_kv=[500, 63, 0], q_heads=16, kv_heads=2, chunk_size=128),
    dict(seq_lens=[3, 1], seq_lens_kv=[130, 1000], q_heads=24, kv_heads=3),            # 24 rows
    dict(seq_lens=[8], seq_lens_kv=[191], q_heads=8, kv_heads=1, chunk_size=-1),       # 64 rows
    dict(seq_lens=[5, 5], seq_lens_kv=[640, 1], q_heads=18, kv_heads=2),               # 45 rows
]
APPEND = [
    dict(seq_lens=[70, 3, 0, 130], seq_lens_kv=[100, 0, 9, 63], q_heads=8, kv_heads=2),
    dict(seq_lens=[65], seq_lens_kv=[0], q_heads=1, kv_heads=1),                       # multi-head, one tile
    dict(seq_lens=[300, 41], seq_lens_kv=[1, 500], q_heads=10, kv_heads=2, chunk_size=128),
    dict(seq_lens=[33, 64], seq_lens_kv=[128, 200], q_heads=14, kv_heads=2, chunk_size=-1),
]


@pytest.mark.parametrize("scale_kind", SCALES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", DECODE + VERIFY + APPEND)
def test_attention(kw, kind, scale_kind):
    p = make(11, kv_dtype=kind, scale_kind=scale_kind, **kw)
    out, lse, *_ = run(p)
    check(p, out, lse)


@pytest.mark.parametrize("kw", [DECODE[3], VERIFY[0], APPEND[0]])
def test_attention_without_causal_mask(kw):
    p = make(12, causal=False, **kw)
    out, lse, *_ = run(p)
    check(p, out, lse)


LONG = [
    dict(seq_lens=[1], seq_lens_kv=[20000], q_heads=2, kv_heads=1),                  # 157 pieces, 32 warps merge a row
    dict(seq_lens=[1, 1], seq_lens_kv=[9000, 513], q_heads=10, kv_heads=2),          # 16 warps
    dict(seq_lens=[2, 1], seq_lens_kv=[3700, 511], q_heads=8, kv_heads=1),           # 16 rows, pieces of one sequence
    dict(seq_lens=[6, 2], seq_lens_kv=[6000, 30], q_heads=16, kv_heads=2),           # 48 rows
    dict(seq_lens=[3], seq_lens_kv=[5000], q_heads=21, kv_heads=3),                  # 21 rows, odd head count
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", LONG)
def test_long_contexts_in_pieces(kw, kind):
    p = make(24, kv_dtype=kind, scale_kind="per_channel", **kw)
    out, lse, _, plan = run(p)
    check(p, out, lse)
    assert plan.describe()["max_chunks"] > 1


def test_per_channel_scales_at_an_odd_address():
    """At most 16 rows: the scales may start at any bf16 address."""
    p = make(28, scale_kind="per_channel", **DECODE[3])
    d = device(p)
    for n in ("k_scale", "v_scale"):
        whole = torch.zeros(d[n].numel() + 1, dtype=torch.bfloat16, device="cuda")
        whole[1:] = d[n]
        d[n] = whole[1:]
    out, lse, *_ = run(p, d)
    check(p, out, lse)


@pytest.mark.parametrize("kw", [DECODE[3], VERIFY[1], APPEND[0]])
def test_negative_tensor_scales(kw):
    """The sign of a tensor scale is part of the value."""
    p = make(25, **kw)
    p.k_scale, p.v_scale = p.k_scale ^ 0x8000, p.v_scale ^ 0x8000
    out, lse, *_ = run(p)
    check(p, out, lse)


@pytest.mark.parametrize("scale_kind", SCALES)
@pytest.mark.parametrize("kw", [DECODE[3], DECODE[6], VERIFY[1], APPEND[0]])
def test_zero_tensor_scales(kw, scale_kind):
    """A K scale of 0 makes every visible position equal; a V scale of 0 the output 0."""
    p = make(26, scale_kind=scale_kind, **kw)
    n = max(1, len(p.k_scale) // 2)
    p.k_scale[:n] = 0
    p.v_scale[n:] = 0
    out, lse, *_ = run(p)
    check(p, out, lse)


@pytest.mark.parametrize("kw", [DECODE[2], VERIFY[0], APPEND[0]])
def test_workspace_of_one_plan_in_two_graphs(pa, kw):
    """Two captured graphs share a plan's workspace: replayed one after the other,
    each gives its own queries' result."""
    p = make(26, **kw)
    ds = [device(p), device(p)]
    other = bf16_bits(np.random.default_rng(3).standard_normal(p.q_bits.shape))
    ds[1]["q"].copy_(torch.from_numpy(other.view(np.int16)).view(torch.bfloat16))
    plan = plan_of(pa, p)
    ws = workspace(plan)
    pa.pa_plan_upload(plan, ws)
    graphs = []
    for d in ds:
        args = args_of(pa, d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_run(plan, args, ws)
            pa.pa_merge(plan, args, ws)
        graphs.append(g)
    for k in (0, 1, 1, 0):
        graphs[k].replay()
    assert pa.pa_check(plan, ws)[0] == 0
    for d, q in zip(ds, (p.q_bits, other)):
        p.q_bits = q
        check(p, d["out"].float().cpu().numpy().astype(np.float64), d["lse"].cpu().numpy().astype(np.float64))


@pytest.mark.parametrize("kw", [DECODE[2], VERIFY[0], APPEND[0]])
def test_bounded_wait_times_out_and_context_survives(pa, kw):
    """The test hook skips the first copy: the waits run out, the run reports it, and
    the next run is right."""
    p = make(27, **kw)
    d = device(p)
    plan = plan_of(pa, p)
    ws, args = workspace(plan), args_of(pa, d)
    pa.pa_plan_upload(plan, ws)
    pa.pa_debug_set_faults(wait_limit_ns=5_000_000, skip_first_load=True)
    try:
        pa.pa_run(plan, args, ws)
        st, _ = pa.pa_check(plan, ws)
    finally:
        pa.pa_debug_set_faults(0, False)
    assert st == pa.PA_ERR_DEVICE_TIMEOUT
    out, lse, *_ = run(p, d)
    check(p, out, lse)


@pytest.mark.parametrize("sms", [1, 5])
@pytest.mark.parametrize("kw", [DECODE[3], DECODE[6], VERIFY[0], APPEND[0]])
def test_few_ctas_take_many_items(kw, sms):
    p = make(13, kv_dtype="int4", **{**kw, "chunk_size": 64})
    out, lse, *_ = run(p, sms=sms)
    check(p, out, lse)


@pytest.mark.parametrize("kv_heads, kv", [(4, [9001, 4032]), (8, [90, 9170])])
def test_pieces_begin_with_a_second_half_page(kv_heads, kv):
    """One CTA, so that the pieces run over more pages than a warp looks up at once."""
    p = make(31, seq_lens=[1, 1], seq_lens_kv=kv, q_heads=16, kv_heads=kv_heads)
    out, lse, _, plan = run(p, sms=1)
    it = np.asarray(plan.describe()["items"])
    odd = it[it[:, 5] % 64 == 32]
    assert len(odd) and (odd[:, 6] - odd[:, 5]).max() > 32 * 64
    check(p, out, lse)


def test_more_items_than_a_cta_keeps_records_of():
    """One CTA, 700 items of one or two pages, and one of 40 pages."""
    p = make(14, seq_lens=[1] * 351, seq_lens_kv=[2500] + [70] * 350, q_heads=4, kv_heads=2)
    out, lse, *_ = run(p, sms=1)
    check(p, out, lse)


@pytest.mark.parametrize("kw", [DECODE[1], VERIFY[1], APPEND[3]])
def test_packed_query_rows(kw):
    p = make(15, q_stride=(kw["q_heads"] + 2 * kw["kv_heads"]) * 128, **kw)
    out, lse, *_ = run(p)
    check(p, out, lse)


@pytest.mark.parametrize("kw", [DECODE[1], VERIFY[0]])
def test_output_at_an_odd_address(kw):
    p = make(16, **kw)
    d = device(p)
    whole = torch.zeros(d["out"].numel() + 1, dtype=torch.bfloat16, device="cuda")
    d["out"] = whole[1:].view(d["out"].shape)
    out, lse, *_ = run(p, d)
    check(p, out, lse)


@pytest.mark.parametrize("kw", [DECODE[4], VERIFY[0]])
def test_single_launch_option_leaves_4_bit_plans_alone(pa, kw):
    pa.pa_set_fused_merge(True)
    try:
        p = make(17, **kw)
        out, lse, *_ = run(p)
    finally:
        pa.pa_set_fused_merge(False)
    check(p, out, lse)


@pytest.mark.parametrize("kw", [dict(seq_lens=[3, 4], seq_lens_kv=[61, 1150], q_heads=4, kv_heads=2),
                                dict(seq_lens=[6, 1], seq_lens_kv=[127, 0], q_heads=16, kv_heads=2),
                                dict(seq_lens=[6, 5], seq_lens_kv=[1021, 63], q_heads=16, kv_heads=2)])
def test_tree_mask_with_rows_that_see_nothing_of_their_chunk(kw):
    p = make(18, **kw)
    M = int(p.seq_lens.max())
    r = np.random.default_rng(5)
    p.attn_mask = np.tril(r.integers(0, 2, (p.bsz, M, M)), -1).astype(np.uint8) + np.eye(M, dtype=np.uint8)[None]
    out, lse, *_ = run(p)
    check(p, out, lse)


def test_tree_mask_that_leaves_a_row_empty():
    """No cached prefix and a mask row of zeros: out 0, lse -inf, others unharmed."""
    p = make(19, seq_lens=[3], seq_lens_kv=[0], q_heads=4, kv_heads=2)
    p.attn_mask = np.array([[[1, 0, 0], [0, 0, 0], [1, 0, 1]]], np.uint8)
    out, lse, *_ = run(p)
    check(p, out, lse)
    assert np.isneginf(lse[1]).all() and (out[1] == 0).all()


@pytest.mark.parametrize("kw", [DECODE[3], VERIFY[0], APPEND[2]])
def test_output_epilogue(kw):
    """shift, smooth and int8 output: the rounded value may be one step off where
    the attention tolerance reaches over a rounding border."""
    p = make(20, **kw)
    d = device(p)
    r = np.random.default_rng(6)
    n = p.q_heads * 128
    sh, sm = bf16_bits(r.uniform(-.2, .2, n)), bf16_bits(r.uniform(.5, 1.5, n))
    bf = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    d["out_all"] = torch.full((p.total_q + 1, p.q_heads, 128), 7, dtype=torch.int8, device="cuda")
    d["out"] = d["out_all"][:-1]
    out, lse, *_ = run(p, d, shift_bias=bf(sh), smooth_weight=bf(sm), out_int8=True, in_scale=0.2,
                       quant_max_bound=127.0, quant_min_bound=-127.0)
    ro, rl, to, tl = reference(p)
    sh, sm = (kv4.bf16_to_f64(a).reshape(p.q_heads, 128) for a in (sh, sm))
    v, dv = (ro + sh) * sm * 127 * 0.2, to * sm * 127 * 0.2 + 1e-4
    lo, hi = (np.clip(np.rint(v + s * dv), -127, 127) for s in (-1, 1))
    assert ((out >= lo) & (out <= hi)).all()


def test_bad_page_is_reported_not_dereferenced(pa):
    for kw in (DECODE[3], VERIFY[0], APPEND[0]):
        p = make(21, **kw)
        d = device(p)
        d["block_table"][0, 0] = p.num_pages
        plan = plan_of(pa, p)
        ws, args = workspace(plan), args_of(pa, d)
        pa.pa_plan_upload(plan, ws)
        pa.pa_run(plan, args, ws)
        st, _ = pa.pa_check(plan, ws)
        assert st == pa.PA_ERR_BAD_PAGE, kw


def test_results_do_not_change_from_run_to_run():
    for kw in (DECODE[5], VERIFY[2], APPEND[3]):
        p = make(22, **kw)
        a = run(p)
        b = run(p)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_chunks_merge_to_the_unsplit_result():
    p = make(23, seq_lens=[1, 2], seq_lens_kv=[900, 130], q_heads=8, kv_heads=2)
    ref = reference(p)
    for cs in (0, 64, 192, -1):
        p.chunk_size = cs
        out, lse, *_ = run(p)
        check(p, out, lse, ref)


# ---------------------------------------------------------------- cross attention
CROSS = [
    dict(seq_lens=[1] * 5, seq_lens_kv=[1500, 0, 1, 64, 333], q_heads=4, kv_heads=4, chunk_size=-1),
    dict(seq_lens=[1, 1], seq_lens_kv=[0, 0], q_heads=8, kv_heads=2),
    dict(seq_lens=[5, 3, 0, 5], seq_lens_kv=[70, 0, 9, 640], q_heads=16, kv_heads=2, chunk_size=128),
    dict(seq_lens=[100, 7, 80], seq_lens_kv=[65, 0, 900], q_heads=6, kv_heads=2),
    dict(seq_lens=[448, 1], seq_lens_kv=[20, 1500], q_heads=2, kv_heads=2, chunk_size=512),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", CROSS)
def test_cross_attention(kw, kind):
    p = make(31, kv_dtype=kind, causal=False, cross=True, **kw)
    out, lse, *_ = run(p)
    check(p, out, lse)


@pytest.mark.parametrize("kind", ["int8", "fp8_e4m3"])
@pytest.mark.parametrize("kw", CROSS)
def test_cross_attention_over_8_bit_caches(kw, kind):
    """The same lengths over the 8-bit caches: rows decoded by their oracle."""
    c = synth.make_case(name="x", seed=32, kv_dtype=kind, causal=False, **{**kw, "seq_lens": kw["seq_lens"]})
    c.cross = True
    p = types.SimpleNamespace(**{n: getattr(c, n) for n in (
        "q_heads", "kv_heads", "kv_dtype", "scale_kind", "layout", "causal", "cross", "chunk_size", "sm_scale",
        "q_stride", "seq_lens", "seq_lens_kv", "bsz", "cu_seqlens_q", "total_q", "num_pages", "max_blocks_per_seq",
        "block_table", "cache_k", "cache_v", "k_scale", "v_scale", "q_bits")})
    p.held = c.seq_lens_kv
    ref = reference(p, rows=lambda w, b, h, n: oa.dequant_kv(c, b, h, n)[w == "v"])
    out, lse, *_ = run(p)
    check(p, out, lse, ref)


def test_cross_epilogue_of_empty_rows(pa):
    """An empty row is 0 before the output epilogue: (0 + shift) * smooth."""
    p = make(33, seq_lens=[2, 1], seq_lens_kv=[0, 40], q_heads=4, kv_heads=2, causal=False, cross=True)
    shift = torch.linspace(-1, 1, 512, device="cuda").bfloat16()
    out, lse, d, _ = run(p, shift_bias=shift)
    assert np.array_equal(out[:2].reshape(2, 512), shift.float().cpu().numpy()[None].repeat(2, 0))


# ---------------------------------------------------------------- write, read back
ROWS = [
    dict(seq_lens=[70, 3, 0, 130], seq_lens_kv=[100, 0, 9, 63], kv_heads=2),
    dict(seq_lens=[1] * 9, seq_lens_kv=[0, 1, 15, 16, 31, 32, 63, 64, 100], kv_heads=3),
    dict(seq_lens=[2, 1, 33], seq_lens_kv=[63, 127, 31], kv_heads=1),
    dict(seq_lens=[200, 64], seq_lens_kv=[0, 64], kv_heads=4),
]
STRIDES = ["plain", "packed", "odd"]


def placed(rows, how):
    """Device rows with a stride of their own: (tensor whose first element is row 0, stride, whole buffer)."""
    T, h = rows.shape[:2]
    x = rows.reshape(T, h * 128)
    if how == "plain":
        return x.contiguous(), h * 128, None
    pad = 2 * h * 128 if how == "packed" else 1
    first = 256 if how == "packed" else 1
    whole = torch.full((T * (h * 128 + pad) + first,), 9.0, dtype=rows.dtype, device="cuda")
    view = whole[first:].view(T, h * 128 + pad)
    view[:, :h * 128] = x
    return view, h * 128 + pad, whole


@pytest.mark.parametrize("how", STRIDES)
@pytest.mark.parametrize("scale_kind", SCALES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", ROWS)
def test_written_bytes_are_the_oracles(pa, kw, kind, scale_kind, how):
    check_written(pa, kw, kind, scale_kind, how)


def check_written(pa, kw, kind, scale_kind, how, sms=None):
    p = make(41, q_heads=kw["kv_heads"], kv_dtype=kind, scale_kind=scale_kind, **kw)
    p.k_new[0, 0, :4] = bf16_bits([np.nan, np.inf, -np.inf, 1.0])
    p.v_new[-1, -1, 16:20] = bf16_bits([np.nan, 3e38, 1e-38, -0.0])
    p.v_new[-1, -1, 32:48] = 0
    d = device(p)
    k, stride, _ = placed(d["k_new"], how)
    v, _, _ = placed(d["v_new"], how)
    plan = plan_of(pa, p, sms)
    ws = workspace(plan)
    pa.pa_plan_upload(plan, ws)
    pa.pa_cache_append(plan, args_of(pa, d), k, v, stride, ws)
    assert pa.pa_check(plan, ws)[0] == 0
    rk, rv = kv4.append(p, p.k_new, p.v_new, p.cache_k, p.cache_v)
    for got, want, w in ((d["cache_k"], rk, "K"), (d["cache_v"], rv, "V")):
        bad = np.argwhere(got.cpu().numpy() != want)
        assert not len(bad), f"{w} bytes differ at {bad[:4].tolist()}"


@pytest.mark.parametrize("how", STRIDES)
@pytest.mark.parametrize("scale_kind", SCALES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", ROWS)
def test_rows_read_back(pa, kw, kind, scale_kind, how):
    check_read(pa, kw, kind, scale_kind, how)


def check_read(pa, kw, kind, scale_kind, how, sms=None):
    p = make(42, q_heads=kw["kv_heads"], kv_dtype=kind, scale_kind=scale_kind, **kw)
    d = device(p)
    k, stride, kw_ = placed(torch.full_like(d["k_new"], 9.0), how)
    v, _, vw_ = placed(torch.full_like(d["v_new"], 9.0), how)
    plan = plan_of(pa, p, sms)
    ws = workspace(plan)
    pa.pa_plan_upload(plan, ws)
    pa.pa_cache_read(plan, args_of(pa, d), k, v, stride, ws)
    assert pa.pa_check(plan, ws)[0] == 0
    n = p.kv_heads * 128
    for got, whole, w in ((k, kw_, "k"), (v, vw_, "v")):
        want = np.concatenate([np.stack([kv4.read_back(p, w, b, h, int(p.seq_lens_kv[b]), int(p.seq_lens[b]))
                                         for h in range(p.kv_heads)], 1) for b in range(p.bsz)])
        bits = got[:, :n].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
        assert np.array_equal(bits, want.reshape(bits.shape)), w
        if whole is not None:       # what lies between the rows is left as it was
            assert bool((got[:, n:] == 9).all()) and bool((whole[:whole.numel() - got.numel()] == 9).all())


# A plan for one SM takes units of 32 positions at these sizes; the first two sets number
# their units by search (a long range beside single rows, empty ranges, more than 32).
LONG_ROWS = [
    dict(seq_lens=[1, 700, 0] + [1] * 40, seq_lens_kv=[5, 33, 7] + [29 + 3 * i for i in range(40)], kv_heads=2),
    dict(seq_lens=[0] * 40 + [2, 600, 0, 31, 1], seq_lens_kv=[1] * 40 + [31, 0, 5, 32, 63], kv_heads=1),
    dict(seq_lens=[200, 64, 97], seq_lens_kv=[0, 64, 31], kv_heads=4),
]


@pytest.mark.parametrize("sms", [1, None])
@pytest.mark.parametrize("scale_kind", ["per_kv_head", "per_channel"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", LONG_ROWS)
def test_long_and_mixed_rows(pa, kw, kind, scale_kind, sms):
    check_written(pa, kw, kind, scale_kind, "plain", sms)
    check_read(pa, kw, kind, scale_kind, "packed", sms)


@pytest.mark.parametrize("kw", [
    dict(q_heads=8, kv_heads=2), dict(q_heads=8, kv_heads=2, scale_kind="per_channel"),
    dict(q_heads=8, kv_heads=2, kv_dtype="fp8_e4m3"),
    dict(q_heads=128, kv_heads=1, head_dim_qk=576, head_dim_v=512, layout="mla", kv_dtype="fp8_e4m3",
         scale_kind="global"),
    dict(q_heads=128, kv_heads=1, head_dim_qk=576, head_dim_v=512, layout="mla", scale_kind="global"),
])
def test_8_bit_rows_read_back(pa, kw):
    check_8_bit_read(pa, kw, [70, 1, 0, 20], [10, 63, 5, 0], 152)


@pytest.mark.parametrize("kw", [
    dict(q_heads=8, kv_heads=2, scale_kind="per_channel"), dict(q_heads=8, kv_heads=2, kv_dtype="fp8_e4m3"),
    dict(q_heads=128, kv_heads=1, head_dim_qk=576, head_dim_v=512, layout="mla", kv_dtype="fp8_e4m3",
         scale_kind="global"),
])
@pytest.mark.parametrize("sms", [1, 152])
def test_8_bit_long_and_mixed_rows_read_back(pa, kw, sms):
    check_8_bit_read(pa, kw, [1, 700, 0] + [1] * 40, [5, 33, 7] + [29 + 3 * i for i in range(40)], sms)
    check_8_bit_read(pa, kw, [300, 364], [0, 31], sms)


def check_8_bit_read(pa, kw, q, kv, sms):
    c = synth.make_case(name="r", seed=43, seq_lens=q, seq_lens_kv=kv, **kw)
    d = to_device(c)
    plan = pa.pa_plan(pa.problem_of(c), c.seq_lens, c.seq_lens_kv, c.cu_seqlens_q, sms)
    ws = workspace(plan)
    pa.pa_plan_upload(plan, ws)
    mla = c.layout == "mla"
    D = c.head_dim_qk
    k = torch.zeros((c.total_q, c.kv_heads, D), dtype=torch.bfloat16, device="cuda")
    v = None if mla else torch.zeros_like(k)
    args = pa.make_args(**{n: d[n] for n in ("q", "cache_k", "cache_v", "k_scale", "v_scale", "block_table", "out",
                                             "lse", "seq_lens", "seq_lens_kv", "cu_seqlens_q")})
    pa.pa_cache_read(plan, args, k, v, c.kv_heads * D, ws)
    assert pa.pa_check(plan, ws)[0] == 0
    table = decode_table(c.kv_dtype).astype(np.float32)
    for b in range(c.bsz):
        t0, n, first = int(c.cu_seqlens_q[b]), int(c.seq_lens[b]), int(c.seq_lens_kv[b])
        for h in range(c.kv_heads):
            K, V = oa.gather_raw(c, b, h, first + n)
            for got, raw, w in ((k, K, "k"), (v, V, "v")):
                if got is None:
                    continue
                g = np.asarray(oa._scales(c, w, h)).astype(np.float32)
                bits = got[t0:t0 + n, h].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
                assert np.array_equal(bits, kv4.to_bf16_bits(table[raw[first:]] * g)), (b, h, w)


@pytest.mark.parametrize("call", ["pa_cache_append", "pa_cache_read"])
def test_row_calls_report_a_bad_page(pa, call):
    p = make(44, q_heads=2, kv_heads=2, seq_lens=[70, 5], seq_lens_kv=[0, 3])
    d = device(p)
    before = d["cache_k"].clone()
    d["block_table"][0, 1] = -5
    plan = plan_of(pa, p)
    ws = workspace(plan)
    pa.pa_plan_upload(plan, ws)
    getattr(pa, call)(plan, args_of(pa, d), d["k_new"], d["v_new"], 256, ws)
    assert pa.pa_check(plan, ws)[0] == pa.PA_ERR_BAD_PAGE
    if call == "pa_cache_read":     # the page's positions read as zeros
        assert bool((d["k_new"][64:70] == 0).all()) and bool((d["v_new"][64:70] == 0).all())
        assert torch.equal(d["cache_k"], before)


def far_pool(p, d):
    """The case's pages at the end of a pool whose offsets pass 32 bits."""
    slabs = (1 << 32) // 4608 + 1000
    first = slabs // p.kv_heads - p.num_pages
    for n in ("cache_k", "cache_v"):
        pool = torch.empty((first + p.num_pages, p.kv_heads, 4608), dtype=torch.uint8, device="cuda")
        pool[first:] = d[n].view(p.num_pages, p.kv_heads, 4608)
        d[n] = pool
    bt = d["block_table"]
    d["block_table"] = torch.where(bt >= 0, bt + first, bt)
    return first


@pytest.mark.parametrize("kw", [DECODE[3], DECODE[6], VERIFY[0], APPEND[0]])
def test_attention_over_a_pool_past_32_bits(kw):
    p = make(32, **kw)
    d = device(p)
    p.num_pages += far_pool(p, d)
    out, lse, *_ = run(p, d)
    check(p, out, lse)


def test_rows_of_a_pool_past_32_bits(pa):
    p = make(33, seq_lens=[70, 3], seq_lens_kv=[40, 100], q_heads=8, kv_heads=2, kv_dtype="int4")
    d = device(p)
    n, first = p.num_pages, far_pool(p, d)
    p.num_pages += first
    plan = plan_of(pa, p)
    ws = workspace(plan)
    pa.pa_plan_upload(plan, ws)
    pa.pa_cache_append(plan, args_of(pa, d), d["k_new"], d["v_new"], 256, ws)
    rk, rv = kv4.append(p, p.k_new, p.v_new, p.cache_k, p.cache_v)
    assert np.array_equal(d["cache_k"][first:].cpu().numpy().reshape(rk.shape), rk)
    assert np.array_equal(d["cache_v"][first:].cpu().numpy().reshape(rv.shape), rv)
    k, v = torch.zeros_like(d["k_new"]), torch.zeros_like(d["v_new"])
    pa.pa_cache_read(plan, args_of(pa, d), k, v, 256, ws)
    assert pa.pa_check(plan, ws)[0] == 0
    p.cache_k, p.cache_v, p.num_pages = rk, rv, n
    for got, w in ((k, "k"), (v, "v")):
        want = np.concatenate([np.stack([kv4.read_back(p, w, b, h, int(p.seq_lens_kv[b]), int(p.seq_lens[b]))
                                         for h in range(p.kv_heads)], 1) for b in range(p.bsz)])
        bits = got.reshape(p.total_q, 256).view(torch.int16).cpu().numpy().view(np.uint16)
        assert np.array_equal(bits, want.reshape(bits.shape)), w


# ---------------------------------------------------------------- together
def serve(pa, p, d, plan, ws, args, read):
    pa.pa_cache_append(plan, args, d["k_new"], d["v_new"], p.kv_heads * 128, ws)
    pa.pa_run(plan, args, ws)
    pa.pa_merge(plan, args, ws)
    pa.pa_cache_read(plan, args, read[0], read[1], p.kv_heads * 128, ws)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kw", [dict(seq_lens=[1, 1], seq_lens_kv=[200, 63], q_heads=8, kv_heads=2, chunk_size=64),
                                dict(seq_lens=[90, 20], seq_lens_kv=[30, 0], q_heads=8, kv_heads=2)])
def test_write_attend_and_read_on_a_side_stream(pa, kw, captured):
    """One serving step as a program makes it: new rows written, attention over the
    updated cache, the rows read back; on another stream, and as a graph that is
    replayed with other queries."""
    p = make(51, kv_dtype="int4", **kw)
    d = device(p)
    plan = plan_of(pa, p)
    ws, args = workspace(plan), args_of(pa, d)
    read = torch.zeros_like(d["k_new"]), torch.zeros_like(d["v_new"])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        pa.pa_plan_upload(plan, ws)
        if captured:
            g = torch.cuda.CUDAGraph()
            s.synchronize()
            with torch.cuda.graph(g, stream=s):
                serve(pa, p, d, plan, ws, args, read)
            p.q_bits = bf16_bits(np.random.default_rng(9).standard_normal(p.q_bits.shape))
            d["q"].copy_(torch.from_numpy(p.q_bits.view(np.int16)).view(torch.bfloat16))
            for _ in range(2):
                g.replay()
        else:
            serve(pa, p, d, plan, ws, args, read)
        assert pa.pa_check(plan, ws)[0] == 0
    p.cache_k, p.cache_v = kv4.append(p, p.k_new, p.v_new, p.cache_k, p.cache_v)
    out, lse = d["out"].float().cpu().numpy().astype(np.float64), d["lse"].cpu().numpy().astype(np.float64)
    check(p, out, lse)
    for got, w in zip(read, "kv"):
        want = np.concatenate([np.stack([kv4.read_back(p, w, b, h, int(p.seq_lens_kv[b]), int(p.seq_lens[b]))
                                         for h in range(p.kv_heads)], 1) for b in range(p.bsz)])
        assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), want)


def test_encoder_states_written_once_and_attended_to(pa):
    """Encoder rows written with a plan of their own lengths, then two decoder steps
    of cross attention with another plan over the same pool."""
    enc = make(52, seq_lens=[90, 0, 130], seq_lens_kv=[0, 0, 0], q_heads=4, kv_heads=4)
    d = device(enc)
    plan = plan_of(pa, enc)
    ws = workspace(plan)
    pa.pa_plan_upload(plan, ws)
    pa.pa_cache_append(plan, args_of(pa, d), d["k_new"], d["v_new"], 512, ws)
    assert pa.pa_check(plan, ws)[0] == 0
    enc.cache_k, enc.cache_v = kv4.append(enc, enc.k_new, enc.v_new, enc.cache_k, enc.cache_v)
    for q_len in (1, 20):
        dec = make(53, seq_lens=[q_len] * 3, seq_lens_kv=enc.seq_lens, q_heads=4, kv_heads=4, causal=False, cross=True)
        for n in ("block_table", "num_pages", "max_blocks_per_seq", "cache_k", "cache_v", "k_scale", "v_scale"):
            setattr(dec, n, getattr(enc, n))
        dd = device(dec)
        dd["cache_k"], dd["cache_v"] = d["cache_k"], d["cache_v"]
        out, lse, *_ = run(dec, dd)
        check(dec, out, lse)


def test_built_in_workspace(pa):
    p = make(54, seq_lens=[1, 1], seq_lens_kv=[200, 63], q_heads=8, kv_heads=2, chunk_size=64)
    d = device(p)
    pa.pa_run_static(plan_of(pa, p), args_of(pa, d), check=True)
    check(p, d["out"].float().cpu().numpy().astype(np.float64), d["lse"].cpu().numpy().astype(np.float64))


def test_debug_library_cases():
    spec = importlib.util.spec_from_file_location(
        "pa_build_for_kv4_debug_test", os.path.join(ROOT, "paged_quantized_kv_gqa_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.build(debug=True)
    env = dict(os.environ, PA_GB300_DEBUG="1")
    env.pop("PA_GB300_TRACE", None)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_kv4_cases.py")], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "all 4-bit cases passed" in r.stdout
