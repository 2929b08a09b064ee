"""The rotated append on the GPU against the oracle: every cache byte equal (the
rotation's roundings are fixed), queries equal to the oracle's rounded to bf16."""
import numpy as np
import pytest
import torch

import rope_helpers as rh
from gpu_helpers import num_sms
from oracle import kv4

pytestmark = pytest.mark.gpu


def dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def launch(p, *, q=True, in_place=False, packed=False, pad=0, rows=None, stream=None, sms=None, cache_at=0):
    """Runs the call (the values' cache cache_at bytes into its buffer); returns (q_out bits,
    cache_k, cache_v, status, detail)."""
    import paged_quantized_kv_gqa_gb300 as pa
    T, mla = rows or p.total_q, p.layout == "mla"
    d = {n: torch.from_numpy(getattr(p, n).copy()).cuda() for n in ("block_table", "seq_lens", "seq_lens_kv", "cu_seqlens_q",
                                                                     "cache_k")}
    if mla:
        d["cache_v"] = d["cache_k"]
    else:
        d["cache_v"] = torch.zeros(p.cache_v.size + cache_at, dtype=torch.uint8, device="cuda")[cache_at:].view(p.cache_v.shape)
        d["cache_v"].copy_(torch.from_numpy(p.cache_v))
    for w in "kv":
        s = getattr(p, w + "_scale")
        d[w + "_scale"] = torch.from_numpy(s).cuda() if p.scale_kind == "global" else dev(s)
    qw, kw = p.q_new[0].size, p.k_new[0].size
    if packed:
        row = np.concatenate([x.reshape(T, -1) for x in (p.q_new, p.k_new, p.v_new)] + [np.full((T, pad), 0x7FC0, np.uint16)], 1)
        row = dev(row)
        qs, ks, vs = row[:, :qw], row[:, qw:qw + kw], row[:, qw + kw:]
    else:
        wide = lambda x: dev(np.concatenate([x.reshape(T, -1), np.full((T, pad), 0x7FC0, np.uint16)], 1))  # noqa: E731
        qs, ks, vs = wide(p.q_new), wide(p.k_new), None if mla else wide(p.v_new)
    out = qs if in_place else torch.full((T, qw + 2 * pad), 7.0, dtype=torch.bfloat16, device="cuda")
    prob = pa.make_problem(**{k: getattr(p, k) for k in (
        "bsz", "q_heads", "kv_heads", "head_dim_qk", "head_dim_v", "block_size", "max_blocks_per_seq", "num_pages", "kv_dtype",
        "scale_kind", "layout", "chunk_size", "sm_scale", "q_stride", "causal")})
    plan = pa.pa_plan(prob, p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, sms or num_sms())
    ws = torch.zeros(max(plan.workspace_size, 256), dtype=torch.uint8, device="cuda")
    pa.pa_plan_upload(plan, ws)
    args = pa.make_args(q=None, cache_k=d["cache_k"], cache_v=d["cache_v"], k_scale=d["k_scale"], v_scale=d["v_scale"],
                        block_table=d["block_table"], out=None, seq_lens=d["seq_lens"], seq_lens_kv=d["seq_lens_kv"],
                        cu_seqlens_q=d["cu_seqlens_q"])
    r = pa.make_rope(cos_sin=torch.from_numpy(p.table).cuda(), table_rows=p.table_rows, rot_dim=p.rot, pairs=p.pairs,
                     positions=torch.from_numpy(p.positions).cuda() if p.given else None, axes=p.axes, pair_axes=p.pair_axis)
    torch.cuda.synchronize()
    pa.pa_rope_append(plan, args, r, qs if q else None, qs.stride(0), out if q else None, out.stride(0), ks,
                      vs, ks.stride(0), ws, stream)
    st, det = pa.pa_check(plan, ws, stream)
    bits = out.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    return bits, d["cache_k"].cpu().numpy(), None if mla else d["cache_v"].cpu().numpy(), st, det


def check(p, **kw):
    bits, ck, cv, st, det = launch(p, **kw)
    assert st == 0, (st, det)
    q, want_k, want_v = rh.expected(p)
    T, n = p.total_q, p.q_new[0].size
    if kw.get("q", True):
        assert (bits[:, :n].reshape(q.shape) == kv4.to_bf16_bits(q.astype(np.float32))).all()
    # beyond the row: as it was
    rest = bits[:, n:]
    if not kw.get("in_place"):
        assert (rest == kv4.to_bf16_bits(np.full(rest.shape, 7.0, np.float32))).all()
    assert (ck == want_k).all()
    assert cv is None or (cv == want_v).all()


@pytest.mark.parametrize("kv_dtype", rh.FORMATS)
@pytest.mark.parametrize("scale_kind", ["per_kv_head", "per_channel", "global"])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_formats(kv_dtype, scale_kind, pairs):
    check(rh.make(seed=1, seq_lens=[1, 70, 0, 9], seq_lens_kv=[63, 30, 5, 0], q_heads=6, kv_heads=2, kv_dtype=kv_dtype,
                  scale_kind=scale_kind, pairs=pairs))


@pytest.mark.parametrize("rot", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_widths(rot, pairs):
    check(rh.make(seed=2, seq_lens=[3, 5], seq_lens_kv=[0, 61], q_heads=3, kv_heads=3, kv_dtype="fp8_e4m3", rot=rot,
                  pairs=pairs))


@pytest.mark.parametrize("pair_axis", ["turns", "runs", "odd"])
@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_axes(axes, pair_axis, pairs):
    order = {"turns": [i % axes for i in range(48)], "runs": [i * axes // 48 // 1 for i in range(48)],
             "odd": [min(axes - 1, i // 7) for i in range(48)]}[pair_axis]
    check(rh.make(seed=3, seq_lens=[9, 1], seq_lens_kv=[2, 200], kv_dtype="fp4_e2m1", rot=96, pairs=pairs, axes=axes,
                  pair_axis=order, table_rows=300))


def test_positions_handed_over_on_one_axis():
    check(rh.make(seed=4, seq_lens=[20], seq_lens_kv=[7], given=True, table_rows=1000))


@pytest.mark.parametrize("kv_dtype", ["int8", "fp8_e4m3"])
@pytest.mark.parametrize("rot", [16, 48, 64])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_latent_rows(kv_dtype, rot, pairs):
    check(rh.make(seed=5, seq_lens=[1, 17, 0, 2], seq_lens_kv=[63, 60, 3, 0], layout="mla", kv_dtype=kv_dtype, rot=rot,
                  pairs=pairs), pad=8)


@pytest.mark.parametrize("kw", [dict(q=False), dict(in_place=True), dict(packed=True, pad=16), dict(pad=8),
                                dict(packed=True, in_place=True)])
def test_rows_in_place_packed_padded_or_without_queries(kw):
    check(rh.make(seed=6, seq_lens=[5, 33], seq_lens_kv=[10, 31], q_heads=10, kv_heads=2, kv_dtype="int4", rot=64), **kw)


@pytest.mark.parametrize("kw", [dict(in_place=True), dict(q=False)])
def test_latent_rows_in_place_or_without_queries(kw):
    check(rh.make(seed=7, seq_lens=[5], seq_lens_kv=[62], layout="mla", kv_dtype="fp8_e4m3", rot=64), **kw)


@pytest.mark.parametrize("kv_dtype", rh.FORMATS)
@pytest.mark.parametrize("spread", [1e-3, 30.0, 1e30])
def test_far_values(kv_dtype, spread):
    """Blocks of scale zero or subnormal, saturated codes and scales."""
    check(rh.make(seed=8, seq_lens=[12], seq_lens_kv=[60], kv_dtype=kv_dtype, scale_kind="per_channel", spread=spread))


# A plan for few SMs takes the launches of large calls (queries by themselves, units of 8
# rows of K and 32 positions of V) at sizes that the oracle can follow
@pytest.mark.parametrize("kv_dtype", rh.FORMATS)
@pytest.mark.parametrize("scale_kind", ["per_kv_head", "per_channel", "global"])
def test_many_rows(kv_dtype, scale_kind):
    check(rh.make(seed=9, seq_lens=[170, 1, 0, 75], seq_lens_kv=[13, 64, 3, 0], q_heads=28, kv_heads=14, kv_dtype=kv_dtype,
                  scale_kind=scale_kind), sms=2)


@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
@pytest.mark.parametrize("rot, axes", [(128, 1), (80, 3), (64, 2)])
def test_many_rows_of_several_axes(rot, axes, pairs):
    check(rh.make(seed=20, seq_lens=[99, 40], seq_lens_kv=[60, 1], q_heads=21, kv_heads=3, kv_dtype="int4", rot=rot, axes=axes,
                  pairs=pairs, table_rows=400), sms=1)


@pytest.mark.parametrize("kw", [dict(q=False), dict(in_place=True), dict(packed=True, pad=16), dict(packed=True, in_place=True)])
def test_many_rows_in_place_packed_or_without_queries(kw):
    check(rh.make(seed=21, seq_lens=[130, 7], seq_lens_kv=[31, 0], q_heads=10, kv_heads=5, kv_dtype="int8"), sms=1, **kw)


@pytest.mark.parametrize("kv_dtype", rh.FORMATS)
@pytest.mark.parametrize("spread", [1e-3, 30.0, 1e30])
def test_many_rows_of_far_values(kv_dtype, spread):
    check(rh.make(seed=22, seq_lens=[150], seq_lens_kv=[60], kv_heads=4, kv_dtype=kv_dtype, scale_kind="per_channel",
                  spread=spread), sms=1)


@pytest.mark.parametrize("sms", [None, 1])
@pytest.mark.parametrize("kv_dtype", ["int4", "fp4_e2m1"])
@pytest.mark.parametrize("q_heads, kv_heads", [(1, 1), (3, 3), (5, 1), (15, 5), (9, 3), (18, 9)])
def test_odd_heads_of_four_bits(kv_dtype, q_heads, kv_heads, sms):
    check(rh.make(seed=24, seq_lens=[300, 2], seq_lens_kv=[31, 64], q_heads=q_heads, kv_heads=kv_heads, kv_dtype=kv_dtype), sms=sms)


@pytest.mark.parametrize("sms", [None, 1])
@pytest.mark.parametrize("scale_kind", ["per_kv_head", "global"])
@pytest.mark.parametrize("kv_dtype", rh.FORMATS)
@pytest.mark.parametrize("spread", [1e-3, 30.0, 1e30])
def test_far_values_of_odd_heads(kv_dtype, scale_kind, spread, sms):
    check(rh.make(seed=25, seq_lens=[160], seq_lens_kv=[60], q_heads=3, kv_heads=3, kv_dtype=kv_dtype, scale_kind=scale_kind,
                  spread=spread), sms=sms)


@pytest.mark.parametrize("kv_dtype", rh.FORMATS)
@pytest.mark.parametrize("q", [True, False])
@pytest.mark.parametrize("sms", [1, 2, 4])
def test_units_of_many_rows(kv_dtype, sms, q):
    check(rh.make(seed=27, seq_lens=[77, 3, 0, 166], seq_lens_kv=[13, 63, 3, 7], q_heads=28, kv_heads=14, kv_dtype=kv_dtype),
          sms=sms, q=q)


@pytest.mark.parametrize("kv_dtype", rh.FORMATS)
def test_a_cache_on_a_boundary_of_16_bytes(kv_dtype):
    check(rh.make(seed=26, seq_lens=[130], seq_lens_kv=[31], kv_dtype=kv_dtype), sms=1, cache_at=16)


@pytest.mark.parametrize("sms", [None, 1])
@pytest.mark.parametrize("kv_dtype", rh.FORMATS)
def test_not_numbers(kv_dtype, sms):
    """NaN and infinities in rows: every other block, and row, as without them; int8 and 4 bits
    store a NaN as 0, E4M3 as its NaN (0x7F), and infinities saturate."""
    import paged_quantized_kv_gqa_gb300 as pa
    p = rh.make(seed=23, seq_lens=[140], seq_lens_kv=[3], q_heads=2, kv_heads=2, kv_dtype=kv_dtype)
    p.k_new, p.v_new, p.q_new = p.k_new.copy(), p.v_new.copy(), p.q_new.copy()
    clean = launch(p, sms=sms)
    for x in (p.k_new, p.v_new, p.q_new):
        x[5, 0, 3] = 0x7FC0
        x[77, 1, 100] = 0x7F80
        x[78, 1, 101] = 0xFF80
    got = launch(p, sms=sms)
    assert got[3] == pa.PA_OK
    rows = [r for r in range(140) if r not in (5, 77, 78)]
    assert (got[0][rows] == clean[0][rows]).all()
    q, want_k, want_v = rh.expected(p)
    assert (got[1] == want_k).all() and (got[2] == want_v).all()


def test_many_latent_rows():
    check(rh.make(seed=10, seq_lens=[300, 1], seq_lens_kv=[13, 64], layout="mla", kv_dtype="int8", rot=64))


def test_no_rows():
    import paged_quantized_kv_gqa_gb300 as pa
    p = rh.make(seed=11, seq_lens=[0, 0], seq_lens_kv=[5, 0])
    for n in ("q_new", "k_new", "v_new"):           # (an empty tensor has no address)
        setattr(p, n, np.zeros((1,) + getattr(p, n).shape[1:], np.uint16))
    bits, ck, cv, st, _ = launch(p, rows=1)
    assert st == pa.PA_OK and (bits == kv4.to_bf16_bits(np.full(bits.shape, 7.0, np.float32))).all()
    assert (ck == p.cache_k).all() and (cv == p.cache_v).all()


@pytest.mark.parametrize("layout", ["gqa", "mla"])
def test_positions_outside_the_table_are_reported_and_their_rows_not_turned(layout):
    import paged_quantized_kv_gqa_gb300 as pa
    p = rh.make(seed=12, seq_lens=[6], seq_lens_kv=[0], rot=64, layout=layout, kv_dtype="fp8_e4m3", given=True, table_rows=50)
    good = p.positions.copy()
    p.positions[0, 2], p.positions[0, 4] = 50, -1
    bits, ck, cv, st, det = launch(p)
    assert st == pa.PA_ERR_BAD_POSITION and det in (2, 4)
    p.positions = good
    p.table = p.table.copy()
    p.positions[0, [2, 4]] = 0                      # position 0: angle 0
    q, want_k, want_v = rh.expected(p)
    n = p.q_new[0].size
    assert (bits[:, :n].reshape(q.shape) == kv4.to_bf16_bits(q.astype(np.float32))).all()
    assert (ck == want_k).all() and (cv is None or (cv == want_v).all())


@pytest.mark.parametrize("layout", ["gqa", "mla"])
def test_a_bad_page_is_reported_and_nothing_of_it_written(layout):
    import paged_quantized_kv_gqa_gb300 as pa
    p = rh.make(seed=13, seq_lens=[10], seq_lens_kv=[60], rot=64, layout=layout, kv_dtype="int8")
    whole = rh.expected(p)
    p.block_table = p.block_table.copy()
    page = int(p.block_table[0, 1])
    p.block_table[0, 1] = p.num_pages
    bits, ck, cv, st, det = launch(p)
    assert st == pa.PA_ERR_BAD_PAGE and det == 0
    want = whole[1].copy()
    want[page] = p.cache_k[page]
    assert (ck == want).all()
    assert (bits[:, :p.q_new[0].size].reshape(whole[0].shape) == kv4.to_bf16_bits(whole[0].astype(np.float32))).all()


def test_on_another_stream_and_captured():
    import paged_quantized_kv_gqa_gb300 as pa
    p = rh.make(seed=14, seq_lens=[9], seq_lens_kv=[60], kv_dtype="fp4_e2m1")
    s = torch.cuda.Stream()
    bits, ck, cv, st, _ = launch(p, stream=s)
    q, want_k, want_v = rh.expected(p)
    assert st == 0 and (ck == want_k).all() and (cv == want_v).all()
    # replayed: the cache of each replay is what the rows hold then
    T = p.total_q
    d = {n: torch.from_numpy(getattr(p, n).copy()).cuda() for n in ("block_table", "seq_lens", "seq_lens_kv", "cu_seqlens_q",
                                                                     "cache_k", "cache_v")}
    qs, ks, vs = dev(p.q_new.reshape(T, -1)), dev(p.k_new.reshape(T, -1)), dev(p.v_new.reshape(T, -1))
    scales = [dev(p.k_scale), dev(p.v_scale)]
    table = torch.from_numpy(p.table).cuda()
    out = torch.zeros_like(qs)
    prob = pa.make_problem(**{k: getattr(p, k) for k in (
        "bsz", "q_heads", "kv_heads", "head_dim_qk", "head_dim_v", "block_size", "max_blocks_per_seq", "num_pages", "kv_dtype",
        "scale_kind", "layout", "chunk_size", "sm_scale", "q_stride", "causal")})
    plan = pa.pa_plan(prob, p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, num_sms())
    ws = torch.zeros(max(plan.workspace_size, 256), dtype=torch.uint8, device="cuda")
    pa.pa_plan_upload(plan, ws)
    args = pa.make_args(q=None, cache_k=d["cache_k"], cache_v=d["cache_v"], k_scale=scales[0], v_scale=scales[1],
                        block_table=d["block_table"], out=None, seq_lens=d["seq_lens"], seq_lens_kv=d["seq_lens_kv"],
                        cu_seqlens_q=d["cu_seqlens_q"])
    r = pa.make_rope(cos_sin=table, table_rows=p.table_rows, rot_dim=p.rot)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_rope_append(plan, args, r, qs, qs.stride(0), out, out.stride(0), ks, vs, ks.stride(0), ws)
    g.replay()
    torch.cuda.synchronize()
    assert (d["cache_k"].cpu().numpy() == want_k).all()
    other = rh.make(seed=15, seq_lens=[9], seq_lens_kv=[60], kv_dtype="fp4_e2m1")
    ks.copy_(dev(other.k_new.reshape(T, -1)))
    p.k_new = other.k_new
    g.replay()
    torch.cuda.synchronize()
    assert (d["cache_k"].cpu().numpy() == rh.expected(p)[1]).all()


@pytest.mark.parametrize("kv_dtype", ["int8", "fp4_e2m1"])
def test_pages_beyond_two_gigabytes(kv_dtype):
    """The last pages of a pool of 4 GB and more a side: the same stored values as in a
    small pool."""
    import paged_quantized_kv_gqa_gb300 as pa
    p = rh.make(seed=16, seq_lens=[70, 3], seq_lens_kv=[0, 61], q_heads=8, kv_heads=8, kv_dtype=kv_dtype)
    got = []
    for pages in (p.num_pages, 140_000 if kv_dtype == "fp4_e2m1" else 70_000):
        prob = pa.make_problem(bsz=p.bsz, q_heads=8, kv_heads=8, head_dim_qk=128, head_dim_v=128, block_size=64,
                               max_blocks_per_seq=p.max_blocks_per_seq, num_pages=pages, kv_dtype=kv_dtype,
                               scale_kind="per_kv_head", layout="gqa", causal=True, chunk_size=0, sm_scale=0.1, q_stride=1024)
        plan = pa.pa_plan(prob, p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, num_sms())
        caches = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in pa.pa_cache_bytes(prob)]
        table = torch.from_numpy(np.where(p.block_table < 0, -1, pages - 1 - p.block_table).astype(np.int32)).cuda()
        lens = [torch.from_numpy(x).cuda() for x in (p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q)]
        scales = [dev(p.k_scale), dev(p.v_scale)]
        args = pa.make_args(q=None, cache_k=caches[0], cache_v=caches[1], k_scale=scales[0], v_scale=scales[1],
                            block_table=table, out=None, seq_lens=lens[0], seq_lens_kv=lens[1], cu_seqlens_q=lens[2])
        ws = torch.zeros(max(plan.workspace_size, 256), dtype=torch.uint8, device="cuda")
        pa.pa_plan_upload(plan, ws)
        r = pa.make_rope(cos_sin=torch.from_numpy(p.table).cuda(), table_rows=p.table_rows, rot_dim=128)
        k, v = dev(p.k_new.reshape(p.total_q, -1)), dev(p.v_new.reshape(p.total_q, -1))
        pa.pa_rope_append(plan, args, r, None, 0, None, 0, k, v, 1024, ws)
        rows = [torch.zeros(p.total_q, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        pa.pa_cache_read(plan, args, *rows, 1024, ws)
        assert pa.pa_check(plan, ws)[0] == 0
        got.append(rows)
        del caches
    assert got[1][0].abs().sum() > 0 and all(torch.equal(a, b) for a, b in zip(*got))
