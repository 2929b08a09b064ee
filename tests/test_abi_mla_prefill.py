"""Plans of expanded latent rows and what pa_mla_prefill refuses (CPU)."""
import numpy as np
import pytest

from test_tmem_order import commit_barriers, source, unfenced

A = 1 << 20


@pytest.fixture(scope="module")
def pa():
    import paged_quantized_kv_gqa_gb300 as m
    return m


def make_plan(pa, q_lens, kv_lens, heads=4, mask="causal", chunk=0, sms=152, **kw):
    a = dict(bsz=len(q_lens), q_heads=heads, kv_heads=heads, head_dim_qk=192, head_dim_v=128, kv_dtype="bf16",
             layout="mla_expanded", causal=mask == "causal", cross=mask == "cross", chunk_size=chunk, sm_scale=0.07,
             q_stride=heads * 192)
    a.update(kw)
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    return pa.pa_plan(pa.make_problem(**a), q_lens, kv_lens, cu, sms)


@pytest.mark.parametrize("mask", ["causal", "full", "cross"])
@pytest.mark.parametrize("chunk", [0, -1, 512])
@pytest.mark.parametrize("sms", [1, 7, 152])
@pytest.mark.parametrize("q_lens, kv_lens, heads", [([1], [0], 1), ([300, 0, 257, 1], [0, 40, 2000, 9000], 3),
                                                      ([256, 512], [100, 0], 16), ([700] * 5, [0, 0, 5000, 1, 64], 128)])
def test_every_row_and_position_is_covered_once(pa, q_lens, kv_lens, heads, chunk, mask, sms):
    plan = make_plan(pa, q_lens, kv_lens, heads, mask, chunk, sms)
    d = plan.describe()
    assert d["family"] == "expanded" and d["num_ctas"] <= sms
    assert (np.diff(d["work_indptr"]) > 0).all() and d["work_indptr"][-1] == len(d["items"])
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    seen = {}
    for b, h, t0, n, base, k0, k1, cc in d["items"]:
        assert 1 <= n <= 256 and cu[b] <= t0 and t0 + n <= cu[b + 1] and k0 < k1 and 0 <= h < heads
        i = t0 - cu[b]
        held = kv_lens[b] + (0 if mask == "cross" else q_lens[b])
        assert base == (kv_lens[b] + i if mask == "causal" else held)
        seen.setdefault((b, h, i, n), []).append((cc & 0xFFFF, cc >> 16, k0, k1))
    tiles = [(b, i, min(256, q - i)) for b, q in enumerate(q_lens) for i in range(0, q, 256)]
    for b, i, n in tiles:
        lim = kv_lens[b] + (i + n if mask == "causal" else 0 if mask == "cross" else q_lens[b])
        for h in range(heads):
            parts = sorted(seen.pop((b, h, i, n), []))
            assert [p[0] for p in parts] == list(range(len(parts))) and all(p[1] == len(parts) for p in parts)
            edges = [0] + [p[3] for p in parts]
            assert [p[2] for p in parts] == edges[:-1] and edges[-1] == lim
            assert d["nch_token"][cu[b] + i] == len(parts)
    assert not seen
    assert chunk != 0 or d["max_chunks"] == 1


def test_plans_are_a_function_of_their_inputs_and_balanced(pa):
    make = lambda: make_plan(pa, [2048, 900, 1700], [0, 0, 300], 128).describe()  # noqa: E731
    a, b = make(), make()
    assert (a["items"] == b["items"]).all() and (a["work_indptr"] == b["work_indptr"]).all()
    cost = [-(-(k1 - k0) // 128) * (21 if n > 128 else 14) + 30 for _, _, _, n, _, k0, k1, _ in a["items"]]
    load = np.add.reduceat(cost, a["work_indptr"][:-1])
    assert load.max() <= load.mean() + max(cost)


def call(pa, plan=None, args=None, **kw):
    a = dict(q=A, out=A, lse=None)
    a.update(args or {})
    r = dict(k=A, v=A, kv_stride=512, k_rope=A, rope_stride=64, ws=A)
    r.update(kw)
    pa.pa_mla_prefill(plan or make_plan(pa, [5], [3]), pa.make_args(cache_k=None, cache_v=None, k_scale=None, v_scale=None,
                                                                    block_table=None, **a),
                      r["k"], r["v"], r["kv_stride"], r["k_rope"], r["rope_stride"], r["ws"], stream=0)


@pytest.mark.parametrize("kw, text", [
    (dict(args=dict(q=None)), "null"),
    (dict(args=dict(q=A + 8)), "aligned"),
    (dict(args=dict(out=None)), "null out"),
    (dict(args=dict(out=A + 8)), "aligned"),
    (dict(args=dict(out_int8=True, quant_max_bound=200.0)), "int8"),
    (dict(k=None), "null"),
    (dict(v=None), "null"),
    (dict(k_rope=None), "null"),
    (dict(ws=None), "workspace"),
    (dict(k=A + 2), "aligned"),
    (dict(v=A + 8), "aligned"),
    (dict(k_rope=A + 4), "aligned"),
    (dict(kv_stride=504), "smaller"),
    (dict(kv_stride=513), "multiples"),
    (dict(rope_stride=56), "smaller"),
    (dict(rope_stride=68), "multiples"),
    (dict(kv_stride=1 << 39), "2\\^40"),
])
def test_refusals(pa, kw, text):
    with pytest.raises(pa.PaError, match=text) as e:
        call(pa, **kw)
    assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_a_tree_mask_is_refused(pa):
    with pytest.raises(pa.PaError, match="tree mask"):
        call(pa, args=dict(attn_mask=A))


@pytest.mark.parametrize("kw", [dict(head_dim_qk=128), dict(head_dim_v=192), dict(kv_heads=2), dict(block_size=128)])
def test_unsupported_shapes(pa, kw):
    with pytest.raises(pa.PaError) as e:
        make_plan(pa, [5], [3], **kw)
    assert e.value.status == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(kv_dtype="int8"), dict(layout="gqa", scale_kind="global", max_blocks_per_seq=4,
                                                             num_pages=4, head_dim_qk=128)])
def test_bf16_rows_and_the_layout_go_together(pa, kw):
    with pytest.raises(pa.PaError) as e:
        make_plan(pa, [5], [3], **kw)
    assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_a_cache_needs_its_sizes(pa):
    with pytest.raises(TypeError):
        make_plan(pa, [5], [3], layout="gqa", kv_dtype="int8")


def test_calls_do_not_take_the_other_kind_of_plan(pa):
    plan = make_plan(pa, [5], [3])
    args = pa.make_args(q=A, cache_k=A, cache_v=A, k_scale=A, v_scale=A, block_table=A, out=A, seq_lens=A, seq_lens_kv=A,
                        cu_seqlens_q=A)
    for f in (lambda: pa.pa_run(plan, args, A, 0), lambda: pa.pa_cache_append(plan, args, A, A, 512, A, 0),
              lambda: pa.pa_cache_read(plan, args, A, A, 512, A, 0), lambda: pa.pa_cache_bytes(plan.problem),
              lambda: pa.pa_rope_append(plan, args, pa.make_rope(cos_sin=A, table_rows=9, rot_dim=64), None, 0, None, 0, A, A,
                                        512, A, 0)):
        with pytest.raises(pa.PaError):
            f()
    gqa = pa.make_problem(bsz=1, q_heads=4, kv_heads=4, head_dim_qk=128, head_dim_v=128, max_blocks_per_seq=1, num_pages=1,
                          kv_dtype="int8", scale_kind="global", layout="gqa", causal=True, chunk_size=0, sm_scale=0.1,
                          q_stride=512)
    with pytest.raises(pa.PaError, match="MLA_EXPANDED"):
        call(pa, plan=pa.pa_plan(gqa, [5], [3], [0, 5], 152))


def test_every_wait_for_mmas_is_followed_by_the_fence():
    for name in ("pa_mla_prefill.cu", "pa_mla_product.cu"):
        text = source(name)
        assert len(commit_barriers(text)) >= 2 and not unfenced(text)
