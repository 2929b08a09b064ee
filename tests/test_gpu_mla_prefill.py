"""Attention to expanded latent rows on the GPU against float64.

Tolerance, per element.  A score is off by ds: 192 products summed in binary32 (a step
of each partial sum, 2^-23 of the magnitudes' sum), its product with the scale and the
subtraction of the maximum (a few 2^-24 of the score).  A weight is off by the factor
e^(2 ds) (its own score and the sum's), 2^-21 for exp2, and P's rounding to bf16, 2^-8;
the row's rounding to bf16 adds 2^-8 of the result.  So |out| may be off by
2^-8 |out| + (2^-8 + 4 ds) sum p |v|, lse by 2 ds + 2^-20 max(1, |lse|).  Split rows are
joined in binary32, within the same bounds."""
import numpy as np
import pytest
import torch

from gpu_helpers import num_sms
from oracle import mla

pytestmark = pytest.mark.gpu


def randn(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16()


def held_of(q_lens, kv_lens, mask):
    return [k + (0 if mask == "cross" else q) for q, k in zip(q_lens, kv_lens)]


def make(seed, q_lens, kv_lens, heads, mask, scale=1.0):
    T, N = sum(q_lens), max(1, sum(held_of(q_lens, kv_lens, mask)))
    return (randn(seed, T, heads, 192, scale=scale), randn(seed + 1, N, heads, 128, scale=scale), randn(seed + 2, N, heads, 128),
            randn(seed + 3, N, 64, scale=scale))


def launch(pa, t, q_lens, kv_lens, heads, mask, chunk=0, pad=0, sm_scale=192 ** -0.5, lse=True, stream=None, sms=None, **ep):
    def wide(x):
        x = x.flatten(1)
        w = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=torch.bfloat16)
        w[:, :x.shape[1]] = x
        return w.cuda()
    q, k, v, kr = (wide(x) for x in t)
    T = sum(q_lens)
    prob = pa.make_problem(bsz=len(q_lens), q_heads=heads, kv_heads=heads, head_dim_qk=192, head_dim_v=128, kv_dtype="bf16",
                           layout="mla_expanded", causal=mask == "causal", cross=mask == "cross", chunk_size=chunk,
                           sm_scale=sm_scale, q_stride=q.stride(0))
    plan = pa.pa_plan(prob, q_lens, kv_lens, np.concatenate([[0], np.cumsum(q_lens)]), sms or num_sms())
    ws = torch.full((plan.workspace_size,), 0xFF, dtype=torch.uint8, device="cuda")
    pa.pa_plan_upload(plan, ws)
    out = torch.full((T + 3, heads, 128), 7, dtype=torch.int8 if ep.get("out_int8") else torch.bfloat16, device="cuda")
    l = torch.full((T + 3, heads), 7.0, device="cuda")
    args = pa.make_args(q=q, cache_k=None, cache_v=None, k_scale=None, v_scale=None, block_table=None, out=out,
                        lse=l if lse else None, **ep)
    torch.cuda.synchronize()
    pa.pa_mla_prefill(plan, args, k, v, k.stride(0), kr, kr.stride(0), ws, stream)
    if chunk != 0:
        pa.pa_merge(plan, args, ws, stream)
    st, det = pa.pa_check(plan, ws, stream)
    assert st == 0, (st, det, pa.pa_last_error())
    assert (out[T:] == 7).all() and (l[T:] == 7).all()
    return out[:T], l[:T], plan


def compare(t, out, lse, q_lens, kv_lens, mask, sm_scale=192 ** -0.5):
    q, k, v, kr = (x.double().numpy() for x in t)
    ref, ref_l, mag = mla.prefill(q, k, v, kr, q_lens, kv_lens, mask, sm_scale)
    key = np.concatenate([k, np.broadcast_to(kr[:, None], (*k.shape[:2], 64))], 2)
    # sum |q k| of the sequence's largest score: by the largest |k| of each dim
    big = np.zeros(ref_l.shape)
    t0 = n0 = 0
    for ql, h in zip(q_lens, held_of(q_lens, kv_lens, mask)):
        if h:
            big[t0:t0 + ql] = np.einsum("thd,hd->th", np.abs(q[t0:t0 + ql]), np.abs(key[n0:n0 + h]).max(0))
        t0, n0 = t0 + ql, n0 + h
    ds = (192 * 2.0 ** -23 + 4 * 2.0 ** -24) * sm_scale * big
    got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 4 * ds[..., None]) * mag
    worst = np.abs(got - ref) / np.maximum(tol, 1e-30)
    assert (np.abs(got - ref) <= tol).all(), float(worst.max())
    none = np.isneginf(ref_l)
    assert (np.isneginf(got_l) == none).all() and (got[none] == 0).all()
    err = np.abs(got_l - np.where(none, 0, ref_l))[~none]
    assert (err <= (2 * ds + 2.0 ** -20 * np.maximum(1, np.abs(np.where(none, 0, ref_l))))[~none]).all()


def check(q_lens, kv_lens, heads, mask, seed=0, scale=1.0, **kw):
    import paged_quantized_kv_gqa_gb300 as pa
    t = make(seed, q_lens, kv_lens, heads, mask, scale)
    out, lse, plan = launch(pa, t, q_lens, kv_lens, heads, mask, **kw)
    compare(t, out, lse, q_lens, kv_lens, mask, kw.get("sm_scale", 192 ** -0.5))
    return plan


@pytest.mark.parametrize("mask", ["causal", "full", "cross"])
@pytest.mark.parametrize("q", [1, 2, 127, 128, 129, 255, 256, 257, 600])
def test_query_lengths(mask, q):
    check([q], [70], 2, mask)


@pytest.mark.parametrize("mask", ["causal", "full", "cross"])
@pytest.mark.parametrize("kv", [1, 63, 64, 65, 127, 128, 129, 500])
def test_prefix_lengths(mask, kv):
    check([5, 130], [kv, kv], 3, mask)


@pytest.mark.parametrize("mask", ["causal", "full", "cross"])
@pytest.mark.parametrize("chunk", [0, -1, 64, 512])
def test_ragged_batches_and_splits(mask, chunk):
    check([300, 0, 1, 257, 64, 3], [0, 5, 0, 1000, 129, 1500], 5, mask, chunk=chunk, pad=8)


@pytest.mark.parametrize("sms", [1, 3])
def test_many_items_a_cta(sms):
    """Items of one and two tiles, one step and many, one after the other on a CTA."""
    check([300, 20, 1, 513, 128, 129], [0, 700, 2, 0, 300, 0], 3, "causal", sms=sms)
    check([300, 20, 1, 513, 128, 129], [0, 700, 2, 0, 300, 0], 3, "causal", sms=sms, chunk=128)
    check([20, 300], [0, 10], 2, "cross", sms=sms, chunk=-1)


@pytest.mark.parametrize("heads", [1, 16, 20, 128])
def test_heads(heads):
    check([40, 150], [100, 0], heads, "causal", chunk=-1)


def test_long_rows():
    check([260], [9000], 2, "causal", chunk=-1)
    check([260], [9000], 2, "full", chunk=0)


@pytest.mark.parametrize("scale", [0.0, 4.0])
def test_flat_and_peaked_scores(scale):
    check([200], [300], 2, "causal", scale=scale)


def test_rising_scores_rescale_the_rows():
    import paged_quantized_kv_gqa_gb300 as pa
    q, k, v, kr = make(3, [140], [900], 2, "causal")
    q = q.abs()
    k = (k.abs().float() * torch.linspace(0.1, 6, k.shape[0])[:, None, None]).bfloat16()   # maxima rise step by step
    out, lse, _ = launch(pa, (q, k, v, kr), [140], [900], 2, "causal")
    compare((q, k, v, kr), out, lse, [140], [900], "causal")


def test_other_sequences_rows_may_hold_anything():
    import paged_quantized_kv_gqa_gb300 as pa
    q_lens, kv_lens = [70, 40, 200], [30, 100, 9]
    t = make(4, q_lens, kv_lens, 2, "causal")
    clean, clean_l, _ = launch(pa, t, q_lens, kv_lens, 2, "causal")
    dirty = [x.clone() for x in t]
    for x in dirty[1:]:
        x[100:240] = float("nan")                   # all of the middle sequence's rows
        x[150] = float("inf")
    dirty[0][70:110] = float("nan")
    out, lse, _ = launch(pa, dirty, q_lens, kv_lens, 2, "causal")
    rows = [r for r in range(310) if not 70 <= r < 110]
    assert torch.equal(out[rows], clean[rows]) and torch.equal(lse[rows], clean_l[rows])


def test_without_lse_and_with_the_output_epilogue():
    import paged_quantized_kv_gqa_gb300 as pa
    q_lens, kv_lens, heads = [150, 20], [700, 0], 3
    t = make(5, q_lens, kv_lens, heads, "causal")
    ref = mla.prefill(*(x.double().numpy() for x in t), q_lens, kv_lens, "causal", 192 ** -0.5)[0]
    shift, smooth = randn(6, heads * 128).cuda(), randn(7, heads * 128).abs().cuda()
    want = (ref + shift.double().cpu().numpy().reshape(heads, 128)) * smooth.double().cpu().numpy().reshape(heads, 128)
    for chunk in (0, 128):
        out, _, _ = launch(pa, t, q_lens, kv_lens, heads, "causal", chunk=chunk, lse=False, shift_bias=shift,
                           smooth_weight=smooth)
        # the attention's own error times the smoothing factors (below 5), and the rounding
        assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 5 * 2.0 ** -6).all()
        codes, _, _ = launch(pa, t, q_lens, kv_lens, heads, "causal", chunk=chunk, lse=False, out_int8=True, in_scale=0.5,
                             quant_max_bound=100.0, quant_min_bound=-90.0)
        assert (np.abs(codes.cpu().numpy() - np.clip(np.rint(ref * 50.0), -90, 100)) <= 50 * 2.0 ** -6 + 1).all()


def test_the_same_call_gives_the_same_bits_on_any_stream():
    import paged_quantized_kv_gqa_gb300 as pa
    t = make(8, [500, 30], [0, 3000], 4, "causal")
    a = launch(pa, t, [500, 30], [0, 3000], 4, "causal", chunk=-1)
    b = launch(pa, t, [500, 30], [0, 3000], 4, "causal", chunk=-1, stream=torch.cuda.Stream())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_nothing_to_see():
    """Cross attention to sequences without rows, alone and among others."""
    check([5, 3], [0, 0], 2, "cross")
    check([5, 3], [0, 0], 2, "cross", chunk=-1)
    check([5, 300, 2], [0, 40, 0], 2, "cross")


def test_ranges_of_two_plans_join_by_their_lse():
    """New tokens against the cached prefix and among themselves, as one range."""
    import paged_quantized_kv_gqa_gb300 as pa
    q_lens, kv_lens, heads = [90, 200], [300, 41], 2
    t = make(9, q_lens, kv_lens, heads, "causal")
    whole = mla.prefill(*(x.double().numpy() for x in t), q_lens, kv_lens, "causal", 192 ** -0.5)
    prefix = [r for n0, kv in ((0, 300), (390, 41)) for r in range(n0, n0 + kv)]
    new = [r for r in range(390 + 241) if r not in set(prefix)]
    part = lambda rows: (t[0], *(x[rows] for x in t[1:]))  # noqa: E731
    o1, l1, _ = launch(pa, part(prefix), q_lens, kv_lens, heads, "cross")
    o2, l2, _ = launch(pa, part(new), q_lens, [0, 0], heads, "causal")
    l = torch.logaddexp(l1.double(), l2.double())
    o = (l1.double() - l).exp()[..., None] * o1.double() + (l2.double() - l).exp()[..., None] * o2.double()
    assert np.abs(l.cpu().numpy() - whole[1]).max() <= 1e-3
    assert (np.abs(o.cpu().numpy() - whole[0]) <= 2.0 ** -7 * (np.abs(whole[0]) + whole[2])).all()


def test_a_missing_load_is_reported_and_the_next_call_works():
    import paged_quantized_kv_gqa_gb300 as pa
    pa.pa_debug_set_faults(wait_limit_ns=2_000_000, skip_first_load=True)
    try:
        t = make(10, [300], [0], 2, "causal")
        with pytest.raises(AssertionError) as e:
            launch(pa, t, [300], [0], 2, "causal")
        assert "4" in str(e.value)
    finally:
        pa.pa_debug_set_faults()
    check([300], [0], 2, "causal")


def test_captured_and_replayed():
    import paged_quantized_kv_gqa_gb300 as pa
    q_lens, kv_lens, heads = [100, 7], [0, 2000], 2
    t = [x.flatten(1).cuda() for x in make(11, q_lens, kv_lens, heads, "causal")]
    prob = pa.make_problem(bsz=2, q_heads=heads, kv_heads=heads, head_dim_qk=192, head_dim_v=128, kv_dtype="bf16",
                           layout="mla_expanded", causal=True, chunk_size=-1, sm_scale=0.1, q_stride=heads * 192)
    plan = pa.pa_plan(prob, q_lens, kv_lens, [0, 100, 107], num_sms())
    assert plan.describe()["max_chunks"] > 1
    ws = torch.zeros(plan.workspace_size, dtype=torch.uint8, device="cuda")
    pa.pa_plan_upload(plan, ws)
    out, lse = torch.zeros(107, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(107, heads, device="cuda")
    args = pa.make_args(q=t[0], cache_k=None, cache_v=None, k_scale=None, v_scale=None, block_table=None, out=out, lse=lse)
    torch.cuda.synchronize()

    def call():
        pa.pa_mla_prefill(plan, args, t[1], t[2], heads * 128, t[3], 64, ws)
        pa.pa_merge(plan, args, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in t:
        x.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    got = out.clone(), lse.clone()
    call()
    torch.cuda.synchronize()
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1]) and out.abs().sum() > 0
