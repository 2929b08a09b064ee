"""How exact the results over the 4-bit cache are: the errors that the kernels' stated
roundings leave, and no larger ones.

What the kernels round: Q' of per-channel K scales up to 64 rows is two fp16 numbers
(exact but for parts below 2^-24), P is fp16 (relative error at most 2^-11), the final
row bf16; sums, maxima and partial rows are 32 bits.  Where a coarser rounding is to be
told from these, its error is worked out in the oracle on the same inputs."""
import numpy as np
import pytest

from kv4_helpers import KINDS, bf16_bits, check, make, reference, run, seen_mask
from oracle import kv4

pytestmark = pytest.mark.gpu

ROWS = [  # packed rows: 4, 8, 16, 21, 48, 64
    dict(seq_lens=[1, 1, 1], seq_lens_kv=[900, 70, 1700], q_heads=8, kv_heads=2),
    dict(seq_lens=[1, 1, 1], seq_lens_kv=[900, 70, 1700], q_heads=16, kv_heads=2),
    dict(seq_lens=[2, 1], seq_lens_kv=[900, 1700], q_heads=16, kv_heads=2),
    dict(seq_lens=[3, 2], seq_lens_kv=[900, 1700], q_heads=14, kv_heads=2),
    dict(seq_lens=[6, 6], seq_lens_kv=[900, 1700], q_heads=16, kv_heads=2),
    dict(seq_lens=[8, 4], seq_lens_kv=[900, 1700], q_heads=16, kv_heads=2),
]


def queries(p, b, h):
    G = p.q_heads // p.kv_heads
    t0, t1 = int(p.cu_seqlens_q[b]), int(p.cu_seqlens_q[b + 1])
    return kv4.bf16_to_f64(p.q_bits[t0:t1, h * G * 128:(h + 1) * G * 128]).reshape(t1 - t0, G, 128)


def lse_with(p, q_of):
    """lse [T, Hq] with Q' = q_of(q, k scales) against the keys without their scales."""
    G = p.q_heads // p.kv_heads
    lse = np.zeros((p.total_q, p.q_heads))
    for b in range(p.bsz):
        t0, t1 = int(p.cu_seqlens_q[b]), int(p.cu_seqlens_q[b + 1])
        seen = seen_mask(p, b)
        for h in range(p.kv_heads):
            c, s = kv4.stored_rows(p, "k", b, h, int(p.held[b]))
            g = kv4.tensor_scale(p, "k", h).astype(np.float64)
            V = np.zeros((int(p.held[b]), 128))
            lse[t0:t1, h * G:(h + 1) * G] = kv4.attend(q_of(queries(p, b, h), g), c * s, V, seen, p.sm_scale)[1]
    return lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", ROWS)
def test_small_channel_scales_keep_their_bits(kw, kind):
    """Channel scales near 1e-3 beside block scales near 448, as a range of 2688 or 3136
    steps a channel gives them.  One fp16 number for Q' has a relative error of up to
    2^-11; two have 2^-22, and 256 additions in 32 bits about 2^-20 at random: at least a
    factor of 2^8 less, of which the test asks for 2^4."""
    p = make(81, kv_dtype=kind, scale_kind="per_channel", **kw)
    r = np.random.default_rng(3)
    n = p.kv_heads * 128
    p.k_scale = bf16_bits(r.uniform(0.5e-3, 1.5e-3, n))
    codes, _ = kv4.unpack_k(p.cache_k)
    p.cache_k = kv4.pack_k(codes, r.integers(0x78, 0x7F, (*codes.shape[:-1], 8)).astype(np.uint8))   # 256 .. 448
    p.q_bits = bf16_bits(6.0 * r.standard_normal(p.q_bits.shape))
    ref = reference(p)
    out, lse, *_ = run(p)
    check(p, out, lse, ref)
    exact = lse_with(p, lambda q, g: q * g)
    one = lse_with(p, lambda q, g: (q * g).astype(np.float16).astype(np.float64))
    assert np.allclose(exact, ref[1], rtol=0, atol=1e-9)
    rms = lambda e: float(np.sqrt(np.mean(e * e)))  # noqa: E731
    print(f"lse: {rms(lse - exact):.2e}, with one fp16 number {rms(one - exact):.2e}")
    assert rms(lse - exact) * 16 <= rms(one - exact)


SPLIT = [
    dict(seq_lens=[1, 1], seq_lens_kv=[4095, 2999], q_heads=8, kv_heads=2),
    dict(seq_lens=[2, 1], seq_lens_kv=[4094, 2999], q_heads=16, kv_heads=2),
    dict(seq_lens=[6, 5], seq_lens_kv=[4090, 8995], q_heads=16, kv_heads=2),
    dict(seq_lens=[70, 3], seq_lens_kv=[1930, 3000], q_heads=8, kv_heads=2, chunk_size=512),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", SPLIT)
def test_partial_rows_keep_32_bits(kw, kind):
    """q = 0: every score is 0, every P exactly 1, so that the sums, the partial rows and
    the last rounding are all there is.  V is positive in a sequence's first half and
    negative in the second: the row is the small difference of large partial rows, which
    bf16 partial rows would be off by 2^-9 of."""
    p = make(82, kv_dtype=kind, scale_kind="global", causal=False, **kw)
    p.q_bits[:] = 0
    codes, sb = kv4.unpack_v(p.cache_v)
    table = kv4.code_table(kind)
    pos, neg = (np.flatnonzero(f(table)) for f in (lambda t: t > 0, lambda t: (t < 0) & (t > -8)))
    r = np.random.default_rng(4)
    for b in range(p.bsz):
        n = int(p.held[b])
        for k in range(-(-n // 64)):
            side = pos if 64 * k < n // 2 else neg
            codes[p.block_table[b, k]] = r.choice(side, codes.shape[1:])
    p.cache_v = kv4.pack_v(codes, sb)
    out, lse, _, plan = run(p)
    d = plan.describe()
    G = p.q_heads // p.kv_heads
    worst = 0.0
    for b in range(p.bsz):
        n, t0, t1 = int(p.held[b]), int(p.cu_seqlens_q[b]), int(p.cu_seqlens_q[b + 1])
        assert d["nch_token"][t0] > 1
        for h in range(p.kv_heads):
            V = kv4.rows(p, "v", b, h, n)
            want = V.mean(0)
            # the last rounding, and 32-bit sums: L / 16 steps of at most 2^-23 of the
            # running sum each, with a few more for the division and the merge
            tol = 2.0 ** -8 * np.abs(want) + (n / 16 + 8) * 2.0 ** -23 * np.abs(V).mean(0)
            got = out[t0:t1, h * G:(h + 1) * G]
            assert (np.abs(got - want) <= tol).all()
            # the same with bf16 partial rows
            it = d["items"]
            pieces = sorted((int(a[5]), int(a[6])) for a in it if a[0] == b and a[1] == h and a[2] == t0)
            assert pieces[0][0] == 0 and pieces[-1][1] == n and len(pieces) == d["nch_token"][t0]
            coarse = sum((c - a) * kv4.bf16_to_f64(bf16_bits(V[a:c].mean(0))) for a, c in pieces) / n
            worst = max(worst, float((np.abs(coarse - want) / tol).max()))
    assert worst > 2.0, "bf16 partial rows would pass this test"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw", ROWS + SPLIT)
def test_errors_are_those_of_the_stated_roundings(kw, kind):
    """The mean square of the outputs' errors against what the roundings give: ulp^2 / 12
    of the row's bf16 numbers, and at most (2^-11 p v)^2 / 3 a position for P in fp16.
    With P in bf16 the second part is 64 times as large and the sum 1.7 times or more."""
    p = make(83, kv_dtype=kind, **{**kw, "causal": True})
    out, lse, *_ = run(p)
    ref, *_ = reference(p)
    ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(ref), 1e-30))) - 7)
    expected = (ulp ** 2 / 12).sum()
    G = p.q_heads // p.kv_heads
    for b in range(p.bsz):
        seen, n = seen_mask(p, b), int(p.held[b])
        for h in range(p.kv_heads):
            K, V = kv4.rows(p, "k", b, h, n), kv4.rows(p, "v", b, h, n)
            s = np.where(seen[:, None, :], p.sm_scale * np.einsum("ngd,ld->ngl", queries(p, b, h), K), -np.inf)
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            expected += (2.0 ** -22 / 3) * np.einsum("ngl,ld->", w * w, V * V)
    # the sum's own scatter: that of a mean of N squares of uniform errors, 2 / sqrt(N)
    # of it at most, four times that allowed
    ratio = ((out - ref) ** 2).sum() / expected
    print(f"{ratio:.3f} of the expected square error")
    assert ratio <= 1.0 + 8.0 / np.sqrt(ref.size) + 0.02


# ---------------------------------------------------------------- what cuts a decode plan
@pytest.mark.parametrize("kv_dtype", KINDS)
def test_the_cut_of_a_decode_plan_does_not_show(kv_dtype):
    """The number of SMs, and a neighbour beyond 512 positions, decide where a 4-bit
    decode plan cuts; whatever they say, the rows are the reference's."""
    kw = dict(seq_lens=[1, 2], seq_lens_kv=[500, 130], q_heads=8, kv_heads=2, kv_dtype=kv_dtype)
    p = make(84, **kw)
    ref, cuts = reference(p), set()
    for sms in (1, 5, 152):
        out, lse, _, plan = run(p, sms=sms)
        check(p, out, lse, ref)
        cuts.add(plan.describe()["max_chunks"])
    assert cuts == {1}           # up to 512 positions: whole
    p = make(84, **{**kw, "seq_lens_kv": [1900, 130]})
    ref, cuts = reference(p), set()
    for sms in (1, 2, 5, 152):
        out, lse, _, plan = run(p, sms=sms)
        check(p, out, lse, ref)
        cuts.add(plan.describe()["max_chunks"])
    assert len(cuts) >= 3 and max(cuts) > 8


@pytest.mark.parametrize("kv_dtype", KINDS)
def test_chunks_of_an_append_plan_do_not_show(kv_dtype):
    p = make(85, seq_lens=[70, 20], seq_lens_kv=[500, 30], q_heads=8, kv_heads=2, kv_dtype=kv_dtype)
    ref, cuts = reference(p), set()
    for cs in (0, 64, 192, 512):
        p.chunk_size = cs
        out, lse, _, plan = run(p)
        check(p, out, lse, ref)
        cuts.add(plan.describe()["max_chunks"])
    assert cuts == {1, 9, 3, 2}
