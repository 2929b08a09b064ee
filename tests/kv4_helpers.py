"""Seeded problems over the 4-bit cache and their comparison with the oracle."""
import math
import types

import numpy as np

from oracle import kv4

KINDS = ["fp4_e2m1", "int4"]
SCALES = ["per_kv_head", "per_channel", "global"]


def bf16_bits(x):
    return kv4.to_bf16_bits(np.asarray(x, np.float32))


def make(seed=0, *, seq_lens, seq_lens_kv, q_heads, kv_heads, kv_dtype="fp4_e2m1", scale_kind="per_kv_head",
         causal=True, cross=False, chunk_size=0, q_stride=None, garbage=True, extra_pages=2):
    """A problem with random codes (every nibble occurs) and block scales.  With
    `garbage`, the bytes of positions that no sequence holds are 0xFF: as block
    scales, NaN."""
    r = np.random.default_rng(seed)
    p = types.SimpleNamespace(q_heads=q_heads, kv_heads=kv_heads, head_dim_qk=128, head_dim_v=128, block_size=64,
                              kv_dtype=kv_dtype, scale_kind=scale_kind, layout="gqa", causal=causal, cross=cross,
                              chunk_size=chunk_size, sm_scale=128 ** -0.5, q_stride=q_stride or q_heads * 128)
    p.seq_lens, p.seq_lens_kv = np.asarray(seq_lens, np.int32), np.asarray(seq_lens_kv, np.int32)
    p.bsz = len(p.seq_lens)
    p.cu_seqlens_q = np.concatenate([[0], np.cumsum(p.seq_lens)]).astype(np.int32)
    p.total_q = int(p.cu_seqlens_q[-1])
    p.held = p.seq_lens_kv + (0 if cross else p.seq_lens)
    need = -(-p.held // 64)
    p.num_pages = int(need.sum()) + extra_pages
    p.max_blocks_per_seq = int(max(1, need.max(initial=1)))
    perm = r.permutation(p.num_pages)
    p.block_table = np.full((p.bsz, p.max_blocks_per_seq), -1, np.int32)
    at = 0
    used = np.zeros((p.num_pages, 64), bool)
    for b, n in enumerate(need):
        p.block_table[b, :n] = perm[at:at + n]
        for k in range(n):
            used[perm[at + k], :min(64, p.held[b] - 64 * k)] = True
        at += n
    for w, pack in (("k", kv4.pack_k), ("v", kv4.pack_v)):
        codes = r.integers(0, 16, (p.num_pages, kv_heads, 64, 128)).astype(np.uint8)
        sb = r.integers(0x28, 0x40, (p.num_pages, kv_heads, 64, 8)).astype(np.uint8)   # 0.25 .. 1.875
        sb[r.random(sb.shape) < 0.02] = 0            # blocks of zeros
        if garbage:
            hole = ~used[:, None, :, None]
            codes, sb = np.where(hole, 15, codes).astype(np.uint8), np.where(hole, 255, sb).astype(np.uint8)
        setattr(p, "cache_" + w, pack(codes, sb))
        n = {"global": 1, "per_kv_head": kv_heads, "per_channel": kv_heads * 128}[scale_kind]
        g = r.uniform(0.1, 0.4, n).astype(np.float32)
        setattr(p, w + "_scale", g if scale_kind == "global" else bf16_bits(g))
    p.q_bits = bf16_bits(r.standard_normal((p.total_q, p.q_stride)))
    p.k_new = bf16_bits(r.standard_normal((p.total_q, kv_heads, 128)))
    p.v_new = bf16_bits(r.standard_normal((p.total_q, kv_heads, 128)))
    return p


def problem(pa, p):
    return pa.make_problem(bsz=p.bsz, q_heads=p.q_heads, kv_heads=p.kv_heads, head_dim_qk=128, head_dim_v=128,
                           block_size=64, max_blocks_per_seq=p.max_blocks_per_seq, num_pages=p.num_pages,
                           kv_dtype=p.kv_dtype, scale_kind=p.scale_kind, layout="gqa", causal=p.causal,
                           cross=p.cross, chunk_size=p.chunk_size, sm_scale=p.sm_scale, q_stride=p.q_stride)


def seen_mask(p, b):
    n, L = int(p.seq_lens[b]), int(p.held[b])
    j, i = np.arange(L)[None, :], np.arange(n)[:, None]
    seen = j <= p.seq_lens_kv[b] + i if p.causal else np.ones((n, L), bool)
    mask = getattr(p, "attn_mask", None)
    if mask is not None:
        pre = int(p.seq_lens_kv[b])
        c = np.clip(j - pre, 0, mask.shape[2] - 1)
        seen = seen & ((j < pre) | (mask[b][i, c] != 0))
    return seen


def reference(p, rows=None):
    """out, lse [T, Hq(, 128)] and their tolerances, in float64.

    Tolerance of an element, from the arithmetic: the final rounding to bf16
    (2^-8 |out|) and, with chunks, the partial rows' (2^-8 sum p|v|); P in fp16
    (2^-11 sum p|v|, and 2^-25 per position below the normal range, the largest
    p being at least 1 / 256 of the row sum's scale); a score error d changes
    every p by at most a factor e^(2d): d = sm_scale * (2^-11 where Q' is rounded
    to fp16 after a per-channel scale, and 2^-14 for 128 additions in fp32) *
    sum |q k|, plus 2^-20 for exp2, log2 and the running maximum; sums over L
    positions in fp32 add L * 2^-22 of their terms' magnitude (L * 2^-24 in lse)."""
    G = p.q_heads // p.kv_heads
    T = p.total_q
    out, lse = np.zeros((T, p.q_heads, 128)), np.full((T, p.q_heads), -np.inf)
    tol_o, tol_l = np.zeros(out.shape), np.zeros(lse.shape)
    rows = rows or (lambda w, b, h, n: kv4.rows(p, w, b, h, n))
    for b in range(p.bsz):
        t0, t1 = int(p.cu_seqlens_q[b]), int(p.cu_seqlens_q[b + 1])
        if t0 == t1:
            continue
        seen, L = seen_mask(p, b), int(p.held[b])
        for h in range(p.kv_heads):
            q = kv4.bf16_to_f64(p.q_bits[t0:t1, h * G * 128:(h + 1) * G * 128]).reshape(t1 - t0, G, 128)
            V = rows("v", b, h, L)
            o, l, absv, mag = kv4.attend(q, rows("k", b, h, L), V, seen, p.sm_scale)
            # up to 16 rows over a 4-bit cache Q' times a per-channel scale is two fp16 numbers
            one_fp16 = p.scale_kind == "per_channel" and (int(max(p.seq_lens)) * G > 16 or p.kv_dtype not in KINDS)
            c = (2.0 ** -11 if one_fp16 else 0.0) + 2.0 ** -14
            d = p.sm_scale * c * mag + 2.0 ** -20
            sl = np.s_[t0:t1, h * G:(h + 1) * G]
            out[sl], lse[sl] = o, l
            tol_o[sl] = (2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -11 + 2 * d[..., None] + L * 2.0 ** -22) * absv
                         + L * 2.0 ** -25 * np.abs(V).max(initial=0.0) + 1e-30)
            tol_l[sl] = d + L * 2.0 ** -24 + 2.0 ** -20 * np.abs(np.where(np.isfinite(l), l, 0.0)) + 2.0 ** -20
    return out, lse, tol_o, tol_l


def device(p):
    import torch
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    raw = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    sc = raw if p.scale_kind == "global" else bf
    d = dict(q=bf(p.q_bits), cache_k=raw(p.cache_k), cache_v=raw(p.cache_v), k_scale=sc(p.k_scale),
             v_scale=sc(p.v_scale), block_table=raw(p.block_table), seq_lens=raw(p.seq_lens),
             seq_lens_kv=raw(p.seq_lens_kv), cu_seqlens_q=raw(p.cu_seqlens_q))
    if hasattr(p, "k_new"):
        d.update(k_new=bf(p.k_new), v_new=bf(p.v_new))
    # one row behind the last token: left as it was
    d["out_all"] = torch.full((p.total_q + 1, p.q_heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    d["lse_all"] = torch.full((p.total_q + 1, p.q_heads), 7.0, device="cuda")
    d["out"], d["lse"] = d["out_all"][:-1], d["lse_all"][:-1]
    if getattr(p, "attn_mask", None) is not None:
        d["attn_mask"] = raw(p.attn_mask.astype(np.uint8))
    return d


def plan_of(pa, p, sms=None):
    from gpu_helpers import num_sms
    return pa.pa_plan(problem(pa, p), p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q, sms or num_sms())


def args_of(pa, d, **kw):
    names = ("q", "cache_k", "cache_v", "k_scale", "v_scale", "block_table", "out", "lse", "seq_lens", "seq_lens_kv",
             "cu_seqlens_q")
    return pa.make_args(**{n: d[n] for n in names}, **{"attn_mask": d.get("attn_mask"), **kw})


def workspace(plan, fill=0xFF):
    import torch
    return torch.full((max(plan.workspace_size, 256),), fill, dtype=torch.uint8, device="cuda")


def run(p, d=None, sms=None, **kw):
    """Plan, upload, run, merge and check; (out, lse) as float64 arrays and the tensors."""
    import paged_quantized_kv_gqa_gb300 as pa
    d = d or device(p)
    plan = plan_of(pa, p, sms)
    ws = workspace(plan)
    args = args_of(pa, d, **kw)
    pa.pa_plan_upload(plan, ws)
    pa.pa_run(plan, args, ws)
    pa.pa_merge(plan, args, ws)
    st, det = pa.pa_check(plan, ws)
    assert st == 0, (st, det, pa.pa_last_error())
    assert bool((d["out_all"][-1] == 7).all()) and bool((d["lse_all"][-1] == 7).all()), "row behind the last token"
    return d["out"].float().cpu().numpy().astype(np.float64), d["lse"].cpu().numpy().astype(np.float64), d, plan


def check(p, out, lse, ref=None):
    ro, rl, to, tl = ref or reference(p)
    assert np.isfinite(out).all(), "non-finite output"
    err = np.abs(out - ro) / to
    assert err.max(initial=0.0) <= 1.0, f"out: {err.max():.2f} of the tolerance at {np.argwhere(err > 1)[:3].tolist()}"
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl)), "rows without a position"
    with np.errstate(invalid="ignore"):
        el = np.where(np.isneginf(rl), 0.0, np.abs(lse - rl) / tl)
    assert el.max(initial=0.0) <= 1.0, f"lse: {el.max():.2f} of the tolerance"
    print(f"out {err.max(initial=0.0):.3f}, lse {el.max(initial=0.0):.3f} of the tolerance")
