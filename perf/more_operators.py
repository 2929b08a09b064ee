"""Measured cases of the operators around latent attention and the rotated append.

Five operators, reached through the package's public calls:

  rope     the step before attention: queries rotated by their positions, new K / V
           rows rotated (K), quantised and written into the paged cache
           (pa_rope_append), and the stored values read back (pa_cache_read).
           Positions may have several axes (time, height, width)
  absorb   latent attention, absorbed form: queries taken into the latent space
           (pa_mla_absorb), q'[t][h] = [q_nope[t][h] W_k[h], q_rope[t][h]]
  project  its outputs taken out of it (pa_mla_project), o[t][h] = W_v[h] o'[t][h]
  expand   latent attention, expanded form: the keys and values of every head from
           latent rows (pa_mla_expand), k[n][h] = W_k[h] c[n], v[n][h] = W_v[h] c[n]
  prefill  attention of new tokens to expanded rows (pa_mla_prefill, pa_merge): keys
           of 128 dims a head and 64 rotated ones that all heads share, values of 128

One weight serves absorb, project and expand: [heads][256][512], the rows of a head
being 128 of W_k and 128 of W_v.

Rotation of a pair (a, b) by cos c and sin s of its angle, from a table in 32 bits,
every product and sum rounded to 32 bits:  a c - b s,  b c + a s.
Pairs of a width r: dims (i, i + r / 2) ("halves") or (2i, 2i + 1) ("adjacent").
Grouped heads rotate the first r of their 128 dims; latent rows (576 wide) the dims
from 512 on, and the queries to them (192 a head) those from 128 on.

Stored values, x rotated, s its scale, in 32 bits, ties to even:
  int8      round(x / s), at most 127 either way
  fp8_e4m3  E4M3(x / s), at most 448 either way
  int4, fp4_e2m1  per block of 16 dims: e = E4M3(min(max |x / s| / M, 448)), M = 7 or 6,
            step = e s, code = nearest to x / step, at most M either way
Pages hold 64 positions: 8-bit K [page][head][64][128], V [page][head][128][64];
latent rows [page][64][576]; 4-bit K and V slabs of 4608 bytes a (page, head), two half
pages of 32 positions: K codes [32][64] then scales [32][8], V codes [128][16] then
scales [8][32], two codes a byte, the lower first.
"""
import math
import random

import torch

own = False

DIM, PAGE, HALF, BLK = 128, 64, 32, 16
NBLK = DIM // BLK
KCODES = HALF * DIM // 2
HBYTES = KCODES + HALF * NBLK
SLAB = 2 * HBYTES
NOPE, ROPE, LAT = 128, 64, 512            # latent attention: key dims, rotated dims, latent
QW, LW, MLA_HEADS = NOPE + ROPE, LAT + ROPE, 128
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TOP = {"int8": 127.0, "fp8_e4m3": 448.0, "int4": 7.0, "fp4_e2m1": 6.0}


# ---------------------------------------------------------------- the cases
def listed():
    c = []
    # a full decode batch of chat lengths: one token a sequence, latency counts
    c.append(dict(name="rope_step", op="rope", layout="gqa", kv="int8", scale="per_channel", bsz=64, q_lo=1, q_hi=1,
                  kv_lo=512, kv_hi=4096, heads=32, kv_heads=8, rot=128, pairs="halves", axes=1, split=0, pad=0, lens=1))
    # prompts of text and images, positions of three axes, packed qkv rows
    c.append(dict(name="rope_prompts_axes", op="rope", layout="gqa", kv="fp4_e2m1", scale="per_kv_head", bsz=8, q_lo=1024,
                  q_hi=8192, kv_lo=0, kv_hi=200, heads=32, kv_heads=8, rot=128, pairs="halves", axes=3, split=2, pad=1,
                  lens=2))
    # chunks of prompts of a latent-attention model: its queries and latent rows
    c.append(dict(name="rope_latent", op="rope", layout="mla", kv="fp8_e4m3", scale="global", bsz=8, q_lo=64, q_hi=512,
                  kv_lo=0, kv_hi=8192, heads=MLA_HEADS, kv_heads=1, rot=64, pairs="adjacent", axes=1, split=0, pad=0,
                  lens=3))
    # one decode step's queries: the weights are what is read
    c.append(dict(name="absorb_step", op="absorb", rows=48, heads=128, pad=0))
    # a verification batch of an odd number of tokens
    c.append(dict(name="absorb_verify", op="absorb", rows=777, heads=128, pad=64))
    # three tokens on one of eight shares of the heads: the call's latency
    c.append(dict(name="project_short", op="project", rows=3, heads=16, pad=0))
    # a verification batch
    c.append(dict(name="project_verify", op="project", rows=777, heads=128, pad=0))
    # a short odd run of rows read from the cache, one share of the heads
    c.append(dict(name="expand_short", op="expand", rows=333, heads=16, pad=64))
    # the latent rows of a prefill batch, every head
    c.append(dict(name="expand_prompts", op="expand", rows=8192, heads=128, pad=64))
    # one short prompt behind a short prefix, one share of the heads
    c.append(dict(name="prefill_short", op="prefill", mask="causal", bsz=1, q_lo=77, q_hi=77, kv_lo=130, kv_hi=130,
                  heads=16, pad=0, lens=4))
    # whole prompts of different lengths
    c.append(dict(name="prefill_prompts", op="prefill", mask="causal", bsz=4, q_lo=512, q_hi=2048, kv_lo=0, kv_hi=0,
                  heads=128, pad=0, lens=5))
    # a chunk of new tokens against long cached ranges, to be joined by its lse; one empty
    c.append(dict(name="prefill_cached", op="prefill", mask="cross", bsz=4, q_lo=128, q_hi=512, kv_lo=0, kv_hi=8192,
                  heads=32, pad=64, lens=6))
    return c


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = [work(c) for c in listed()]
    bytes_max, flops_max = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        op = rng.choice(["rope", "rope", "absorb", "project", "expand", "prefill", "prefill"])
        pad = rng.choice([0, 0, 8, 64])
        if op == "rope":
            mla = rng.random() < 0.3
            hi = _log_int(rng, 1, 4096 if mla else 8192)
            axes = rng.choice([1, 1, 2, 3])
            kv_heads = 1 if mla else rng.choice([1, 2, 3, 4, 8, 16])
            case = dict(op=op, layout="mla" if mla else "gqa",
                        kv=rng.choice(["int8", "fp8_e4m3"] if mla else list(TOP)),
                        scale="global" if mla else rng.choice(["global", "per_kv_head", "per_channel"]),
                        bsz=_log_int(rng, 1, 64), q_lo=max(1, hi // rng.choice([1, 2, 5, 9])), q_hi=hi, kv_lo=0,
                        kv_hi=rng.choice([0, 77, 200, 4096]), kv_heads=kv_heads,
                        heads=MLA_HEADS if mla else kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8]),
                        rot=rng.choice([32, 48, 64] if mla else [32, 64, 80, 96, 128, 128]),
                        pairs=rng.choice(["halves", "adjacent"]), axes=axes, split=rng.randrange(3), pad=rng.randrange(2),
                        lens=rng.randrange(1 << 30))
        elif op == "prefill":
            mask = rng.choice(["causal", "causal", "full", "cross"])
            q, kv = _log_int(rng, 1, 2048), rng.choice([0, _log_int(rng, 1, 8192)])
            case = dict(op=op, mask=mask, bsz=_log_int(rng, 1, 8), q_lo=max(1, q // rng.choice([1, 2, 6])), q_hi=q,
                        kv_lo=kv // rng.choice([1, 2, 8]), kv_hi=kv, heads=rng.choice([1, 2, 5, 8, 16, 20, 32, 64, 128]),
                        pad=pad, lens=rng.randrange(1 << 30))
            # what the plain form holds at once: padded scores
            if case["bsz"] * q * (q + kv) * case["heads"] > 2_200_000_000:
                continue
        else:
            case = dict(op=op, rows=_log_int(rng, 1, 8192 if op == "expand" else 2048),
                        heads=rng.choice([1, 2, 5, 8, 16, 20, 32, 64, 128]), pad=pad)
        w = work(case)
        if w["bytes"] <= bytes_max and w["flops"] <= flops_max:
            return case


# ---------------------------------------------------------------- lengths, floors
def _lens(case):
    r = random.Random(case["lens"])
    ql = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["bsz"])]
    kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["bsz"])]
    if case.get("mask") == "cross" and case["bsz"] > 2:
        kv[1] = 0                                     # one sequence without rows
    return ql, kv


def _held(case):
    ql, kv = _lens(case)
    return kv if case.get("mask") == "cross" else [a + b for a, b in zip(ql, kv)]


def work(case):
    op, h = case["op"], case["heads"]
    if op == "absorb":
        return {"bytes": case["rows"] * h * (QW + LW) * 2 + h * NOPE * LAT * 2, "flops": 2.0 * case["rows"] * h * NOPE * LAT}
    if op == "project":
        return {"bytes": case["rows"] * h * (LAT + DIM) * 2 + h * DIM * LAT * 2, "flops": 2.0 * case["rows"] * h * DIM * LAT}
    if op == "expand":
        return {"bytes": case["rows"] * (LAT + h * (NOPE + DIM)) * 2 + h * (NOPE + DIM) * LAT * 2,
                "flops": 2.0 * case["rows"] * h * (NOPE + DIM) * LAT}
    ql, kv = _lens(case)
    T = sum(ql)
    if op == "prefill":
        n = sum(_held(case))
        if case["mask"] == "cross":
            pairs = sum(q * k for q, k in zip(ql, kv))
        elif case["mask"] == "full":
            pairs = sum(q * (q + k) for q, k in zip(ql, kv))
        else:
            pairs = sum(q * k + q * (q + 1) // 2 for q, k in zip(ql, kv))
        return {"bytes": T * h * ((QW + DIM) * 2 + 4) + n * (h * (NOPE + DIM) + ROPE) * 2,
                "flops": 2.0 * (QW + DIM) * pairs * h}
    # rows in, rotated queries, stored bytes and read values out
    rot = case["rot"]
    if case["layout"] == "mla":
        return {"bytes": T * (h * QW * 4 + LW * 5 + rot * 4), "flops": 3.0 * T * (h + 1) * rot + 4.0 * T * LW}
    row = case["kv_heads"] * DIM * 2
    stored = row * (1.0 if case["kv"] in ("int8", "fp8_e4m3") else 0.5 + 1.0 / BLK)
    return {"bytes": T * (h * DIM * 4 + row * 4 + stored + rot * 4),
            "flops": 3.0 * T * (h + case["kv_heads"]) * rot + 4.0 * T * row}


# ---------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


def _padded(x, pad):
    """The same rows in a wider tensor: [rows][width + pad], and its view of `width`."""
    wide = torch.zeros((x.shape[0], x.shape[1] + pad), dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _pair_axes(case):
    """The axis of every pair: runs of pairs, or the axes in turn."""
    n, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return [0] * n
    if case["split"] == 0:                            # axes in turn
        return [i % axes for i in range(n)]
    first = n // (2 * case["split"])                  # a shorter or longer run of the first, the rest shared out
    rest = n - first
    return [0] * first + [1 + i * (axes - 1) // rest for i in range(rest)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, gen)
    st = dict(case=case)
    h, pad = case["heads"], case["pad"]
    if case["op"] == "prefill":
        ql, kv = _lens(case)
        held = _held(case)
        T, N = sum(ql), sum(held)
        st.update(q_lens=ql, kv_lens=kv, held=held, scale=QW ** -0.5,
                  q=_padded(_randn(gen, T, h * QW), pad),
                  k=_padded(_randn(gen, max(N, 1), h * NOPE), pad), v=_padded(_randn(gen, max(N, 1), h * DIM), pad),
                  k_rope=_padded(_randn(gen, max(N, 1), ROPE), pad),
                  q_lens_d=torch.tensor(ql, device="cuda"), kv_lens_d=torch.tensor(kv, device="cuda"),
                  held_d=torch.tensor(held, device="cuda"),
                  out=torch.empty((T, h, DIM), dtype=torch.bfloat16, device="cuda"), lse=torch.empty((T, h), device="cuda"))
        if own:
            import paged_quantized_kv_gqa_gb300 as pa
            st["pa"] = pa
            prob = pa.make_problem(bsz=case["bsz"], q_heads=h, kv_heads=h, head_dim_qk=QW, head_dim_v=DIM, kv_dtype="bf16",
                                   layout="mla_expanded", causal=case["mask"] == "causal", cross=case["mask"] == "cross",
                                   chunk_size=-1, sm_scale=st["scale"], q_stride=h * QW + pad)
            cu = [sum(ql[:i]) for i in range(len(ql) + 1)]
            st["plan"] = pa.pa_plan(prob, ql, kv, cu, torch.cuda.get_device_properties(0).multi_processor_count)
            st["ws"] = torch.empty(st["plan"].workspace_size, dtype=torch.uint8, device="cuda")
            pa.pa_plan_upload(st["plan"], st["ws"])
            st["args"] = pa.make_args(q=st["q"], cache_k=None, cache_v=None, k_scale=None, v_scale=None, block_table=None,
                                      out=st["out"], lse=st["lse"])
        return st
    n = case["rows"]
    # weights of a trained projection's size: outputs of about unit variance
    width = NOPE if case["op"] == "absorb" else LAT
    st["w"] = (torch.randn((h, NOPE + DIM, LAT), generator=gen, device="cuda") * width ** -0.5).bfloat16()
    if case["op"] == "absorb":
        st["x"] = _padded(_randn(gen, n, h * QW), pad)
        st["out"] = torch.empty((n, h, LW), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "project":
        st["x"] = _padded(_randn(gen, n, h * LAT), pad)
        st["out"] = torch.empty((n, h, DIM), dtype=torch.bfloat16, device="cuda")
    else:
        st["x"] = _padded(_randn(gen, n, LAT), pad)
        st["k"] = torch.empty((n, h, NOPE), dtype=torch.bfloat16, device="cuda")
        st["v"] = torch.empty((n, h, DIM), dtype=torch.bfloat16, device="cuda")
    if own:
        import paged_quantized_kv_gqa_gb300 as pa
        st["pa"] = pa
        st["ws"] = torch.zeros(pa.PA_STATUS_BYTES, dtype=torch.uint8, device="cuda")   # where a kernel reports errors
    return st


def _prepare_rope(case, gen):
    ql, kv = _lens(case)
    h, hk, bsz, T, mla = case["heads"], case["kv_heads"], case["bsz"], sum(ql), case["layout"] == "mla"
    held = _held(case)
    pages = [-(-n // PAGE) for n in held]
    num_pages, mb = sum(pages) + 3, max(pages)
    order = torch.randperm(num_pages, generator=gen, device="cuda").int()
    bt, at = torch.full((bsz, mb), -1, dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(pages):
        bt[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in ql:
        cu.append(cu[-1] + n)
    st = dict(case=case, block_table=bt, q_lens=ql, kv_lens=kv, seq_lens=torch.tensor(ql, dtype=torch.int32, device="cuda"),
              seq_lens_kv=torch.tensor(kv, dtype=torch.int32, device="cuda"),
              cu_seqlens_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    tok_b = torch.repeat_interleave(torch.arange(bsz, device="cuda"), st["seq_lens"].long())
    st["tok_b"] = tok_b
    st["pos"] = st["seq_lens_kv"].long()[tok_b] + torch.arange(T, device="cuda") - st["cu_seqlens_q"].long()[tok_b]
    # positions of the first axis count the tokens; the others are places within an image
    last = max(held)
    st["positions"] = torch.cat([st["pos"].int()[None], torch.randint(0, min(last, 300), (case["axes"] - 1, T), generator=gen,
                                                                       device="cuda").int()])
    st["pair_axes"] = _pair_axes(case)
    n = case["rot"] // 2
    angle = torch.arange(last, dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    fmt = {"int8": 0.02, "fp8_e4m3": 0.01, "int4": 0.3, "fp4_e2m1": 0.3}[case["kv"]]   # values within the format's range
    for side in ("k", "v"):
        if case["scale"] == "global":
            s = torch.full((1,), 1.1 * fmt, device="cuda")
        else:
            s = ((torch.rand(hk if case["scale"] == "per_kv_head" else hk * DIM, generator=gen, device="cuda") + 1.0)
                 * fmt).bfloat16()
        st[side + "_scale"] = s
    if case["scale"] == "global":
        st["v_scale"] = st["k_scale"]
    if mla:
        st["q"] = _padded(_randn(gen, T, h * QW), 0)
        st["k_new"], st["v_new"] = _padded(_randn(gen, T, LW), 64 * case["pad"]), None
        st["cache_k"] = torch.zeros((num_pages, PAGE, LW), dtype=torch.uint8, device="cuda")
        st["cache_v"] = st["cache_k"]
    else:
        if case["pad"]:                               # one packed row of q, k and v a token
            qkv = _randn(gen, T, (h + 2 * hk) * DIM)
            st["q"], st["k_new"], st["v_new"] = qkv[:, :h * DIM], qkv[:, h * DIM:(h + hk) * DIM], qkv[:, (h + hk) * DIM:]
        else:
            st["q"], st["k_new"], st["v_new"] = (_randn(gen, T, k * DIM) for k in (h, hk, hk))
        four = case["kv"] in ("int4", "fp4_e2m1")
        for side in ("k", "v"):
            shape = (SLAB,) if four else (PAGE, DIM) if side == "k" else (DIM, PAGE)
            st["cache_" + side] = torch.zeros((num_pages, hk) + shape, dtype=torch.uint8, device="cuda")
    st["q_out"] = torch.empty((T, st["q"].shape[1]), dtype=torch.bfloat16, device="cuda")
    width = LW if mla else hk * DIM
    st["k_out"] = torch.empty((T, width), dtype=torch.bfloat16, device="cuda")
    st["v_out"] = None if mla else torch.empty_like(st["k_out"])
    if own:
        import paged_quantized_kv_gqa_gb300 as pa
        st["pa"] = pa
        prob = pa.make_problem(bsz=bsz, q_heads=h, kv_heads=hk, head_dim_qk=LW if mla else DIM, head_dim_v=LAT if mla else DIM,
                               block_size=PAGE, max_blocks_per_seq=mb, num_pages=num_pages, kv_dtype=case["kv"],
                               scale_kind=case["scale"], layout=case["layout"], causal=True, chunk_size=-1,
                               sm_scale=(QW if mla else DIM) ** -0.5, q_stride=h * (LW if mla else DIM))
        st["plan"] = pa.pa_plan(prob, ql, kv, cu, torch.cuda.get_device_properties(0).multi_processor_count)
        st["ws"] = torch.empty(st["plan"].workspace_size, dtype=torch.uint8, device="cuda")
        pa.pa_plan_upload(st["plan"], st["ws"])
        st["args"] = pa.make_args(q=None, cache_k=st["cache_k"], cache_v=st["cache_v"], k_scale=st["k_scale"],
                                  v_scale=st["v_scale"], block_table=bt, out=None, seq_lens=st["seq_lens"],
                                  seq_lens_kv=st["seq_lens_kv"], cu_seqlens_q=st["cu_seqlens_q"])
        st["rope"] = pa.make_rope(cos_sin=st["cos_sin"], table_rows=last, rot_dim=case["rot"], pairs=case["pairs"],
                                  positions=st["positions"] if case["axes"] > 1 else None, axes=case["axes"],
                                  pair_axes=st["pair_axes"])
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state)
    if op == "rope":
        return _rope(state)
    if op == "prefill":
        return _prefill(state)
    h, x, w = case["heads"], state["x"].float(), state["w"].float()
    if op == "absorb":
        x = x.unflatten(1, (h, QW))
        y = torch.matmul(x[..., :NOPE].transpose(0, 1), w[:, :NOPE]).transpose(0, 1)
        return {"q": torch.cat([y, x[..., NOPE:]], -1).bfloat16()}
    if op == "project":
        y = torch.matmul(x.unflatten(1, (h, LAT)).transpose(0, 1), w[:, NOPE:].transpose(1, 2)).transpose(0, 1)
        return {"o": y.bfloat16()}
    y = torch.matmul(x, w.flatten(0, 1).t()).unflatten(1, (h, NOPE + DIM))
    return {"k": y[:, :, :NOPE].bfloat16(), "v": y[:, :, NOPE:].bfloat16()}


def _run_own(state):
    pa, case = state["pa"], state["case"]
    op, h = case["op"], case["heads"]
    if op == "rope":
        k = state["k_new"]
        pa.pa_rope_append(state["plan"], state["args"], state["rope"], state["q"], state["q"].stride(0), state["q_out"],
                          state["q_out"].stride(0), k, state["v_new"], k.stride(0), state["ws"])
        pa.pa_cache_read(state["plan"], state["args"], state["k_out"], state["v_out"], state["k_out"].stride(0), state["ws"])
        got = {"q": state["q_out"], "k": state["k_out"]}
        return got if state["v_out"] is None else dict(got, v=state["v_out"])
    if op == "prefill":
        pa.pa_mla_prefill(state["plan"], state["args"], state["k"], state["v"], state["k"].stride(0), state["k_rope"],
                          state["k_rope"].stride(0), state["ws"])
        pa.pa_merge(state["plan"], state["args"], state["ws"])
        return {"out": state["out"], "lse": state["lse"]}
    x, w, n = state["x"], state["w"], case["rows"]
    if op == "absorb":
        pa.pa_mla_absorb(n, h, x, x.stride(0), w, w.stride(0), state["out"], state["out"].stride(0), state["ws"])
        return {"q": state["out"]}
    if op == "project":
        pa.pa_mla_project(n, h, x, x.stride(0), w[:, NOPE:], w.stride(0), state["out"], state["out"].stride(0), state["ws"])
        return {"o": state["out"]}
    pa.pa_mla_expand(n, h, x, x.stride(0), w, w.stride(0), state["k"], state["v"], state["k"].stride(0), state["ws"])
    return {"k": state["k"], "v": state["v"]}


def _prefill(state):
    """Scores of the padded batch, sequences side by side."""
    case, h, bsz = state["case"], state["case"]["heads"], state["case"]["bsz"]
    Q, L = max(state["q_lens"]), max(1, max(state["held"]))
    i, j = torch.arange(Q, device="cuda"), torch.arange(L, device="cuda")
    real, held = i < state["q_lens_d"][:, None], j < state["held_d"][:, None]            # [bsz][Q], [bsz][L]
    q0, k0 = state["q_lens_d"].cumsum(0) - state["q_lens_d"], state["held_d"].cumsum(0) - state["held_d"]
    qi = (q0[:, None] + i).clamp(max=state["q"].shape[0] - 1)
    ki = (k0[:, None] + j).clamp(max=state["k"].shape[0] - 1)
    q = state["q"].float()[qi].unflatten(2, (h, QW)).transpose(1, 2)
    k = state["k"].float()[ki].unflatten(2, (h, NOPE)).transpose(1, 2)
    v = state["v"].float()[ki].unflatten(2, (h, DIM)).transpose(1, 2)
    kr = state["k_rope"].float()[ki][:, None]
    S = (torch.matmul(q[..., :NOPE], k.transpose(2, 3)) + torch.matmul(q[..., NOPE:], kr.transpose(2, 3))) * state["scale"]
    seen = held[:, None, :].expand(bsz, Q, L)
    if case["mask"] == "causal":
        seen = seen & (j <= (state["kv_lens_d"][:, None] + i)[..., None])
    S.masked_fill_(~seen[:, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    P = S.sub_(m).exp_()
    total = P.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    O = torch.matmul(P, v * held[:, None, :, None]) / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": O.transpose(1, 2)[real].bfloat16(), "lse": lse.transpose(1, 2)[real]}


def _angles(state):
    """cos and sin of every token's pairs, [T][rot / 2] each."""
    n = state["case"]["rot"] // 2
    axis = torch.tensor(state["pair_axes"], device="cuda")
    row = state["positions"].long()[axis].t()                                            # [T][pairs]
    pair = torch.arange(n, device="cuda").expand_as(row)
    return state["cos_sin"][row, pair], state["cos_sin"][row, pair + n]


def _rotate(x, cos, sin, pairs, first):
    """Rows [T][heads][dims] in 32 bits, rotated from dim `first` on."""
    n = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    y, part = x.clone(), x[..., first:first + 2 * n]
    if pairs == "halves":
        a, b, out = part[..., :n], part[..., n:], y[..., first:first + 2 * n]
        out[..., :n], out[..., n:] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b, out = part[..., 0::2], part[..., 1::2], y[..., first:first + 2 * n]
        out[..., 0::2], out[..., 1::2] = a * cos - b * sin, b * cos + a * sin
    return y


def _scales(case, s):
    """The tensor's scale of every kv head and dim, in 32 bits."""
    if case["layout"] == "mla":
        return s.float().expand(1, LW)
    if case["scale"] == "per_channel":
        return s.float().view(case["kv_heads"], DIM)
    return s.float().reshape(-1, 1).expand(case["kv_heads"], DIM)


def _codes8(x, g, kind):
    y = x / g
    if kind == "int8":
        return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _values8(b, kind):
    return b.view(torch.int8 if kind == "int8" else torch.float8_e4m3fn).float()


def _codes4(x, g, kind):
    """Rows [..., 128] -> codes [..., 128], block scales [..., 8] as E4M3 bytes."""
    blocks = x.unflatten(-1, (NBLK, BLK))
    y = (x / g).unflatten(-1, (NBLK, BLK))
    # a tensor as divisor: by a Python number, torch multiplies with a rounded reciprocal
    s = (y.abs().amax(-1) / torch.tensor(TOP[kind], device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s.float()[..., None] * g.expand_as(x).unflatten(-1, (NBLK, BLK))
    q = torch.where(step > 0, blocks / step, torch.zeros_like(step))
    if kind == "int4":
        codes = (q.round().clamp(-7, 7).to(torch.int8) & 15).to(torch.uint8)
    else:
        a = q.abs()
        mag = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
        codes = (mag + 8 * torch.signbit(q)).to(torch.uint8)
    return codes.flatten(-2), s.view(torch.uint8)


def _values4(codes, s, kind):
    t = (LEVELS + [-x for x in LEVELS]) if kind == "fp4_e2m1" else [float(i - 16 * (i > 7)) for i in range(16)]
    v = torch.tensor(t, device=codes.device)[codes.int()].unflatten(-1, (NBLK, BLK))
    return v, s.contiguous().view(torch.float8_e4m3fn).float()[..., None]


def _pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _unpack(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _rope(state):
    case, kind = state["case"], state["case"]["kv"]
    cos, sin = _angles(state)
    mla, h, hk = case["layout"] == "mla", case["heads"], case["kv_heads"]
    page = state["block_table"][state["tok_b"], state["pos"] // PAGE].long()
    off = state["pos"] % PAGE
    g = _scales(case, state["k_scale"])
    if mla:
        q = _rotate(state["q"].float().unflatten(1, (h, QW)), cos, sin, case["pairs"], NOPE)
        k = _rotate(state["k_new"].float()[:, None], cos, sin, case["pairs"], LAT)
        state["cache_k"][page, off] = _codes8(k, g, kind)[:, 0]
        return {"q": q.flatten(1).bfloat16(), "k": (_values8(state["cache_k"][page, off], kind) * g).bfloat16()}
    q = _rotate(state["q"].float().unflatten(1, (h, DIM)), cos, sin, case["pairs"], 0)
    k = _rotate(state["k_new"].float().unflatten(1, (hk, DIM)), cos, sin, case["pairs"], 0)
    v, gv = state["v_new"].float().unflatten(1, (hk, DIM)), _scales(case, state["v_scale"])
    ck, cv = state["cache_k"], state["cache_v"]
    if kind in ("int8", "fp8_e4m3"):
        ck[page, :, off] = _codes8(k, g, kind)
        cv[page, :, :, off] = _codes8(v, gv, kind)
        k, v = _values8(ck[page, :, off], kind) * g, _values8(cv[page, :, :, off], kind) * gv
    else:
        half, r = off // HALF, off % HALF
        kh, vh = (c.view(c.shape[0], hk, 2, HBYTES) for c in (ck, cv))
        kc, ks = kh[..., :KCODES].unflatten(-1, (HALF, DIM // 2)), kh[..., KCODES:].unflatten(-1, (HALF, NBLK))
        vc, vs = vh[..., :KCODES].unflatten(-1, (DIM, HALF // 2)), vh[..., KCODES:].unflatten(-1, (NBLK, HALF))
        codes, s = _codes4(k, g, kind)
        kc[page, :, half, r], ks[page, :, half, r] = _pack(codes), s
        codes, s = _codes4(v, gv, kind)
        nibbles = _unpack(vc)
        nibbles[page, :, half, :, r] = codes
        vc.copy_(_pack(nibbles))
        vs[page, :, half, :, r] = s
        val, s = _values4(_unpack(kc[page, :, half, r]), ks[page, :, half, r], kind)
        k = (val * (s * g.unflatten(-1, (NBLK, BLK)))).flatten(-2)
        val, s = _values4(_unpack(vc)[page, :, half, :, r], vs[page, :, half, :, r], kind)
        v = (val * (s * gv.unflatten(-1, (NBLK, BLK)))).flatten(-2)
    return {"q": q.flatten(1).bfloat16(), "k": k.flatten(1).bfloat16(), "v": v.flatten(1).bfloat16()}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, h = case["op"], case["heads"]
    if op == "prefill":
        return _exact_prefill(st)
    if op == "rope":
        return _exact_rope(st)
    x, w = st["x"].double(), st["w"].double()
    if op == "absorb":
        x = x.reshape(-1, h, QW)
        y = torch.empty(x.shape[0], h, LW, dtype=torch.float64, device="cuda")
        y[..., LAT:] = x[..., NOPE:]
        for i in range(h):
            y[:, i, :LAT] = x[:, i, :NOPE] @ w[i, :NOPE]
        return {"q": y}
    if op == "project":
        x = x.reshape(-1, h, LAT)
        return {"o": torch.stack([x[:, i] @ w[i, NOPE:].T for i in range(h)], 1)}
    return {"k": torch.stack([x @ w[i, :NOPE].T for i in range(h)], 1),
            "v": torch.stack([x @ w[i, NOPE:].T for i in range(h)], 1)}


def _exact_prefill(st):
    case, h = st["case"], st["case"]["heads"]
    outs, lses, t, n = [], [], 0, 0
    for ql, prefix, held in zip(st["q_lens"], st["kv_lens"], st["held"]):
        q = st["q"][t:t + ql].double().reshape(ql, h, QW)
        k, v = (st[s][n:n + held].double().reshape(held, h, DIM) for s in ("k", "v"))
        kr = st["k_rope"][n:n + held].double()
        o = torch.zeros(ql, h, DIM, dtype=torch.float64, device="cuda")
        lse = torch.full((ql, h), -math.inf, dtype=torch.float64, device="cuda")
        late = torch.arange(held, device="cuda") > prefix + torch.arange(ql, device="cuda")[:, None]
        for i in range(h if held else 0):
            s = torch.cat([q[:, i, :NOPE], q[:, i, NOPE:]], 1) @ torch.cat([k[:, i], kr], 1).T / math.sqrt(QW)
            if case["mask"] == "causal":
                s = s.masked_fill(late, -math.inf)
            lse[:, i] = torch.logsumexp(s, -1)
            o[:, i] = torch.exp(s - lse[:, i, None]) @ v[:, i]
        outs.append(o)
        lses.append(lse)
        t, n = t + ql, n + held
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _fl(x):
    """Rounded to 32 bits: exact here, where 64 bits hold a product of two 32-bit
    numbers whole and round their sums and quotients far below 32 bits' last place."""
    return x.float().double()


def _exact_rope(st):
    case = st["case"]
    T, n, mla = st["q"].shape[0], case["rot"] // 2, case["layout"] == "mla"
    table = st["cos_sin"].double()
    c, s = (torch.empty(T, n, dtype=torch.float64, device="cuda") for _ in range(2))
    for p, axis in enumerate(st["pair_axes"]):
        row = st["positions"][axis].long()
        c[:, p], s[:, p] = table[row, p], table[row, n + p]
    i = torch.arange(n, device="cuda")
    a_dim, b_dim = (i, i + n) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)

    def turned(x, first):
        y, a, b = x.double(), x[..., first + a_dim].double(), x[..., first + b_dim].double()
        cc, ss = c[:, None], s[:, None]
        y[..., first + a_dim], y[..., first + b_dim] = _fl(_fl(a * cc) - _fl(b * ss)), _fl(_fl(b * cc) + _fl(a * ss))
        return y

    def kept(x, g):
        if case["kv"] == "int8":
            return _fl(x / g).round().clamp(-127, 127) * g
        if case["kv"] == "fp8_e4m3":
            e = torch.arange(127, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
            y = _fl(x / g)
            return torch.sign(y) * _nearest(y.abs().clamp(max=448.0), e) * g
        blocks = lambda t: t.reshape(*t.shape[:-1], NBLK, BLK)  # noqa: E731
        grid = torch.tensor(LEVELS if case["kv"] == "fp4_e2m1" else [float(k) for k in range(8)], dtype=torch.float64,
                            device="cuda")
        e = torch.arange(127, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        gg = g.expand_as(x)
        top = _fl(blocks(x / gg)).abs().amax(-1)
        bs = _nearest(_fl(top / grid[-1]).clamp(max=448.0), e)
        step = _fl(bs[..., None] * blocks(gg))
        q = torch.where(step > 0, _fl(blocks(x) / step), torch.zeros_like(step))
        return (torch.sign(q) * _nearest(q.abs().clamp(max=float(grid[-1])), grid) * bs[..., None] * blocks(gg)).reshape(x.shape)

    h, hk = case["heads"], case["kv_heads"]
    if mla:
        q = turned(st["q"].reshape(T, h, QW), NOPE)
        k = kept(turned(st["k_new"].reshape(T, 1, LW), LAT), st["k_scale"].double())
        return {"q": q.reshape(T, -1), "k": k.reshape(T, -1)}
    got = {"q": turned(st["q"].reshape(T, h, DIM), 0).reshape(T, -1)}
    for side in ("k", "v"):
        x = st[side + "_new"].reshape(T, hk, DIM)
        x = turned(x, 0) if side == "k" else x.double()
        g = _scales(case, st[side + "_scale"]).double()
        got[side] = torch.cat([kept(part, g) for part in x.split(8192)]).reshape(T, -1)
    return got


def _nearest(x, grid):
    """The nearest value of an ascending grid, halfway to the even index."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - x, x - grid[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])
