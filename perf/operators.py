"""Measured cases of the operators on a cache held in 4 bits.

Three operators, reached through the package's public calls:

  attend  attention of decode, verification and prefill tokens over a paged
          4-bit cache (pa_run, pa_merge), and cross attention of decoder tokens
          to encoder states held in such a cache (mask="cross")
  store   quantising new K / V rows into the cache as they are written
          (pa_cache_append) and reading the stored values back (pa_cache_read)
  load    reading a stored range back as bf16 rows (pa_cache_read)

The cache: a page holds 64 positions.  K and V of one (page, kv head) are a
slab of 4608 bytes each, two half pages of 32 positions one after the other,
2304 bytes each:
  K half: codes [32 positions][64 bytes], byte i holding dims 2i (low nibble)
          and 2i + 1; then E4M3 scales [32 positions][8 blocks of 16 dims]
  V half: codes [128 dims][16 bytes], byte i holding positions 2i (low) and
          2i + 1; then E4M3 scales [8 blocks of 16 dims][32 positions]
A stored value is code * block scale * g, g being the scale of the tensor (per
kv head, per channel or one for all).  Codes: "fp4_e2m1" (sign, two exponent
bits, one mantissa bit: 0 .5 1 1.5 2 3 4 6) or "int4" (two's complement, -7..7
when written).  Writing a block of 16 values x of one position:
  y = x / g; s = E4M3(min(max|y| / M, 448)), M = 6 (fp4_e2m1) or 7 (int4);
  step = s * g; code = nearest code to x / step, ties to even, saturated
with every quotient and product in 32 bits.
"""
import math
import random

import torch

own = False

DIM, PAGE, HALF, BLK = 128, 64, 32, 16
NBLK = DIM // BLK
KCODES = HALF * DIM // 2          # code bytes of a half page
HBYTES = KCODES + HALF * NBLK     # bytes of a half page of K or of V
SLAB = 2 * HBYTES
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TOP = {"fp4_e2m1": 6.0, "int4": 7.0}


# ---------------------------------------------------------------- the cases
def listed():
    c = []
    # two short sequences, one token each: the call's latency is what counts
    c.append(dict(name="decode_two_short", op="attend", mask="causal", kv="fp4_e2m1", scale="per_kv_head",
                  bsz=2, q_lo=1, q_hi=1, kv_lo=36, kv_hi=99, heads=4, kv_heads=1, chunk=0, lens=1))
    # a full decode batch of chat lengths, chunks of 512 positions
    c.append(dict(name="decode_batch", op="attend", mask="causal", kv="int4", scale="per_channel",
                  bsz=64, q_lo=1, q_hi=1, kv_lo=512, kv_hi=4096, heads=32, kv_heads=8, chunk=512, lens=2))
    # a few sequences of book length: the largest cache that is read
    c.append(dict(name="decode_long", op="attend", mask="causal", kv="fp4_e2m1", scale="global",
                  bsz=8, q_lo=1, q_hi=1, kv_lo=32768, kv_hi=131072, heads=64, kv_heads=8, chunk=-1, lens=3))
    # an odd group of five heads, lengths from one position on
    c.append(dict(name="decode_ragged", op="attend", mask="causal", kv="fp4_e2m1", scale="per_channel",
                  bsz=24, q_lo=1, q_hi=1, kv_lo=0, kv_hi=2999, heads=40, kv_heads=8, chunk=-1, lens=4))
    # verification of five draft tokens after long prefixes
    c.append(dict(name="verify_drafts", op="attend", mask="causal", kv="int4", scale="per_kv_head",
                  bsz=32, q_lo=6, q_hi=6, kv_lo=8192, kv_hi=32768, heads=64, kv_heads=8, chunk=1024, lens=5))
    # chunked prefill after cached prefixes: a dense contraction
    c.append(dict(name="prefill_chunks", op="attend", mask="causal", kv="fp4_e2m1", scale="per_kv_head",
                  bsz=8, q_lo=64, q_hi=512, kv_lo=0, kv_hi=8192, heads=32, kv_heads=8, chunk=0, lens=6))
    # one decoder token against encoder states of another length, some empty
    c.append(dict(name="cross_step", op="attend", mask="cross", kv="int4", scale="per_kv_head",
                  bsz=64, q_lo=1, q_hi=1, kv_lo=0, kv_hi=1500, heads=16, kv_heads=16, chunk=-1, lens=7))
    # a decoder prompt against its encoder states
    c.append(dict(name="cross_prompt", op="attend", mask="cross", kv="fp4_e2m1", scale="global",
                  bsz=16, q_lo=65, q_hi=448, kv_lo=100, kv_hi=1500, heads=16, kv_heads=16, chunk=0, lens=8))
    # the rows of one decode step written
    c.append(dict(name="store_step", op="store", kv="fp4_e2m1", scale="global",
                  bsz=64, q_lo=1, q_hi=1, kv_lo=0, kv_hi=4096, kv_heads=8, lens=9))
    # whole prompts written
    c.append(dict(name="store_prompts", op="store", kv="int4", scale="per_kv_head",
                  bsz=8, q_lo=1024, q_hi=8192, kv_lo=0, kv_hi=200, kv_heads=8, lens=10))
    # cached prefixes read back, for a program that works on the rows
    c.append(dict(name="load_prefixes", op="load", kv="fp4_e2m1", scale="per_channel",
                  bsz=8, q_lo=4096, q_hi=16384, kv_lo=0, kv_hi=0, kv_heads=8, lens=11))
    # a short odd range of two heads
    c.append(dict(name="load_short", op="load", kv="int4", scale="global",
                  bsz=3, q_lo=1, q_hi=100, kv_lo=0, kv_hi=77, kv_heads=2, lens=12))
    return c


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = [work(c) for c in listed()]
    bytes_max, flops_max = max(w["bytes"] for w in most), max(w["flops"] for w in most)
    while True:
        kv = rng.choice(["fp4_e2m1", "int4"])
        scale = rng.choice(["global", "per_kv_head", "per_channel"])
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        bsz = _log_int(rng, 1, 64)
        kind = rng.choice(["decode", "decode", "verify", "prefill", "cross", "store", "load"])
        case = dict(kv=kv, scale=scale, bsz=bsz, kv_heads=kv_heads, lens=rng.randrange(1 << 30))
        if kind in ("store", "load"):
            hi = _log_int(rng, 1, 16384 if kind == "load" else 8192)
            case.update(op=kind, q_lo=max(1, hi // rng.choice([1, 2, 5, 9])), q_hi=hi, kv_lo=0,
                        kv_hi=rng.choice([0, 77, 200, 4096]))
        else:
            group = rng.choice([1, 2, 3, 4, 5, 7, 8])
            hi = _log_int(rng, 1, 131072 if kind == "decode" else 32768 if kind == "verify" else 8192)
            q = (1 if kind == "decode" else rng.randint(2, 6) if kind == "verify" else
                 _log_int(rng, 16, 512) if kind == "prefill" else _log_int(rng, 1, 448))
            case.update(op="attend", mask="cross" if kind == "cross" else "causal",
                        q_lo=q if kind in ("decode", "verify") else max(1, q // rng.choice([1, 2, 6])), q_hi=q,
                        kv_lo=hi // rng.choice([1, 2, 4, 8, 64]), kv_hi=hi, heads=kv_heads * group,
                        chunk=rng.choice([-1, -1, 0, 512, 1024]))
            if case["chunk"] == 0 and hi > 16384:     # one CTA would walk a long row alone
                case["chunk"] = -1
            padded = bsz * (q + hi)
            # what the plain form holds at once: rows of 32 bits and the scores
            if padded * kv_heads > 12_000_000 or padded * q * case["heads"] > 1_500_000_000:
                continue
        w = work(case)
        if w["bytes"] <= bytes_max and w["flops"] <= flops_max:
            return case


# ---------------------------------------------------------------- lengths, floors
def _lens(case):
    r = random.Random(case["lens"])
    ql = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["bsz"])]
    kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["bsz"])]
    if case.get("mask") == "cross" and case["kv_lo"] == 0 and case["bsz"] > 2:
        kv[1] = 0                                     # one sequence without states
    return ql, kv


def work(case):
    ql, kv = _lens(case)
    T, row = sum(ql), case["kv_heads"] * DIM
    stored = row * 2 * (0.5 + 1.0 / BLK)              # K and V bytes of one position
    if case["op"] == "attend":
        hq = case["heads"]
        if case["mask"] == "cross":
            n, pairs = sum(kv), sum(q * k for q, k in zip(ql, kv))
        else:
            n = sum(k + q for q, k in zip(ql, kv))
            pairs = sum(q * k + q * (q + 1) // 2 for q, k in zip(ql, kv))
        return {"bytes": n * stored + T * hq * (DIM * 4 + 4), "flops": 4.0 * DIM * pairs * hq}
    if case["op"] == "store":                         # rows in, slabs and values out
        return {"bytes": T * (row * 2 * 4 + stored), "flops": 4.0 * T * row * 2}
    return {"bytes": T * (row * 2 * 2 + stored), "flops": 2.0 * T * row * 2}


# ---------------------------------------------------------------- inputs
def _round_codes(q, kind):
    """Quotients -> 4-bit codes, ties to even, saturated."""
    if kind == "int4":
        return (q.round().clamp(-7, 7).to(torch.int8) & 15).to(torch.uint8)
    a = q.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (mag + 8 * torch.signbit(q)).to(torch.uint8)


def _quantise(x, g, kind):
    """x, g [..., 128] in 32 bits -> codes [..., 128] uint8, scales [..., 8] E4M3."""
    y = (x / g).unflatten(-1, (NBLK, BLK))
    # a tensor as divisor: by a Python number, torch multiplies with a rounded reciprocal
    s = (y.abs().amax(-1) / torch.tensor(TOP[kind], device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s.float()[..., None] * g.expand_as(x).unflatten(-1, (NBLK, BLK))
    q = torch.where(step > 0, x.unflatten(-1, (NBLK, BLK)) / step, torch.zeros_like(step))
    return _round_codes(q, kind).flatten(-2), s


def _pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _slabs(x, g, kind, value_side):
    """Pages of rows x [n, 64, 128] -> slabs [n, 4608]."""
    n = x.shape[0]
    codes, s = _quantise(x, g, kind)
    codes, s = codes.view(n, 2, HALF, DIM), s.view(torch.uint8).view(n, 2, HALF, NBLK)
    if value_side:
        codes, s = codes.transpose(2, 3), s.transpose(2, 3)
    return torch.cat([_pack(codes).reshape(n, 2, KCODES), s.reshape(n, 2, -1)], -1).view(n, SLAB)


def _channel_scales(case, s):
    """The tensor's scale of every kv head and dim, in 32 bits: [kv_heads, 128]."""
    h = case["kv_heads"]
    if case["scale"] == "per_channel":
        return s.float().view(h, DIM)
    return s.float().reshape(-1, 1).expand(h, DIM)


def _tensor_scale(case, gen, dev):
    h = case["kv_heads"]
    if case["scale"] == "global":
        return torch.rand(1, generator=gen, device=dev) * 0.3 + 0.02
    n = h if case["scale"] == "per_kv_head" else h * DIM
    return (torch.rand(n, generator=gen, device=dev) * 0.3 + 0.02).bfloat16()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    ql, kv = _lens(case)
    h, bsz, T = case["kv_heads"], case["bsz"], sum(ql)
    cross = case.get("mask") == "cross"
    held = kv if cross else [a + b for a, b in zip(ql, kv)]
    pages = [-(-n // PAGE) for n in held]
    num_pages, mb = sum(pages) + 3, max(1, max(pages))
    order = torch.randperm(num_pages, generator=gen, device=dev).int()
    bt, at = torch.full((bsz, mb), -1, dtype=torch.int32, device=dev), 0
    for b, n in enumerate(pages):
        bt[b, :n] = order[at:at + n]
        at += n
    st = dict(case=case, k_scale=_tensor_scale(case, gen, dev), v_scale=_tensor_scale(case, gen, dev),
              block_table=bt, q_lens=ql, kv_lens=kv, held=held,
              seq_lens=torch.tensor(ql, dtype=torch.int32, device=dev),
              seq_lens_kv=torch.tensor(kv, dtype=torch.int32, device=dev))
    cu = [0]
    for n in ql:
        cu.append(cu[-1] + n)
    st["cu"] = cu
    st["cu_seqlens_q"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    # the sequence and the index within it of every token row
    st["tok_b"] = torch.repeat_interleave(torch.arange(bsz, device=dev), st["seq_lens"].long())
    st["tok_i"] = torch.arange(T, device=dev) - st["cu_seqlens_q"].long()[st["tok_b"]]
    for side in ("k", "v"):
        cache = torch.zeros((num_pages * h, SLAB), dtype=torch.uint8, device=dev)
        if case["op"] != "store":                     # keys and values of unit variance
            g = _channel_scales(case, st[side + "_scale"])
            some = max(1, (1 << 26) // (PAGE * DIM))
            for i in range(0, num_pages * h, some):
                n = min(some, num_pages * h - i)
                x = torch.randn((n, PAGE, DIM), generator=gen, device=dev).bfloat16().float()
                heads = torch.arange(i, i + n, device=dev) % h
                cache[i:i + n] = _slabs(x, g[heads][:, None, :], case["kv"], side == "v")
        st["cache_" + side] = cache.view(num_pages, h, SLAB)
    if case["op"] == "attend":
        st["q"] = torch.randn((T, case["heads"], DIM), generator=gen, device=dev).bfloat16()
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((T, case["heads"]), device=dev)
    else:
        st["k_new"] = torch.randn((T, h, DIM), generator=gen, device=dev).bfloat16()
        st["v_new"] = torch.randn((T, h, DIM), generator=gen, device=dev).bfloat16()
        st["k_out"], st["v_out"] = torch.empty_like(st["k_new"]), torch.empty_like(st["v_new"])
    if own:
        import paged_quantized_kv_gqa_gb300 as pa
        st["pa"] = pa
        hq = case.get("heads", h)
        prob = pa.make_problem(bsz=bsz, q_heads=hq, kv_heads=h, head_dim_qk=DIM, head_dim_v=DIM, block_size=PAGE,
                               max_blocks_per_seq=mb, num_pages=num_pages, kv_dtype=case["kv"],
                               scale_kind=case["scale"], layout="gqa", causal=not cross, cross=cross,
                               chunk_size=case.get("chunk", 0), sm_scale=DIM ** -0.5, q_stride=hq * DIM)
        st["plan"] = pa.pa_plan(prob, ql, kv, cu, torch.cuda.get_device_properties(dev).multi_processor_count)
        st["ws"] = torch.empty(st["plan"].workspace_size, dtype=torch.uint8, device=dev)
        pa.pa_plan_upload(st["plan"], st["ws"])
        st["args"] = pa.make_args(q=st.get("q"), cache_k=st["cache_k"], cache_v=st["cache_v"], k_scale=st["k_scale"],
                                  v_scale=st["v_scale"], block_table=bt, out=st.get("out"), lse=st.get("lse"),
                                  seq_lens=st["seq_lens"], seq_lens_kv=st["seq_lens_kv"],
                                  cu_seqlens_q=st["cu_seqlens_q"])
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        pa = state["pa"]
        if case["op"] == "attend":
            pa.pa_run(state["plan"], state["args"], state["ws"])
            pa.pa_merge(state["plan"], state["args"], state["ws"])
            return {"out": state["out"], "lse": state["lse"]}
        stride = case["kv_heads"] * DIM
        if case["op"] == "store":
            pa.pa_cache_append(state["plan"], state["args"], state["k_new"], state["v_new"], stride, state["ws"])
        pa.pa_cache_read(state["plan"], state["args"], state["k_out"], state["v_out"], stride, state["ws"])
        return {"k": state["k_out"], "v": state["v_out"]}
    if case["op"] == "attend":
        return _attend(state)
    if case["op"] == "store":
        _store(state, "k")
        _store(state, "v")
    return {"k": _load(state, "k"), "v": _load(state, "v")}


def _values(codes, kind):
    """4-bit codes -> the values they stand for, 32 bits."""
    t = (LEVELS + [-x for x in LEVELS]) if kind == "fp4_e2m1" else [float(i - 16 * (i > 7)) for i in range(16)]
    return torch.tensor(t, device=codes.device)[codes.int()]


def _unpack(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _rows_of_slabs(state, slabs, side):
    """Slabs [..., kv_heads, 4608] -> rows [..., kv_heads, 64, 128] in 32 bits."""
    case = state["case"]
    halves = slabs.unflatten(-1, (2, HBYTES))
    codes, s = halves[..., :KCODES], halves[..., KCODES:].contiguous().view(torch.float8_e4m3fn).float()
    if side == "k":
        x = _values(_unpack(codes.unflatten(-1, (HALF, DIM // 2))), case["kv"])
        s = s.unflatten(-1, (HALF, NBLK))
    else:
        x = _values(_unpack(codes.unflatten(-1, (DIM, HALF // 2))), case["kv"]).transpose(-1, -2)
        s = s.unflatten(-1, (NBLK, HALF)).transpose(-1, -2)
    x = (x.unflatten(-1, (NBLK, BLK)) * s[..., None]).flatten(-2).flatten(-3, -2)
    return x * _channel_scales(case, state[side + "_scale"])[:, None, :]


def _attend(state):
    case, bt = state["case"], state["block_table"].clamp(min=0).long()
    h, G, bsz = case["kv_heads"], case["heads"] // case["kv_heads"], case["bsz"]
    K, V = (_rows_of_slabs(state, state["cache_" + s][bt], s).transpose(1, 2).flatten(2, 3) for s in ("k", "v"))
    L, Q = K.shape[2], max(state["q_lens"])           # padded lengths
    tb, ti = state["tok_b"], state["tok_i"]
    q = torch.zeros((bsz, h, Q, G, DIM), device=bt.device)
    q[tb, :, ti] = state["q"].float().unflatten(1, (h, G))
    S = (q.flatten(2, 3) @ K.transpose(2, 3)).unflatten(2, (Q, G)) * DIM ** -0.5
    pos, i = torch.arange(L, device=bt.device), torch.arange(Q, device=bt.device)
    kv = state["seq_lens_kv"].long()[:, None, None]
    if case["mask"] == "cross":
        seen = (pos < kv).expand(bsz, Q, L)
    else:
        seen = pos <= kv + i[:, None]
    seen = seen & (pos < torch.tensor(state["held"], device=bt.device)[:, None, None])
    S = S.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    P = (S - m).exp()
    total = P.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    V = V.masked_fill(~(seen.any(1)[:, None, :, None]), 0.0)
    O = (P.flatten(2, 3) @ V).unflatten(2, (Q, G)) / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": O[tb, :, ti].flatten(1, 2).bfloat16(), "lse": lse[tb, :, ti].flatten(1, 2)}


def _places(state):
    """Page, half page and place within it of every new token row."""
    pos = state["seq_lens_kv"].long()[state["tok_b"]] + state["tok_i"]
    return state["block_table"][state["tok_b"], pos // PAGE].long(), pos % PAGE // HALF, pos % HALF


def _store(state, side):
    case, cache = state["case"], state["cache_" + side]
    x = state[side + "_new"].float()
    codes, s = _quantise(x, _channel_scales(case, state[side + "_scale"]), case["kv"])
    page, half, r = _places(state)
    halves = cache.view(*cache.shape[:2], 2, HBYTES)
    if side == "k":
        halves[..., :KCODES].unflatten(-1, (HALF, DIM // 2))[page, :, half, r] = _pack(codes)
        halves[..., KCODES:].unflatten(-1, (HALF, NBLK))[page, :, half, r] = s.view(torch.uint8)
    else:
        held = _unpack(halves[..., :KCODES].unflatten(-1, (DIM, HALF // 2)))
        held[page, :, half, :, r] = codes
        halves[..., :KCODES].unflatten(-1, (DIM, HALF // 2)).copy_(_pack(held))
        halves[..., KCODES:].unflatten(-1, (NBLK, HALF))[page, :, half, :, r] = s.view(torch.uint8)


def _load(state, side):
    case, cache = state["case"], state["cache_" + side]
    page, half, r = _places(state)
    halves = cache.view(*cache.shape[:2], 2, HBYTES)
    if side == "k":
        codes = _unpack(halves[..., :KCODES].unflatten(-1, (HALF, DIM // 2))[page, :, half, r])
        s = halves[..., KCODES:].unflatten(-1, (HALF, NBLK))[page, :, half, r]
    else:
        pair = halves[..., :KCODES].unflatten(-1, (DIM, HALF // 2))[page, :, half, :, r // 2]
        codes = torch.where((r % 2 == 1)[:, None, None], pair >> 4, pair & 15)
        s = halves[..., KCODES:].unflatten(-1, (NBLK, HALF))[page, :, half, :, r]
    step = s.contiguous().view(torch.float8_e4m3fn).float()[..., None] \
        * _channel_scales(case, state[side + "_scale"]).unflatten(-1, (NBLK, BLK))
    return (_values(codes, case["kv"]).unflatten(-1, (NBLK, BLK)) * step).flatten(-2).bfloat16()


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attention(st)
    out = {}
    for side in ("k", "v"):
        g = _channel_scales(case, st[side + "_scale"]).double()
        if case["op"] == "store":
            parts = [_exact_stored(x, g, case["kv"]) for x in st[side + "_new"].split(8192)]
        else:
            parts = []
            for b, (n, first) in enumerate(zip(st["q_lens"], st["kv_lens"])):
                rows = _exact_rows(st, side, b, first + n)
                parts.append(rows[first:] * g)
        out[side] = torch.cat(parts)
    return out


def _grid(kind, dev):
    pos = LEVELS if kind == "fp4_e2m1" else [float(i) for i in range(8)]
    return torch.tensor(pos, dtype=torch.float64, device=dev)


def _exact_stored(x, g, kind):
    """The value that every element of rows x [n, kv_heads, 128] is stored as.
    Quotients are rounded to 32 bits where the definition says so: a quotient
    of two 32-bit numbers, rounded from 64 bits, is the correctly rounded one."""
    x = x.double()
    grid = _grid(kind, x.device)
    blocks = lambda t: t.reshape(*t.shape[:-1], NBLK, BLK)  # noqa: E731
    y = blocks(x / g).float().abs().amax(-1).double()
    want = (y / (6.0 if kind == "fp4_e2m1" else 7.0)).float().double().clamp(max=448.0)
    e4m3 = torch.arange(127, device=x.device, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    hi = torch.searchsorted(e4m3, want).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = e4m3[hi] - want, want - e4m3[lo]
    s = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), e4m3[hi], e4m3[lo])
    step = (s[..., None] * blocks(g)).float().double()
    q = torch.where(step > 0, blocks(x) / step, torch.zeros_like(step)).float().double()
    mag = q.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, mag).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - mag, mag - grid[lo]
    c = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])
    return (c * torch.sign(q) * s[..., None] * blocks(g)).reshape(x.shape)


def _exact_rows(st, side, b, n):
    """Positions 0 .. n-1 of sequence b without the tensor's scale: [n, kv_heads, 128]."""
    kind, h = st["case"]["kv"], st["case"]["kv_heads"]
    grid = _grid(kind, st["block_table"].device)
    table = torch.cat([grid, -grid]) if kind == "fp4_e2m1" else torch.cat([grid, grid - 8.0])
    slabs = st["cache_" + side][st["block_table"][b, :-(-n // PAGE)].long()].reshape(-1, h, 2, HBYTES)
    m = slabs.shape[0]
    raw, sc = slabs[..., :KCODES], slabs[..., KCODES:].contiguous()
    nib = torch.empty(*raw.shape, 2, dtype=torch.long, device=raw.device)
    nib[..., 0], nib[..., 1] = raw % 16, raw // 16
    val = table[nib.reshape(m, h, 2, -1)]
    sc = sc.view(torch.float8_e4m3fn).double()
    if side == "k":
        val, sc = val.reshape(m, h, 2, HALF, DIM), sc.reshape(m, h, 2, HALF, NBLK)
    else:
        val = val.reshape(m, h, 2, DIM, HALF).permute(0, 1, 2, 4, 3)
        sc = sc.reshape(m, h, 2, NBLK, HALF).permute(0, 1, 2, 4, 3)
    val = val * sc.repeat_interleave(BLK, -1)
    return val.permute(0, 2, 3, 1, 4).reshape(m * PAGE, h, DIM)[:n]


def _exact_attention(st):
    case = st["case"]
    h, G = case["kv_heads"], case["heads"] // case["kv_heads"]
    gk, gv = (_channel_scales(case, st[s + "_scale"]).double() for s in ("k", "v"))
    outs, lses = [], []
    for b, (n, prefix, held) in enumerate(zip(st["q_lens"], st["kv_lens"], st["held"])):
        q = st["q"][st["cu"][b]:st["cu"][b] + n].double().reshape(n, h, G, DIM)
        if held == 0:
            outs.append(torch.zeros(n, h * G, DIM, dtype=torch.float64, device=q.device))
            lses.append(torch.full((n, h * G), -math.inf, dtype=torch.float64, device=q.device))
            continue
        K, V = _exact_rows(st, "k", b, held) * gk, _exact_rows(st, "v", b, held) * gv
        s = torch.einsum("nhgd,lhd->hgnl", q, K) / math.sqrt(DIM)
        if case["mask"] == "causal":
            late = torch.arange(held, device=q.device) > prefix + torch.arange(n, device=q.device)[:, None]
            s = s.masked_fill(late, -math.inf)
        lse = torch.logsumexp(s, -1)
        o = torch.einsum("hgnl,lhd->nhgd", torch.exp(s - lse[..., None]), V)
        outs.append(o.reshape(n, h * G, DIM))
        lses.append(lse.permute(2, 0, 1).reshape(n, h * G))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
