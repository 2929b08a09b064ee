"""Seeded problems of the rotated append."""
import types

import numpy as np

from oracle import kv4, rope
from oracle.formats import bf16_to_f64

FORMATS = ["int8", "fp8_e4m3", "int4", "fp4_e2m1"]


def make(seed=0, *, seq_lens, seq_lens_kv, q_heads=4, kv_heads=2, kv_dtype="int8", scale_kind="per_kv_head", layout="gqa",
         rot=128, pairs="halves", axes=1, pair_axis=None, given=False, table_rows=None, spread=1.0):
    """`given`: positions handed over instead of counted; `spread` scales the rows."""
    r = np.random.default_rng(seed)
    mla = layout == "mla"
    p = types.SimpleNamespace(q_heads=128 if mla else q_heads, kv_heads=1 if mla else kv_heads,
                              head_dim_qk=576 if mla else 128, head_dim_v=512 if mla else 128, block_size=64,
                              kv_dtype=kv_dtype, scale_kind="global" if mla else scale_kind, layout=layout, causal=True,
                              chunk_size=0, sm_scale=0.1, rot=rot, pairs=pairs, axes=axes)
    p.q_stride = p.q_heads * p.head_dim_qk
    p.seq_lens, p.seq_lens_kv = np.asarray(seq_lens, np.int32), np.asarray(seq_lens_kv, np.int32)
    p.bsz = len(p.seq_lens)
    p.cu_seqlens_q = np.concatenate([[0], np.cumsum(p.seq_lens)]).astype(np.int32)
    p.total_q = T = int(p.cu_seqlens_q[-1])
    need = -(-(p.seq_lens_kv + p.seq_lens) // 64)
    p.num_pages = int(need.sum()) + 2
    p.max_blocks_per_seq = int(max(1, need.max(initial=1)))
    perm, at = r.permutation(p.num_pages), 0
    p.block_table = np.full((p.bsz, p.max_blocks_per_seq), -1, np.int32)
    for b, n in enumerate(need):
        p.block_table[b, :n] = perm[at:at + n]
        at += n
    four = kv_dtype in ("int4", "fp4_e2m1")
    shape = {"k": (p.num_pages, 64, 576) if mla else (p.num_pages, kv_heads) + ((kv4.SLAB,) if four else (64, 128)),
             "v": (p.num_pages, kv_heads) + ((kv4.SLAB,) if four else (128, 64))}
    top = {"int8": 127.0, "fp8_e4m3": 448.0, "int4": 7.0, "fp4_e2m1": 6.0}[kv_dtype]
    for w in "kv":
        setattr(p, "cache_" + w, None if mla and w == "v" else r.integers(0, 256, shape[w]).astype(np.uint8))
        n = {"global": 1, "per_kv_head": p.kv_heads, "per_channel": p.kv_heads * 128}[p.scale_kind]
        g = (r.uniform(2.0, 4.0, n) / top).astype(np.float32)
        setattr(p, w + "_scale", g if p.scale_kind == "global" else kv4.to_bf16_bits(g))
    bits = lambda *s: kv4.to_bf16_bits((spread * r.standard_normal(s)).astype(np.float32))  # noqa: E731
    p.q_new, p.k_new = bits(T, p.q_heads, 192 if mla else 128), bits(T, p.kv_heads, p.head_dim_qk)
    p.v_new = None if mla else bits(T, kv_heads, 128)
    pos = np.concatenate([s + np.arange(n) for s, n in zip(p.seq_lens_kv, p.seq_lens)] or [[]]).astype(np.int32)
    p.table_rows = table_rows or int((p.seq_lens + p.seq_lens_kv).max(initial=1)) + 5
    p.positions = np.stack([pos] + [r.integers(0, p.table_rows, T).astype(np.int32) for _ in range(axes - 1)])
    p.given = given or axes > 1
    if given:
        p.positions[0] = r.integers(0, p.table_rows, T)
    p.pair_axis = pair_axis if pair_axis is not None else [i % axes for i in range(rot // 2)]
    angle = np.arange(p.table_rows)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    p.table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    return p


def expected(p):
    """q_out (float64, before its rounding to bf16) and the caches."""
    mla = p.layout == "mla"
    args = (p.table, p.positions, p.pair_axis, p.pairs)
    q = rope.turned(bf16_to_f64(p.q_new), 128 if mla else 0, *args)
    k = rope.turned(bf16_to_f64(p.k_new), 512 if mla else 0, *args)
    return (q, *rope.append(p, k, p.v_new, p.cache_k, p.cache_v))
