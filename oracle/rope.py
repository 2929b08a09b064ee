"""Rotary positions and the rotated cache append (oracle side), shares no code with
the CUDA path.

A pair (a, b) turns by an angle with cos c and sin s from a table row: a c - b s and
b c + a s, each product and sum rounded to binary32.  In float64 a product of two
binary32 numbers is exact and a sum rounds far below binary32's last place, so rounding
each step's float64 result gives the binary32 step."""
from __future__ import annotations

import numpy as np

from . import cache_append as ca
from . import kv4
from .formats import bf16_to_f64


def _fl(x):
    with np.errstate(over="ignore"):
        return x.astype(np.float32).astype(np.float64)


def turned(x, first, table, positions, pair_axis, pairs):
    """Rows x [T, heads, dims] (float64) with dims first .. first + rot_dim - 1 turned;
    table [rows, rot_dim] fp32, positions [axes, T]."""
    rot = table.shape[1]
    n = rot // 2
    y = x.copy()
    for i in range(n):
        a, b = (first + i, first + i + n) if pairs == "halves" else (first + 2 * i, first + 2 * i + 1)
        row = table[positions[pair_axis[i]]].astype(np.float64)
        c, s = row[:, i, None], row[:, n + i, None]
        with np.errstate(invalid="ignore"):            # infinities of a pair
            y[:, :, a] = _fl(_fl(x[:, :, a] * c) - _fl(x[:, :, b] * s))
            y[:, :, b] = _fl(_fl(x[:, :, b] * c) + _fl(x[:, :, a] * s))
    return y


def _codes8(x, s, kind):
    """A NaN becomes E4M3's NaN, and 0 as int8."""
    q = x.astype(np.float32) / s
    lost, q = np.isnan(q), np.where(np.isnan(q), np.float32(0), q)
    codes = ca.e4m3_encode(q) if kind == "fp8_e4m3" else ca.int8_encode(q)
    return np.where(lost, np.uint8(0x7F if kind == "fp8_e4m3" else 0), codes)


def append(p, k, v_bits, cache_k, cache_v):
    """Turned keys k (float64 [T, kv_heads, D]) and values (bf16 bits) written into copies."""
    ck, cv = cache_k.copy(), None if cache_v is None else cache_v.copy()
    four = p.kv_dtype in ("int4", "fp4_e2m1")
    codes = {"k": kv4.unpack_k(ck), "v": kv4.unpack_v(cv)} if four else None
    for b in range(len(p.seq_lens)):
        for i in range(int(p.seq_lens[b])):
            t, j = int(p.cu_seqlens_q[b]) + i, int(p.seq_lens_kv[b]) + i
            page, off = int(p.block_table[b, j // 64]), j % 64
            if p.layout == "mla":
                ck[page, off] = _codes8(k[t, 0], ca._scales(p, p.k_scale, 0, k.shape[2]), p.kv_dtype)
                continue
            for h in range(p.kv_heads):
                v = bf16_to_f64(v_bits[t, h])
                if four:
                    for w, x in (("k", k[t, h]), ("v", v)):
                        c, s = kv4.quantise_rows(x.astype(np.float32)[None], kv4.tensor_scale(p, w, h), p.kv_dtype)
                        codes[w][0][page, h, off], codes[w][1][page, h, off] = c[0], s[0]
                else:
                    ck[page, h, off] = _codes8(k[t, h], ca._scales(p, p.k_scale, h, 128), p.kv_dtype)
                    cv[page, h, :, off] = _codes8(v, ca._scales(p, p.v_scale, h, 128), p.kv_dtype)
    return (kv4.pack_k(*codes["k"]), kv4.pack_v(*codes["v"])) if four else (ck, cv)
