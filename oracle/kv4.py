"""The 4-bit cache in float64 (oracle side): codes, slabs, quantisation and
attention over dequantised rows.

Shares no code with the CUDA path.  A page holds 64 positions; K and V of one
(page, kv head) are slabs of 4608 bytes, two half pages of 32 positions:
  K half: codes [32][64] (byte i = dims 2i low nibble, 2i + 1), scales [32][8]
  V half: codes [128][16] (byte i = positions 2i low, 2i + 1), scales [8][32]
value = code * E4M3 scale of its 16 dims * tensor scale.
"""
from __future__ import annotations

import math

import numpy as np

from .cache_append import e4m3_encode
from .formats import bf16_to_f64, e4m3_value

HALF, DIM, BLK = 32, 128, 16
KCODES = HALF * DIM // 2
HBYTES = KCODES + HALF * (DIM // BLK)
SLAB = 2 * HBYTES
E4M3 = np.array([e4m3_value(c) for c in range(256)])


def fp4_value(code: int) -> float:
    """OCP E2M1: sign, exponent (bias 1), mantissa; exponent 0 is subnormal."""
    s, e, m = code >> 3, (code >> 1) & 3, code & 1
    v = 0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)
    return -v if s else v


def code_table(kind: str) -> np.ndarray:
    if kind == "fp4_e2m1":
        return np.array([fp4_value(c) for c in range(16)])
    return np.array([float(c - 16 if c >= 8 else c) for c in range(16)])


def unpack_k(slabs):
    """[..., 4608] bytes -> codes [..., 64, 128], scale bytes [..., 64, 8]."""
    lead = slabs.shape[:-1]
    h = slabs.reshape(*lead, 2, HBYTES)
    b = h[..., :KCODES].reshape(*lead, 2, HALF, DIM // 2)
    codes = np.stack([b & 15, b >> 4], -1).reshape(*lead, 64, DIM)
    return codes, h[..., KCODES:].reshape(*lead, 64, DIM // BLK)


def unpack_v(slabs):
    lead = slabs.shape[:-1]
    h = slabs.reshape(*lead, 2, HBYTES)
    b = h[..., :KCODES].reshape(*lead, 2, DIM, HALF // 2)
    codes = np.stack([b & 15, b >> 4], -1).reshape(*lead, 2, DIM, HALF)
    scales = h[..., KCODES:].reshape(*lead, 2, DIM // BLK, HALF)
    return (np.moveaxis(codes, -1, -2).reshape(*lead, 64, DIM),
            np.moveaxis(scales, -1, -2).reshape(*lead, 64, DIM // BLK))


def pack_k(codes, scales):
    lead = codes.shape[:-2]
    b = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(*lead, 2, KCODES)
    return np.concatenate([b, scales.reshape(*lead, 2, -1)], -1).reshape(*lead, SLAB).astype(np.uint8)


def pack_v(codes, scales):
    lead = codes.shape[:-2]
    c = np.moveaxis(codes.reshape(*lead, 2, HALF, DIM), -1, -2)
    b = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(*lead, 2, KCODES)
    s = np.moveaxis(scales.reshape(*lead, 2, HALF, DIM // BLK), -1, -2).reshape(*lead, 2, -1)
    return np.concatenate([b, s], -1).reshape(*lead, SLAB).astype(np.uint8)


def tensor_scale(p, which: str, kvh: int) -> np.ndarray:
    """fp32 scale of each of the 128 channels of kv head kvh."""
    s = p.k_scale if which == "k" else p.v_scale
    if p.scale_kind == "global":
        return np.full(DIM, np.float32(np.asarray(s, np.float32).reshape(-1)[0]))
    f = bf16_to_f64(np.asarray(s, np.uint16)).astype(np.float32)
    return np.full(DIM, f[kvh]) if p.scale_kind == "per_kv_head" else f[kvh * DIM:(kvh + 1) * DIM]


def quantise_rows(x, g, kind: str):
    """x [n, 128] float32, g [128] float32 -> codes [n, 128], scale bytes [n, 8],
    every quotient and product in binary32."""
    top = np.float32(6.0 if kind == "fp4_e2m1" else 7.0)
    table = code_table(kind)
    x = np.where(np.isnan(x), np.float32(0), x.astype(np.float32))
    with np.errstate(all="ignore"):
        y = np.abs(x / g).reshape(len(x), -1, BLK).max(-1)
        sb = e4m3_encode(np.minimum(y / top, np.float32(448.0)))
        step = np.repeat(E4M3[sb].astype(np.float32), BLK, axis=1) * g
        q = np.where(step > 0, x / np.where(step > 0, step, np.float32(1)), np.float32(0))
    a = np.minimum(np.abs(q.astype(np.float64)), float(top))
    mags = table[:8] if kind == "fp4_e2m1" else np.arange(8.0)
    d = np.abs(a[..., None] - mags)
    best = d == d.min(-1, keepdims=True)
    even = best & (np.arange(8) % 2 == 0)
    mag = np.argmax(np.where(even.any(-1, keepdims=True), even, best), -1)
    neg = np.signbit(q)
    code = mag + 8 * neg if kind == "fp4_e2m1" else np.where(neg, -mag, mag) & 15
    return code.astype(np.uint8), sb


def append(p, k_bits, v_bits, cache_k, cache_v):
    """The appended tokens' rows (bf16 bits [T, kv_heads, 128]) written into copies."""
    ck, cv = cache_k.copy(), cache_v.copy()
    codes = {"k": unpack_k(ck), "v": unpack_v(cv)}
    new = {"k": k_bits, "v": v_bits}
    for b in range(len(p.seq_lens)):
        for i in range(int(p.seq_lens[b])):
            t, j = int(p.cu_seqlens_q[b]) + i, int(p.seq_lens_kv[b]) + i
            page, off = int(p.block_table[b, j // 64]), j % 64
            for h in range(p.kv_heads):
                for w in ("k", "v"):
                    x = bf16_to_f64(new[w][t, h]).astype(np.float32)[None]
                    c, s = quantise_rows(x, tensor_scale(p, w, h), p.kv_dtype)
                    codes[w][0][page, h, off], codes[w][1][page, h, off] = c[0], s[0]
    return pack_k(*codes["k"]), pack_v(*codes["v"])


def stored_rows(p, which: str, b: int, kvh: int, n: int):
    """Codes [n, 128] and block scales [n, 128] (float64) of positions 0 .. n-1."""
    pages = [int(x) for x in p.block_table[b, :math.ceil(n / 64)]]
    cache = p.cache_k if which == "k" else p.cache_v
    un = unpack_k if which == "k" else unpack_v
    if not pages:
        return np.zeros((0, DIM)), np.zeros((0, DIM))
    codes, sb = un(cache[pages, kvh])
    codes, sb = codes.reshape(-1, DIM)[:n], sb.reshape(-1, DIM // BLK)[:n]
    return code_table(p.kv_dtype)[codes], np.repeat(E4M3[sb], BLK, axis=1)


def rows(p, which: str, b: int, kvh: int, n: int) -> np.ndarray:
    c, s = stored_rows(p, which, b, kvh, n)
    return c * s * tensor_scale(p, which, kvh).astype(np.float64)


def read_back(p, which: str, b: int, kvh: int, first: int, n: int) -> np.ndarray:
    """bf16 bits of positions first .. first + n - 1 as pa_cache_read gives them."""
    c, s = stored_rows(p, which, b, kvh, first + n)
    step = s.astype(np.float32) * tensor_scale(p, which, kvh)
    return to_bf16_bits((c.astype(np.float32) * step)[first:])


def to_bf16_bits(x) -> np.ndarray:
    """float32 -> bf16 bits, nearest, ties to even (finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def attend(q, K, V, seen, sm_scale):
    """q [n, G, 128], K / V [L, 128], seen [n, L] -> out, lse and what a tolerance
    needs: sum p |v| per element and the largest sum |q k| per row."""
    s = np.where(seen[:, None, :], sm_scale * np.einsum("ngd,ld->ngl", q, K), -np.inf)
    if K.shape[0] == 0:
        z = np.zeros(q.shape)
        return z, np.full(q.shape[:2], -np.inf), z, np.zeros(q.shape[:2])
    m = s.max(-1, keepdims=True)
    m0 = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - m0)
    z = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(z > 0, m0 + np.log(z), -np.inf)[..., 0]
    w = e / np.where(z > 0, z, 1.0)
    mag = np.where(seen[:, None, :], np.einsum("ngd,ld->ngl", np.abs(q), np.abs(K)), 0.0).max(-1)
    return np.einsum("ngl,ld->ngd", w, V), lse, np.einsum("ngl,ld->ngd", w, np.abs(V)), mag
