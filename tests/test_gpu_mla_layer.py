"""The calls of a latent-attention layer one after the other, absorbed and expanded, against
float64.

Both forms compute out = W_v sum_j p_j c_j, s_j = scale (<W_k^T q_nope, c_j> + <q_rope, r_j>)
over the rows (c, r) that the cache holds, whose values the reference takes as stored.  Every
rounding to bf16 is 2^-8 of a value at most (fp16's smaller ones, two a value, 2^-10
together).  Absorbed: the latent query (576 of them in a score), the latent output, the
result; expanded: the keys and values, P, the result.  So a score is off by at most
ds = (2^-8 + 2^-10) scale sum |q'| |k|, out by 3 * 2^-8 |out|-like terms and 4 ds sum p |v|.
That is what a single element may be off; the roundings are independent, so the root mean
square of the error, over that of the result, is far smaller: a score's error is about
2^-8 / sqrt(12) sqrt(sum (q' k)^2) scale < 0.01, as much of p, with the three roundings
less than 1.5 % in all."""
import numpy as np
import pytest
import torch

from gpu_helpers import num_sms
from oracle import rope
from oracle.formats import decode_table
from test_gpu_rope_append import dev

import rope_helpers as rh

pytestmark = pytest.mark.gpu

H, SCALE = 128, 192 ** -0.5


def setup(seed, seq_lens, seq_lens_kv, kv_dtype):
    """A problem of the rotated append whose cache holds codes of ordinary size."""
    p = rh.make(seed=seed, seq_lens=seq_lens, seq_lens_kv=seq_lens_kv, layout="mla", kv_dtype=kv_dtype, rot=64, pairs="adjacent")
    r = np.random.default_rng(seed + 100)
    g = np.float32(0.02 if kv_dtype == "int8" else 0.01)
    p.k_scale = np.array([g], np.float32)
    p.v_scale = p.k_scale
    x = r.standard_normal(p.cache_k.shape).astype(np.float32)
    p.cache_k = rope._codes8(x, g, kv_dtype)
    p.sm_scale = SCALE
    p.w = torch.from_numpy((r.standard_normal((H, 256, 512)) * 512 ** -0.5).astype(np.float32)).bfloat16()
    return p


def reference(p):
    q, cache, _ = rh.expected(p)
    table = decode_table(p.kv_dtype)
    w = p.w.double().numpy()
    outs, spreads = [], []
    for b, (ql, kv) in enumerate(zip(p.seq_lens, p.seq_lens_kv)):
        n = ql + kv
        pages = p.block_table[b, :-(-n // 64)]
        rows = table[cache[pages].reshape(-1, 576)[:n]] * float(p.k_scale[0])
        t = slice(int(p.cu_seqlens_q[b]), int(p.cu_seqlens_q[b + 1]))
        lat = np.concatenate([np.einsum("thd,hdc->thc", q[t, :, :128], w[:, :128]), q[t, :, 128:]], 2)
        s = SCALE * np.einsum("thc,nc->thn", lat, rows)
        late = np.arange(n) > kv + np.arange(ql)[:, None]
        s[np.broadcast_to(late[:, None], s.shape)] = -np.inf
        e = np.exp(s - s.max(-1, keepdims=True))
        e /= e.sum(-1, keepdims=True)
        v = np.einsum("nc,hdc->nhd", rows[:, :512], w[:, 128:])
        outs.append(np.einsum("thn,nhd->thd", e, v))
        ds = (2.0 ** -8 + 2.0 ** -10) * SCALE * np.einsum("thc,nc->thn", np.abs(lat), np.abs(rows)).max(-1)
        mag = np.einsum("thn,nhd->thd", e, np.einsum("nc,hdc->nhd", np.abs(rows[:, :512]), np.abs(w[:, 128:])))
        spreads.append(3 * 2.0 ** -8 * mag + 4 * ds[..., None] * np.einsum("thn,nhd->thd", e, np.abs(v)))
    return np.concatenate(outs), np.concatenate(spreads)


class Layer:
    """What a program keeps: plans, workspaces, weights and rows."""

    def __init__(self, pa, p):
        self.pa, self.p, T = pa, p, p.total_q
        self.d = {n: torch.from_numpy(getattr(p, n).copy()).cuda() for n in
                  ("block_table", "seq_lens", "seq_lens_kv", "cu_seqlens_q", "cache_k", "table")}
        self.scale = torch.from_numpy(p.k_scale).cuda()
        self.w = p.w.cuda()
        self.q, self.k = dev(p.q_new.reshape(T, -1)), dev(p.k_new.reshape(T, -1))
        self.rope = pa.make_rope(cos_sin=self.d["table"], table_rows=p.table_rows, rot_dim=64, pairs="adjacent")
        held = p.seq_lens + p.seq_lens_kv
        self.N = int(held.sum())
        cu = np.concatenate([[0], np.cumsum(held)]).astype(np.int32)
        paged = dict(bsz=p.bsz, q_heads=H, kv_heads=1, head_dim_qk=576, head_dim_v=512, block_size=64,
                     max_blocks_per_seq=p.max_blocks_per_seq, num_pages=p.num_pages, kv_dtype=p.kv_dtype, scale_kind="global",
                     layout="mla", causal=True, chunk_size=-1, sm_scale=SCALE, q_stride=H * 576)
        self.plan = self.planned(paged, p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q)
        self.range = self.planned(paged, held, 0 * held, cu)      # every position, to be read back
        self.fill = self.planned(dict(bsz=p.bsz, q_heads=H, kv_heads=H, head_dim_qk=192, head_dim_v=128, kv_dtype="bf16",
                                      layout="mla_expanded", causal=True, chunk_size=-1, sm_scale=SCALE, q_stride=H * 192),
                                 p.seq_lens, p.seq_lens_kv, p.cu_seqlens_q)
        self.held, self.none, self.cu_held = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (held, 0 * held, cu))
        bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.ql, self.ol, self.out = bf(T, H, 576), bf(T, H, 512), bf(T, H, 128)
        self.rows, self.kx, self.vx, self.out2 = bf(self.N, 576), bf(self.N, H, 128), bf(self.N, H, 128), bf(T, H, 128)
        c = dict(cache_k=self.d["cache_k"], cache_v=self.d["cache_k"], k_scale=self.scale, v_scale=self.scale,
                 block_table=self.d["block_table"])
        self.args = pa.make_args(q=self.ql, out=self.ol, seq_lens=self.d["seq_lens"], seq_lens_kv=self.d["seq_lens_kv"],
                                 cu_seqlens_q=self.d["cu_seqlens_q"], **c)
        self.range_args = pa.make_args(q=None, out=None, seq_lens=self.held, seq_lens_kv=self.none, cu_seqlens_q=self.cu_held, **c)
        self.fill_args = pa.make_args(q=self.q, out=self.out2, cache_k=None, cache_v=None, k_scale=None, v_scale=None,
                                      block_table=None)
        torch.cuda.synchronize()

    def planned(self, problem, *lens):
        plan = self.pa.pa_plan(self.pa.make_problem(**problem), *lens, num_sms())
        ws = torch.zeros(max(plan.workspace_size, 256), dtype=torch.uint8, device="cuda")
        self.pa.pa_plan_upload(plan, ws)
        return plan, ws

    def run(self, append=True):
        pa, T = self.pa, self.p.total_q
        plan, ws = self.plan
        if append:
            pa.pa_rope_append(plan, self.args, self.rope, self.q, H * 192, self.q, H * 192, self.k, None, 576, ws)
        pa.pa_mla_absorb(T, H, self.q, H * 192, self.w, 256 * 512, self.ql, H * 576, ws)
        pa.pa_run(plan, self.args, ws)
        pa.pa_merge(plan, self.args, ws)
        pa.pa_mla_project(T, H, self.ol, H * 512, self.w[:, 128:], 256 * 512, self.out, H * 128, ws)
        rplan, rws = self.range
        pa.pa_cache_read(rplan, self.range_args, self.rows, None, 576, rws)
        pa.pa_mla_expand(self.N, H, self.rows, 576, self.w, 256 * 512, self.kx, self.vx, H * 128, rws)
        fplan, fws = self.fill
        pa.pa_mla_prefill(fplan, self.fill_args, self.kx, self.vx, H * 128, self.rows[:, 512:], 576, fws)
        pa.pa_merge(fplan, self.fill_args, fws)

    def check(self):
        for plan, ws in (self.plan, self.range, self.fill):
            st, det = self.pa.pa_check(plan, ws)
            assert st == 0, (st, det, self.pa.pa_last_error())
        ref, tol = reference(self.p)
        for out in (self.out, self.out2):
            got = out.double().cpu().numpy()
            assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()
            rel = np.sqrt(((got - ref) ** 2).mean() / (ref ** 2).mean())
            assert rel <= 0.015, rel


@pytest.mark.parametrize("kv_dtype", ["fp8_e4m3", "int8"])
@pytest.mark.parametrize("seq_lens, seq_lens_kv", [([1, 1, 2], [70, 0, 500]), ([40, 1, 7], [0, 129, 64])])
def test_a_layer_absorbed_and_expanded(kv_dtype, seq_lens, seq_lens_kv):
    import paged_quantized_kv_gqa_gb300 as pa
    layer = Layer(pa, setup(1, seq_lens, seq_lens_kv, kv_dtype))
    layer.run()
    layer.check()


def test_a_layer_captured():
    """The whole layer as a graph; its rows change between replays."""
    import paged_quantized_kv_gqa_gb300 as pa
    layer = Layer(pa, setup(2, [1, 3], [100, 300], "fp8_e4m3"))
    layer.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = layer.q.clone(), layer.d["cache_k"].clone()
    with torch.cuda.graph(graph):
        layer.run()
    other = setup(3, [1, 3], [100, 300], "fp8_e4m3")
    p = layer.p
    p.q_new, p.k_new = other.q_new, other.k_new
    layer.q.copy_(dev(p.q_new.reshape(p.total_q, -1)))
    layer.k.copy_(dev(p.k_new.reshape(p.total_q, -1)))
    graph.replay()
    torch.cuda.synchronize()
    layer.check()
    assert not torch.equal(keep[0], layer.q)
