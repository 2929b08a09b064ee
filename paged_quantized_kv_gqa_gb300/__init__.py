"""Paged, quantised-KV GQA / MLA attention on GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/pa.h`` (``libpa_gb300.so``,
built in-tree by ``paged_quantized_kv_gqa_gb300.build``).  The functions keep
the C names: pa_plan, pa_plan_upload, pa_run, pa_merge, pa_check,
pa_debug_gather, pa_debug_set_faults.  They only marshal arguments; every step
of the attention runs in the library's CUDA kernels.  There is no fallback:
importing this package fails if the library has not been built.

Device buffers may be given as torch tensors (their data_ptr is used) or as
raw integer addresses; streams as torch.cuda.Stream, raw integers or None (the
current torch stream when torch has CUDA, else the legacy default stream).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# PA_GB300_TRACE=1 selects the library built with the pipeline trace (the
# trace module sets it); PA_GB300_DEBUG=1 the debug library (work-item bounds
# checks, poisoned shared and tensor memory); the default library has neither
LIB_PATH = os.path.join(_HERE, "libpa_gb300_trace.so" if os.environ.get("PA_GB300_TRACE") == "1"
                        else "libpa_gb300_debug.so" if os.environ.get("PA_GB300_DEBUG") == "1"
                        else "libpa_gb300.so")

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_CUDA = 0, 1, 2, 3
PA_ERR_DEVICE_TIMEOUT, PA_ERR_BAD_PAGE, PA_ERR_BAD_ITEM, PA_ERR_BAD_POSITION = 4, 5, 6, 7
KV_DTYPES = {"int8": 0, "fp8_e4m3": 1, "int4": 2, "fp4_e2m1": 3, "bf16": 4}
MASK_FULL, MASK_CAUSAL, MASK_CROSS = 0, 1, 2
SCALE_KINDS = {"per_kv_head": 0, "per_channel": 1, "global": 2}
LAYOUTS = {"gqa": 0, "mla": 1, "mla_expanded": 2}
PA_STATUS_BYTES = 256     # the status block at the start of a workspace
ROPE_PAIRS = {"halves": 0, "adjacent": 1}
FAMILIES = {0: "decode", 1: "append", 2: "mla", 3: "expanded"}


class PaProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "bsz", "q_heads", "kv_heads", "head_dim_qk", "head_dim_v", "block_size",
        "max_blocks_per_seq", "num_pages", "kv_dtype", "scale_kind", "layout", "causal",
        "chunk_size")] + [("sm_scale", ctypes.c_float), ("q_stride", ctypes.c_int64)]


class PaArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "q", "cache_k", "cache_v", "k_scale", "v_scale", "block_table", "seq_lens",
        "seq_lens_kv", "cu_seqlens_q", "out", "lse", "attn_mask", "shift_bias",
        "smooth_weight")] + [("out_int8", ctypes.c_int32), ("in_scale", ctypes.c_float),
                             ("quant_max_bound", ctypes.c_float),
                             ("quant_min_bound", ctypes.c_float)]


class PaRope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p)] + [
        (n, ctypes.c_int32) for n in ("table_rows", "rot_dim", "pairs", "axes")] + [
        ("pair_axis", ctypes.c_uint8 * 64)]


class PaPlanDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "family", "chunk_size", "tokens_per_tile", "num_items", "num_ctas", "total_q",
        "max_chunks", "n_merge")] + [
        ("items", ctypes.POINTER(ctypes.c_int32)),
        ("work_indptr", ctypes.POINTER(ctypes.c_int32)),
        ("nch_token", ctypes.POINTER(ctypes.c_int32)),
        ("merge_tokens", ctypes.POINTER(ctypes.c_int32)),
        ("workspace_bytes", ctypes.c_size_t),
        ("kv_bytes", ctypes.c_int64),
        ("flops", ctypes.c_double),
        ("fused_merge", ctypes.c_int32),
        ("plan_bytes", ctypes.c_size_t)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    P32 = ctypes.POINTER(ctypes.c_int32)
    sig = {
        "pa_plan": ([ctypes.POINTER(PaProblem), P32, P32, P32, i32, ctypes.POINTER(vp)], i32),
        "pa_plan_describe": ([vp, ctypes.POINTER(PaPlanDesc)], i32),
        "pa_workspace_size": ([vp], ctypes.c_size_t),
        "pa_plan_upload": ([vp, vp, vp], i32),
        "pa_run": ([vp, ctypes.POINTER(PaArgs), vp, vp], i32),
        "pa_merge": ([vp, ctypes.POINTER(PaArgs), vp, vp], i32),
        "pa_check": ([vp, vp, vp, P32], i32),
        "pa_plan_destroy": ([vp], None),
        "pa_last_error": ([], ctypes.c_char_p),
        "pa_debug_gather": ([ctypes.POINTER(PaProblem), ctypes.POINTER(PaArgs), i32, i32, i32,
                             i32, vp, vp, vp], i32),
        "pa_debug_set_faults": ([i64, i32], i32),
        "pa_run_static": ([vp, ctypes.POINTER(PaArgs), vp, i32], i32),
        "pa_debug_set_trace": ([vp, i32, i32], i32),
        "pa_set_fused_merge": ([i32], i32),
        "pa_cache_append": ([vp, ctypes.POINTER(PaArgs), vp, vp, i64, vp, vp], i32),
        "pa_cache_read": ([vp, ctypes.POINTER(PaArgs), vp, vp, i64, vp, vp], i32),
        "pa_rope_append": ([vp, ctypes.POINTER(PaArgs), ctypes.POINTER(PaRope), vp, i64, vp, i64, vp, vp, i64, vp,
                            vp], i32),
        "pa_mla_absorb": ([i32, i32, vp, i64, vp, i64, vp, i64, vp, vp], i32),
        "pa_mla_project": ([i32, i32, vp, i64, vp, i64, vp, i64, vp, vp], i32),
        "pa_mla_expand": ([i32, i32, vp, i64, vp, i64, vp, vp, i64, vp, vp], i32),
        "pa_mla_prefill": ([vp, ctypes.POINTER(PaArgs), vp, vp, i64, vp, i64, vp, vp], i32),
        "pa_cache_bytes": ([ctypes.POINTER(PaProblem), ctypes.POINTER(ctypes.c_size_t),
                            ctypes.POINTER(ctypes.c_size_t)], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


lib = _load()


class PaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"pa status {status}: {msg}")
        self.status = status


def _check(status: int):
    if status != PA_OK:
        raise PaError(status, lib.pa_last_error().decode(errors="replace"))


def _i32(x, what: str) -> int:
    """A number that fits the C argument (ctypes would cut it to 32 bits)."""
    x = int(x)
    if not -1 << 31 <= x < 1 << 31:
        raise OverflowError(f"{what} = {x} does not fit 32 bits")
    return x


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


# torch's current-stream lookup, kept from the first call that found it
# (torch.cuda.is_available() and a Stream object a call cost more host time than a
# small launch).  Only a lookup that worked is kept: without torch or a device every
# call looks again, and an error of the lookup is raised, since a stream guessed
# instead of the current one would race with the caller's work.
_current_raw_stream = None


def _resolve_current_stream():
    global _current_raw_stream
    try:
        import torch
    except ImportError:
        return
    if not torch.cuda.is_available():
        return
    torch.cuda.current_stream()     # initialises torch's CUDA state
    raw, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
    if raw is not None:
        _current_raw_stream = lambda: int(raw(dev()))
    else:
        _current_raw_stream = lambda: int(torch.cuda.current_stream().cuda_stream)


def _stream(s) -> Optional[int]:
    if s is None:
        if _current_raw_stream is None:
            _resolve_current_stream()
        return _current_raw_stream() if _current_raw_stream else None
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def make_problem(*, bsz, q_heads, kv_heads, head_dim_qk, head_dim_v, block_size=64,
                 max_blocks_per_seq=None, num_pages=None, kv_dtype, scale_kind=None, layout, causal,
                 chunk_size, sm_scale, q_stride, cross=False) -> PaProblem:
    """cross=True: cross attention to seq_lens_kv cached states, the query tokens
    not being in the cache (causal must be False then).  The "mla_expanded" layout has
    no cache and needs no max_blocks_per_seq, num_pages and scale_kind."""
    if layout in ("mla_expanded", LAYOUTS["mla_expanded"]):
        max_blocks_per_seq, num_pages = max_blocks_per_seq or 1, num_pages or 1
        scale_kind = "global" if scale_kind is None else scale_kind
    elif max_blocks_per_seq is None or num_pages is None or scale_kind is None:
        raise TypeError("a cache needs max_blocks_per_seq, num_pages and scale_kind")
    if cross and causal:
        raise ValueError("cross attention has no causal mask")
    p = PaProblem()
    p.bsz, p.q_heads, p.kv_heads = bsz, q_heads, kv_heads
    p.head_dim_qk, p.head_dim_v, p.block_size = head_dim_qk, head_dim_v, block_size
    p.max_blocks_per_seq, p.num_pages = max_blocks_per_seq, num_pages
    p.kv_dtype = KV_DTYPES[kv_dtype] if isinstance(kv_dtype, str) else kv_dtype
    p.scale_kind = SCALE_KINDS[scale_kind] if isinstance(scale_kind, str) else scale_kind
    p.layout = LAYOUTS[layout] if isinstance(layout, str) else layout
    p.causal = MASK_CROSS if cross else int(bool(causal))
    p.chunk_size = chunk_size
    p.sm_scale = sm_scale
    p.q_stride = q_stride
    return p


def problem_of(case) -> PaProblem:
    """PaProblem from any object carrying the problem fields (e.g. synth.Case)."""
    return make_problem(bsz=case.bsz, q_heads=case.q_heads, kv_heads=case.kv_heads,
                        head_dim_qk=case.head_dim_qk, head_dim_v=case.head_dim_v,
                        block_size=case.block_size, max_blocks_per_seq=case.max_blocks_per_seq,
                        num_pages=case.num_pages, kv_dtype=case.kv_dtype,
                        scale_kind=case.scale_kind, layout=case.layout, causal=case.causal,
                        chunk_size=case.chunk_size, sm_scale=case.sm_scale,
                        q_stride=case.q_stride, cross=getattr(case, "cross", False))


class Plan:
    """Owns a pa_plan_t handle."""

    def __init__(self, handle: int, problem: PaProblem):
        self.handle = handle
        self.problem = problem

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h:
            lib.pa_plan_destroy(h)

    def describe(self) -> dict:
        d = PaPlanDesc()
        _check(lib.pa_plan_describe(self.handle, ctypes.byref(d)))
        arr = lambda p, n: np.ctypeslib.as_array(p, shape=(n,)).copy() if n else np.zeros(0, np.int32)
        return dict(family=FAMILIES[d.family], chunk=d.chunk_size,
                    tokens_per_tile=d.tokens_per_tile, num_items=d.num_items,
                    num_ctas=d.num_ctas, total_q=d.total_q, max_chunks=d.max_chunks,
                    items=arr(d.items, d.num_items * 8).reshape(-1, 8),
                    work_indptr=arr(d.work_indptr, d.num_ctas + 1),
                    nch_token=arr(d.nch_token, d.total_q),
                    merge_tokens=arr(d.merge_tokens, d.n_merge),
                    workspace_bytes=int(d.workspace_bytes), kv_bytes=int(d.kv_bytes),
                    flops=float(d.flops), fused_merge=bool(d.fused_merge),
                    plan_bytes=int(d.plan_bytes))

    @property
    def workspace_size(self) -> int:
        return int(lib.pa_workspace_size(self.handle))


def pa_plan(problem: PaProblem, seq_lens, seq_lens_kv, cu_seqlens_q, num_sms: int) -> Plan:
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    sk = np.ascontiguousarray(seq_lens_kv, dtype=np.int32)
    cu = np.ascontiguousarray(cu_seqlens_q, dtype=np.int32)
    P32 = ctypes.POINTER(ctypes.c_int32)
    h = ctypes.c_void_p()
    _check(lib.pa_plan(ctypes.byref(problem), sl.ctypes.data_as(P32), sk.ctypes.data_as(P32),
                       cu.ctypes.data_as(P32), int(num_sms), ctypes.byref(h)))
    return Plan(h.value, problem)


def make_args(*, q, cache_k, cache_v, k_scale, v_scale, block_table, out, lse=None,
              seq_lens=None, seq_lens_kv=None, cu_seqlens_q=None, attn_mask=None,
              shift_bias=None, smooth_weight=None, out_int8=False, in_scale=1.0,
              quant_max_bound=127.0, quant_min_bound=-127.0) -> PaArgs:
    """The arguments of one call.  Tensors stay alive as long as the returned object;
    memory behind raw addresses is the caller's to keep."""
    a = PaArgs()
    a.tensors = [t for t in (q, cache_k, cache_v, k_scale, v_scale, block_table, out, lse, seq_lens, seq_lens_kv,
                             cu_seqlens_q, attn_mask, shift_bias, smooth_weight) if hasattr(t, "data_ptr")]
    a.q, a.cache_k, a.cache_v = _ptr(q), _ptr(cache_k), _ptr(cache_v)
    a.k_scale, a.v_scale, a.block_table = _ptr(k_scale), _ptr(v_scale), _ptr(block_table)
    a.seq_lens, a.seq_lens_kv, a.cu_seqlens_q = _ptr(seq_lens), _ptr(seq_lens_kv), _ptr(cu_seqlens_q)
    a.out, a.lse = _ptr(out), _ptr(lse)
    a.attn_mask = _ptr(attn_mask)
    a.shift_bias, a.smooth_weight = _ptr(shift_bias), _ptr(smooth_weight)
    a.out_int8 = 1 if out_int8 else 0
    a.in_scale, a.quant_max_bound, a.quant_min_bound = in_scale, quant_max_bound, quant_min_bound
    return a


def pa_plan_upload(plan: Plan, workspace, stream=None):
    _check(lib.pa_plan_upload(plan.handle, _ptr(workspace), _stream(stream)))


def pa_run(plan: Plan, args: PaArgs, workspace, stream=None):
    _check(lib.pa_run(plan.handle, ctypes.byref(args), _ptr(workspace), _stream(stream)))


def pa_merge(plan: Plan, args: PaArgs, workspace, stream=None):
    _check(lib.pa_merge(plan.handle, ctypes.byref(args), _ptr(workspace), _stream(stream)))


def pa_check(plan: Optional[Plan], workspace, stream=None):
    """Synchronises the stream; returns (status, detail) of the workspace status word."""
    detail = ctypes.c_int32(0)
    st = lib.pa_check(plan.handle if plan else None, _ptr(workspace), _stream(stream),
                      ctypes.byref(detail))
    return int(st), int(detail.value)


def pa_debug_gather(problem: PaProblem, args: PaArgs, b: int, kv_head: int, pos0: int, n: int,
                    dst_k, dst_v, stream=None):
    _check(lib.pa_debug_gather(ctypes.byref(problem), ctypes.byref(args), b, kv_head, pos0, n,
                               _ptr(dst_k), _ptr(dst_v), _stream(stream)))


def pa_debug_set_faults(wait_limit_ns: int = 0, skip_first_load: bool = False):
    _check(lib.pa_debug_set_faults(int(wait_limit_ns), int(bool(skip_first_load))))


def pa_run_static(plan: Plan, args: PaArgs, stream=None, check: bool = False):
    """Upload, run and merge with the library's built-in 32 MiB device workspace
    (for callers that cannot allocate device memory; see include/pa.h).
    check=True synchronises the stream and raises on a device-side error."""
    _check(lib.pa_run_static(plan.handle, ctypes.byref(args), _stream(stream), int(bool(check))))


def pa_cache_append(plan: Plan, args: PaArgs, k_new, v_new, kv_stride: int, workspace,
                    stream=None):
    """Quantise the appended tokens' K / V rows (bf16, token stride kv_stride
    elements) into the paged cache of args (see include/pa.h)."""
    _check(lib.pa_cache_append(plan.handle, ctypes.byref(args), _ptr(k_new), _ptr(v_new),
                               int(kv_stride), _ptr(workspace), _stream(stream)))


def pa_cache_read(plan: Plan, args: PaArgs, k_out, v_out, kv_stride: int, workspace,
                  stream=None):
    """Read the plan's position ranges (seq_lens_kv[b] .. + seq_lens[b]) of the
    cache back as bf16 rows, token stride kv_stride elements (see include/pa.h)."""
    _check(lib.pa_cache_read(plan.handle, ctypes.byref(args), _ptr(k_out), _ptr(v_out),
                             int(kv_stride), _ptr(workspace), _stream(stream)))


def make_rope(*, cos_sin, table_rows, rot_dim, pairs="halves", positions=None, axes=1, pair_axes=None) -> PaRope:
    """Rotary positions of pa_rope_append (see include/pa.h): a device fp32 table
    [table_rows][rot_dim] of cosines, then sines; with several axes, device int32
    positions [axes][T] and pair_axes, the axis of each of the rot_dim / 2 pairs
    (pair_axes=None: every pair by the first).  Tensors stay alive with the returned object."""
    r = PaRope()
    pair_axes = [int(a) for a in pair_axes] if pair_axes is not None else [0] * max(0, rot_dim // 2)
    if len(pair_axes) != rot_dim // 2 or len(pair_axes) > 64:
        raise ValueError("pair_axes needs one axis per pair, rot_dim / 2 of at most 64")
    if any(a < 0 or a > 255 for a in pair_axes):
        raise ValueError("an axis is a small non-negative number")
    r.tensors = [t for t in (cos_sin, positions) if hasattr(t, "data_ptr")]
    r.cos_sin, r.positions = _ptr(cos_sin), _ptr(positions)
    r.table_rows, r.rot_dim, r.axes = _i32(table_rows, "table_rows"), _i32(rot_dim, "rot_dim"), _i32(axes, "axes")
    r.pairs = ROPE_PAIRS[pairs] if isinstance(pairs, str) else pairs
    r.pair_axis[:len(pair_axes)] = pair_axes
    return r


def pa_rope_append(plan: Plan, args: PaArgs, rope: PaRope, q_new, q_stride: int, q_out, q_out_stride: int, k_new,
                   v_new, kv_stride: int, workspace, stream=None):
    """Rotate the new tokens' queries into q_out (None with q_new=None: no queries) and
    write their rotated keys and their values into the cache of args (see include/pa.h)."""
    _check(lib.pa_rope_append(plan.handle, ctypes.byref(args), ctypes.byref(rope), _ptr(q_new), int(q_stride),
                              _ptr(q_out), int(q_out_stride), _ptr(k_new), _ptr(v_new), int(kv_stride),
                              _ptr(workspace), _stream(stream)))


def pa_mla_absorb(rows: int, heads: int, q, q_stride: int, w, w_head_stride: int, out, out_stride: int, workspace,
                  stream=None):
    """Queries [rows][heads][128 + 64] into the latent space, [rows][heads][512 + 64]
    (see include/pa.h; workspace: a status block of PA_STATUS_BYTES or more)."""
    _check(lib.pa_mla_absorb(_i32(rows, "rows"), _i32(heads, "heads"), _ptr(q), int(q_stride), _ptr(w),
                             int(w_head_stride), _ptr(out), int(out_stride), _ptr(workspace), _stream(stream)))


def pa_mla_project(rows: int, heads: int, o, o_stride: int, w, w_head_stride: int, out, out_stride: int, workspace,
                   stream=None):
    """Latent outputs [rows][heads][512] out of the latent space, [rows][heads][128]
    (see include/pa.h; w: the first W_v row of head 0)."""
    _check(lib.pa_mla_project(_i32(rows, "rows"), _i32(heads, "heads"), _ptr(o), int(o_stride), _ptr(w),
                              int(w_head_stride), _ptr(out), int(out_stride), _ptr(workspace), _stream(stream)))


def pa_mla_expand(rows: int, heads: int, c, c_stride: int, w, w_head_stride: int, k_out, v_out, kv_stride: int,
                  workspace, stream=None):
    """Keys and values [rows][heads][128] of every head from latent rows [rows][512]
    (see include/pa.h)."""
    _check(lib.pa_mla_expand(_i32(rows, "rows"), _i32(heads, "heads"), _ptr(c), int(c_stride), _ptr(w),
                             int(w_head_stride), _ptr(k_out), _ptr(v_out), int(kv_stride), _ptr(workspace),
                             _stream(stream)))


def pa_mla_prefill(plan: Plan, args: PaArgs, k_nope, v, kv_stride: int, k_rope, rope_stride: int, workspace,
                   stream=None):
    """Attention of the plan's tokens to expanded latent rows (an "mla_expanded" plan;
    see include/pa.h); pa_merge joins the ranges of split rows."""
    _check(lib.pa_mla_prefill(plan.handle, ctypes.byref(args), _ptr(k_nope), _ptr(v), int(kv_stride), _ptr(k_rope),
                              int(rope_stride), _ptr(workspace), _stream(stream)))


def pa_cache_bytes(problem: PaProblem):
    """(bytes of cache_k, bytes of cache_v) of the problem's page pool."""
    k, v = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.pa_cache_bytes(ctypes.byref(problem), ctypes.byref(k), ctypes.byref(v)))
    return int(k.value), int(v.value)


def pa_debug_set_trace(buf=None, ctas: int = 0, tiles_per_cta: int = 0):
    """Enable (device uint64 buffer of ctas * tiles_per_cta * 16) or disable (None)
    the kernels' %globaltimer pipeline trace (traced library only: see
    PA_GB300_TRACE; the default library raises PA_ERR_UNSUPPORTED)."""
    _check(lib.pa_debug_set_trace(_ptr(buf), int(ctas), int(tiles_per_cta)))


def pa_set_fused_merge(on: bool):
    """Decode-family plans built afterwards merge split rows inside pa_run (True)
    or leave them to pa_merge's separate kernel (False, the default)."""
    _check(lib.pa_set_fused_merge(1 if on else 0))


def pa_last_error() -> str:
    return lib.pa_last_error().decode(errors="replace")
