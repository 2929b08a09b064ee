"""4-bit cases for the debug library (shared and tensor memory filled with NaN
bytes before first use, work items checked against the problem's bounds).  Run as
a script in a process with PA_GB300_DEBUG=1; tests/test_gpu_kv4.py does that.  A
kernel that read shared or tensor memory it never wrote would carry the poison
into its output.  Exits non-zero on the first failure."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

from kv4_helpers import check, make, run  # noqa: E402
import paged_quantized_kv_gqa_gb300 as pa  # noqa: E402

CASES = [
    ("warp decode, split", dict(seq_lens=[1, 1], seq_lens_kv=[1500, 3], q_heads=8, kv_heads=2)),
    ("warp decode, 16 rows", dict(seq_lens=[2, 1], seq_lens_kv=[700, 64], q_heads=16, kv_heads=2)),
    ("verify, 48 rows, split", dict(seq_lens=[6, 6], seq_lens_kv=[1500, 300], q_heads=64, kv_heads=8)),
    ("verify, 21 rows", dict(seq_lens=[3, 0, 1], seq_lens_kv=[130, 5, 7], q_heads=14, kv_heads=2)),
    ("append", dict(seq_lens=[150, 70], seq_lens_kv=[400, 33], q_heads=32, kv_heads=8)),
    ("append, chunks", dict(seq_lens=[65, 3], seq_lens_kv=[200, 700], q_heads=10, kv_heads=2, chunk_size=128)),
    ("cross", dict(seq_lens=[1, 2, 1], seq_lens_kv=[900, 0, 31], q_heads=4, kv_heads=4, causal=False, cross=True)),
    ("cross prompt", dict(seq_lens=[80, 65], seq_lens_kv=[0, 130], q_heads=4, kv_heads=4, causal=False, cross=True)),
]


if __name__ == "__main__":
    assert os.path.basename(pa.LIB_PATH) == "libpa_gb300_debug.so", pa.LIB_PATH
    for i, (label, kw) in enumerate(CASES):
        for kind in ("int4", "fp4_e2m1"):
            for scale in ("per_kv_head", "per_channel"):
                p = make(60 + i, kv_dtype=kind, scale_kind=scale, **kw)
                out, lse, *_ = run(p)
                check(p, out, lse)
                print("ok", label, kind, scale)
    print("debug library: all 4-bit cases passed")
