"""Cases of expanded latent rows for the debug library (kernels compiled with PA_DEBUG: shared
and tensor memory filled with NaN bytes before first use, work items checked against the
problem's bounds).  Run as a script in a process with PA_GB300_DEBUG=1;
tests/test_gpu_debug_expanded.py does that.

1. Plans of one and two query tiles, ragged, split and joined, against float64: a kernel that
   read memory it never wrote would carry the poison into its output.
2. Items altered in the uploaded plan, which the check reports as PA_ERR_BAD_ITEM with their
   index: the last sequence's rows one further on (its range then ends behind the last row,
   which the loads would fill with zeros), a range that ends a row later, a first row before
   the rows.  A clean run afterwards reports PA_OK.

Exits non-zero on the first failure."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import numpy as np  # noqa: E402
import torch  # noqa: E402

import paged_quantized_kv_gqa_gb300 as pa  # noqa: E402
from gpu_helpers import num_sms  # noqa: E402
from test_gpu_mla_prefill import check, make  # noqa: E402

CASES = [
    ("one tile", [77], [130], "causal", dict()),
    ("two tiles", [300, 256, 129], [0, 40, 500], "causal", dict()),
    ("ragged, split", [300, 0, 1, 257], [0, 5, 0, 1000], "causal", dict(chunk=128)),
    ("full, chosen split", [64, 3], [129, 1500], "full", dict(chunk=-1)),
    ("cross, rows that see nothing", [200, 5, 1], [700, 0, 63], "cross", dict(chunk=256)),
    ("an SM for all", [300, 40], [90, 300], "causal", dict(sms=1)),
]


def bad_items():
    q_lens, kv_lens, heads = [5, 40], [70, 100], 2
    t = [x.flatten(1).cuda() for x in make(3, q_lens, kv_lens, heads, "causal")]
    prob = pa.make_problem(bsz=2, q_heads=heads, kv_heads=heads, head_dim_qk=192, head_dim_v=128, kv_dtype="bf16",
                           layout="mla_expanded", causal=True, chunk_size=0, sm_scale=0.07, q_stride=heads * 192)
    plan = pa.pa_plan(prob, q_lens, kv_lens, [0, 5, 45], num_sms())
    ws = torch.zeros(plan.workspace_size, dtype=torch.uint8, device="cuda")
    out = torch.zeros(45, heads, 128, dtype=torch.bfloat16, device="cuda")
    args = pa.make_args(q=t[0], cache_k=None, cache_v=None, k_scale=None, v_scale=None, block_table=None, out=out, lse=None)

    def run(words=None):
        pa.pa_plan_upload(plan, ws)
        torch.cuda.synchronize()
        if words is not None:
            ws.copy_(torch.from_numpy(words.view(np.uint8)).cuda())
            torch.cuda.synchronize()
        pa.pa_mla_prefill(plan, args, t[1], t[2], heads * 128, t[3], 64, ws)
        return pa.pa_check(plan, ws)

    assert run()[0] == pa.PA_OK
    good = ws.cpu().numpy().view(np.int32).copy()
    # an item of the last sequence: rows 75 .. 214 of 215, tokens 5 .. 44
    win = np.lib.stride_tricks.sliding_window_view(good, 8)
    pos = [i for i in range(len(win)) if win[i][0] == 75 and win[i][2] == 5 and win[i][3] & 0xFFFF == 40 and win[i][6] == 140]
    assert len(pos) == heads, pos
    k = [i for i, x in enumerate(plan.describe()["items"]) if x[0] == 1]
    for word, by in ((0, 1), (6, 1), (0, -76)):
        bad = good.copy()
        bad[pos[0] + word] += by
        st, det = run(bad)
        assert st == pa.PA_ERR_BAD_ITEM and det in k, (word, by, st, det)
    assert run()[0] == pa.PA_OK


if __name__ == "__main__":
    print("library", os.path.basename(pa.LIB_PATH))
    assert os.path.basename(pa.LIB_PATH) == "libpa_gb300_debug.so", pa.LIB_PATH
    for i, (label, q_lens, kv_lens, mask, kw) in enumerate(CASES):
        check(q_lens, kv_lens, 3, mask, seed=80 + i, **kw)
        print("ok", label)
    bad_items()
    print("debug library: all expanded cases passed")
