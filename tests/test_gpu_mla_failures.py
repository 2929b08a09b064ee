"""A load that never comes, in the kernels of latent attention: the waits end within their limit,
the status and its detail say so, and the next call is as if nothing had been."""
import numpy as np
import pytest
import torch

from gpu_helpers import num_sms
from test_gpu_mla_ops import run
from test_gpu_mla_prefill import check, make

pytestmark = pytest.mark.gpu


def prefill_status(pa, q_lens, kv_lens, heads, mask, sms=None):
    t = [x.flatten(1).cuda() for x in make(10, q_lens, kv_lens, heads, mask)]
    prob = pa.make_problem(bsz=len(q_lens), q_heads=heads, kv_heads=heads, head_dim_qk=192, head_dim_v=128, kv_dtype="bf16",
                           layout="mla_expanded", causal=mask == "causal", cross=mask == "cross", chunk_size=0, sm_scale=0.1,
                           q_stride=heads * 192)
    plan = pa.pa_plan(prob, q_lens, kv_lens, np.concatenate([[0], np.cumsum(q_lens)]), sms or num_sms())
    ws = torch.zeros(plan.workspace_size, dtype=torch.uint8, device="cuda")
    pa.pa_plan_upload(plan, ws)
    out = torch.zeros(sum(q_lens), heads, 128, dtype=torch.bfloat16, device="cuda")
    args = pa.make_args(q=t[0], cache_k=None, cache_v=None, k_scale=None, v_scale=None, block_table=None, out=out, lse=None)
    torch.cuda.synchronize()
    pa.pa_mla_prefill(plan, args, t[1], t[2], heads * 128, t[3], 64, ws)
    st, det = pa.pa_check(plan, ws)
    return st, det, plan.describe()["num_items"]


@pytest.mark.parametrize("q_lens, kv_lens, heads, mask, sms", [([300], [0], 2, "causal", None), ([77], [130], 3, "causal", None),
                                                               ([600, 3], [900, 40], 4, "full", 1), ([5], [700], 1, "cross", None)])
def test_prefill(q_lens, kv_lens, heads, mask, sms):
    import paged_quantized_kv_gqa_gb300 as pa
    pa.pa_debug_set_faults(wait_limit_ns=2_000_000, skip_first_load=True)
    try:
        st, det, items = prefill_status(pa, q_lens, kv_lens, heads, mask, sms)
    finally:
        pa.pa_debug_set_faults()
    assert st == pa.PA_ERR_DEVICE_TIMEOUT and 0 <= det < items
    assert prefill_status(pa, q_lens, kv_lens, heads, mask, sms)[0] == pa.PA_OK
    check(q_lens, kv_lens, heads, mask, sms=sms)


# one tile a pair; runs of several tiles of one head, and of several heads
@pytest.mark.parametrize("rows, heads", [(300, 192), (5000, 20), (33000, 3)])
def test_expand_by_pairs(rows, heads):
    import paged_quantized_kv_gqa_gb300 as pa
    want = run("expand", rows, heads)[2]
    for _ in range(3):
        pa.pa_debug_set_faults(wait_limit_ns=2_000_000, skip_first_load=True)
        try:
            assert run("expand", rows, heads)[3] == pa.PA_ERR_DEVICE_TIMEOUT
        finally:
            pa.pa_debug_set_faults()
        got, st = run("expand", rows, heads)[2:4]
        assert st == pa.PA_OK and all(torch.equal(a, b) for a, b in zip(got, want))
