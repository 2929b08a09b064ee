"""Tensor memory is touched only behind the fence that the memory model asks for.

A thread that learns of finished MMAs through an mbarrier (tcgen05.commit arrives on
it) has to execute tcgen05.fence::after_thread_sync before its own tensor-memory
loads, stores or MMAs are ordered behind them.  The kernels are read as text: behind
every wait on a barrier that some tc_commit names, the fence comes before the next
access."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_quantized_kv_gqa_gb300",
                    "csrc")
KERNELS = ["pa_decode.cu", "pa_decode.cuh", "pa_append.cuh", "pa_mla.cu"]
WAIT = re.compile(r"\b(?:wait_or_abort|dwait|mwait|mbar_test_wait)\(\s*&?(\w+)")
# the fence, an access, or the next warp role (the branches of a kernel's body)
EVENT = re.compile(r"(?P<fence>\btc_fence_after\(\))|(?P<use>\b(?:tmem_(?:st|ld)\d+|mma_(?:ts|ss)\w*)\()|(?P<role>\n  \} else)")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), f.read())


def commit_barriers(text):
    """Names of the barriers that tc_commit arrives on, pointers made from them included."""
    names = set(re.findall(r"\btc_commit\w*\(\s*&?(\w+)", text))
    for alias, of in re.findall(r"uint64_t\*\s*(\w+)\s*=\s*(\w+)\s*\+\s*2 \* X", text):
        if of in names:
            names.add(alias)
    return names


def unfenced(text):
    """(line, barrier) of the waits whose next tensor-memory access has no fence before it."""
    names, bad = commit_barriers(text), []
    for w in WAIT.finditer(text):
        if w.group(1) in names:
            e = EVENT.search(text, w.end())
            if e is not None and e.group("use"):
                bad.append((text.count("\n", 0, w.start()) + 1, w.group(1)))
    return bad


@pytest.mark.parametrize("name", KERNELS)
def test_every_wait_for_mmas_is_followed_by_the_fence(name):
    text = source(name)
    assert len(commit_barriers(text)) >= 2
    assert not unfenced(text)


def test_a_missing_fence_is_seen():
    text = """tc_commit(&done[0]);
      if (!dwait(&done[g & 1], 0, limit, abort_any)) return;
      %s
      tmem_st16(dst, w);"""
    assert unfenced(text % "") == [(2, "done")] and not unfenced(text % "tc_fence_after();")
