"""A wait that a whole warp takes part in has one answer for all of its lanes.

Lanes that poll a barrier, the clock and the abort flag by themselves may give up at
different times.  What follows a wait in the roles of whole warps (an elected issue,
tensor-memory access, __syncwarp) asks for all lanes.  The kernels are read as text:
outside the branches of a single lane every wait_or_abort is the one for whole warps, and
what looks at the abort flag to leave a loop or a role does so by a vote."""
import re

import pytest

from test_pair_signals import block
from test_tmem_order import source

KERNELS = ["pa_mla_expand.cu", "pa_mla_prefill.cu", "pa_mla_product.cu"]


def unvoted(text):
    """Lines of waits by whole warps whose lanes may go different ways."""
    single = [(m.start(), block(text, m.end())) for m in re.finditer(r"if \(lane == 0\) (?=\{)", text)]
    bad = [m.start() for m in re.finditer(r"\bwait_or_abort\([^;{]*?abort_any(, whole_warp)?\)", text) if not m.group(1)]
    for m in re.finditer(r"\*abort_any(?! = )", text):     # reads: a vote's, or those of a plain branch
        if not re.search(r"(?:__any_sync\(0xffffffffu, |\bif \(!?)$", text[:m.start()]):
            bad.append(m.start())
    return sorted({text.count("\n", 0, at) + 1 for at in bad if not any(a <= at < b for a, b in single)})


@pytest.mark.parametrize("name", KERNELS)
def test_waits_of_whole_warps_are_voted_on(name):
    text = source(name)
    assert "wait_or_abort(" in text and not unvoted(text)


def test_lanes_that_part_are_seen():
    assert unvoted("x = wait_or_abort(bar, 0, limit, abort_any);\n") == [1]
    assert not unvoted("x = wait_or_abort(bar, 0, limit, abort_any, whole_warp);\n")
    assert not unvoted("if (lane == 0) { wait_or_abort(bar, 0, limit, abort_any); }")
    assert unvoted("while (ok && *s_done < n) ok = !*abort_any && globaltimer() - t0 <= limit;") == [1]
    assert unvoted("const bool ok = f() && !*abort_any;") == [1]
    assert not unvoted("ok = !__any_sync(0xffffffffu, *abort_any || late);")
    assert not unvoted("if (!*abort_any) record_status(a, b, c);\n*abort_any = 1;")
