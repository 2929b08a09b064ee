"""What follows a wait in the roles of whole warps is done by whole warps.

Lanes that poll a barrier, the clock and the abort flag by themselves may give up at
different times, and an elected issue, tensor-memory access or __syncwarp asks for all of
them.  The kernels are read as text.  Outside the branches of a single lane a wait is either
the one for whole warps, whose lanes get one answer, or it goes into the lane's own `ok`
(`ok = ok && wait_or_abort(..)`): then no branch hangs on a wait, MMAs are issued under
`leader && ok` by a lane elected once, with the warp together again behind them, and the lanes
vote on ok before the warp branches on it."""
import re

import pytest

from test_pair_signals import block
from test_tmem_order import source

KERNELS = ["pa_mla_expand.cu", "pa_mla_prefill.cu", "pa_mla_product.cu"]


def unvoted(text):
    """Lines where a warp's lanes may go different ways."""
    single = [(m.start(), block(text, m.end())) for m in re.finditer(r"if \(lane == 0\) (?=\{)", text)]
    bad, own_ok = [], False
    for m in re.finditer(r"\bwait_or_abort\([^;{]*?abort_any(, whole_warp)?\)", text):
        if m.group(1) or any(a <= m.start() < b for a, b in single):
            continue
        if text[:m.start()].endswith(" ok = ok && "):
            own_ok = True
        else:
            bad.append(m.start())
    for m in re.finditer(r"\*abort_any(?! = )", text):     # reads: a vote's, a plain branch's, or into the lane's ok
        before = text[:m.start()]
        if not (re.search(r"(?:__any_sync\(0xffffffffu, |\bif \(!?)$", before) or
                own_ok and re.search(r" ok = !$", before)):
            bad.append(m.start())
    if own_ok:
        bad += [m.start() for m in re.finditer(r"(?:!|&& |return )wait\(", text) if not any(a <= m.start() < b for a, b in single)]
        for m in re.finditer(r"if \((?:elect_one\(\)|leader)[^{;]*(?=\{)", text):
            end = block(text, m.end())
            if "mma_" in text[m.end():end]:
                if m.group() != "if (leader && ok) " or "bool leader = elect_one();" not in text or not re.match(r"\s*(?:ok = warp_all\(ok\)|__syncwarp\(\));", text[end:]):
                    bad.append(m.start())
    return sorted({text.count("\n", 0, at) + 1 for at in bad if not any(a <= at < b for a, b in single)})


@pytest.mark.parametrize("name", KERNELS)
def test_no_lane_goes_its_own_way(name):
    text = source(name)
    assert "wait_or_abort(" in text and not unvoted(text)


def test_the_lanes_vote_before_their_warp_branches():
    """pa_mla_prefill's MMA warps: each way through a step ends in a vote, as does the last product."""
    text = source("pa_mla_prefill.cu")
    issue_s = text.index("auto issue_s = ")
    assert re.search(r"ok = warp_all\(ok\);\s*\}$", text[issue_s:block(text, text.index(") {", issue_s))])
    loop = text.index("for (int i = 0; i < w.n && ok; ++i, ++g) {", issue_s)
    body = text[loop:block(text, loop)]
    assert re.search(r"if \(i < steps\) \{[\s\S]*\bissue_s\([^;]*;(?:\s*due\w* = [^;]*;)*\s*\} else \{", body)
    assert re.search(r"ok = warp_all\(ok\);\s*\}\s*\}$", body)
    assert re.search(r"if \(ok\) flush\(\);\s*ok = warp_all\(ok\);", text)


def test_lanes_that_part_are_seen():
    call = "wait_or_abort(bar, 0, limit, abort_any"
    assert unvoted(f"x = {call});\n") == [1]
    assert not unvoted(f"x = {call}, whole_warp);\n")
    assert not unvoted(f"if (lane == 0) {{ {call}); }}")
    assert unvoted("while (ok && *s_done < n) ok = !*abort_any && globaltimer() - t0 <= limit;") == [1]
    assert unvoted("const bool ok = f() && !*abort_any;") == [1]
    assert not unvoted("ok = !__any_sync(0xffffffffu, *abort_any || late);")
    assert not unvoted("if (!*abort_any) record_status(a, b, c);\n*abort_any = 1;")
    own = f"const bool leader = elect_one(); ok = ok && {call});\n"
    issue = "if (leader && ok) { mma_ss(d); }\n"
    assert not unvoted(own + issue + " ok = warp_all(ok);")
    assert unvoted(own + issue) == [2]
    assert unvoted(own + "if (elect_one() && ok) { mma_ss(d); }\n ok = warp_all(ok);") == [2]
    assert unvoted(own + "if (leader) { mma_ss(d); }\n ok = warp_all(ok);") == [2]
    assert unvoted(own + "if (!wait(bar)) return;") == [2]
