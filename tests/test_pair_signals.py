"""What a CTA pair's MMAs signal is waited for in both CTAs before either leaves.

A commit of a pair arrives at barriers in the shared memory of both CTAs, some time after
the MMAs before it are done; a CTA that has left may have a successor in that memory.  The
kernel is read as text: every barrier that such a commit names has a wait that both CTAs
reach, and none is signalled once more than it is waited for."""
import re

from test_tmem_order import commit_barriers, source, unfenced

WAIT = re.compile(r"\b(?:wait_or_abort\w*|mbar_wait|wait)\(\s*&?(\w+)")


def block(text, start):
    """End of the braces that open at or behind `start`."""
    depth = 0
    for i in range(text.index("{", start), len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return i + 1
    raise ValueError("open braces")


def one_cta(text):
    """Ranges of the text that only one CTA of the pair runs."""
    return [(m.start(), block(text, m.end())) for m in re.finditer(r"if \(rank == [01]\) (?=\{)", text)]


def unwaited(text):
    ranges = one_cta(text)
    both = {w.group(1) for w in WAIT.finditer(text) if not any(a <= w.start() < b for a, b in ranges)}
    return set(re.findall(r"\btc_commit_pair\(\s*&?(\w+)", text)) - both


def test_both_ctas_wait_for_every_commit_of_a_pair():
    text = source("pa_mla_expand.cu")
    assert len(set(re.findall(r"\btc_commit_pair\(\s*&?(\w+)", text))) >= 4
    assert not unwaited(text)


def test_weights_are_given_back_only_for_a_head_that_follows():
    """bfree is waited for when another head's weights are loaded: once a head but the first."""
    text = source("pa_mla_expand.cu")
    guard = re.search(r"if \((\w+)\) tc_commit_pair\(bfree\)", text).group(1)
    rule = re.search(r"const bool %s = ([^;]*);" % guard, text).group(1)
    assert re.match(r"t \+ 1 < end && ", rule) and "||" not in rule


def test_a_wait_of_one_cta_is_seen():
    text = "if (rank == 0) { tc_commit_pair(drain); mbar_wait(drain, 0, 1); }"
    assert unwaited(text) == {"drain"}
    assert not unwaited(text + " mbar_wait(drain, 0, 1);")


def test_every_wait_for_mmas_is_followed_by_the_fence():
    """As in the other kernels of latent attention (test_abi_mla_prefill.py)."""
    text = source("pa_mla_expand.cu")
    assert {"drain", "dfull", "empty", "bfree"} <= commit_barriers(text) and not unfenced(text)
    assert unfenced(text.replace("tc_fence_after();", ";"))
