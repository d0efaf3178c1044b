"""Every bounded wait of a kernel may give up, so none of its answers may be dropped: a warp that goes on would use
what has not arrived, and a block that leaves would leave copies in flight behind it."""
import glob
import os
import re

import routed_expert_ffn_moe_gb300 as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")
WAIT = re.compile(r"\b(wait_phase|wait_bar|wait_bar_pair)\s*\(")


def dropped(text):
    """Calls of a wait that stand as a statement of their own."""
    text = re.sub(r"//[^\n]*", "", text)
    out = []
    for m in WAIT.finditer(text):
        before = text[:m.start()].rstrip()
        while before.endswith("::"):  # a qualified name
            before = re.sub(r"\w*::$", "", before).rstrip()
        if re.search(r"([;{}]|\belse|\bdo)$", before) or re.search(r"\b(if|for|while)\s*\([^;{}]*\)$", before):
            out.append(text[m.start():].split(";")[0])
    return out


def test_the_check_finds_dropped_waits():
    assert dropped("{ wait_phase(a, b); }") and dropped("if (RES && vec) wait_bar(x);") and dropped("a(); tc::wait_bar(x);")
    assert dropped("else\n  wait_bar(x, y);")
    assert not dropped("ok = wait_bar(x);") and not dropped("if (!wait_phase(a, b)) break;")
    assert not dropped("return tc::wait_bar(x);") and not dropped("bool wait_phase(uint64_t* bar) {")
    assert not dropped("__all_sync(m, wait_phase(a)); // wait_bar(x)") and not dropped("if (a ||\n !wait_bar(x)) {")


def test_no_answer_of_a_wait_is_dropped():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
    texts = {os.path.basename(f): open(f, encoding="utf-8").read() for f in files}
    assert sum(len(WAIT.findall(t)) for t in texts.values()) > 40
    assert {f: d for f, t in texts.items() if (d := dropped(t))} == {}
