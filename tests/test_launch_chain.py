"""Every kernel is launched so that it may start before the one ahead of it has ended, and a kernel's
wait covers that one alone. So each block has to wait, whatever it then has to do: a grid whose
blocks left without waiting would end early, and the kernel behind it would start on top of the one
ahead. Checked in the sources; no GPU needed."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "routed_expert_ffn_moe_gb300", "csrc")


def span(s, i, pair):
    """[i, end) of the bracket that opens at s[i]."""
    depth = 0
    for j in range(i, len(s)):
        depth += (s[j] == pair[0]) - (s[j] == pair[1])
        if depth == 0:
            return j + 1
    raise ValueError("unbalanced")


def kernels(path):
    """(name, body) of the __global__ functions of a source file, comments dropped."""
    s = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__", s):
        at = m.end()
        while True:  # past __launch_bounds__(...) to the parameter list
            k = re.compile(r"(\w+)\s*\(").search(s, at)
            at = span(s, k.end() - 1, "()")
            if not k.group(1).startswith("__"):
                break
        if s[at:].lstrip().startswith("{"):
            b = s.index("{", at)
            yield k.group(1), s[b:span(s, b, "{}")]


ALL = [(os.path.basename(f), n, b) for f in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
       for n, b in kernels(f) if "selftest" not in f]


def test_the_kernels_are_found():
    assert {"k_attn_decode", "k_attn_join", "k_attn_prefill_join", "k_combine"} <= {n for _, n, _ in ALL}


@pytest.mark.parametrize("name,body", [a[1:] for a in ALL], ids=[f"{f}:{n}" for f, n, _ in ALL])
def test_no_block_leaves_before_it_has_waited(name, body):
    wait = re.search(r"pdl_wait_then_release\(\)", body)
    assert wait, name
    early = re.search(r"\breturn\s*;", body)
    assert not early or wait.start() < early.start(), name
