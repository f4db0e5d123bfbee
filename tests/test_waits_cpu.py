"""Waits of the kernels, read from their source: no GPU can be made to lose a copy.

A wait on an mbarrier gives up after a limit, each lane by its own clock.  Near the
limit some lanes of a warp may see the phase and others not, and what follows is done
by whole warps (votes, shuffles, matrix products): the answer has to be one for all."""

import glob
import os
import re

import pytest

import gqa_attention_learned_gb300 as sa

CSRC = os.path.join(os.path.dirname(sa.__file__), "csrc")
FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu")) if "mbar_wait" in open(f).read())
VOTE = "__all_sync(0xffffffffu, "


def uses(source):
    """What stands before each wait whose answer is used, and the wait's first words."""
    source = re.sub(r"//[^\n]*", "", source)
    # a file's own `wait` is one more of them, unless it votes itself
    names = "mbar_wait|wait" if "bool wait(" in source else "mbar_wait"
    for m in re.finditer(rf"\b(?:{names})\(", source):
        before = source[:m.start()]
        if before.rstrip().endswith(("bool", "inline", ";", "{", "}")):
            continue                                       # its definition; a statement
        if before.rstrip().endswith(")") and before.rstrip()[-2:] != "))":
            continue                                       # for (..) mbar_wait(..); if (..) mbar_wait(..);
        yield before[-60:], source[m.start():m.start() + 60]


@pytest.mark.parametrize("name", FILES)
def test_a_warp_has_one_answer(name):
    with open(os.path.join(CSRC, name)) as f:
        found = list(uses(f.read()))
    assert found
    for before, call in found:
        assert before.endswith(VOTE), f"{name}: {' '.join((before + call).split())}"


def test_the_search_finds_what_it_looks_for():
    one = "bool wait(int *b) { return true; }\n" \
          "if (!mbar_wait(&b, 0)) return; for (int i = 0; i < 3; ++i) wait(&c, 1);\n"
    assert [c[:9] for _, c in uses(one)] == ["mbar_wait"]
    assert not list(uses("bool mbar_wait(x) { wait(&a, 0); }"))
    assert [b[-9:] for b, _ in uses(f"ok = {VOTE}mbar_wait(&a, 0));")] == ["ffffffu, "]
