"""A bounded wait ends for each lane by its own clock, so a warp that waits as a whole agrees on
the outcome before its next warp-wide instruction (a TMEM load, a shuffle).  When the lanes
disagree cannot be arranged on a GPU; that no such wait is left to its lanes is read here."""

import os
import re

from conftest import ROOT

SOURCE = os.path.join(ROOT, "fp8_delayed_scaling_02_b200", "csrc", "mm_fp8.cu")


def _headers(src, at):
    """The text in front of each brace that is open at ``at``."""
    opened = []
    for m in re.finditer(r"[{}]", src[:at]):
        if m.group() == "{":
            opened.append(re.split(r"[;{}]", src[:m.start()])[-1])
        elif opened:
            opened.pop()
    return opened


def test_every_wait_of_a_whole_warp_is_agreed_on():
    src = re.sub(r'"(?:\\.|[^"\\\n])*"', '""', open(SOURCE).read())  # PTX text has braces of its own
    src = re.sub(r"//[^\n]*", "", src)
    calls = [m.start() for m in re.finditer(r"\bmbar_wait\(", src)]
    whole = 0
    assert len(calls) > 8
    for at in calls:
        if "bool mbar_wait" in src[at - 12:at + 10]:
            continue  # its definition
        if any("lane == 0" in h for h in _headers(src, at)):
            continue  # one lane waits
        whole += 1
        line = src[:at].count("\n") + 1
        assert src[:at].rstrip().endswith("bool ok ="), f"line {line}: the lanes act on their own outcomes"
        after = src[src.index(";", at) + 1:].lstrip()
        assert after.startswith("ok = __all_sync(0xFFFFFFFFu, ok);"), f"line {line}: the outcome is not agreed on"
    assert whole == 4  # accumulators of the three epilogues, the operand of one
