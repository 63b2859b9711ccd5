"""Roles whose warps meet at named barriers leave their loops by a joint vote, read from the kernels' sources: a
warp that left by itself, after a wait that ran out, would keep the others at the barrier for ever."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_attention_gb300", "csrc")


def loop_exits(text, head):
    """Statements that leave the loop that starts with `head`: its breaks and returns outside of the loops and
    lambdas within it, one that stands alone with the statement before it."""
    text = " ".join(re.sub(r"//[^\n]*", "", text).split())
    at = text.index(head)
    out, inner, words, last, parens = [], [], "", "", 0
    for ch in text[text.index("{", at):]:
        parens += (ch == "(") - (ch == ")")
        if parens or ch not in "{};":
            words += ch
            continue
        loop = re.search(r"\b(for|while|do|switch)\b|\[[&=]?\]", words)
        if ch == "{":
            inner.append(bool(inner and loop))
        elif ch == "}":
            inner.pop()
            if not inner:
                return out
        elif re.search(r"\b(break|return)\b", words) and not loop and not any(inner):
            out.append(f"{last}; {words.strip()}" if words.strip() == "break" else words.strip())
        words, last = "", words.strip()
    raise AssertionError("the loop does not end")


@pytest.mark.parametrize("source, head", [("tq_paged_tree.cu", "for (uint32_t items = 0;; ++items)")])
def test_the_item_loop_is_left_by_all_warps_together(source, head):
    exits = loop_exits(open(os.path.join(CSRC, source), encoding="utf-8").read(), head)
    assert exits and all("both_or(" in e for e in exits), exits


def test_the_check_sees_a_warp_that_leaves_alone():
    text = "for (;;) { if (!next()) break; for (;;) { if (x) break; } while (y) break; if (both_or(!ok)) { z(); break; } }"
    assert loop_exits(text, "for (;;)") == ["if (!next()) break", "z(); break"]
