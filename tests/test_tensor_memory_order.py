"""Order of tensor memory accesses in the kernels' sources, which no run shows reliably.

A wait on a barrier that tensor products arrive on (tc_commit) orders what follows behind those products only
together with tc_fence_after: the sources are read block by block, and a load or store of tensor memory, or a
product, has to find a fence on every way from the last such wait to it.

Loads and stores of tensor memory are a whole warp's. A `continue` of some lanes in the loop that they stand in would
leave it to the compiler whether the others wait for them.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_diffusion_speculative_project_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and "tc_commit(" in open(os.path.join(CSRC, f)).read())

TOKEN = re.compile(r"[{}]|\b(?:mbar_wait|mbar_wait_warp|wait)\(\s*&?(\w+)|\btc_fence_after\(|\btmem_(?:ld|st)\d\w*\(|\btc_mma_\w+\(")


def plain(text):
    """Comments and strings out, lines kept."""
    text = re.sub(r"/\*.*?\*/", lambda m: "\n" * m.group().count("\n"), text, flags=re.S)
    return re.sub(r'"(?:\\.|[^"\\\n])*"', '""', re.sub(r"//[^\n]*", "", text))


def unfenced(text):
    """Lines with an access to tensor memory that a wait may reach without a fence between them."""
    text = plain(text)
    barriers = set(re.findall(r"\btc_commit\(\s*&?(\w+)", text))
    found, outer, waiting, branch = [], [], False, None
    for m in TOKEN.finditer(text):
        t = m.group()
        if t == "{":   # at the block's begin, and at the ends of the branches before it
            outer.append((waiting, branch or False))
            branch = None
        elif t == "}":
            begin, ends = outer.pop()
            if re.match(r"\s*else\b", text[m.end():]):
                waiting, branch = begin, ends or waiting
            else:      # the block may have been passed by
                waiting = (begin or ends or waiting) and bool(outer)
        elif t.startswith("tc_fence_after"):
            waiting = False
        elif m.group(1):
            waiting |= m.group(1) in barriers
        elif waiting:
            found.append(text.count("\n", 0, m.start()) + 1)
    return found


def test_the_reading_finds_what_it_looks_for():
    head = "void f() { tc_commit(&done[0]);"
    for body, lines in (("mbar_wait(&done[1], 0); tc_fence_after(); tmem_ld32(a, v); }", []),
                        ("mbar_wait(&done[1], 0); tmem_ld32(a, v); }", [1]),
                        ("mbar_wait(&other, 0); tmem_ld32(a, v); }", []),
                        ("mbar_wait_warp(&done[1], 0);\nif (x) { tc_fence_after(); tmem_ld32(a, v); }\ntmem_st16_raw(a, v); }", [3]),
                        ("for (;;) { ok = mbar_wait(&done[1], 0); if (!ok) break; } tc_fence_after(); tmem_st32(a, v); }", []),
                        ("if (x) { mbar_wait(&done[1], 0); } else { tmem_ld32(a, v); }\ntmem_ld32(a, v); }", [2]),
                        ("if (x) { ok = mbar_wait(&done[1], 0); } /* tc_fence_after(); */\ntc_mma_bf16(a, v); }", [2])):
        assert unfenced(head + body) == lines, body


@pytest.mark.parametrize("name", FILES)
def test_tensor_memory_is_touched_behind_a_fence(name):
    assert unfenced(open(os.path.join(CSRC, name)).read()) == []


def skipped(text):
    """Lines with a `continue` in a loop that accesses tensor memory itself, not by a loop inside it."""
    text = plain(text)
    found, blocks = [], []   # a block: is it a loop's or a lambda's, has it accesses, lines of its `continue`
    for m in re.finditer(r"[{}]|\bcontinue\b|\btmem_(?:ld|st)\d\w*\(|\bfetch\(", text):
        t, inner = m.group(), next((b for b in reversed(blocks) if b[0]), None)
        if t == "{":
            head = text[:m.start()].rstrip()
            at, depth = len(head), 0
            while head.endswith(")") and at > 0:
                at -= 1
                depth += (head[at] == ")") - (head[at] == "(")
                if depth == 0:
                    break
            blocks.append([bool(re.search(r"(\b(for|while)|\])\s*$", head[:at])), False, []])
        elif t == "}":
            _, touches, lines = blocks.pop()
            found += lines if touches else []
        elif inner is not None:
            if t == "continue":
                inner[2].append(text.count("\n", 0, m.start()) + 1)
            else:
                inner[1] = True
    return found


def test_the_reading_finds_lanes_that_skip():
    for text, lines in (("void f() { for (int i = 0; i < 4; ++i) { tmem_ld16(a, v);\nif (!real) continue;\nx = v; } }", [2]),
                        ("void f() { for (int i = 0; i < 4; ++i) { if (x) {\ncontinue; }\ntmem_st16_raw(a, v); } }", [2]),
                        ("void f() { while (g(1)) { for (;;) { tmem_ld16(a, v); }\nif (x) continue; } }", []),
                        ("void f() { for (;;) { if (x) continue; } tmem_ld16(a, v); }", [])):
        assert skipped(text) == lines, text


@pytest.mark.parametrize("name", FILES)
def test_no_lane_skips_a_warps_access(name):
    assert skipped(open(os.path.join(CSRC, name)).read()) == []
