"""The 4-bit cache's kernel sources, read as text: orderings that no run can show
to be missing.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_attention_sequence_gated_gb300", "csrc")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["gdn_kv4.cuh", "gdn_kv4.cu", "gdn_kv4_attn.cu"])
def test_kernels_that_start_early_read_with_ordinary_loads(name):
    """They run while the kernel before them still writes lengths, pages, rows, queries and masks, so
    non-coherent loads are undefined; and neither those nor the cache-hint intrinsics are ordered behind
    the wait for that kernel's end, as an ordinary load or a volatile one is."""
    text = code(name)
    assert not re.findall(r"\b__ld(?:g|cg|ca|cs|lu|cv)\s*\(", text)
    assert not re.findall(r"ld\.global(?:\.\w+)*\.nc", text)
    for load in re.finditer(r'asm\s*(volatile)?\s*\(\s*"ld\.', text):
        assert load.group(1), text[load.start():load.start() + 80]


def blocks(text):
    """Every innermost-to-outermost { } block of a source text, as (start, end)."""
    open_at, found = [], []
    for i, c in enumerate(text):
        if c == "{":
            open_at.append(i)
        elif c == "}":
            found.append((open_at.pop(), i))
    return found


@pytest.mark.parametrize("name", ["gdn_kv4_attn.cu", "gdn_chunked.cu"])
def test_the_thread_that_initialises_a_barrier_fences_it(name):
    """fence.mbarrier_init orders the initialisations of the thread that executes it, and no others', before the
    asynchronous copies that signal the barriers: the fence follows in the block of the condition that the
    initialisation stands under (or in that of a loop's)."""
    text = code(name)
    every = sorted(blocks(text), key=lambda b: b[1] - b[0])
    inits = list(re.finditer(r"\bmbar_init\s*\(", text))
    assert inits
    for init in inits:
        at = init.start()
        line = text[text.rfind("\n", 0, at) + 1:at]
        assert not re.search(r"\bif\s*\(", line), line        # a condition of its own, without the fence
        for lo, hi in every:
            if lo < at < hi:
                head = text[text.rfind("\n", 0, lo) + 1:lo]
                if not re.search(r"\bfor\s*\(", head):
                    break
        assert "fence_mbar_init()" in text[at:hi], text[lo:hi][:200]
