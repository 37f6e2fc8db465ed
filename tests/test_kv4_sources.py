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
