"""Sizes at the end of 32 bits that the calls of the 16- and 32-bit paged cache must refuse, and what the compiler must give
their kernels, without a GPU.  The addresses are made up: none of these calls reaches a launch.
"""
import os
import re

import pytest

import linear_attention_sequence_gated_gb300 as gdn
from linear_attention_sequence_gated_gb300 import _build
from test_paged_host import BASE, L, attend, turn  # noqa: F401

FAR = dict(q=1 << 45, qo=1 << 46, k=None, ko=None, pos=1 << 47, plan=BASE)


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 31])
def test_tokens_whose_last_warp_would_pass_32_bits(L, T):  # noqa: F811
    """A warp takes up to 32 rows of 32 bytes, so the last one's tokens end up to 31 behind the last token."""
    assert turn(L, T=T, H=1, Hk=0, d=16, r=16, **FAR) == gdn.ERR_ARG


def test_tables_whose_tiles_fill_31_bits(L):  # noqa: F811
    """Room for 2^31 - 2 steps (126 * 11 sequences of 16 + 1549395 tiles): rounding their number up to a CTA's groups would wrap."""
    size = dict(B=1386, H=4, Hkv=1, page=16, max_pages=31 * 151 * 331 - 16)
    assert size["B"] * (size["max_pages"] + 16) == 2 ** 31 - 2
    assert attend(L, table=1 << 50, **size) == gdn.ERR_ARG
    assert L.gdn_flash_attn_paged_workspace_bytes(1386, 4, 1, 1, 128, 128, 16, size["max_pages"], 1) == 0
    assert L.gdn_flash_attn_paged_workspace_bytes(1386, 4, 1, 1, 128, 128, 16, size["max_pages"] - 1, 1) > 0


def test_kernels_have_the_registers_that_their_warps_share_out(L):  # noqa: F811
    """The attention's warps redistribute what the launch has (setmaxnreg); with fewer registers the library refuses to launch, so
    the compiler has to have given each kernel the full number: 128 beside 12 warps that compute, 168 beside 8."""
    seen = 0
    for t in ("bf16", "f16", "f32"):
        for d in (64, 128, 256):
            with open(os.path.join(_build.BUILD, f"gdn_paged_attn_{t}_{d}.log")) as f:
                log = f.read()
            for warps, used in re.findall(r"Compiling entry function '\S*attn_kernelI\w*?Li\d+ELi\d+ELi(\d+)ELi\d+ELb[01]E.*?"
                                          r"Used (\d+) registers", log, flags=re.S):
                assert int(used) == {12: 128, 8: 168}[int(warps)]
                seen += 1
    assert seen == 9 * 6
